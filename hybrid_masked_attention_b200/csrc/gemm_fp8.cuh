// Pieces shared by the kernels of the block-scaled e4m3 product (gemm_fp8.cu, gemm_fp8_rows.cu).
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "fp8.cuh"
#include "mma_util.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace mtfm {

// kind::f8f6f4, e4m3 x e4m3 -> fp32 (formats 0), both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Test of a TMA coordinate in the bounds-checked build (MTFM_DEBUG_BOUNDS, mtfm_internal.cuh): a
// failed one sets the error word, and the caller skips the copy.  `true` in other builds.
__device__ __forceinline__ bool tma_inbounds(int32_t* err, bool ok) {
#ifdef MTFM_DEBUG_BOUNDS
  if (!ok) atomicOr(err, kErrBounds);
  return ok;
#else
  return true;
#endif
}
// A load's box may reach past its matrix, in x and y; its start is aligned, and not negative.
__device__ __forceinline__ bool load_ok(int32_t* err, int x, int cols, int size, int y) {
  return tma_inbounds(err, x >= 0 && (int64_t)x * size % 16 == 0 && x < cols && y >= 0);
}
// A store starts inside its matrix.
__device__ __forceinline__ bool store_ok(int32_t* err, int x, int cols, int size, int y, int rows) {
  return tma_inbounds(err, x >= 0 && (int64_t)x * size % 16 == 0 && x < cols && y >= 0 && y < rows);
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// shared::cluster address of a shared::cta address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
constexpr float kLog2E = 1.44269504088896341f;
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// SiLU without a cancellation at either end: with e = exp(-|x|) in [0, 1],
//   SiLU(x) = x / (1 + e) for x >= 0,  x e / (1 + e) below.
// Relative error at most (13 + 2 |x|) 2^-24 (the exponential's argument is rounded twice, 2 |x|;
// exponential 4, four shared reciprocals 7, products 2); results below 2^-119 in magnitude are 0.
// NaN gives NaN, and so does minus infinity (0 times infinity).
__device__ __forceinline__ float silu_exp(float x) { return ex2_approx(-fabsf(x * kLog2E)); }
__device__ __forceinline__ float silu_top(float x, float e) { return x < 0.f ? x * e : x; }
__device__ __forceinline__ float silu1(float x) {
  const float e = silu_exp(x);
  return silu_top(x, e) * rcp_approx(1.f + e);
}
// Four values with one reciprocal, 1/a = (b c d) / (a b c d): 1.25 special-function operations a
// value.  The denominators lie in [1, 2]; a NaN's is taken as 2, which keeps it out of the others.
// 53133 x 1280 x 512 takes 76 us with it.  h + h tanh(h), h = x / 2, with the hardware's tanh (one
// operation, and half the instructions) took 65, but loses SiLU of negative values to
// cancellation: an error of up to 2^-12 |x|, 1 % of SiLU at x = -4 and all of it at -12.
__device__ __forceinline__ void silu4(float2& x, float2& y) {
  const float e0 = silu_exp(x.x), e1 = silu_exp(x.y), e2 = silu_exp(y.x), e3 = silu_exp(y.y);
  const float a = fminf(1.f + e0, 2.f), b = fminf(1.f + e1, 2.f), c = fminf(1.f + e2, 2.f), d = fminf(1.f + e3, 2.f);
  const float ab = a * b, cd = c * d, r = rcp_approx(ab * cd);
  const float rab = r * cd, rcd = r * ab;
  x = __fmul2_rn(make_float2(silu_top(x.x, e0), silu_top(x.y, e1)), __fmul2_rn(make_float2(rab, rab), make_float2(b, a)));
  y = __fmul2_rn(make_float2(silu_top(y.x, e2), silu_top(y.y, e3)), __fmul2_rn(make_float2(rcd, rcd), make_float2(d, c)));
}
// ---------------------------------------------------------------- host
// Row-major e4m3 matrix [rows, cols], row pitch ld bytes; boxes of box_rows x 128 columns.
inline bool make_map_e4m3(CUtensorMap* map, const uint8_t* base, int rows, int cols, int64_t ld, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {(cuuint32_t)kGroup, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Few rows of A (gemm_fp8_rows.cu): whether that kernel takes the product, and its launch.
bool gemm_fp8_rows_takes(int M, int N, int K);
cudaError_t launch_gemm_fp8_rows(int32_t* err, int M, int N, int K, const Fp8In& a, const Fp8In& b, const Fp8Epi& epi,
                                 cudaStream_t st);

}  // namespace mtfm
