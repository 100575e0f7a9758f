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
// SiLU of two values, for fp32 outputs: x / (1 + exp(-x)) with one reciprocal for both, 1/a =
// b / (a b).  The exponentials are held below 2^63 (x > -43.6) so that a b stays finite; beyond
// that |SiLU| < 5e-18 is off by no more than that.  Otherwise within a few roundings of fp32.
__device__ __forceinline__ void silu2(float& x0, float& x1) {
  const float a = 1.f + fminf(ex2_approx(x0 * -kLog2E), 0x1p63f), b = 1.f + fminf(ex2_approx(x1 * -kLog2E), 0x1p63f);
  const float r = rcp_approx(a * b);
  x0 = x0 * (r * b);
  x1 = x1 * (r * a);
}
// For bf16 outputs: h + h tanh(h), h = x / 2, with the hardware's tanh (one special-function
// operation instead of 1.5, and half the instructions; they bound a K = 512 projection:
// 53133 x 1280 takes 72 us with silu2 and 62 with this).  tanh's relative error of 2^-11 makes an
// error of at most 2^-12 |x|, a sixteenth of bf16's half step at |x|: phi_1 of the bf16
// projections (gemm_tc.cu) is the same function.
template <typename OT>
__device__ __forceinline__ void silu_pair(float& x0, float& x1) {
  if constexpr (sizeof(OT) == 2) {
    x0 = silu_fast(x0);
    x1 = silu_fast(x1);
  } else {
    silu2(x0, x1);
  }
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
