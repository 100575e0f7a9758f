// The 8-bit form shared by the producers (norm, gate, quantiser) and the block-scaled
// product: e4m3 values (4 exponent, 3 mantissa bits, largest 448) with one fp32 scale for
// each group.  A group is 128 consecutive columns of one row, or a block of 128 x 128; the
// last ones are ragged.  With m = max(max |v|, 2^-100) over the group
//     scale = m / 448,   q = e4m3(v * (448 (1 / m)))   (round to nearest even, saturating),
// every operation rounded to nearest fp32, so that v ~ scale * q with an error of at most half a step of e4m3 (2^-4 relative) for
// |v| >= m * 2^-6 / 448 and of m * 2^-10 / 448 below that.  The floor keeps 1 / m finite
// for a group of zeros (q = 0).  A NaN does not enter m; it stays a NaN of its own element.
// An infinity makes the scale infinite, and the whole group reads back as NaN.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "mtfm_internal.cuh"
#include "tma_host.cuh"

namespace mtfm {

constexpr int kGroup = 128;
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 0x1p-100f;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// max |x| over the warp (NaN operands are passed over), on every lane.
__device__ __forceinline__ float warp_absmax(float x) {
  float y;
  asm("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float absmax4(const float (&v)[4]) {
  return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
}
__device__ __forceinline__ float warp_sum32(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Index of the warp in its block, known to the compiler as equal in all of its lanes: row
// pointers then live in uniform registers.  The quantiser's time was mostly address arithmetic
// (12345 x 1000 bf16: 12.6 us, with it 9.6); the norm, whose next row is loaded under a
// condition, lost its overlap by it and a quarter of its speed.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// 1 / x to one unit in the last place, subnormal results included.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sum of the partial sums of a row's W warps (a power of two, at least 2), in their order.
__device__ __forceinline__ float row_sum(const float* part, int W) {
  if (W < 4) return part[0] + part[1];
  float s = 0.f;
  for (int k = 0; k < W; k += 4) {
    const float4 t = *reinterpret_cast<const float4*>(part + k);
    s += (t.x + t.y) + (t.z + t.w);
  }
  return s;
}

// Four columns of a 128-column group per lane, of which the group's row has n.
// VEC (rows of a multiple of 4 columns that start on 4-element boundaries): columns 4 lane ..
// 4 lane + 3 as one vector.  Otherwise columns lane, lane + 32, lane + 64, lane + 96, which
// keeps element-wise accesses coalesced for rows at any offset.
// Raw: the four elements as loaded.  Nothing is computed from them before unpack(), so that a row
// fetched ahead stays in flight (with single bf16 loads packed into words at once, the backward of
// 30000 x 1001 took 107 us; without, 68).
template <typename T, bool VEC>
struct Raw;
template <bool VEC>
struct Raw<float, VEC> { float4 v; };
template <>
struct Raw<__nv_bfloat16, true> { uint2 v; };
template <>
struct Raw<__nv_bfloat16, false> { uint16_t v[4]; };

template <bool VEC>
__device__ __forceinline__ bool lane_has(int lane, int j, int n) { return (VEC ? 4 * lane : lane + 32 * j) < n; }
template <bool VEC>
__device__ __forceinline__ int lane_col(int lane, int j) { return VEC ? 4 * lane + j : lane + 32 * j; }

template <bool VEC>
__device__ __forceinline__ Raw<float, VEC> load_raw(const float* p, int lane, int n) {
  Raw<float, VEC> r{make_float4(0.f, 0.f, 0.f, 0.f)};
  if (VEC) {
    if (4 * lane < n) r.v = *reinterpret_cast<const float4*>(p + 4 * lane);
  } else {
    if (lane < n) r.v.x = p[lane];
    if (lane + 32 < n) r.v.y = p[lane + 32];
    if (lane + 64 < n) r.v.z = p[lane + 64];
    if (lane + 96 < n) r.v.w = p[lane + 96];
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ Raw<__nv_bfloat16, VEC> load_raw(const __nv_bfloat16* p, int lane, int n) {
  Raw<__nv_bfloat16, VEC> r;
  if constexpr (VEC) {
    r.v = make_uint2(0, 0);
    if (4 * lane < n) r.v = *reinterpret_cast<const uint2*>(p + 4 * lane);
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = lane + 32 * j < n ? h[lane + 32 * j] : 0;
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ void unpack(const Raw<float, VEC>& r, float (&v)[4]) {
  v[0] = r.v.x; v[1] = r.v.y; v[2] = r.v.z; v[3] = r.v.w;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, true>& r, float (&v)[4]) {
  v[0] = __uint_as_float(r.v.x << 16);
  v[1] = __uint_as_float(r.v.x & 0xffff0000u);
  v[2] = __uint_as_float(r.v.y << 16);
  v[3] = __uint_as_float(r.v.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, false>& r, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __uint_as_float((uint32_t)r.v[j] << 16);
}
template <bool VEC, typename T>
__device__ __forceinline__ void load4(const T* p, int lane, int n, float (&v)[4]) {
  unpack(load_raw<VEC>(p, lane, n), v);
}
// The same of an array that nothing writes meanwhile (a norm's weight): such loads may move up
// past the stores of other columns, which they otherwise wait behind one group after the other.
template <bool VEC>
__device__ __forceinline__ Raw<float, VEC> load_const(const float* p, int lane, int n) {
  Raw<float, VEC> r{make_float4(0.f, 0.f, 0.f, 0.f)};
  if (VEC) {
    if (4 * lane < n) r.v = __ldg(reinterpret_cast<const float4*>(p + 4 * lane));
  } else {
    if (lane < n) r.v.x = __ldg(p + lane);
    if (lane + 32 < n) r.v.y = __ldg(p + lane + 32);
    if (lane + 64 < n) r.v.z = __ldg(p + lane + 64);
    if (lane + 96 < n) r.v.w = __ldg(p + lane + 96);
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ void put4(float* p, int lane, int n, const float (&v)[4]) {
  if (VEC) {
    if (4 * lane < n) *reinterpret_cast<float4*>(p + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < n) p[lane + 32 * j] = v[j];
  }
}
template <bool VEC>
__device__ __forceinline__ void put4(__nv_bfloat16* p, int lane, int n, const float (&v)[4]) {
  if (VEC) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    uint2 t;
    t.x = *reinterpret_cast<uint32_t*>(&lo);
    t.y = *reinterpret_cast<uint32_t*>(&hi);
    if (4 * lane < n) *reinterpret_cast<uint2*>(p + 4 * lane) = t;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < n) p[lane + 32 * j] = __float2bfloat16_rn(v[j]);
  }
}
// q = e4m3(v * inv)
template <bool VEC>
__device__ __forceinline__ void put4_e4m3(uint8_t* p, int lane, int n, const float (&v)[4], float inv) {
  const uint32_t t = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  if (VEC) {
    if (4 * lane < n) *reinterpret_cast<uint32_t*>(p + 4 * lane) = t;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < n) p[lane + 32 * j] = (uint8_t)(t >> (8 * j));
  }
}

// The factor of a group, 448 (1 / m): reciprocal and product each rounded to nearest, which is
// what `448.0 / m` is in torch, so that the quantiser's bytes are those of the plain form.  (With
// an approximate reciprocal single values fell on the other side of a rounding border.)
__device__ __forceinline__ float quant_factor(float m) { return kE4m3Max * __frcp_rn(m); }

// Quantises the warp's C neighbouring 128-column groups of a row, of which n columns are left
// (columns past them hold zeros), and writes their bytes.  Lane i < C returns group i's m =
// max(max |v|, 2^-100), from which the caller writes the scale m / 448.  Lane i also computes the
// factor of group i: one reciprocal for the row instead of one a group.
template <bool VEC, int C>
__device__ __forceinline__ float quant_groups(const float (&v)[C][4], int lane, int n, uint8_t* q) {
  float mine = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i * kGroup < n) {
      const float m = fmaxf(warp_absmax(absmax4(v[i])), kAmaxFloor);
      if (lane == i) mine = m;
    }
  const float f = quant_factor(mine);
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i * kGroup < n) put4_e4m3<VEC>(q + i * kGroup, lane, n - i * kGroup, v[i], __shfl_sync(0xffffffffu, f, i));
  return mine;
}

// Matrices of the 8-bit entry points.  ld: row pitch in elements.
struct MatIn {
  const void* p;
  int64_t ld;
  int type;  // mtfm_dtype
};
struct MatOut {
  void* p;
  int64_t ld;
  int type;
};
struct Fp8Out {
  uint8_t* q;
  int64_t ld;
  float* scale;
  int64_t ld_scale;
};
struct Fp8In {
  const uint8_t* q;
  int64_t ld;
  const float* scale;
  int64_t ld_scale;
};

constexpr int kMaxNormDim = 16384;

// Every row starts on a boundary of 4 elements of `size` bytes.
inline bool rows_vec4(const void* p, int64_t ld, int size) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(4 * size - 1)) == 0 && ld % 4 == 0;
}
inline int dtype_size(int type) { return type == MTFM_BF16 ? 2 : 4; }

// err (may be NULL): a device error word; the kernel does nothing while it is not zero.
// With a row_map, rows from `mapped` on read row row_map[row - mapped] of x (a kernel of its own:
// the test in the other one's loads cost it a third of its speed); x must then be fp32, delta and
// x_out NULL.
cudaError_t launch_add_rmsnorm_fp8(const int32_t* err, int rows, int dim, const MatIn& x, const MatIn& delta,
                                   int mapped, const int32_t* row_map, const float* w, float eps, const MatOut& x_out,
                                   const Fp8Out& out, float* rstd, cudaStream_t st);
// Blocks of the backward's row pass at most (2 an SM of 148): each writes one partial row of dw.
constexpr int kNormBwdBlocks = 296;
cudaError_t launch_rmsnorm_bwd(int rows, int dim, const MatIn& x, const float* w, const float* rstd, const MatIn& dy,
                               const MatIn& dres, const MatOut& dx, float* dw, float* partials, cudaStream_t st);
cudaError_t launch_gate_fwd_fp8(const MetaView& m, bool target, int rows, int D, float eps, const float* a,
                                const __nv_bfloat16* u, const float* gamma, const float* beta, const Fp8Out& out,
                                float* stats, cudaStream_t st);
cudaError_t launch_fp8_quant(int rows, int cols, const MatIn& x, int block_rows, const Fp8Out& out, cudaStream_t st);

// Epilogue of the block-scaled product: out = act(C) + res, written into up to four column
// segments (each its own matrix, borders at multiples of 32) and, with a row map, into row
// row_map[i] of out and res for output row i.
struct Fp8Epi {
  int act;       // mtfm_act
  int out_type;  // mtfm_dtype of the segments and of res
  int n_seg;
  int seg_begin[5];
  void* seg_ptr[4];
  int64_t seg_ld[4];
  const void* res;  // NULL: none (one segment only)
  int64_t ld_res;
  const int32_t* row_map;
};
cudaError_t launch_gemm_fp8(int32_t* err, int M, int N, int K, const Fp8In& a, const Fp8In& b, const Fp8Epi& epi,
                            cudaStream_t st);

}  // namespace mtfm
