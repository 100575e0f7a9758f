// Residual addition, RMSNorm and quantisation in one pass over the row.
//
//   h = x + delta,  r = 1 / sqrt(mean_j h_j^2 + eps),  v = h r w  ->  (q, scale) of fp8.cuh
//   x_out = h rounded to x's type (the residual stream; v is taken from h before it)
//
// Each element is moved once and takes about ten operations: bound by memory.  A 128-column
// group is one warp's 32 lanes x 4 columns, so the group's largest magnitude is one redux
// instruction and nothing goes through shared memory for the scales.
//
// Up to 1024 columns a warp holds its whole row (C groups); wider rows are split over W warps,
// which exchange one partial sum.  Warps stride over the rows.
// 57023 x 768 fp32 with a bf16 delta: 81 us, 5.9 TB/s; 8191 x 4096 bf16 with a bf16 delta: 46 us.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"

namespace mtfm {
namespace {

struct None {};    // no delta
struct Mapped {};  // no delta, and rows from `mapped` on gathered

template <typename XT, typename DT>
struct NormArgs {
  const int32_t* err;
  int rows, dim, W;
  const XT* x;
  int64_t ldx;
  const DT* delta;
  int64_t ld_delta;
  int mapped;  // rows from this one on read row row_map[row - mapped] of x
  const int32_t* row_map;
  const float* w;
  float eps;
  XT* x_out;
  int64_t ld_xout;
  Fp8Out out;
  float* rstd;
};

// Threads of a block: 4 rows of one warp each, or the W <= 16 warps of rows of up to C groups
// a warp (8 warps, two blocks an SM, at C = 4; 16 warps at C = 8).
template <int C, bool MULTI>
constexpr int kThreadsN = !MULTI ? 128 : C == 4 ? 256 : 512;

template <typename XT, typename DT, int C, bool MULTI, bool VEC>
__global__ void __launch_bounds__(kThreadsN<C, MULTI>)
add_rmsnorm_fp8_kernel(const __grid_constant__ NormArgs<XT, DT> p) {
  constexpr bool kMapped = std::is_same<DT, Mapped>::value;
  constexpr bool kDelta = !kMapped && !std::is_same<DT, None>::value;
  using DRaw = typename std::conditional<kDelta, DT, XT>::type;
  constexpr int kWarps = kThreadsN<C, MULTI> / 32;
  __shared__ __align__(16) float s_part[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = MULTI ? p.W : 1;
  const int sub = MULTI ? warp % W : 0, slot = MULTI ? warp / W : warp;
  const int R = kWarps / W;  // rows of a block at a time
  // the warp's C groups are neighbours: their addresses differ by constants
  const int col0 = sub * C * kGroup, n0 = p.dim - col0;  // first column, and columns from there on
  pdl_wait();
  pdl_trigger();
  if (p.err && *p.err) return;
  Raw<XT, VEC> xr[C];
  Raw<DRaw, VEC> dr[C];
  auto load_row = [&](int64_t row) {
    if (row >= p.rows) return;
    int64_t src = row;
    if constexpr (kMapped) src = row >= p.mapped ? (int64_t)p.row_map[row - p.mapped] : row;
    const XT* px = p.x + src * p.ldx + col0;
    // No test of the group around a load or its use (past the row the lanes' own predicates load
    // nothing, and zeros are held): where both stood under the same test, the compiler joined them
    // in some instances and the row's loads were waited for one by one (40000 x 1000, fp32 and an
    // fp32 delta: 236 us against 84).
#pragma unroll
    for (int i = 0; i < C; ++i)
      xr[i] = load_raw<VEC>(px + i * kGroup, lane, n0 - i * kGroup);
    if constexpr (kDelta) {
      const DT* pd = p.delta + row * p.ld_delta + col0;
#pragma unroll
      for (int i = 0; i < C; ++i)
        dr[i] = load_raw<VEC>(pd + i * kGroup, lane, n0 - i * kGroup);
    }
  };
  // The next row is loaded before the present one is reduced, and one-warp rows hold the weight in
  // registers.  (Groups of eight a warp of a split row leave no registers for either.)
  constexpr bool kAhead = !(C == 8 && MULTI);
  constexpr bool kHoldW = !MULTI;
  const float* pw = p.w + col0;
  Raw<float, VEC> wr[kHoldW ? C : 1];
  if constexpr (kHoldW) {
#pragma unroll
    for (int i = 0; i < C; ++i) wr[i] = load_const<VEC>(pw + i * kGroup, lane, n0 - i * kGroup);
  }
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t row = (int64_t)blockIdx.x * R + slot;
  if (kAhead) load_row(row);
  int flip = 0;
  // every warp of a block makes the same number of rounds (the barrier below)
  for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < p.rows; row0 += step, row += step, flip ^= 1) {
    if (!kAhead) load_row(row);
    float h[C][4];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      unpack(xr[i], h[i]);
      if constexpr (kDelta) {
        float d[4];
        unpack(dr[i], d);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] += d[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fmaf(h[i][j], h[i][j], s);
    }
    if (kAhead) load_row(row + step);
    s = warp_sum32(s);
    if (MULTI) {
      if (lane == 0) s_part[flip][warp] = s;
      __syncthreads();
      s = row_sum(s_part[flip] + warp - sub, W);
    }
    if (row >= p.rows) continue;
    const float r = 1.f / sqrtf(s / (float)p.dim + p.eps);
    if (p.rstd && sub == 0 && lane == 0) p.rstd[row] = r;
    uint8_t* qr = p.out.q + row * p.out.ld + col0;
    XT* xo = p.x_out + row * p.ld_xout + col0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int n = n0 - i * kGroup;
      if (n > 0) {
        if (kDelta && p.x_out) put4<VEC>(xo + i * kGroup, lane, n, h[i]);
        float ww[4];
        if constexpr (kHoldW) unpack(wr[i], ww);
        else unpack(load_const<VEC>(pw + i * kGroup, lane, n), ww);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = h[i][j] * r * ww[j];
      }
    }
    const float mine = quant_groups<VEC>(h, lane, n0, qr);
    if (lane < C && n0 > lane * kGroup) p.out.scale[row * p.out.ld_scale + sub * C + lane] = mine / kE4m3Max;
  }
}

template <typename XT, typename DT, int C, bool MULTI, bool VEC>
cudaError_t go(const NormArgs<XT, DT>& a, cudaStream_t st) {
  constexpr int threads = kThreadsN<C, MULTI>;
  const int R = threads / 32 / a.W;
  static int per_sm = 0;  // blocks an SM holds: a property of the kernel
  if (per_sm == 0) {
    int n = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, add_rmsnorm_fp8_kernel<XT, DT, C, MULTI, VEC>,
                                                                  threads, 0);
    if (e != cudaSuccess) return e;
    per_sm = n > 0 ? n : 1;
  }
  const int64_t blocks = std::min<int64_t>(((int64_t)a.rows + R - 1) / R, (int64_t)per_sm * sm_count());
  return launch_pdl(add_rmsnorm_fp8_kernel<XT, DT, C, MULTI, VEC>, dim3((unsigned)blocks), dim3(threads), 0, st, a);
}

inline int pow2_ceil(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

// Element-wise rows (VEC false) of more than two groups go to the split form at once: eight groups
// are 64 single loads a lane.
template <typename XT, typename DT, bool VEC>
cudaError_t shape(NormArgs<XT, DT>& a, cudaStream_t st) {
  const int G = (a.dim + kGroup - 1) / kGroup;
  a.W = 1;
  if (G <= 2) return go<XT, DT, 2, false, VEC>(a, st);
  if constexpr (VEC) {
    if (G <= 4) return go<XT, DT, 4, false, VEC>(a, st);
    if (G <= 6) return go<XT, DT, 6, false, VEC>(a, st);
    if (G <= 8) return go<XT, DT, 8, false, VEC>(a, st);
  }
  if (G <= 32) {
    a.W = std::max(2, pow2_ceil((G + 3) / 4));
    return go<XT, DT, 4, true, VEC>(a, st);
  }
  a.W = pow2_ceil((G + 7) / 8);
  return go<XT, DT, 8, true, VEC>(a, st);
}

template <typename XT, typename DT>
cudaError_t types(const int32_t* err, int rows, int dim, const MatIn& x, const MatIn& delta, int mapped, const int32_t* row_map,
                  const float* w, float eps, const MatOut& x_out, const Fp8Out& out, float* rstd, cudaStream_t st) {
  NormArgs<XT, DT> a{err, rows, dim, 1, static_cast<const XT*>(x.p), x.ld, static_cast<const DT*>(delta.p), delta.ld,
                     mapped, row_map, w, eps, static_cast<XT*>(x_out.p), x_out.ld, out, rstd};
  const bool vec = dim % 4 == 0 && rows_vec4(x.p, x.ld, sizeof(XT)) &&
                   (!delta.p || rows_vec4(delta.p, delta.ld, dtype_size(delta.type))) &&
                   (!x_out.p || rows_vec4(x_out.p, x_out.ld, sizeof(XT))) && rows_vec4(w, 4, 4) &&
                   rows_vec4(out.q, out.ld, 1);
  return vec ? shape<XT, DT, true>(a, st) : shape<XT, DT, false>(a, st);
}

template <typename XT, typename... Args>
cudaError_t with_delta(const MatIn& delta, const int32_t* row_map, Args&&... args) {
  if (row_map) {  // the layers' residual stream, which is fp32
    if constexpr (std::is_same<XT, float>::value) return types<XT, Mapped>(args...);
    else return cudaErrorInvalidValue;
  }
  if (!delta.p) return types<XT, None>(args...);
  if (delta.type == MTFM_BF16) return types<XT, __nv_bfloat16>(args...);
  return types<XT, float>(args...);
}

}  // namespace

cudaError_t launch_add_rmsnorm_fp8(const int32_t* err, int rows, int dim, const MatIn& x, const MatIn& delta,
                                   int mapped, const int32_t* row_map, const float* w, float eps, const MatOut& x_out,
                                   const Fp8Out& out, float* rstd, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  if (x.type == MTFM_BF16)
    return with_delta<__nv_bfloat16>(delta, row_map, err, rows, dim, x, delta, mapped, row_map, w, eps, x_out, out, rstd, st);
  return with_delta<float>(delta, row_map, err, rows, dim, x, delta, mapped, row_map, w, eps, x_out, out, rstd, st);
}

}  // namespace mtfm
