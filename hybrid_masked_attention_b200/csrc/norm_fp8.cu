// Residual addition, RMSNorm and quantisation in one pass over the row, and the backward
// pass of the norm.
//
//   h = x + delta,  r = 1 / sqrt(mean_j h_j^2 + eps),  v = h r w  ->  (q, scale) of fp8.cuh
//   x_out = h rounded to x's type (the residual stream; v is taken from h before it)
//
// Backward, with g = dy w and x the stream that was normalised:
//   dx = r (g - x r^2 mean_j(g_j x_j)) + dres,      dw_j = sum_rows dy_j x_j r
//
// Both move each element once and do a handful of operations on it, so memory bounds them.
// A 128-column group is one warp's 32 lanes x 4 columns: the group's largest magnitude is
// one redux instruction and a row needs no shared memory for its scales.  W warps share a
// row, each holding up to C groups of it in registers.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"

namespace mtfm {
namespace {

struct None {};  // no delta, no dres

// Groups a warp holds: 4 (rows of up to 8 warps, 4096 columns, in blocks of 8 warps) or 8
// (up to 16 warps, 16384 columns, in blocks of 16: the registers of a row of 8 groups do
// not fit four times into a thread of a larger block).
template <int C>
constexpr int kThreads = C == 4 ? 256 : 512;

template <typename XT, typename DT, int C, bool VEC>
__global__ void __launch_bounds__(kThreads<C>)
add_rmsnorm_fp8_kernel(const int32_t* err, int rows, int dim, int W, const XT* x, int64_t ldx, const DT* delta,
                       int64_t ld_delta, const int32_t* __restrict__ row_map, const float* __restrict__ w, float eps,
                       XT* x_out, int64_t ld_xout, Fp8Out out, float* __restrict__ rstd) {
  constexpr bool kDelta = !std::is_same<DT, None>::value;
  __shared__ float s_part[32];
  pdl_wait();
  pdl_trigger();
  if (err && *err) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % W;
  const int row = blockIdx.x * ((int)(blockDim.x >> 5) / W) + warp / W;
  const int G = (dim + kGroup - 1) / kGroup;
  const bool live = row < rows;
  float h[C][4];
  float s = 0.f;
  if (live) {
    const XT* xr = x + (int64_t)(row_map ? row_map[row] : row) * ldx;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int g = i * W + sub;
      if (g < G) load4<VEC>(xr + g * kGroup, lane, dim - g * kGroup, h[i]);
    }
    if constexpr (kDelta) {
      const DT* dr = delta + (int64_t)row * ld_delta;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int g = i * W + sub;
        if (g < G) {
          float d[4];
          load4<VEC>(dr + g * kGroup, lane, dim - g * kGroup, d);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[i][j] += d[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i * W + sub < G)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(h[i][j], h[i][j], s);
  }
  s = warp_sum32(s);
  if (W > 1) {
    if (lane == 0) s_part[warp] = s;
    __syncthreads();
    s = 0.f;
    for (int k = 0; k < W; ++k) s += s_part[warp - sub + k];
  }
  if (!live) return;
  const float r = 1.f / sqrtf(s / (float)dim + eps);
  if (rstd && sub == 0 && lane == 0) rstd[row] = r;
  uint8_t* qr = out.q + (int64_t)row * out.ld;
  float* sr = out.scale + (int64_t)row * out.ld_scale;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int g = i * W + sub;
    if (g < G) {
      const int n = dim - g * kGroup;
      if (kDelta && x_out) put4<VEC>(x_out + (int64_t)row * ld_xout + g * kGroup, lane, n, h[i]);
      float ww[4], v[4];
      load4<VEC>(w + g * kGroup, lane, n, ww);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = h[i][j] * r * ww[j];
      quant_group<VEC>(v, lane, n, qr + g * kGroup, sr + g);
    }
  }
}

// Row pass of the backward.  Each block strides over the rows; a lane keeps the same columns
// for all of them, so dw is summed in registers, in a fixed order, and leaves the block as
// one partial row.
template <typename XT, typename YT, typename RT, int C, bool VEC>
__global__ void __launch_bounds__(kThreads<C>)
rmsnorm_bwd_kernel(int rows, int dim, int W, const XT* x, int64_t ldx, const float* __restrict__ w,
                   const float* __restrict__ rstd, const YT* dy, int64_t ld_dy, const RT* dres, int64_t ld_dres, XT* dx,
                   int64_t ld_dx, float* __restrict__ partials) {
  constexpr bool kRes = !std::is_same<RT, None>::value;
  extern __shared__ float s_dw[];  // [rows per block - 1][dim]
  __shared__ float s_part[2][32];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % W, slot = warp / W, R = (int)(blockDim.x >> 5) / W;
  const int G = (dim + kGroup - 1) / kGroup;
  float ww[C][4], dw[C][4];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int g = i * W + sub;
#pragma unroll
    for (int j = 0; j < 4; ++j) ww[i][j] = dw[i][j] = 0.f;
    if (g < G) load4<VEC>(w + g * kGroup, lane, dim - g * kGroup, ww[i]);
  }
  int flip = 0;
  // every warp of the block makes the same number of rounds (the barrier below)
  for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < rows; row0 += (int64_t)gridDim.x * R, flip ^= 1) {
    const int64_t row = row0 + slot;
    const bool live = row < rows;
    float xv[C][4], gv[C][4];
    float s = 0.f, r = 0.f;
    if (live) {
      r = rstd[row];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int g = i * W + sub;
        if (g < G) {
          load4<VEC>(x + row * ldx + g * kGroup, lane, dim - g * kGroup, xv[i]);
          load4<VEC>(dy + row * ld_dy + g * kGroup, lane, dim - g * kGroup, gv[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i * W + sub < G)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[i][j] = fmaf(gv[i][j], xv[i][j] * r, dw[i][j]);
            gv[i][j] *= ww[i][j];
            s = fmaf(gv[i][j], xv[i][j], s);
          }
    }
    s = warp_sum32(s);
    if (W > 1) {
      if (lane == 0) s_part[flip][warp] = s;
      __syncthreads();
      s = 0.f;
      for (int k = 0; k < W; ++k) s += s_part[flip][warp - sub + k];
    }
    if (live) {
      const float c = s / (float)dim * r * r;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int g = i * W + sub;
        if (g < G) {
          const int n = dim - g * kGroup;
          float o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = r * fmaf(-xv[i][j], c, gv[i][j]);
          if constexpr (kRes) {
            float t[4];
            load4<VEC>(dres + row * ld_dres + g * kGroup, lane, n, t);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += t[j];
          }
          put4<VEC>(dx + row * ld_dx + g * kGroup, lane, n, o);
        }
      }
    }
  }
  // the block's partial row: slots 1.. hand theirs over through shared memory
  if (R > 1) {
    if (slot > 0)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int g = i * W + sub;
        if (g < G)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = g * kGroup + lane_col<VEC>(lane, j);
            if (c < dim) s_dw[(size_t)(slot - 1) * dim + c] = dw[i][j];
          }
      }
    __syncthreads();
  }
  if (slot == 0)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int g = i * W + sub;
      if (g < G)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = g * kGroup + lane_col<VEC>(lane, j);
          if (c < dim) {
            float t = dw[i][j];
            for (int k = 0; k < R - 1; ++k) t += s_dw[(size_t)k * dim + c];
            partials[(size_t)blockIdx.x * dim + c] = t;
          }
        }
    }
}

// dw = sum of the partial rows: 32 columns a block, 32 rows of threads, fixed order.
__global__ void __launch_bounds__(1024)
dw_reduce_kernel(const float* __restrict__ partials, int n_part, int dim, float* __restrict__ dw) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float t = 0.f;
  if (c < dim)
    for (int b = threadIdx.y; b < n_part; b += 32) t += partials[(size_t)b * dim + c];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  t = warp_sum32(s[threadIdx.x][threadIdx.y]);
  const int co = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && co < dim) dw[co] = t;
}

inline int pow2_ceil(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

template <typename XT, typename DT, int C, bool VEC>
cudaError_t norm_go(const int32_t* err, int rows, int dim, int W, const MatIn& x, const MatIn& delta,
                    const int32_t* row_map, const float* w, float eps, const MatOut& x_out, const Fp8Out& out, float* rstd,
                    cudaStream_t st) {
  constexpr int warps = kThreads<C> / 32;
  const int R = warps / W;
  return launch_pdl(add_rmsnorm_fp8_kernel<XT, DT, C, VEC>, dim3((unsigned)(((int64_t)rows + R - 1) / R)), dim3(32 * warps),
                    0, st, err, rows, dim, W, static_cast<const XT*>(x.p), x.ld, static_cast<const DT*>(delta.p), delta.ld,
                    row_map, w, eps, static_cast<XT*>(x_out.p), x_out.ld, out, rstd);
}

template <typename XT, typename DT>
cudaError_t norm_shape(const int32_t* err, int rows, int dim, const MatIn& x, const MatIn& delta, const int32_t* row_map,
                       const float* w, float eps, const MatOut& x_out, const Fp8Out& out, float* rstd, cudaStream_t st) {
  const int G = (dim + kGroup - 1) / kGroup;
  const bool vec = rows_vec4(x.p, x.ld, sizeof(XT)) && (!delta.p || rows_vec4(delta.p, delta.ld, dtype_size(delta.type))) &&
                   (!x_out.p || rows_vec4(x_out.p, x_out.ld, sizeof(XT))) && rows_vec4(w, 4, 4) &&
                   rows_vec4(out.q, out.ld, 1);
  if (G <= 32) {
    const int W = pow2_ceil((G + 3) / 4);
    return vec ? norm_go<XT, DT, 4, true>(err, rows, dim, W, x, delta, row_map, w, eps, x_out, out, rstd, st)
               : norm_go<XT, DT, 4, false>(err, rows, dim, W, x, delta, row_map, w, eps, x_out, out, rstd, st);
  }
  const int W = pow2_ceil((G + 7) / 8);
  return vec ? norm_go<XT, DT, 8, true>(err, rows, dim, W, x, delta, row_map, w, eps, x_out, out, rstd, st)
             : norm_go<XT, DT, 8, false>(err, rows, dim, W, x, delta, row_map, w, eps, x_out, out, rstd, st);
}

template <typename XT>
cudaError_t norm_delta(const int32_t* err, int rows, int dim, const MatIn& x, const MatIn& delta, const int32_t* row_map,
                       const float* w, float eps, const MatOut& x_out, const Fp8Out& out, float* rstd, cudaStream_t st) {
  if (!delta.p) return norm_shape<XT, None>(err, rows, dim, x, delta, row_map, w, eps, x_out, out, rstd, st);
  if (delta.type == MTFM_BF16)
    return norm_shape<XT, __nv_bfloat16>(err, rows, dim, x, delta, row_map, w, eps, x_out, out, rstd, st);
  return norm_shape<XT, float>(err, rows, dim, x, delta, row_map, w, eps, x_out, out, rstd, st);
}

template <typename XT, typename YT, typename RT, int C, bool VEC>
cudaError_t bwd_go(int rows, int dim, const MatIn& x, const float* w, const float* rstd, const MatIn& dy, const MatIn& dres,
                   const MatOut& dx, float* dw, float* partials, cudaStream_t st) {
  const int G = (dim + kGroup - 1) / kGroup;
  constexpr int warps = kThreads<C> / 32;
  const int W = pow2_ceil((G + C - 1) / C), R = warps / W;
  const size_t smem = sizeof(float) * (size_t)(R - 1) * dim;  // R W C 128 columns at most: under 33 KB
  const int blocks = (int)std::min<int64_t>(kNormBwdBlocks, ((int64_t)rows + R - 1) / R);
  cudaError_t e = launch_pdl(rmsnorm_bwd_kernel<XT, YT, RT, C, VEC>, dim3(blocks), dim3(32 * warps), smem, st, rows, dim, W,
                             static_cast<const XT*>(x.p), x.ld, w, rstd, static_cast<const YT*>(dy.p), dy.ld,
                             static_cast<const RT*>(dres.p), dres.ld, static_cast<XT*>(dx.p), dx.ld, partials);
  if (e != cudaSuccess) return e;
  return launch_pdl(dw_reduce_kernel, dim3((dim + 31) / 32), dim3(32, 32), 0, st, (const float*)partials, blocks, dim, dw);
}

template <typename XT, typename YT, typename RT>
cudaError_t bwd_vec(int rows, int dim, const MatIn& x, const float* w, const float* rstd, const MatIn& dy, const MatIn& dres,
                    const MatOut& dx, float* dw, float* partials, cudaStream_t st) {
  const bool vec = rows_vec4(x.p, x.ld, sizeof(XT)) && rows_vec4(dy.p, dy.ld, sizeof(YT)) && rows_vec4(w, 4, 4) &&
                   (!dres.p || rows_vec4(dres.p, dres.ld, dtype_size(dres.type))) && rows_vec4(dx.p, dx.ld, sizeof(XT));
  if (dim <= 32 * kGroup)
    return vec ? bwd_go<XT, YT, RT, 4, true>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st)
               : bwd_go<XT, YT, RT, 4, false>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
  return vec ? bwd_go<XT, YT, RT, 8, true>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st)
             : bwd_go<XT, YT, RT, 8, false>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
}

template <typename XT, typename YT>
cudaError_t bwd_res(int rows, int dim, const MatIn& x, const float* w, const float* rstd, const MatIn& dy, const MatIn& dres,
                    const MatOut& dx, float* dw, float* partials, cudaStream_t st) {
  if (!dres.p) return bwd_vec<XT, YT, None>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
  if (dres.type == MTFM_BF16) return bwd_vec<XT, YT, __nv_bfloat16>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
  return bwd_vec<XT, YT, float>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm_fp8(const int32_t* err, int rows, int dim, const MatIn& x, const MatIn& delta,
                                   const int32_t* row_map, const float* w, float eps, const MatOut& x_out,
                                   const Fp8Out& out, float* rstd, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  if (x.type == MTFM_BF16)
    return norm_delta<__nv_bfloat16>(err, rows, dim, x, delta, row_map, w, eps, x_out, out, rstd, st);
  return norm_delta<float>(err, rows, dim, x, delta, row_map, w, eps, x_out, out, rstd, st);
}

cudaError_t launch_rmsnorm_bwd(int rows, int dim, const MatIn& x, const float* w, const float* rstd, const MatIn& dy,
                               const MatIn& dres, const MatOut& dx, float* dw, float* partials, cudaStream_t st) {
  if (rows <= 0) return cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)dim, st);
  if (x.type == MTFM_BF16)
    return dy.type == MTFM_BF16
               ? bwd_res<__nv_bfloat16, __nv_bfloat16>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st)
               : bwd_res<__nv_bfloat16, float>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
  return dy.type == MTFM_BF16 ? bwd_res<float, __nv_bfloat16>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st)
                              : bwd_res<float, float>(rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
}

}  // namespace mtfm
