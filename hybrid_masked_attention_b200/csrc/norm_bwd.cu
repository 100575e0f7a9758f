// Backward of the RMSNorm.  With g = dy w and x the stream that was normalised:
//   dx = r (g - x r^2 mean_j(g_j x_j)) + dres,      dw_j = sum_rows dy_j x_j r
//
// One pass over x, dy and dres (bound by memory).  Blocks stride over the rows; a lane keeps
// the same columns for all of its rows, so dw is summed in registers, in an order that depends
// on the sizes alone, and leaves a block as one partial row; a second kernel adds those up.
// 25959 x 512 fp32: 40 us, 5.3 TB/s; 8191 x 4096 bf16: 49 us, 5.5 TB/s.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"

namespace mtfm {
namespace {

struct None {};  // no dres

template <typename XT, typename YT, typename RT>
struct BwdArgs {
  int rows, dim, W;
  const XT* x;
  int64_t ldx;
  const float* w;
  const float* rstd;
  const YT* dy;
  int64_t ld_dy;
  const RT* dres;
  int64_t ld_dres;
  XT* dx;
  int64_t ld_dx;
  float* partials;
};

template <typename R>
__device__ __forceinline__ void unpack2(const R& r, float2 (&v)[2]) {
  float t[4];
  unpack(r, t);
  v[0] = make_float2(t[0], t[1]);
  v[1] = make_float2(t[2], t[3]);
}

template <bool VEC>
__device__ __forceinline__ void load_shared(const float* p, int lane, int n, float (&v)[4]) {
  if (VEC) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (4 * lane < n) t = *reinterpret_cast<const float4*>(p + 4 * lane);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = lane + 32 * j < n ? p[lane + 32 * j] : 0.f;
  }
}

// C groups a warp: 4 with the next row's loads in flight (blocks of 8 warps, rows of up to
// 4096 columns), 8 without (16 warps, 16384 columns; 128 registers hold neither a second row nor dw,
// which is kept in shared memory: 2000 x 16384 bf16, 86 us).
template <int C>
constexpr int kThreadsB = C == 8 ? 512 : 256;

template <typename XT, typename YT, typename RT, int C, bool VEC>
__global__ void __launch_bounds__(kThreadsB<C>, C == 8 ? 1 : 2)
rmsnorm_bwd_kernel(const __grid_constant__ BwdArgs<XT, YT, RT> p) {
  constexpr bool kRes = !std::is_same<RT, None>::value;
  constexpr bool kAhead = C < 8;
  constexpr bool kResEarly = kAhead || VEC;  // dres is fetched with x and dy, not where it is added
  constexpr bool kDwShared = C == 8;  // dw of a thread's 32 columns in shared memory instead of registers
  constexpr int kWarps = kThreadsB<C> / 32;
  using RRaw = typename std::conditional<kRes, RT, XT>::type;
  // [rows of a block - 1][dim], to join dw at the end; kDwShared: [rows of a block][dim], the sums
  extern __shared__ __align__(16) float s_dw[];
  __shared__ __align__(16) float s_part[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.W, sub = warp % W, slot = warp / W, R = kWarps / W;
  // the warp's C groups are neighbours: their addresses differ by constants
  const int col0 = sub * C * kGroup, n0 = p.dim - col0;  // first column, and columns from there on
  pdl_wait();
  pdl_trigger();
  const float inv_dim = 1.f / (float)p.dim;
  float2 dw[kDwShared ? 1 : C][2];
  if constexpr (kDwShared) {  // (every element belongs to one thread)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      put4<VEC>(s_dw + slot * p.dim + col0 + i * kGroup, lane, n0 - i * kGroup, zero);
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) dw[i][0] = dw[i][1] = make_float2(0.f, 0.f);
  }
  Raw<XT, VEC> xr[C];
  Raw<YT, VEC> yr[C];
  Raw<RRaw, VEC> rr[C];
  float r_next = 0.f;
  auto load_row = [&](int64_t row) {
    if (row >= p.rows) return;
    r_next = p.rstd[row];
    const XT* px = p.x + row * p.ldx + col0;
    const YT* py = p.dy + row * p.ld_dy + col0;
#pragma unroll
    for (int i = 0; i < C; ++i) {  // (a group past the row loads nothing, and holds zeros: norm_fp8.cu)
      xr[i] = load_raw<VEC>(px + i * kGroup, lane, n0 - i * kGroup);
      yr[i] = load_raw<VEC>(py + i * kGroup, lane, n0 - i * kGroup);
    }
    if constexpr (kRes && kResEarly) {
      const RT* pr = p.dres + row * p.ld_dres + col0;
#pragma unroll
      for (int i = 0; i < C; ++i) rr[i] = load_raw<VEC>(pr + i * kGroup, lane, n0 - i * kGroup);
    }
  };
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t row = (int64_t)blockIdx.x * R + slot;
  if (kAhead) load_row(row);
  int flip = 0;
  // every warp of the block makes the same number of rounds (the barrier below)
  for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < p.rows; row0 += step, row += step, flip ^= 1) {
    const bool live = row < p.rows;
    if (!kAhead) load_row(row);
    const float r = r_next;
    float2 xv[C][2], gv[C][2];
    const float2 r2 = make_float2(r, r);
    float2 s2 = make_float2(0.f, 0.f);
    Raw<RRaw, VEC> res[C];
    float s = 0.f;
    if (live) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int n = n0 - i * kGroup;
        unpack2(xr[i], xv[i]);
        unpack2(yr[i], gv[i]);
        res[i] = rr[i];
        float2 ww[2], part[2];
        float* sd = s_dw + slot * p.dim + col0 + i * kGroup;
        if constexpr (kDwShared) {
          float t[4];
          load_shared<VEC>(sd, lane, n, t);
          part[0] = make_float2(t[0], t[1]);
          part[1] = make_float2(t[2], t[3]);
        }
        unpack2(load_const<VEC>(p.w + col0 + i * kGroup, lane, n), ww);
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // two columns an instruction
          if constexpr (!kDwShared) dw[i][j] = __ffma2_rn(gv[i][j], __fmul2_rn(xv[i][j], r2), dw[i][j]);
          else part[j] = __ffma2_rn(gv[i][j], __fmul2_rn(xv[i][j], r2), part[j]);
          gv[i][j] = __fmul2_rn(gv[i][j], ww[j]);
          s2 = __ffma2_rn(gv[i][j], xv[i][j], s2);
        }
        if constexpr (kDwShared) {
          const float t[4] = {part[0].x, part[0].y, part[1].x, part[1].y};
          put4<VEC>(sd, lane, n, t);
        }
      }
    }
    if (kAhead) load_row(row + step);
    s = warp_sum32(s2.x + s2.y);
    if (W > 1) {
      if (lane == 0) s_part[flip][warp] = s;
      __syncthreads();
      s = row_sum(s_part[flip] + warp - sub, W);
    }
    if (live) {
      const float c = s * inv_dim * r * r;
      const float2 c2 = make_float2(-c, -c);
      XT* pdx = p.dx + row * p.ld_dx + col0;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int n = n0 - i * kGroup;
        if (n > 0) {
          float2 o[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) o[j] = __fmul2_rn(r2, __ffma2_rn(xv[i][j], c2, gv[i][j]));
          if constexpr (kRes) {
            float2 t[2];
            if constexpr (kResEarly) unpack2(res[i], t);
            else unpack2(load_raw<VEC>(p.dres + row * p.ld_dres + col0 + i * kGroup, lane, n), t);
#pragma unroll
            for (int j = 0; j < 2; ++j) o[j] = __fadd2_rn(o[j], t[j]);
          }
          const float ov[4] = {o[0].x, o[0].y, o[1].x, o[1].y};
          put4<VEC>(pdx + i * kGroup, lane, n, ov);
        }
      }
    }
  }
  // the block's partial row: slots 1.. hand theirs over through shared memory
  if constexpr (kDwShared) {
    if (R > 1) __syncthreads();
  } else if (R > 1) {
    if (slot > 0)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = col0 + i * kGroup + lane_col<VEC>(lane, j);
          if (c < p.dim) s_dw[(size_t)(slot - 1) * p.dim + c] = j & 1 ? dw[i][j >> 1].y : dw[i][j >> 1].x;
        }
    __syncthreads();
  }
  if (slot == 0)
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = col0 + i * kGroup + lane_col<VEC>(lane, j);
        if (c < p.dim) {
          float t;
          if constexpr (kDwShared) t = s_dw[c];
          else t = j & 1 ? dw[i][j >> 1].y : dw[i][j >> 1].x;
          for (int k = kDwShared; k < R - !kDwShared; ++k) t += s_dw[(size_t)k * p.dim + c];
          p.partials[(size_t)blockIdx.x * p.dim + c] = t;
        }
      }
}

// dw = sum of the partial rows: 8 columns (one 32-byte sector) a block, 32 threads down each,
// fixed order.
__global__ void __launch_bounds__(256)
dw_reduce_kernel(const float* __restrict__ partials, int n_part, int dim, float* __restrict__ dw) {
  __shared__ float s[8][33];
  pdl_wait();
  pdl_trigger();
  const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
  const int c = blockIdx.x * 8 + cx;
  float t = 0.f;
  if (c < dim) {
#pragma unroll 8
    for (int b = ry; b < n_part; b += 32) t += partials[(size_t)b * dim + c];
  }
  s[cx][ry] = t;
  __syncthreads();
  t = warp_sum32(s[threadIdx.x >> 5][threadIdx.x & 31]);
  const int co = blockIdx.x * 8 + (threadIdx.x >> 5);
  if ((threadIdx.x & 31) == 0 && co < dim) dw[co] = t;
}

inline int pow2_ceil(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

template <typename XT, typename YT, typename RT, int C, bool VEC>
cudaError_t go(BwdArgs<XT, YT, RT>& a, float* dw, cudaStream_t st) {
  constexpr int warps = kThreadsB<C> / 32;
  const int G = (a.dim + kGroup - 1) / kGroup;
  a.W = pow2_ceil((G + C - 1) / C);
  const int R = warps / a.W;
  // C = 4: R W 512 columns, 4096 at most, less a row; C = 8: R W 1024, 16384 at most
  const size_t smem = sizeof(float) * (size_t)(C == 8 ? R : R - 1) * a.dim;
  cudaError_t e = cudaSuccess;
  // C = 8 always: what a block may have without the attribute, 48 KB, counts s_part too (with the
  // test on `smem` alone, dims 6129..6144 and 12257..12288 were refused at their launch)
  if constexpr (C == 8) {
    e = cudaFuncSetAttribute(rmsnorm_bwd_kernel<XT, YT, RT, C, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  const int per_sm = C == 8 ? 1 : 2;  // the kernel's launch bound
  const int blocks = (int)std::min<int64_t>(std::min(kNormBwdBlocks, per_sm * sm_count()), ((int64_t)a.rows + R - 1) / R);
  e = launch_pdl(rmsnorm_bwd_kernel<XT, YT, RT, C, VEC>, dim3(blocks), dim3(32 * warps), smem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(dw_reduce_kernel, dim3((a.dim + 7) / 8), dim3(256), 0, st, (const float*)a.partials, blocks, a.dim, dw);
}

template <typename XT, typename YT, typename RT>
cudaError_t types(int rows, int dim, const MatIn& x, const float* w, const float* rstd, const MatIn& dy, const MatIn& dres,
                  const MatOut& dx, float* dw, float* partials, cudaStream_t st) {
  BwdArgs<XT, YT, RT> a{rows, dim, 1, static_cast<const XT*>(x.p), x.ld, w, rstd, static_cast<const YT*>(dy.p), dy.ld,
                        static_cast<const RT*>(dres.p), dres.ld, static_cast<XT*>(dx.p), dx.ld, partials};
  const bool vec = dim % 4 == 0 && rows_vec4(x.p, x.ld, sizeof(XT)) && rows_vec4(dy.p, dy.ld, sizeof(YT)) &&
                   rows_vec4(w, 4, 4) && (!dres.p || rows_vec4(dres.p, dres.ld, dtype_size(dres.type))) &&
                   rows_vec4(dx.p, dx.ld, sizeof(XT));
  if (dim <= 32 * kGroup)
    return vec ? go<XT, YT, RT, 4, true>(a, dw, st) : go<XT, YT, RT, 4, false>(a, dw, st);
  return vec ? go<XT, YT, RT, 8, true>(a, dw, st) : go<XT, YT, RT, 8, false>(a, dw, st);
}

template <typename XT, typename YT, typename... Args>
cudaError_t with_res(const MatIn& dres, Args&&... args) {
  if (!dres.p) return types<XT, YT, None>(args...);
  if (dres.type == MTFM_BF16) return types<XT, YT, __nv_bfloat16>(args...);
  return types<XT, YT, float>(args...);
}
template <typename XT, typename... Args>
cudaError_t with_dy(const MatIn& dy, const MatIn& dres, Args&&... args) {
  if (dy.type == MTFM_BF16) return with_res<XT, __nv_bfloat16>(dres, args...);
  return with_res<XT, float>(dres, args...);
}

}  // namespace

cudaError_t launch_rmsnorm_bwd(int rows, int dim, const MatIn& x, const float* w, const float* rstd, const MatIn& dy,
                               const MatIn& dres, const MatOut& dx, float* dw, float* partials, cudaStream_t st) {
  if (rows <= 0) return cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)dim, st);
  if (x.type == MTFM_BF16) return with_dy<__nv_bfloat16>(dy, dres, rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
  return with_dy<float>(dy, dres, rows, dim, x, w, rstd, dy, dres, dx, dw, partials, st);
}

}  // namespace mtfm
