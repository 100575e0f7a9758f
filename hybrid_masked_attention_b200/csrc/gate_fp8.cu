// GLN gate with its output in 8 bits: (q, scale) of v = GLN(A) (*) U, the operand of the
// output projection, one scale for each 128-column group of a row (fp8.cuh).
//   z = (a - mean a) / sqrt(var a + eps),  v = (gamma_type z + beta_type) u   (v = a u without gamma)
// GLN and the type's parameter rows are those of gate.cu (Meituan tech blog §6.1).
//
// Bound by memory: 7 bytes an element (a 4, u 2, q 1).  A warp holds its row (C groups of 128
// columns, 4 a lane, so a group's scale costs one redux), strides over the rows and loads the
// next row before it reduces the present one.  53055 x 768: 55 us, 5.2 TB/s; 0.62 of the issue
// slots are taken, and a warp's own dependent instructions are the largest stall.
#include <algorithm>

#include "fp8.cuh"

namespace mtfm {
namespace {

constexpr int kDbgFile = 8;  // site id of this file's bounds checks

template <int C>
__global__ void __launch_bounds__(128)
gate_fwd_fp8_kernel(const MetaHeader* hdr, const uint8_t* __restrict__ row_type, bool target, int rows, int D, float eps,
                    const float* __restrict__ a, const __nv_bfloat16* __restrict__ u, const float* __restrict__ gamma,
                    const float* __restrict__ beta, Fp8Out out, float* __restrict__ stats) {
  const int lane = threadIdx.x & 31;
  const int G = (D + kGroup - 1) / kGroup;
  pdl_wait();
  pdl_trigger();
  if (hdr->error) return;
  Raw<float, true> ar[C];
  Raw<__nv_bfloat16, true> ur[C];
  int type_next = kRowT;
  auto load_row = [&](int64_t row) {
    if (row >= rows) return;
    if (!target) type_next = row_type[row];
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < G) {
        ar[i] = load_raw<true>(a + row * D + i * kGroup, lane, D - i * kGroup);
        ur[i] = load_raw<true>(u + row * D + i * kGroup, lane, D - i * kGroup);
      }
  };
  const int64_t step = (int64_t)gridDim.x * 4;
  int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (!MTFM_INBOUNDS(hdr, rows <= (target ? hdr->total_t : hdr->total_tokens))) return;
  load_row(row);
  for (; row < rows; row += step) {
    float x[C][4];
    Raw<__nv_bfloat16, true> uu[C];
    const int type = type_next;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < G) {
        unpack(ar[i], x[i]);
        uu[i] = ur[i];
      }
    load_row(row + step);
    if (gamma) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < G) s += (x[i][0] + x[i][1]) + (x[i][2] + x[i][3]);
      const float mean = warp_sum32(s) / (float)D;
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i * kGroup + 4 * lane < D)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[i][j] -= mean;
            s2 = fmaf(x[i][j], x[i][j], s2);
          }
      const float rstd = 1.f / sqrtf(warp_sum32(s2) / (float)D + eps);
      const float* gr = gamma + (size_t)type * D;
      const float* br = beta + (size_t)type * D;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (i < G) {
          float gg[4], bb[4];
          load4<true>(gr + i * kGroup, lane, D - i * kGroup, gg);
          load4<true>(br + i * kGroup, lane, D - i * kGroup, bb);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] = fmaf(x[i][j] * rstd, gg[j], bb[j]);
        }
      if (lane == 0) *reinterpret_cast<float2*>(stats + 2 * row) = make_float2(mean, rstd);
    }
    uint8_t* q = out.q + row * out.ld;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < G) {
        float t[4];
        unpack(uu[i], t);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] *= t[j];
      }
    const float mine = quant_groups<true>(x, lane, D, q);
    if (lane < G) out.scale[row * out.ld_scale + lane] = mine / kE4m3Max;
  }
}

template <int C>
cudaError_t go(const MetaView& m, bool target, int rows, int D, float eps, const float* a, const __nv_bfloat16* u,
               const float* gamma, const float* beta, const Fp8Out& out, float* stats, cudaStream_t st) {
  static int per_sm = 0;  // blocks an SM holds: a property of the kernel
  if (per_sm == 0) {
    int n = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, gate_fwd_fp8_kernel<C>, 128, 0);
    if (e != cudaSuccess) return e;
    per_sm = n > 0 ? n : 1;
  }
  const int blocks = std::min((rows + 3) / 4, per_sm * sm_count());
  return launch_pdl(gate_fwd_fp8_kernel<C>, dim3(blocks), dim3(128), 0, st, (const MetaHeader*)m.hdr,
                    (const uint8_t*)m.row_type, target, rows, D, eps, a, u, gamma, beta, out, stats);
}

}  // namespace

cudaError_t launch_gate_fwd_fp8(const MetaView& m, bool target, int rows, int D, float eps, const float* a,
                                const __nv_bfloat16* u, const float* gamma, const float* beta, const Fp8Out& out,
                                float* stats, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const int G = (D + kGroup - 1) / kGroup;
  if (G <= 2) return go<2>(m, target, rows, D, eps, a, u, gamma, beta, out, stats, st);
  if (G <= 4) return go<4>(m, target, rows, D, eps, a, u, gamma, beta, out, stats, st);
  if (G <= 6) return go<6>(m, target, rows, D, eps, a, u, gamma, beta, out, stats, st);
  return go<8>(m, target, rows, D, eps, a, u, gamma, beta, out, stats, st);
}

}  // namespace mtfm
