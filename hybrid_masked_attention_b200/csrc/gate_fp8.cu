// GLN gate with its output in 8 bits: (q, scale) of v = GLN(A) (*) U, the operand of the
// output projection, one scale for each 128-column group of a row (fp8.cuh).
//   z = (a - mean a) / sqrt(var a + eps),  v = (gamma_type z + beta_type) u   (v = a u without gamma)
// GLN and the type's parameter rows are those of gate.cu (Meituan tech blog §6.1).
//
// One warp per row; group i of the row is the warp's i-th 128-column access, so a scale
// costs one redux.  Bound by memory: 7 bytes an element (a 4, u 2, q 1).
#include "fp8.cuh"

namespace mtfm {
namespace {

constexpr int kDbgFile = 8;  // site id of this file's bounds checks

template <int C>
__global__ void __launch_bounds__(256)
gate_fwd_fp8_kernel(const MetaHeader* hdr, const uint8_t* __restrict__ row_type, bool target, int rows, int D, float eps,
                    const float* __restrict__ a, const __nv_bfloat16* __restrict__ u, const float* __restrict__ gamma,
                    const float* __restrict__ beta, Fp8Out out, float* __restrict__ stats) {
  pdl_wait();
  pdl_trigger();
  if (hdr->error) return;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  if (!MTFM_INBOUNDS(hdr, row < (target ? hdr->total_t : hdr->total_tokens))) return;
  const int G = (D + kGroup - 1) / kGroup;
  const float* ar = a + (size_t)row * D;
  const __nv_bfloat16* ur = u + (size_t)row * D;
  float x[C][4], uu[C][4];
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i < G) {
      load4<true>(ar + i * kGroup, lane, D - i * kGroup, x[i]);
      load4<true>(ur + i * kGroup, lane, D - i * kGroup, uu[i]);
    }
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
    const int type = target ? kRowT : (int)row_type[row];
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
    if (lane == 0) *reinterpret_cast<float2*>(stats + 2 * (size_t)row) = make_float2(mean, rstd);
  }
  uint8_t* q = out.q + (int64_t)row * out.ld;
  float* sc = out.scale + (int64_t)row * out.ld_scale;
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i < G) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = x[i][j] * uu[i][j];
      quant_group<true>(v, lane, D - i * kGroup, q + i * kGroup, sc + i);
    }
}

}  // namespace

cudaError_t launch_gate_fwd_fp8(const MetaView& m, bool target, int rows, int D, float eps, const float* a,
                                const __nv_bfloat16* u, const float* gamma, const float* beta, const Fp8Out& out,
                                float* stats, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const dim3 grid((rows + 7) / 8), block(256);
  auto kern = D <= 4 * kGroup ? gate_fwd_fp8_kernel<4> : gate_fwd_fp8_kernel<8>;
  return launch_pdl(kern, grid, block, 0, st, (const MetaHeader*)m.hdr, (const uint8_t*)m.row_type, target, rows, D, eps, a,
                    u, gamma, beta, out, stats);
}

}  // namespace mtfm
