// Quantisation of a matrix to e4m3 with one scale for each 128-column group of a row
// (activations, gradients) or for each 128 x 128 block (weights); the form is in fp8.cuh.
// Every element is read once and held in registers until its group's scale is known.
// 8192 x 8192 fp32 in blocks: 53 us, 6.3 TB/s (memory).  12345 x 1000 bf16 in groups: 9.7 us; its
// 37 MB stay in L2 between calls, and 0.69 of the issue slots are taken.
#include <algorithm>

#include "fp8.cuh"

namespace mtfm {
namespace {

// 1 x 128 groups.  A unit is kPer consecutive groups of one row; warps stride over the units
// and load the next one before they reduce the present one.
constexpr int kPer = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
quant_rows_kernel(int rows, int cols, int parts, int step_rows, int step_parts, const T* __restrict__ x, int64_t ldx,
                  Fp8Out out) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + warp_index();
  int64_t row = unit / parts;
  int part = (int)(unit % parts);
  Raw<T, VEC> next[kPer];
  auto load_unit = [&](int64_t r, int c0) {
    if (r >= rows) return;
    const T* xr = x + r * ldx + c0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) next[i] = load_raw<VEC>(xr + i * kGroup, lane, cols - c0 - i * kGroup);
  };
  load_unit(row, part * kPer * kGroup);
  while (row < rows) {
    const int c0 = part * kPer * kGroup;
    float v[kPer][4];
#pragma unroll
    for (int i = 0; i < kPer; ++i) unpack(next[i], v[i]);
    uint8_t* q = out.q + row * out.ld + c0;
    float* s = out.scale + row * out.ld_scale + c0 / kGroup;
    row += step_rows;
    part += step_parts;
    if (part >= parts) {
      part -= parts;
      ++row;
    }
    load_unit(row, part * kPer * kGroup);
    const float mine = quant_groups<VEC>(v, lane, cols - c0, q);
    if (lane < kPer && c0 + lane * kGroup < cols) s[lane] = mine / kE4m3Max;
  }
}

// 128 x 128 blocks: one block of threads each, a warp on 16 of its rows.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
quant_blocks_kernel(int rows, int cols, int G, const T* __restrict__ x, int64_t ldx, Fp8Out out) {
  __shared__ float s_max[8];
  pdl_wait();
  pdl_trigger();
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rb = blockIdx.x / G, g = blockIdx.x % G;
  const int64_t r0 = (int64_t)rb * kGroup;
  const int c0 = g * kGroup, n = cols - c0;
  float v[16][4];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t row = r0 + warp + 8 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
    if (row < rows) load4<VEC>(x + row * ldx + c0, lane, n, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, absmax4(v[i]));
  m = warp_absmax(m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  m = kAmaxFloor;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, s_max[k]);
  const float f = quant_factor(m);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t row = r0 + warp + 8 * i;
    if (row < rows) put4_e4m3<VEC>(out.q + row * out.ld + c0, lane, n, v[i], f);
  }
  if (threadIdx.x == 0) out.scale[rb * out.ld_scale + g] = m / kE4m3Max;
}

template <typename T, bool VEC>
cudaError_t quant_go(int rows, int cols, const MatIn& x, int block_rows, const Fp8Out& out, cudaStream_t st) {
  const T* p = static_cast<const T*>(x.p);
  const int G = (cols + kGroup - 1) / kGroup;
  if (block_rows == 1) {
    const int parts = (G + kPer - 1) / kPer;
    const int64_t units = (int64_t)rows * parts;
    const int blocks = (int)std::min<int64_t>((units + 7) / 8, 4 * sm_count());
    return launch_pdl(quant_rows_kernel<T, VEC>, dim3(blocks), dim3(256), 0, st, rows, cols, parts, 8 * blocks / parts,
                      8 * blocks % parts, p, x.ld, out);
  }
  return launch_pdl(quant_blocks_kernel<T, VEC>, dim3((unsigned)((rows + (int64_t)kGroup - 1) / kGroup * G)), dim3(256), 0, st,
                    rows, cols, G, p, x.ld, out);
}

}  // namespace

cudaError_t launch_fp8_quant(int rows, int cols, const MatIn& x, int block_rows, const Fp8Out& out, cudaStream_t st) {
  if (rows <= 0 || cols <= 0) return cudaSuccess;
  const bool vec = cols % 4 == 0 && rows_vec4(x.p, x.ld, dtype_size(x.type)) && rows_vec4(out.q, out.ld, 1);
  if (x.type == MTFM_BF16)
    return vec ? quant_go<__nv_bfloat16, true>(rows, cols, x, block_rows, out, st)
               : quant_go<__nv_bfloat16, false>(rows, cols, x, block_rows, out, st);
  return vec ? quant_go<float, true>(rows, cols, x, block_rows, out, st)
             : quant_go<float, false>(rows, cols, x, block_rows, out, st);
}

}  // namespace mtfm
