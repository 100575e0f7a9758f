// extern "C" entry points of the 8-bit operators that take plain matrices: host-side
// argument checks, then launches.  See include/mtfm.h for the contract.
#include "fp8.cuh"

using namespace mtfm;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline mtfm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MTFM_OK : MTFM_ERR_CUDA; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool known_type(int32_t t) { return t == MTFM_F32 || t == MTFM_BF16; }

// A matrix of `cols` columns: present, of a known type, aligned to its element, rows apart.
bool mat_ok(const void* p, int32_t type, int64_t ld, int64_t rows, int64_t cols) {
  return p && known_type(type) && aligned(p, dtype_size(type)) && (rows <= 1 || ld >= cols);
}
bool scales_ok(const float* p, int64_t ld, int64_t rows, int64_t groups) {
  return p && aligned(p, 4) && (rows <= 1 || ld >= groups);
}
// An output in the place of an input: element for element, or a warp would write what another has
// yet to read.
bool in_place_ok(const void* out, int32_t out_type, int64_t ld_out, const void* in, int32_t in_type, int64_t ld_in,
                 int64_t rows) {
  return out != in || !out || (out_type == in_type && (rows <= 1 || ld_out == ld_in));
}
// The pitch of a single row is never used: one that suits every access.
inline int64_t pitch(int64_t rows, int64_t ld, int64_t cols) { return rows <= 1 ? ceil_div(cols, 16) * 16 : ld; }

}  // namespace

extern "C" {

mtfm_status mtfm_add_rmsnorm_fp8(int32_t rows, int32_t dim, const void* d_x, int32_t x_type, int64_t ldx,
                                 const void* d_delta, int32_t delta_type, int64_t ld_delta, const float* d_w,
                                 float eps, void* d_x_out, int64_t ld_x_out, uint8_t* d_out, int64_t ld_out,
                                 float* d_scale, int64_t ld_scale, float* d_rstd, void* stream) {
  if (rows < 0 || dim <= 0) return MTFM_ERR_INVALID_ARG;
  if (dim > kMaxNormDim) return MTFM_ERR_UNSUPPORTED;
  if (rows == 0) return MTFM_OK;
  if (!mat_ok(d_x, x_type, ldx, rows, dim) || !d_w || !aligned(d_w, 4)) return MTFM_ERR_INVALID_ARG;
  if (d_delta ? !mat_ok(d_delta, delta_type, ld_delta, rows, dim) : d_x_out != nullptr) return MTFM_ERR_INVALID_ARG;
  if (d_x_out && !mat_ok(d_x_out, x_type, ld_x_out, rows, dim)) return MTFM_ERR_INVALID_ARG;
  if (!d_out || (rows > 1 && ld_out < dim)) return MTFM_ERR_INVALID_ARG;
  if (!scales_ok(d_scale, ld_scale, rows, ceil_div(dim, kGroup)) || !aligned(d_rstd, 4)) return MTFM_ERR_INVALID_ARG;
  if (!in_place_ok(d_x_out, x_type, ld_x_out, d_x, x_type, ldx, rows) ||
      !in_place_ok(d_x_out, x_type, ld_x_out, d_delta, delta_type, ld_delta, rows))
    return MTFM_ERR_INVALID_ARG;
  return cuda_status(launch_add_rmsnorm_fp8(
      nullptr, rows, dim, MatIn{d_x, pitch(rows, ldx, dim), x_type}, MatIn{d_delta, pitch(rows, ld_delta, dim), delta_type},
      rows, nullptr, d_w, eps > 0.f ? eps : kRmsEps, MatOut{d_x_out, pitch(rows, ld_x_out, dim), x_type},
      Fp8Out{d_out, pitch(rows, ld_out, dim), d_scale, ld_scale}, d_rstd, static_cast<cudaStream_t>(stream)));
}

size_t mtfm_rmsnorm_bwd_workspace_bytes(int32_t rows, int32_t dim) {
  if (rows < 0 || dim <= 0 || dim > kMaxNormDim) return 0;
  return align256(sizeof(float) * (size_t)kNormBwdBlocks * dim);
}

mtfm_status mtfm_rmsnorm_bwd(int32_t rows, int32_t dim, const void* d_x, int32_t x_type, int64_t ldx,
                             const float* d_w, const float* d_rstd, const void* d_dy, int32_t dy_type,
                             int64_t ld_dy, const void* d_dres, int32_t dres_type, int64_t ld_dres, void* d_dx,
                             int64_t ld_dx, float* d_dw, void* d_ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || dim <= 0) return MTFM_ERR_INVALID_ARG;
  if (dim > kMaxNormDim) return MTFM_ERR_UNSUPPORTED;
  if (!d_dw || !aligned(d_dw, 4)) return MTFM_ERR_INVALID_ARG;
  if (rows > 0) {
    if (!mat_ok(d_x, x_type, ldx, rows, dim) || !d_w || !aligned(d_w, 4) || !d_rstd || !aligned(d_rstd, 4))
      return MTFM_ERR_INVALID_ARG;
    if (!mat_ok(d_dy, dy_type, ld_dy, rows, dim) || !mat_ok(d_dx, x_type, ld_dx, rows, dim)) return MTFM_ERR_INVALID_ARG;
    if (d_dres && !mat_ok(d_dres, dres_type, ld_dres, rows, dim)) return MTFM_ERR_INVALID_ARG;
    if (!d_ws || !aligned(d_ws, 16)) return MTFM_ERR_INVALID_ARG;
    if (ws_bytes < mtfm_rmsnorm_bwd_workspace_bytes(rows, dim)) return MTFM_ERR_WORKSPACE_TOO_SMALL;
    if (!in_place_ok(d_dx, x_type, ld_dx, d_x, x_type, ldx, rows) ||
        !in_place_ok(d_dx, x_type, ld_dx, d_dy, dy_type, ld_dy, rows) ||
        !in_place_ok(d_dx, x_type, ld_dx, d_dres, dres_type, ld_dres, rows))
      return MTFM_ERR_INVALID_ARG;
  }
  return cuda_status(launch_rmsnorm_bwd(
      rows, dim, MatIn{d_x, pitch(rows, ldx, dim), x_type}, d_w, d_rstd, MatIn{d_dy, pitch(rows, ld_dy, dim), dy_type},
      MatIn{d_dres, pitch(rows, ld_dres, dim), dres_type}, MatOut{d_dx, pitch(rows, ld_dx, dim), x_type}, d_dw,
      static_cast<float*>(d_ws), static_cast<cudaStream_t>(stream)));
}

mtfm_status mtfm_fp8_quant(int32_t rows, int32_t cols, const void* d_x, int32_t x_type, int64_t ldx,
                           int32_t block_rows, uint8_t* d_out, int64_t ld_out, float* d_scale, int64_t ld_scale,
                           void* stream) {
  if (rows < 0 || cols < 0 || (block_rows != 1 && block_rows != kGroup)) return MTFM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return MTFM_OK;
  if (!mat_ok(d_x, x_type, ldx, rows, cols) || !d_out || (rows > 1 && ld_out < cols)) return MTFM_ERR_INVALID_ARG;
  if (!scales_ok(d_scale, ld_scale, ceil_div(rows, block_rows), ceil_div(cols, kGroup))) return MTFM_ERR_INVALID_ARG;
  return cuda_status(launch_fp8_quant(rows, cols, MatIn{d_x, pitch(rows, ldx, cols), x_type}, block_rows,
                                      Fp8Out{d_out, pitch(rows, ld_out, cols), d_scale, ld_scale},
                                      static_cast<cudaStream_t>(stream)));
}

mtfm_status mtfm_fp8_gemm(int32_t m, int32_t n, int32_t k, const uint8_t* d_a, int64_t lda, const float* d_a_scale,
                          int64_t ld_a_scale, const uint8_t* d_b, int64_t ldb, const float* d_b_scale,
                          int64_t ld_b_scale, int32_t act, const void* d_res, int64_t ld_res, void* d_out,
                          int32_t out_type, int64_t ld_out, int32_t* d_status, void* stream) {
  if (m < 0 || n < 0 || k <= 0) return MTFM_ERR_INVALID_ARG;
  if (act != MTFM_ACT_NONE && act != MTFM_ACT_SILU) return MTFM_ERR_INVALID_ARG;
  constexpr int32_t kMost = 2147483647 - 8192;  // tile coordinates stay int32
  if (m > kMost || n > kMost || k > kMost) return MTFM_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return MTFM_OK;
  if (!d_a || !d_b || !aligned(d_a, 16) || !aligned(d_b, 16)) return MTFM_ERR_INVALID_ARG;
  lda = pitch(m, lda, k);
  ldb = pitch(n, ldb, k);
  if (lda < k || ldb < k || lda % 16 != 0 || ldb % 16 != 0) return MTFM_ERR_INVALID_ARG;
  if (!scales_ok(d_a_scale, ld_a_scale, m, ceil_div(k, kGroup)) ||
      !scales_ok(d_b_scale, ld_b_scale, ceil_div(n, kGroup), ceil_div(k, kGroup)))
    return MTFM_ERR_INVALID_ARG;
  if (!mat_ok(d_out, out_type, ld_out, m, n) || (d_res && !mat_ok(d_res, out_type, ld_res, m, n)))
    return MTFM_ERR_INVALID_ARG;
  if (!in_place_ok(d_out, out_type, ld_out, d_res, out_type, ld_res, m)) return MTFM_ERR_INVALID_ARG;
  if (!d_status || !aligned(d_status, 4)) return MTFM_ERR_INVALID_ARG;
  const Fp8Epi epi{act, out_type, 1, {0, n, n, n, n}, {d_out, nullptr, nullptr, nullptr},
                   {pitch(m, ld_out, n), 0, 0, 0}, d_res, pitch(m, ld_res, n), nullptr};
  return cuda_status(launch_gemm_fp8(d_status, m, n, k, Fp8In{d_a, lda, d_a_scale, ld_a_scale},
                                     Fp8In{d_b, ldb, d_b_scale, ld_b_scale}, epi, static_cast<cudaStream_t>(stream)));
}

mtfm_status mtfm_fp8_check(const int32_t* d_status, void* stream) {
  if (!d_status) return MTFM_ERR_INVALID_ARG;
  int32_t word = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&word, d_status, sizeof(word), cudaMemcpyDeviceToHost, st) != cudaSuccess) return MTFM_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MTFM_ERR_CUDA;
  if (word & kErrBounds) return MTFM_ERR_BOUNDS;
  return word != 0 ? MTFM_ERR_TIMEOUT : MTFM_OK;
}

}  // extern "C"
