// Block-scaled product of two e4m3 matrices (fp8.cuh):
//   C[i, j] = sum_b sa[i, b] sb[j / 128, b] sum_{k in block b} qa[i, k] qb[j, k],   b = k / 128
//   out = act(C) + res
// TMA brings 128-byte K blocks of A and B (128-byte swizzle, both K-major) into a ring;
// tcgen05 MMAs (kind::f8f6f4) form the partial product of one 128-deep block in TMEM, and
// the epilogue warps add it, times its scale, to fp32 sums in registers.  A block's scale is
// one factor per row of the tile (the tile's columns of one weight block share sb), so the
// whole scaling costs one FMA an element and block.  TMEM holds 2 to 4 partial products: the
// MMAs of the next block run while the last one is read.
//
// Persistent CTAs (one per SM) stride over 128 x BN tiles.  Warp 0 issues TMA, warp 1 the
// MMAs; warps 4..11 are two warpgroups, each on half of the tile's columns, one TMEM lane
// (row) a thread.  The sums take BN / 2 registers a thread; for BN = 256 the registers of
// the first four warps are handed over (setmaxnreg).  Every wait is bounded; a wait that
// gives up raises the CTA's abort flag, the roles drain what they issued, and the error
// word gets the timeout bit.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "fp8.cuh"
#include "mma_util.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace mtfm {
namespace {

using namespace sm100;

constexpr int kBM = 128;
constexpr uint32_t kABytes = kBM * kGroup;
constexpr int kEpiWarps = 8;
constexpr int kThreadsG = 128 + 32 * kEpiWarps;

struct Args {
  int32_t* err;
  int M, N, K;
  const float* sa;
  int64_t ld_sa;
  const float* sb;
  int64_t ld_sb;
  Fp8Epi epi;
  bool vec;  // every output (and res) row starts on a 16-byte boundary
};

template <int BN>
constexpr uint32_t stage_bytes_g() { return kABytes + (uint32_t)BN * kGroup; }
template <int BN>
constexpr int stages_g() { return BN == 256 ? 4 : BN == 128 ? 6 : 8; }
template <int BN>
constexpr int acc_bufs() { return BN == 256 ? 2 : 4; }
template <int BN>
constexpr size_t smem_g() { return (size_t)stages_g<BN>() * stage_bytes_g<BN>() + 1024; }

// kind::f8f6f4, e4m3 x e4m3 -> fp32 (formats 0), both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 da, db; mov.b64 da, {%1, %3}; mov.b64 db, {%2, %3};"
      " setp.ne.b32 p, %5, 0;"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %4, p; }" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// SiLU in fp32 accuracy: the product's callers compare it with the definition, and its
// rounding to bf16 is the only one.
__device__ __forceinline__ float silu_full(float x) { return __fdividef(x, 1.f + __expf(-x)); }

// 32 consecutive columns of one output row.
template <typename OT>
__device__ __forceinline__ void store_row32(const Args& p, int row, int col, float (&v)[32]) {
  const Fp8Epi& e = p.epi;
  if (e.act == MTFM_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = silu_full(v[j]);
  }
  const int64_t orow = e.row_map ? e.row_map[row] : row;
  const int n = p.N - col;
  if (e.res) {
    const OT* r = static_cast<const OT*>(e.res) + orow * e.ld_res + col;
    if (p.vec && n >= 32) {
      if constexpr (sizeof(OT) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 t = reinterpret_cast<const float4*>(r)[j];
          v[4 * j] += t.x; v[4 * j + 1] += t.y; v[4 * j + 2] += t.z; v[4 * j + 3] += t.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 t = reinterpret_cast<const uint4*>(r)[j];
          const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[8 * j + 2 * k] += __uint_as_float(w[k] << 16);
            v[8 * j + 2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) v[j] += (float)r[j];
    }
  }
  void* base = e.seg_ptr[0];
  int64_t ld = e.seg_ld[0];
  int c0 = 0;
#pragma unroll
  for (int s = 1; s < 4; ++s)
    if (s < e.n_seg && col >= e.seg_begin[s]) {
      base = e.seg_ptr[s];
      ld = e.seg_ld[s];
      c0 = e.seg_begin[s];
    }
  OT* o = static_cast<OT*>(base) + orow * ld + (col - c0);
  if (p.vec && n >= 32) {
    if constexpr (sizeof(OT) == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        reinterpret_cast<float4*>(o)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<uint4*>(o)[j] =
            make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                       pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) o[j] = (OT)v[j];
  }
}

template <int BN, typename OT>
__global__ void __launch_bounds__(kThreadsG, 1)
gemm_fp8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, Args p) {
  constexpr int kStages = stages_g<BN>(), kAcc = acc_bufs<BN>();
  constexpr uint32_t kStage = stage_bytes_g<BN>();
  constexpr uint32_t kTmemCols = kAcc * BN;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages];
  __shared__ __align__(8) uint64_t bar_acc_full[kAcc], bar_acc_empty[kAcc], bar_drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nN = (p.N + BN - 1) / BN, nK = (p.K + kGroup - 1) / kGroup;
  const int64_t n_tiles = (int64_t)((p.M + kBM - 1) / kBM) * nN;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  auto b_full = [&](int s) { return smem_addr(&bar_full[s]); };
  auto b_empty = [&](int s) { return smem_addr(&bar_empty[s]); };
  auto b_accf = [&](int a) { return smem_addr(&bar_acc_full[a]); };
  auto b_acce = [&](int a) { return smem_addr(&bar_acc_empty[a]); };
  const uint32_t b_drain = smem_addr(&bar_drain);
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), 1);
    }
    for (int a = 0; a < kAcc; ++a) {
      mbar_init(b_accf(a), 1);
      mbar_init(b_acce(a), kEpiWarps);
    }
    mbar_init(b_drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  pdl_wait();
  // an earlier kernel on this error word failed: nothing is loaded or stored (TMEM is freed below)
  const bool skip = *p.err != 0;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  const int64_t first = skip ? n_tiles : (int64_t)blockIdx.x;

  if (warp < 4) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ----------------------------------------------------------- TMA producer
      int64_t G = 0;  // K blocks issued by this CTA (ring position and phase)
      bool ok = true;
      for (int64_t t = first; ok && t < n_tiles; t += gridDim.x) {
        const int m0 = (int)(t / nN) * kBM, n0 = (int)(t % nN) * BN;
        for (int kb = 0; kb < nK; ++kb, ++G) {
          const int s = (int)(G % kStages);
          if (G >= kStages && !mbar_wait(b_empty(s), (uint32_t)((G / kStages) - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          // boxes that reach past the matrix are filled with zeros and count in full
          mbar_expect_tx(b_full(s), kStage);
          tma_load_2d(sbase + s * kStage, &tm_a, b_full(s), kb * kGroup, m0);
          tma_load_2d(sbase + s * kStage + kABytes, &tm_b, b_full(s), kb * kGroup, n0);
        }
      }
      // no copy may land after the CTA leaves: wait (bounded) for the last one of each stage
      const long long t0 = clock64();
      for (int64_t g = G > kStages ? G - kStages : 0; g < G; ++g)
        while (!mbar_try(b_full((int)(g % kStages)), (uint32_t)(g / kStages) & 1) && clock64() - t0 < kWaitCycles) {
        }
    } else if (warp == 1) {
      // ----------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc = idesc_e4m3_f32(kBM, BN);
      const uint32_t dhi = sw128_desc_hi(1024);
      const uint32_t a_lo = sw128_desc_lo(sbase, 16), b_lo = sw128_desc_lo(sbase + kABytes, 16);
      bool ok = true;
      int64_t G = 0;
      for (int64_t t = first; ok && t < n_tiles; t += gridDim.x) {
        for (int kb = 0; kb < nK; ++kb, ++G) {
          const int s = (int)(G % kStages), a = (int)(G % kAcc);
          ok = (G < kAcc || mbar_wait(b_acce(a), (uint32_t)((G / kAcc) - 1) & 1, abort_flag)) &&
               mbar_wait(b_full(s), (uint32_t)(G / kStages) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t ao = a_lo + s * (kStage >> 4), bo = b_lo + s * (kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < kGroup / 32; ++kk)
              mma_f8(tmem + (uint32_t)(a * BN), ao + kk * 2, bo + kk * 2, dhi, idesc, kk > 0 ? 1u : 0u);
            mma_commit(b_empty(s));
            mma_commit(b_accf(a));
          }
          __syncwarp();
        }
      }
      if (!ok) {
        // drain every MMA issued so far before TMEM is released
        if (elect_one()) mma_commit(b_drain);
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try(b_drain, 0) && clock64() - t0 < kWaitCycles) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------- scaling and epilogue
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    constexpr int kHalf = BN / 2, kChunks = kHalf / 32;
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tlane = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * kHalf);
    bool ok = true;
    int64_t G = 0;
    for (int64_t t = first; ok && t < n_tiles; t += gridDim.x) {
      const int row = (int)(t / nN) * kBM + quad * 32 + lane;
      const int col0 = (int)(t % nN) * BN + half * kHalf;
      const float* sa = p.sa + (int64_t)(row < p.M ? row : 0) * p.ld_sa;
      // the warpgroup's columns lie in one 128-row block of B; columns past N read no scale of their own
      const float* sb = p.sb + (int64_t)((col0 < p.N ? col0 : p.N - 1) / kGroup) * p.ld_sb;
      float acc[kHalf];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) acc[j] = 0.f;
      float sa_next = sa[0], sb_next = sb[0];
      for (int kb = 0; kb < nK; ++kb, ++G) {
        const int a = (int)(G % kAcc);
        const float sc = sa_next * sb_next;
        if (kb + 1 < nK) {
          sa_next = sa[kb + 1];
          sb_next = sb[kb + 1];
        }
        if (!__all_sync(0xffffffffu, mbar_wait(b_accf(a), (uint32_t)(G / kAcc) & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t raw[32];
          tmem_ld32(tlane + (uint32_t)(a * BN + c * 32), raw);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c * 32 + j] = fmaf(__uint_as_float(raw[j]), sc, acc[c * 32 + j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_acce(a));
      }
      if (ok && row < p.M) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = acc[c * 32 + j];
          if (col0 + c * 32 < p.N) store_row32<OT>(p, row, col0 + c * 32, v);
        }
      }
    }
  }
  pdl_trigger();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && s_abort) atomicOr(p.err, kErrTimeout);
}

// Row-major e4m3 matrix [rows, cols], row pitch ld bytes; boxes of box_rows x 128 columns.
bool make_map_e4m3(CUtensorMap* map, const uint8_t* base, int rows, int cols, int64_t ld, uint32_t box_rows) {
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

template <int BN, typename OT>
cudaError_t go(const Fp8In& a, const Fp8In& b, const Args& args, cudaStream_t st) {
  CUtensorMap ma, mb;
  if (!make_map_e4m3(&ma, a.q, args.M, args.K, a.ld, kBM) || !make_map_e4m3(&mb, b.q, args.N, args.K, b.ld, BN))
    return cudaErrorInvalidValue;
  const size_t smem = smem_g<BN>();
  cudaError_t e = cudaFuncSetAttribute(gemm_fp8_kernel<BN, OT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)args.M + kBM - 1) / kBM * (((int64_t)args.N + BN - 1) / BN);
  return launch_pdl(gemm_fp8_kernel<BN, OT>, dim3((unsigned)std::min<int64_t>(tiles, sm_count())), dim3(kThreadsG), smem, st,
                    ma, mb, args);
}

}  // namespace

cudaError_t launch_gemm_fp8(int32_t* err, int M, int N, int K, const Fp8In& a, const Fp8In& b, const Fp8Epi& epi,
                            cudaStream_t st) {
  if (M <= 0 || N <= 0) return cudaSuccess;
  const int size = dtype_size(epi.out_type);
  auto rows16 = [&](const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0;
  };
  bool vec = !epi.res || rows16(epi.res, epi.ld_res);
  for (int s = 0; s < epi.n_seg; ++s) vec = vec && rows16(epi.seg_ptr[s], epi.seg_ld[s]);
  const Args args{err, M, N, K, a.scale, a.ld_scale, b.scale, b.ld_scale, epi, vec};
  return epi.out_type == MTFM_BF16 ? go<128, __nv_bfloat16>(a, b, args, st) : go<128, float>(a, b, args, st);
}

}  // namespace mtfm
