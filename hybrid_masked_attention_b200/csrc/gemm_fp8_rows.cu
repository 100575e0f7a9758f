// Block-scaled e4m3 product for few rows of A (a candidate or a handful at serving):
// out = act(A B^T) + res as gemm_fp8.cu, with M up to 32.
//
// Nothing but reading B counts: every byte of it is used for M rows only.  So the roles are
// swapped: 128 rows of B are the MMA's M side, the rows of A its N side (BT = 16 or 32, zero-
// filled past M), and the depth is split over the CTAs of a cluster until all SMs have
// loads in flight.  A CTA streams its K blocks through a TMA ring; an MMA sums one 128-deep
// block into a TMEM buffer of its own; four warps (a row of B a thread) add it, times the
// block's scales, to fp32 registers.  The cluster's partial sums meet in shared memory: CTA q
// receives every CTA's sums of BT / S rows of A, adds them in the order of the depth, so that
// the result does not depend on timing, and finishes those rows.
// 1 x 8192 x 4096 on the device: 6.8 us with B in L2, 9.0 us from HBM (3.7 TB/s; 256 CTAs of 8
// blocks).
#include <algorithm>

#include "gemm_fp8.cuh"

namespace mtfm {
namespace {

using namespace sm100;

constexpr int kRows = 128;  // rows of B a CTA
constexpr uint32_t kWBytes = kRows * kGroup;
constexpr int kThreadsR = 192;  // warp 0 TMA, warp 1 MMA, warps 2..5 scaling and epilogue
constexpr int kMaxBlocks = 64;  // K blocks of a CTA (their scales are held in shared memory)
constexpr int kMaxSplit = 8;

struct RowArgs {
  int32_t* err;
  int M, N, K;
  const float* sa;
  int64_t ld_sa;
  const float* sb;
  int64_t ld_sb;
  Fp8Epi epi;
};

template <int BT>
constexpr uint32_t stage_bytes_r() { return kWBytes + (uint32_t)BT * kGroup; }
// 80 to 90 KB of loads in flight for each of two CTAs an SM.
template <int BT>
constexpr int stages_r() { return BT == 16 ? 5 : 4; }
// TMEM of the CTAs that fit on an SM together has to fit too, whatever their BT: a CTA that
// waited for columns while its cluster's peer holds another's would wait for good.  128 or 256
// columns for each of two; three do not fit into shared memory.
constexpr int kAcc = 8;
// Dynamic shared memory: the ring, the cluster's partial sums [S][BT / S][128], the scales
// [blocks][BT].
template <int BT>
constexpr uint32_t part_off() { return stages_r<BT>() * stage_bytes_r<BT>(); }
template <int BT>
constexpr uint32_t scale_off_r() { return part_off<BT>() + BT * kRows * 4; }

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
static_assert(2 * (scale_off_r<32>() + kMaxBlocks * 32 * 4 + 2048) <= 233472 && 3 * scale_off_r<32>() > 233472 &&
                  3 * scale_off_r<16>() > 233472, "two CTAs an SM");

// The two halves of a cluster barrier, for threads that need not be converged.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void st_cluster(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

template <int BT, int S, typename OT>
__global__ void __launch_bounds__(kThreadsR)
gemm_fp8_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ RowArgs p) {
  constexpr int kStages = stages_r<BT>();
  constexpr uint32_t kStage = stage_bytes_r<BT>();
  constexpr uint32_t kTmemCols = kAcc * BT;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages], bar_accf[kAcc], bar_acce[kAcc], bar_drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(ring);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = S > 1 ? (int)cluster_rank() : 0;
  const int n0 = (int)(blockIdx.x / S) * kRows;
  const int nK = (p.K + kGroup - 1) / kGroup;
  const int k_lo = (int)((int64_t)nK * rank / S), k_hi = (int)((int64_t)nK * (rank + 1) / S);
  auto b_full = [&](int s) { return smem_addr(&bar_full[s]); };
  auto b_empty = [&](int s) { return smem_addr(&bar_empty[s]); };
  auto b_accf = [&](int a) { return smem_addr(&bar_accf[a]); };
  auto b_acce = [&](int a) { return smem_addr(&bar_acce[a]); };
  const uint32_t b_drain = smem_addr(&bar_drain);
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), 1);
    }
    for (int a = 0; a < kAcc; ++a) {
      mbar_init(b_accf(a), 1);
      mbar_init(b_acce(a), 4);
    }
    mbar_init(b_drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  pdl_wait();
  const bool skip = *p.err != 0;  // an earlier kernel on this error word failed
  __syncthreads();
  pdl_trigger();  // where this grid leaves SMs free, the next kernel sets itself up there meanwhile
  if (S > 1) cluster_arrive();  // this CTA has started: its peers may store into it once they have waited
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  const int lo = skip ? k_hi : k_lo;
  float acc[BT];

  if (warp == 0) {
    if (lane == 0) {
      // ----------------------------------------------------------- TMA producer
      int s = 0;
      uint32_t ph = 0;
      int issued = 0;
      for (int kb = lo; kb < k_hi; ++kb, ++issued) {
        if (!mbar_wait(b_empty(s), ph ^ 1, abort_flag)) break;
        // boxes that reach past a matrix are filled with zeros and count in full
        mbar_expect_tx(b_full(s), kStage);
        if (load_ok(p.err, kb * kGroup, p.K, 1, n0)) tma_load_2d(sbase + s * kStage, &tm_w, b_full(s), kb * kGroup, n0);
        tma_load_2d(sbase + s * kStage + kWBytes, &tm_x, b_full(s), kb * kGroup, 0);
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      // no copy may land after the CTA leaves: wait (bounded) for the last one of each stage
      const long long t0 = clock64();
      for (int g = issued > kStages ? issued - kStages : 0; g < issued; ++g)
        while (!mbar_try(b_full(g % kStages), (uint32_t)(g / kStages) & 1) && clock64() - t0 < kWaitCycles) {
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = idesc_e4m3_f32(kRows, BT);
    const uint64_t w_desc = sw128_desc(sbase, 16, 1024), x_desc = sw128_desc(sbase + kWBytes, 16, 1024);
    bool ok = true;
    int s = 0, a = 0;
    uint32_t ph_s = 0, ph_a = 0;
    for (int kb = lo; kb < k_hi; ++kb) {
      ok = mbar_wait(b_acce(a), ph_a ^ 1, abort_flag) && mbar_wait(b_full(s), ph_s, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint64_t wd = w_desc + (uint32_t)(s * (kStage >> 4)), xd = x_desc + (uint32_t)(s * (kStage >> 4));
#pragma unroll
        for (int kk = 0; kk < kGroup / 32; ++kk) mma_f8(tmem + (uint32_t)(a * BT), wd + 2 * kk, xd + 2 * kk, idesc, kk > 0);
        mma_commit(b_empty(s));
        mma_commit(b_accf(a));
      }
      __syncwarp();
      if (++s == kStages) {
        s = 0;
        ph_s ^= 1;
      }
      if (++a == kAcc) {
        a = 0;
        ph_a ^= 1;
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
  } else {
    // ------------------------------------------------------------- scaling
    const int quad = warp & 3;  // TMEM lanes [32 quad, 32 quad + 32)
    const int r_in = quad * 32 + lane;
    float* s_scale = reinterpret_cast<float*>(ring + scale_off_r<BT>());
    // sa sb of the CTA's blocks, [block][row of A]
    const int nb = k_hi - lo;
    const float* sb = p.sb + (int64_t)(n0 / kGroup) * p.ld_sb + lo;
    for (int i = threadIdx.x - 64; i < nb * BT; i += 128) {
      const int b = i / BT, m = i % BT;
      s_scale[b * BT + m] = m < p.M ? p.sa[m * p.ld_sa + lo + b] * sb[b] : 0.f;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
    for (int j = 0; j < BT; ++j) acc[j] = 0.f;
    const uint32_t tlane = tmem + ((uint32_t)(quad * 32) << 16);
    int a = 0;
    uint32_t ph_a = 0;
    for (int b = 0; b < nb; ++b) {
      if (!__all_sync(0xffffffffu, mbar_wait(b_accf(a), ph_a, abort_flag))) break;
      tc_fence_after();
      const float4* sc = reinterpret_cast<const float4*>(s_scale + b * BT);
      constexpr int kW = BT < 32 ? BT : 32;
#pragma unroll
      for (int c = 0; c < BT / kW; ++c) {
        uint32_t raw[kW];
        if constexpr (kW == 32) tmem_ld32(tlane + (uint32_t)(a * BT + c * kW), raw);
        else tmem_ld16(tlane + (uint32_t)(a * BT + c * kW), raw);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kW / 4; ++j) {
          const float4 f = sc[c * (kW / 4) + j];
          float* o = acc + c * kW + 4 * j;
          o[0] = fmaf(__uint_as_float(raw[4 * j]), f.x, o[0]);
          o[1] = fmaf(__uint_as_float(raw[4 * j + 1]), f.y, o[1]);
          o[2] = fmaf(__uint_as_float(raw[4 * j + 2]), f.z, o[2]);
          o[3] = fmaf(__uint_as_float(raw[4 * j + 3]), f.w, o[3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_acce(a));
      if (++a == kAcc) {
        a = 0;
        ph_a ^= 1;
      }
    }
    if (S > 1) {
      cluster_wait();
      // rows q BT / S .. of A go to CTA q, at [this rank][row there][row of B]
      constexpr int kShare = BT / S;
#pragma unroll
      for (int q = 0; q < S; ++q) {
        if (q * kShare < p.M) {
          const uint32_t at = map_rank(sbase + part_off<BT>() + (uint32_t)((rank * kShare * kRows + r_in) * 4), (uint32_t)q);
#pragma unroll
          for (int j = 0; j < kShare; ++j) st_cluster(at + (uint32_t)(j * kRows * 4), acc[q * kShare + j]);
        }
      }
    }
  }
  if (S > 1) {
    if (warp < 2) cluster_wait();
    cluster_arrive();
    cluster_wait();  // the partial sums have arrived; no CTA leaves before its peers' stores
  }
  if (warp >= 2 && !skip) {
    // ------------------------------------------------------------- epilogue
    const int r_in = (warp & 3) * 32 + lane;
    const int col = n0 + r_in;  // column of out
    if (col < p.N) {
      const Fp8Epi& e = p.epi;
      OT* base = static_cast<OT*>(e.seg_ptr[0]);
      int64_t ld = e.seg_ld[0];
      int c0 = 0;
#pragma unroll
      for (int q = 1; q < 4; ++q)
        if (q < e.n_seg && col >= e.seg_begin[q]) {
          base = static_cast<OT*>(e.seg_ptr[q]);
          ld = e.seg_ld[q];
          c0 = e.seg_begin[q];
        }
      auto finish = [&](int m, float v) {
        if (e.act == MTFM_ACT_SILU) v = silu1(v);
        const int64_t orow = e.row_map ? e.row_map[m] : m;
        if (e.res) v += (float)static_cast<const OT*>(e.res)[orow * e.ld_res + col];
        base[orow * ld + (col - c0)] = (OT)v;
      };
      if (S == 1) {
#pragma unroll
        for (int j = 0; j < BT; ++j)
          if (j < p.M) finish(j, acc[j]);
      } else {
        constexpr int kShare = BT / S;
        const float* part = reinterpret_cast<const float*>(ring + part_off<BT>()) + r_in;
#pragma unroll
        for (int j = 0; j < kShare; ++j) {
          const int m = rank * kShare + j;
          if (m < p.M) {
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < S; ++q) v += part[(q * kShare + j) * kRows];
            finish(m, v);
          }
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && s_abort) atomicOr(p.err, kErrTimeout);
}

template <int BT, int S, typename OT>
cudaError_t go(const RowArgs& args, const Fp8In& a, const Fp8In& b, cudaStream_t st) {
  CUtensorMap mw, mx;
  if (!make_map_e4m3(&mw, b.q, args.N, args.K, b.ld, kRows) || !make_map_e4m3(&mx, a.q, args.M, args.K, a.ld, BT))
    return cudaErrorInvalidValue;
  const int nN = (args.N + kRows - 1) / kRows, nK = (args.K + kGroup - 1) / kGroup;
  const size_t smem = scale_off_r<BT>() + (size_t)((nK + S - 1) / S) * BT * 4 + 1024;
  auto kern = gemm_fp8_rows_kernel<BT, S, OT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nN * S));
  cfg.blockDim = dim3(kThreadsR);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, args);
}

template <int BT, typename OT>
cudaError_t by_split(const RowArgs& args, const Fp8In& a, const Fp8In& b, cudaStream_t st) {
  // split the depth until there are three CTAs for two SMs, as long as each keeps a block.  Splits
  // of 1 / 2 / 4 (/ 8), us on the device, B from HBM: N 8192, K 4096 (4 taken) 11.4 / 9.3 / 9.0 with
  // one row and 15.7 / 12.3 / 10.9 with 32; N 2048, K 1024 (8 taken) 4.7 / 4.4 / 3.7 / 3.6 and 7.8 /
  // 6.5 / 5.2 / 4.8; N 1024, K 512 (4 taken) 3.3 / 3.6 / 3.3 and 6.4 / 5.4 / 4.6.
  const int64_t nN = ((int64_t)args.N + kRows - 1) / kRows;
  const int nK = (args.K + kGroup - 1) / kGroup;
  int S = 1;
  while (S < kMaxSplit && 2 * S <= nK && (2 * nN * S < 3 * sm_count() || (nK + S - 1) / S > kMaxBlocks)) S *= 2;
  switch (S) {
    case 1: return go<BT, 1, OT>(args, a, b, st);
    case 2: return go<BT, 2, OT>(args, a, b, st);
    case 4: return go<BT, 4, OT>(args, a, b, st);
    default: return go<BT, 8, OT>(args, a, b, st);
  }
}

template <typename OT>
cudaError_t by_rows(const RowArgs& args, const Fp8In& a, const Fp8In& b, cudaStream_t st) {
  return args.M <= 16 ? by_split<16, OT>(args, a, b, st) : by_split<32, OT>(args, a, b, st);
}

}  // namespace

// Up to 32 rows, on the device with B from HBM: at N 8192, K 4096 this kernel takes 9.7 us (16 rows)
// and 10.9 (32) against 17.4 and 15.2 of the pairs' tiles, at N 1024, K 512 3.6 and 4.6 against 5.4.
// From 33 rows on the pairs take over, 15.2 us there for up to 64 rows and 15.7 for 128: a thread here
// would need that many sums.
bool gemm_fp8_rows_takes(int M, int N, int K) {
  const int64_t nN = ((int64_t)N + kRows - 1) / kRows;
  return M <= 32 && K <= kMaxBlocks * kMaxSplit * kGroup && nN * kMaxSplit < (1ll << 31);
}

cudaError_t launch_gemm_fp8_rows(int32_t* err, int M, int N, int K, const Fp8In& a, const Fp8In& b, const Fp8Epi& epi,
                                 cudaStream_t st) {
  const RowArgs args{err, M, N, K, a.scale, a.ld_scale, b.scale, b.ld_scale, epi};
  return epi.out_type == MTFM_BF16 ? by_rows<__nv_bfloat16>(args, a, b, st) : by_rows<float>(args, a, b, st);
}

}  // namespace mtfm
