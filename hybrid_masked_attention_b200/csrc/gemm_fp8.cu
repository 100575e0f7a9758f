// Block-scaled product of two e4m3 matrices (fp8.cuh):
//   C[i, j] = sum_b sa[i, b] sb[j / 128, b] sum_{k in block b} qa[i, k] qb[j, k],   b = k / 128
//   out = act(C) + res
//
// Pairs of CTAs (a cluster of 2, one SM each) compute 256 x BN tiles with tcgen05.mma
// cta_group::2 (kind::f8f6f4): each CTA brings its 128 rows of A and half of the tile's rows
// of B by TMA (128-byte K blocks, 128-byte swizzle), the MMA reads both CTAs' B, and each CTA's
// TMEM receives its 128 rows.  Halving the B traffic of a CTA is what the pair is for: at
// 8192^3 the L2 would have to deliver 8.6 GB to single CTAs with 128 x 128 tiles, and delivers
// 4.3 GB to pairs with 256 x 256.
//
// The MMAs sum one 128-deep block of 128 columns at a time; the epilogue warps add it, times
// its scale, to fp32 sums in registers: one packed FMA for two elements and block, since a
// thread has one row (sa) and its columns lie in one weight block (sb).  Four warpgroups of 64
// columns each: 16 warps hide more of the epilogue's latency than 8 of 128 columns did (53133 x
// 1280 x 512 with SiLU 82 against 97 us, 8192^3 alike).
//
// BN = 256: the tile is two halves, each with its own MMA-issuing warp, two TMEM buffers and
// two warpgroups, so that one half's block is read while the tensor pipe works on the other's.
// BN = 128: four TMEM buffers; two warpgroups take the even tiles and two the odd ones.
//
// Warp 0 issues TMA; warps 1 and 3 of the leading CTA issue the MMAs of the pair (one warp for
// both halves kept the tensor pipe waiting: 412 against 311 us at 8192^3 with nothing else in
// the way); warp 2 brings the scales, 128 rows of A a block, to shared memory (read from global
// memory by the epilogue warps themselves, 32 rows a warp and each row in 4 warpgroups, they
// cost 100 us of 560); warps 4..19 are the warpgroups, one TMEM lane (row) a thread.  Their 64
// sums a thread take registers that the first four warps hand over (setmaxnreg).
// What bounds it: at 8192^3 (523 us alone, 595 in a loop under the power
// cap) the hand-over of TMEM buffers, 950 cycles a block as the epilogue's warps count them where the
// tensor pipe needs 512 (it is active for 0.60 of the time, the issue slots for 0.74); at 53133 x 1280
// x 512 with SiLU (75 to 78 us) instruction issue (0.72): a tile's four blocks take 3700 cycles, SiLU
// and the store 3600, which only two blocks of the next tile overlap.
//
// Every wait is bounded; a wait that gives up raises its CTA's abort flag, the other CTA's own
// waits then run out too, both meet at the cluster barrier, and the error word gets the
// timeout bit.  The epilogue's barriers within a warpgroup have no limit: its warps leave their
// tiles together (gemm_fp8_flow.cuh).
#include <cuda.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "gemm_fp8.cuh"
#include "gemm_fp8_flow.cuh"

namespace mtfm {
namespace {

using namespace sm100;

constexpr int kBM = 128;  // rows of a CTA; a pair's tile has 256
constexpr uint32_t kABytes = kBM * kGroup;
constexpr int kGroupsWG = 4;  // epilogue warpgroups, 64 columns each
constexpr int kCols = 64;
constexpr int kThreadsG = 128 + 128 * kGroupsWG;
// Registers: 640 threads are launched with 96 (61440); 128 x 32 + 512 x 112 are as many.
constexpr int kRegsFew = 32, kRegsMany = 112;
constexpr uint32_t kBoxBytes = 128 * 128;  // a warpgroup's staged box: 128 rows x 128 bytes

struct Args {
  int32_t* err;
  int M, N, K;
  const float* sa;
  int64_t ld_sa;
  const float* sb;
  int64_t ld_sb;
  Fp8Epi epi;
  int n_group;  // tiles are walked in bands of n_group tile columns (see launch)
  bool vec;     // every output (and res) row starts on a 16-byte boundary
};

template <int BN>
constexpr uint32_t stage_bytes_g() { return kABytes + (uint32_t)(BN / 2) * kGroup; }
// How the output leaves a tile.
//   kOutTma    : boxes of 128 rows x 128 bytes staged in shared memory, TMA stores.
//   kOutTmaRes : the same with a residual, whose boxes TMA brings into the staging while the tile
//                is computed (BN = 128: the second fp32 box of a warpgroup takes two ring stages).
//   kOutStaged : with a row map: staged, then each warp adds the residual to, and stores, whole
//                128-byte pieces of rows (a thread's own row, from its registers, would touch 32
//                rows at a time: 4911 x 1000 x 1000 took 40 us that way and 23 this way).
//   kOutDirect : rows that do not start, or whose end does not fall, on 16-byte boundaries
//                (4911 x 1001 x 1000, fp32 / bf16: 43 / 68 us, 82 / 83 with a residual, where 1000
//                columns take 15 / 14 and 20 / 15).
constexpr int kOutTma = 0, kOutStaged = 1, kOutDirect = 2, kOutTmaRes = 3;
template <int BN, int OUT>
constexpr int stages_g() { return BN == 256 ? 5 : OUT == kOutTmaRes ? 4 : 6; }
template <int OUT>
constexpr int boxes_g() { return OUT == kOutTmaRes ? 2 : 1; }  // staged boxes of a warpgroup
// Parts of a tile with their own MMAs, and TMEM buffers of a part (512 columns in all).
template <int BN>
constexpr int parts_g() { return BN / 128; }
template <int BN>
constexpr int acc_bufs() { return 512 / BN; }
constexpr int kSlots = 5;  // blocks of A scales in shared memory
// Dynamic shared memory (there is no static): the ring, the staged boxes, the scales, barriers.
template <int BN, int OUT>
constexpr uint32_t stage_off() { return stages_g<BN, OUT>() * stage_bytes_g<BN>(); }
template <int BN, int OUT>
constexpr uint32_t scale_off() { return stage_off<BN, OUT>() + kGroupsWG * boxes_g<OUT>() * kBoxBytes; }
template <int BN, int OUT>
constexpr uint32_t bars_off() { return scale_off<BN, OUT>() + kSlots * 128 * 4; }
template <int BN, int OUT>
constexpr size_t smem_g() { return bars_off<BN, OUT>() + 512; }
struct Bars {
  uint64_t full[6], empty[6];           // ring stages
  uint64_t acc_full[8], acc_empty[4];   // TMEM buffers (acc_full: per part, or per set)
  uint64_t sc_full[2 * kSlots], sc_empty[kSlots];  // scales (sc_full: per set)
  uint64_t res_full[kGroupsWG];  // a warpgroup's residual boxes have landed
  uint64_t drain[2];
  float sb[kSlots][2];                  // B scales of a block, one for each 128 columns of the tile
  uint32_t tmem, skip;
  int abort;
};
static_assert(sizeof(Bars) <= 512 && smem_g<256, kOutTma>() <= 232448 && smem_g<128, kOutTmaRes>() <= 232448,
              "shared memory of an SM");

// ---------------------------------------------------------------- CTA pairs
// Relaxed: what it hands over is TMEM that this warp has finished reading (tcgen05.wait::ld and
// the fence before the arrival); no write to memory has to become visible.  (A release at
// cluster scope is a memory fence: 4096^3 took 182 us with it and 105 without.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// TMA load into this CTA's shared memory, completion counted on a barrier of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void act32(const Args& p, float (&v)[32]) {
  if (p.epi.act == MTFM_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float2 x = make_float2(v[j], v[j + 1]), y = make_float2(v[j + 2], v[j + 3]);
      silu4(x, y);
      v[j] = x.x, v[j + 1] = x.y, v[j + 2] = y.x, v[j + 3] = y.y;
    }
  }
}
// The residual of a row whose 32 columns start at col.
template <typename OT>
__device__ __forceinline__ void residual32(const Args& p, int64_t orow, int col, float (&v)[32]) {
  const Fp8Epi& e = p.epi;
  if (!e.res) return;
  const int n = p.N - col;
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

// 32 finished columns of one row, stored directly.
template <typename OT>
__device__ __forceinline__ void store32(const Args& p, int64_t orow, int col, const float (&v)[32]) {
  const Fp8Epi& e = p.epi;
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
  const int n = p.N - col;
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

// A barrier of the warpgroup (waits without a limit: every warp has to come, gemm_fp8_flow.cuh),
// and one that says whether `ok` holds in all of its threads.
__device__ __forceinline__ bool wg_vote(int id, bool ok) {
  uint32_t all;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.and.pred q, %2, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(all) : "r"((uint32_t)ok), "r"(id) : "memory");
  return all != 0;
}
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// 4-byte asynchronous copy global -> shared, zero-filled past `bytes`; and an arrival on an
// mbarrier once this thread's copies so far have landed.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// First row and column of tile t: bands of n_group tile columns, walked row by row, so that
// the pairs at work share a band of B and few rows of A in L2.
struct Tile {
  int m0, n0;
};
template <int BN>
__device__ __forceinline__ Tile tile_at(const Args& p, int t, int nM, int nN) {
  const int band = nM * p.n_group;
  const int b = t / band;
  const int in = t - b * band;
  const int w = min(p.n_group, nN - b * p.n_group);
  const int m = in / w;
  return {m * (2 * kBM), (b * p.n_group + in - m * w) * BN};
}

template <int BN, typename OT, int OUT>
__global__ void __launch_bounds__(kThreadsG, 1)
gemm_fp8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const __grid_constant__ CUtensorMap tm_o0, const __grid_constant__ CUtensorMap tm_o1,
                const __grid_constant__ CUtensorMap tm_o2, const __grid_constant__ CUtensorMap tm_o3,
                const __grid_constant__ Args p) {
  constexpr int kStages = stages_g<BN, OUT>(), kParts = parts_g<BN>(), kAcc = acc_bufs<BN>();
  constexpr uint32_t kStage = stage_bytes_g<BN>();
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + bars_off<BN, OUT>());

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int nM = (p.M + 2 * kBM - 1) / (2 * kBM), nN = (p.N + BN - 1) / BN, nK = (p.K + kGroup - 1) / kGroup;
  const int n_tiles = nM * nN;  // (an output of 2^31 tiles does not fit in memory)
  const int step = (int)(gridDim.x >> 1);
  const uint32_t sbase = smem_addr(smem);
  const uint32_t b_full = smem_addr(bars.full), b_empty = smem_addr(bars.empty);
  const uint32_t b_accf = smem_addr(bars.acc_full), b_acce = smem_addr(bars.acc_empty);
  const uint32_t b_scf = smem_addr(bars.sc_full), b_sce = smem_addr(bars.sc_empty);
  if (threadIdx.x == 0) {
    bars.abort = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b_full + s * 8, 1);
      mbar_init(b_empty + s * 8, kParts);  // one commit of each part's issuer
    }
    // a buffer is announced to the set of warpgroups whose tile it belongs to (a waiting set must
    // not miss a phase of its barrier while the other set's tile goes through the buffers)
    for (int a = 0; a < 2 * kAcc; ++a) mbar_init(b_accf + a * 8, 1);
    for (int a = 0; a < kParts * kAcc; ++a) mbar_init(b_acce + a * 8, 16);  // two warpgroups of both CTAs
    for (int a = 0; a < 2 * kSlots; ++a) mbar_init(b_scf + a * 8, 32);      // the lanes of warp 2
    for (int a = 0; a < kSlots; ++a) mbar_init(b_sce + a * 8, 8 * kParts);  // the warps of the tile's set
    for (int a = 0; a < kGroupsWG; ++a) mbar_init(smem_addr(&bars.res_full[a]), 1);
    mbar_init(smem_addr(&bars.drain[0]), 1);
    mbar_init(smem_addr(&bars.drain[1]), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc2(smem_addr(&bars.tmem), kTmemCols);
    tc_fence_before();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  pdl_wait();
  // an earlier kernel on this error word failed: nothing is loaded or stored (the pair goes by
  // the leader's reading of it)
  if (threadIdx.x == 0) {
    if (sbase & 1023) bars.abort = 1;  // the swizzled tiles need what the declaration asks for
    bars.skip = *p.err != 0 || (sbase & 1023) != 0;
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  volatile int* abort_flag = &bars.abort;
  pdl_trigger();  // where this grid leaves SMs free, the next kernel sets itself up there meanwhile
  const bool skip = ld_cluster(map_rank(smem_addr(&bars.skip), 0)) != 0;
  const int first = skip ? n_tiles : (int)(blockIdx.x >> 1);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0 && lane == 0) {
      // ----------------------------------------------------------- TMA producer (each CTA)
      int s = 0;
      uint32_t phase = 0;  // of the stage's use (waiting for the phase before the first returns at once)
      const uint32_t full0 = map_rank((b_full + 0 * 8), 0);
      bool ok = true;
      int64_t issued = 0;
      for (int t = first; ok && t < n_tiles; t += step) {
        const Tile tl = tile_at<BN>(p, t, nM, nN);
        const int m0 = tl.m0 + (int)rank * kBM, n0 = tl.n0 + (int)rank * 64;
        for (int kb = 0; kb < nK; ++kb) {
          if (!mbar_wait((b_empty + s * 8), phase ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + (uint32_t)s * 8;
          // boxes that reach past a matrix are filled with zeros and count in full
          if (rank == 0) mbar_expect_tx((b_full + s * 8), 2 * kStage);
          if (load_ok(p.err, kb * kGroup, p.K, 1, m0)) tma_load_pair(sbase + s * kStage, &tm_a, full, kb * kGroup, m0);
#pragma unroll
          for (int part = 0; part < kParts; ++part)  // this CTA's 64 of the part's 128 rows of B
            if (load_ok(p.err, kb * kGroup, p.K, 1, n0 + part * 128))
              tma_load_pair(sbase + s * kStage + kABytes + part * (64 * kGroup), &tm_b, full, kb * kGroup, n0 + part * 128);
          ++issued;
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // no copy may land after the pair leaves: the leader, whose barriers count both CTAs'
      // copies, waits (bounded) for the last one of each stage
      if (rank == 0) {
        const long long t0 = clock64();
        for (int64_t g = issued > kStages ? issued - kStages : 0; g < issued; ++g)
          while (!mbar_try(b_full + (uint32_t)(g % kStages) * 8, (uint32_t)(g / kStages) & 1) && clock64() - t0 < kWaitCycles) {
          }
      } else if (!ok) {
        // after a wait that gave up the leader may have stopped counting before this CTA's last
        // copies: half a millisecond for them to land
        const long long t0 = clock64();
        while (clock64() - t0 < (1 << 20)) {
        }
      }
    } else if (rank == 0 && (warp == 1 || (warp == 3 && kParts > 1))) {
      // ----------------------------------------------------------- MMA issuers (leader), one a part
      constexpr uint32_t idesc = idesc_e4m3_f32(2 * kBM, 128);
      const int part = warp >> 1;
      const uint64_t a_desc = sw128_desc(sbase, 16, 1024);
      const uint64_t b_desc = sw128_desc(sbase + kABytes + part * (64 * kGroup), 16, 1024);
      const uint32_t b_drain = smem_addr(&bars.drain[part]);
      bool ok = true;
      int s = 0, set = 0;  // set: whose tile it is (BN = 128)
      uint32_t ph_s = 0, n = 0;  // n: blocks issued: buffer n % kAcc, round n / kAcc
      for (int t = first; ok && t < n_tiles; t += step, set ^= 1) {
        for (int kb = 0; kb < nK; ++kb, ++n) {
          const int a = (int)(n % kAcc);
          ok = mbar_wait((b_full + s * 8), ph_s, abort_flag) && mbar_wait(b_acce + (uint32_t)(part * kAcc + a) * 8, (n / kAcc - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = a_desc + (uint32_t)(s * (kStage >> 4)), bd = b_desc + (uint32_t)(s * (kStage >> 4));
            const uint32_t d = tmem + (uint32_t)((part * kAcc + a) * 128);
            mma_f8_pair<false>(d, ad, bd, idesc);  // 32 columns of K each
            mma_f8_pair<true>(d, ad + 2, bd + 2, idesc);
            mma_f8_pair<true>(d, ad + 4, bd + 4, idesc);
            mma_f8_pair<true>(d, ad + 6, bd + 6, idesc);
            commit_pair(b_accf + (uint32_t)((kParts > 1 ? part : set) * kAcc + a) * 8);
            commit_pair((b_empty + s * 8));
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph_s ^= 1;
          }
        }
      }
      if (!ok) {
        // drain every MMA issued so far before TMEM is released
        if (elect_one()) commit_pair(b_drain);
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try(b_drain, 0) && clock64() - t0 < kWaitCycles) {
        }
      }
    } else if (warp == 2) {
      // ----------------------------------------------------------- scales (each CTA): lane l copies
      // those of rows l, l + 32, l + 64, l + 96 of a block; rows past M become 0
      bool ok = true;
      int slot = 0, set = 0;
      uint32_t ph = 0;
      for (int t = first; ok && t < n_tiles; t += step, set ^= 1) {
        const Tile tl = tile_at<BN>(p, t, nM, nN);
        const int row = tl.m0 + (int)rank * kBM + lane;
        const float* src = p.sa + (int64_t)row * p.ld_sa;
        const int bcol = tl.n0 + lane * 128;  // of lanes 0 .. kParts - 1: columns past N have no scale
        const float* src_b = p.sb + (int64_t)((bcol < p.N ? bcol : p.N - 1) / kGroup) * p.ld_sb;
        for (int kb = 0; kb < nK; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(b_sce + slot * 8, ph ^ 1, abort_flag))) {
            ok = false;
            break;
          }
          const uint32_t dst = sbase + scale_off<BN, OUT>() + (uint32_t)(slot * 128 + lane) * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = row + 32 * i < p.M;
            copy4(dst + i * 128, in ? src + (int64_t)(32 * i) * p.ld_sa + kb : p.sa, in ? 4 : 0);
          }
          if (lane < kParts) copy4(smem_addr(&bars.sb[slot][lane]), src_b + kb, 4);
          copy_arrive(b_scf + (uint32_t)((kParts > 1 ? 0 : set) * kSlots + slot) * 8);
          if (++slot == kSlots) {
            slot = 0;
            ph ^= 1;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ------------------------------------------------------------- scaling and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    constexpr int kSets = 256 / BN;  // sets of warpgroups that take turns on tiles
    const int quad = warp & 3, wg = (warp - 4) >> 2;
    const int r_in = quad * 32 + lane;
    const int set = kSets > 1 ? wg >> 1 : 0;
    const int part = kParts > 1 ? wg >> 1 : 0;
    const int tcol = kSets > 1 ? (wg & 1) * kCols : wg * kCols;  // first column within the tile
    const uint32_t tlane = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(part * (kAcc * 128) + (wg & 1) * kCols);
    uint8_t* stage = smem + stage_off<BN, OUT>() + wg * (boxes_g<OUT>() * kBoxBytes);
    const uint32_t sstage = smem_addr(stage);
    const int bar_id = 2 + wg;
    const uint32_t accf0 = b_accf + (uint32_t)((wg >> 1) * kAcc) * 8;            // BN = 256: by part; 128: by set
    const uint32_t acce0 = map_rank(b_acce + (uint32_t)(part * kAcc) * 8, 0);  // (mapped once: mapa in the loop cost 140 cycles a block)
    const bool issuer = quad == 0 && lane == 0;
    const int tid = threadIdx.x & 127;
    constexpr int kOutCols = 128 / (int)sizeof(OT);       // columns of a box of the output's type
    constexpr int kResBoxes = kCols / kOutCols;
    constexpr uint32_t kResBytes = kResBoxes * kBoxBytes;
    const uint32_t b_res = smem_addr(&bars.res_full[wg]);
    uint32_t res_issued = 0, ph_res = 0;
    auto orow = [&](int m) { return (int64_t)(p.epi.row_map ? p.epi.row_map[m] : m); };
    uint32_t n = (uint32_t)(set * nK);  // blocks before this set's next one: buffer n % kAcc
    uint32_t phases = 0;                // of this set's barriers, one bit a buffer
    const uint32_t scf0 = b_scf + (uint32_t)((kParts > 1 ? 0 : set) * kSlots) * 8;
    const volatile float* s_scale = reinterpret_cast<const volatile float*>(smem + scale_off<BN, OUT>());
    int slot = set * nK % kSlots;
    uint32_t sc_phases = 0;
    float sc = 0.f;  // sa sb of this thread's row and columns for the next block
    auto next_scale = [&]() {
      __all_sync(0xffffffffu, mbar_wait(scf0 + (uint32_t)slot * 8, (sc_phases >> slot) & 1, abort_flag));
      sc = s_scale[slot * 128 + r_in] * *const_cast<const volatile float*>(&bars.sb[slot][part]);
      sc_phases ^= 1u << slot;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_sce + (uint32_t)slot * 8);
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    };
    // A warp's way through the tiles is epilogue_tiles() below.
    // BN = 256: a tile's first scale is fetched in the last block of the one before.  With sets it
    // is fetched when the tile begins: a set that waited for it while it holds a TMEM buffer would
    // wait for the other set's tile, which needs that buffer.
    float2 acc[kCols / 2];
    int m0 = 0, col0 = 0;  // of the tile
    auto begin = [&](int t) {
      const Tile tl = tile_at<BN>(p, t, nM, nN);
      m0 = tl.m0 + (int)rank * kBM;
      col0 = tl.n0 + tcol;
      // (after a wait that gave up the barrier may be half done: not armed again)
      if (OUT == kOutTmaRes && issuer && *abort_flag == 0) {
        bulk_wait_read<0>();  // the last tile's stores have read the staging
        mbar_expect_tx(b_res, kResBytes);
#pragma unroll
        for (int b = 0; b < kResBoxes; ++b)
          if (load_ok(p.err, col0 + b * kOutCols, nN * BN, (int)sizeof(OT), m0))
            tma_load_2d(sstage + b * kBoxBytes, &tm_o1, b_res, col0 + b * kOutCols, m0);
        ++res_issued;
      }
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    };
    auto blocks = [&](int t) {
      for (int kb = 0; kb < nK; ++kb, ++n) {
        const float2 s2 = make_float2(sc, sc);
        const int a = (int)(n % kAcc);
        if (!__all_sync(0xffffffffu, mbar_wait(accf0 + (uint32_t)a * 8, (phases >> a) & 1, abort_flag))) return;
        phases ^= 1u << a;
        tc_fence_after();
        const uint32_t ta = tlane + (uint32_t)(a * 128);
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t raw[32];
          tmem_ld32(ta + (uint32_t)(c * 32), raw);
          if (c == 0) {  // the next block's scale is fetched while this one is on its way from TMEM
            if (kb + 1 < nK || (kSets == 1 && t + step < n_tiles)) next_scale();
          }
          tmem_ld_wait();
          if (c + 1 == kCols / 32) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acce0 + (uint32_t)a * 8);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[c * 16 + j] = __ffma2_rn(make_float2(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1])), s2,
                                         acc[c * 16 + j]);
        }
      }
    };
    auto vote = [&]() {
      if constexpr (OUT == kOutDirect) return (bool)__all_sync(0xffffffffu, *abort_flag == 0);  // no barriers: by warps
      else return wg_vote(bar_id, *abort_flag == 0);
    };
    auto finish = [&](int) {
      if constexpr (OUT == kOutTmaRes) {
        mbar_wait(b_res, ph_res, abort_flag);
        ph_res ^= 1;
#pragma unroll
        for (int b = 0; b < kResBoxes; ++b) {
          uint8_t* rowp = stage + b * kBoxBytes + r_in * 128;
#pragma unroll
          for (int c = 0; c < kOutCols / 32; ++c) {
            const int wc = b * kOutCols + c * 32;  // within the warpgroup's columns
            float v[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[2 * j] = acc[wc / 2 + j].x, v[2 * j + 1] = acc[wc / 2 + j].y;
            act32(p, v);
#pragma unroll
            for (int i = 0; i < 2 * (int)sizeof(OT); ++i) {
              uint4* at = reinterpret_cast<uint4*>(rowp + (((c * 2 * (int)sizeof(OT) + i) ^ (r_in & 7)) << 4));
              uint4 w = *at;
              if constexpr (sizeof(OT) == 4) {
                w.x = __float_as_uint(v[4 * i] + __uint_as_float(w.x));
                w.y = __float_as_uint(v[4 * i + 1] + __uint_as_float(w.y));
                w.z = __float_as_uint(v[4 * i + 2] + __uint_as_float(w.z));
                w.w = __float_as_uint(v[4 * i + 3] + __uint_as_float(w.w));
              } else {
                auto sum = [&](uint32_t r, int j) {
                  return pack_bf16x2(v[8 * i + j] + __uint_as_float(r << 16),
                                     v[8 * i + j + 1] + __uint_as_float(r & 0xffff0000u));
                };
                w = make_uint4(sum(w.x, 0), sum(w.y, 2), sum(w.z, 4), sum(w.w, 6));
              }
              *at = w;
            }
          }
        }
        fence_proxy_async();
        wg_sync(bar_id);
        // (after a wait that gave up the staging may hold no sums; the barrier orders the flag)
        if (issuer && *abort_flag == 0 && m0 < p.M) {
#pragma unroll
          for (int b = 0; b < kResBoxes; ++b)
            if (col0 + b * kOutCols < p.N && store_ok(p.err, col0 + b * kOutCols, p.N, (int)sizeof(OT), m0, p.M))
              tma_store_2d(&tm_o0, sstage + b * kBoxBytes, col0 + b * kOutCols, m0);
          bulk_commit();
        }
      } else if constexpr (OUT != kOutDirect) {
        using BT = typename std::conditional<OUT == kOutTma, OT, float>::type;  // staged before a residual: unrounded
        constexpr int kBoxCols = 128 / (int)sizeof(BT);  // 64 bf16 or 32 fp32
        uint8_t* rowp = stage + r_in * 128;
#pragma unroll
        for (int b = 0; b < kCols / kBoxCols; ++b) {
          const int col = col0 + b * kBoxCols;
          if constexpr (OUT == kOutTma) {
            if (issuer) bulk_wait_read<0>();  // the last store has read the staging
          }
          wg_sync(bar_id);
#pragma unroll
          for (int c = 0; c < kBoxCols / 32; ++c) {
            const int wc = b * kBoxCols + c * 32;  // within the warpgroup's columns
            float v[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[2 * j] = acc[wc / 2 + j].x, v[2 * j + 1] = acc[wc / 2 + j].y;
            act32(p, v);
#pragma unroll
            for (int i = 0; i < 2 * (int)sizeof(BT); ++i) {
              const int chunk = c * 2 * (int)sizeof(BT) + i;
              uint4 w;
              if constexpr (sizeof(BT) == 4)
                w = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                               __float_as_uint(v[4 * i + 3]));
              else
                w = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                               pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
              *reinterpret_cast<uint4*>(rowp + ((chunk ^ (r_in & 7)) << 4)) = w;
            }
          }
          if constexpr (OUT == kOutTma) {
            fence_proxy_async();
            wg_sync(bar_id);
            if (issuer && m0 < p.M && col < p.N) {
              const CUtensorMap* om = &tm_o0;
              int begin = 0;
#pragma unroll
              for (int q = 1; q < 4; ++q)
                if (q < p.epi.n_seg && col >= p.epi.seg_begin[q]) {
                  begin = p.epi.seg_begin[q];
                  om = q == 1 ? &tm_o1 : q == 2 ? &tm_o2 : &tm_o3;
                }
              if (store_ok(p.err, col - begin, p.N, (int)sizeof(OT), m0, p.M)) tma_store_2d(om, sstage, col - begin, m0);
              bulk_commit();
            }
          } else {
            // piece i of this thread: 4 columns of row 16 i + tid / 8; four pieces at a time, loaded once
            // the box's sums have left their registers
            wg_sync(bar_id);
#pragma unroll 1
            for (int i0 = 0; i0 < 8; i0 += 4) {
              const int r0 = 16 * i0 + (tid >> 3), c = col + (tid & 7) * 4;
              Raw<OT, true> res[4];
              if (p.epi.res) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int m = m0 + r0 + 16 * i;
                  if (m < p.M && c < p.N)
                    res[i] = load_raw<true>(static_cast<const OT*>(p.epi.res) + orow(m) * p.epi.ld_res + c, 0, 4);
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = r0 + 16 * i, m = m0 + r;
                const float4 w = *reinterpret_cast<const float4*>(stage + r * 128 + (((tid & 7) ^ (r & 7)) << 4));
                float v[4] = {w.x, w.y, w.z, w.w};
                if (m < p.M && c < p.N) {
                  if (p.epi.res) {
                    float t[4];
                    unpack(res[i], t);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] += t[j];
                  }
                  put4<true>(static_cast<OT*>(p.epi.seg_ptr[0]) + orow(m) * p.epi.seg_ld[0] + c, 0, 4, v);
                }
              }
            }
          }
        }
      } else if (const int row = m0 + r_in; row < p.M) {
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          if (col0 + c * 32 < p.N) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[2 * j] = acc[c * 16 + j].x, v[2 * j + 1] = acc[c * 16 + j].y;
            act32(p, v);
            residual32<OT>(p, orow(row), col0 + c * 32, v);
            store32<OT>(p, orow(row), col0 + c * 32, v);
          }
        }
      }
    };
    auto next = [&]() {  // past the other sets' blocks
      n += (uint32_t)((kSets - 1) * nK);
      slot = (slot + (kSets - 1) * nK) % kSlots;
    };
    epilogue_tiles<kSets == 1>(first + set * step, n_tiles, kSets * step, next_scale, begin, blocks, vote, finish, next);
    if (issuer) {
      if (OUT == kOutTma || OUT == kOutTmaRes) bulk_wait<0>();  // every store has completed before the CTA leaves
      // and no copy may land after it: after a wait that gave up, the residual's boxes may be on their way
      const long long t0 = clock64();
      while (OUT == kOutTmaRes && res_issued > 0 && !mbar_try(b_res, (res_issued - 1) & 1) && clock64() - t0 < kWaitCycles) {
      }
    }
  }
  __syncthreads();
  cluster_sync();  // the other CTA's MMAs, copies and arrivals reach into this one
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && bars.abort) atomicOr(p.err, kErrTimeout);
}

// Output matrix [rows, cols] in boxes of 128 rows x 128 bytes.
bool make_map_out(CUtensorMap* map, void* base, int type, int rows, int cols, int64_t ld) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int size = dtype_size(type);
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * size)};
  cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)kBM};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, type == MTFM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename OT, int OUT>
cudaError_t go(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap (&mo)[4], const Args& args, int64_t tiles,
               cudaStream_t st) {
  auto kern = gemm_fp8_kernel<BN, OT, OUT>;
  const size_t smem = smem_g<BN, OUT>();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(tiles, sm_count() / 2));
  cfg.blockDim = dim3(kThreadsG);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, ma, mb, mo[0], mo[1], mo[2], mo[3], args);
}

template <int BN>
cudaError_t launch(const Fp8In& a, const Fp8In& b, Args& args, cudaStream_t st) {
  CUtensorMap ma, mb, mo[4];
  memset(mo, 0, sizeof(mo));
  if (!make_map_e4m3(&ma, a.q, args.M, args.K, a.ld, kBM) || !make_map_e4m3(&mb, b.q, args.N, args.K, b.ld, 64))
    return cudaErrorInvalidValue;
  const Fp8Epi& e = args.epi;
  const int box_cols = 128 / dtype_size(e.out_type);
  // a TMA store writes whole 16-byte pieces of a row: a row that ends inside one is stored directly
  bool whole = args.vec;
  for (int s = 0; s < e.n_seg; ++s)
    whole = whole && (e.seg_begin[s + 1] - e.seg_begin[s]) * dtype_size(e.out_type) % 16 == 0;
  int out = !whole ? kOutDirect : e.row_map ? kOutStaged : e.res ? kOutTmaRes : kOutTma;
  if (out == kOutStaged && e.n_seg > 1) out = kOutDirect;
  for (int s = 0; s < e.n_seg && (out == kOutTma || out == kOutTmaRes); ++s)
    if (e.seg_begin[s] % box_cols != 0 ||
        !make_map_out(&mo[s], e.seg_ptr[s], e.out_type, args.M, e.seg_begin[s + 1] - e.seg_begin[s], e.seg_ld[s]))
      out = kOutDirect;
  if (out == kOutTmaRes && !make_map_out(&mo[1], const_cast<void*>(e.res), e.out_type, args.M, args.N, e.ld_res)) out = kOutDirect;
  if (out == kOutTmaRes && BN == 256) return launch<128>(a, b, args, st);
  const int64_t nM = ((int64_t)args.M + 2 * kBM - 1) / (2 * kBM), nN = ((int64_t)args.N + BN - 1) / BN;
  args.n_group = (int)std::min<int64_t>(nN, 8);
  auto by_out = [&](auto type) {
    using OT = decltype(type);
    return out == kOutTma      ? go<BN, OT, kOutTma>(ma, mb, mo, args, nM * nN, st)
           : out == kOutTmaRes ? go<128, OT, kOutTmaRes>(ma, mb, mo, args, nM * nN, st)
           : out == kOutStaged ? go<BN, OT, kOutStaged>(ma, mb, mo, args, nM * nN, st)
                               : go<BN, OT, kOutDirect>(ma, mb, mo, args, nM * nN, st);
  };
  return e.out_type == MTFM_BF16 ? by_out(__nv_bfloat16{}) : by_out(float{});
}

}  // namespace

cudaError_t launch_gemm_fp8(int32_t* err, int M, int N, int K, const Fp8In& a, const Fp8In& b, const Fp8Epi& epi,
                            cudaStream_t st) {
  if (M <= 0 || N <= 0) return cudaSuccess;
  if (gemm_fp8_rows_takes(M, N, K)) return launch_gemm_fp8_rows(err, M, N, K, a, b, epi, st);
  const int size = dtype_size(epi.out_type);
  auto rows16 = [&](const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0;
  };
  bool vec = !epi.res || rows16(epi.res, epi.ld_res);
  for (int s = 0; s < epi.n_seg; ++s) vec = vec && rows16(epi.seg_ptr[s], epi.seg_ld[s]);
  Args args{err, M, N, K, a.scale, a.ld_scale, b.scale, b.ld_scale, epi, 1, vec};
  // Tile width by the rounds the pairs make: a round of 256 x 128 tiles takes 0.55 (short K) to
  // 0.62 (long K) of one of 256 x 256 (8192^3 forced to 128 columns: 647 against 520 us; 4911 x
  // 1000 x 1000, 3 rounds against 2: 17 and 19).
  const int64_t pairs = sm_count() / 2, nM = ((int64_t)M + 255) / 256;
  const int64_t r256 = (nM * (((int64_t)N + 255) / 256) + pairs - 1) / pairs;
  const int64_t r128 = (nM * (((int64_t)N + 127) / 128) + pairs - 1) / pairs;
  return 10 * r256 <= 6 * r128 ? launch<256>(a, b, args, st) : launch<128>(a, b, args, st);
}

}  // namespace mtfm
