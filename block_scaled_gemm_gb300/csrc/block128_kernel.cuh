// block128_kernel.cuh -- the product with one FP32 scale per block of 128 on
// sm_103a:
//
//   C[m,n] (+)= sum over K blocks kb of  sA[m,kb] * sB[n,kb] * P_kb[m,n],
//   P_kb[m,n] = sum over the 128 k of block kb of A[m,k] B[n,k]
//
// The tensor cores form each P_kb unscaled (tcgen05.mma.kind::f8f6f4, 8-bit
// operands, FP32 accumulator in TMEM, cleared for every block), and the
// epilogue warps read it from TMEM and add it, scaled, to FP32 sums that stay
// in registers for the whole of K: FP32 scales cannot enter the MMA, whose
// own block scales are powers of two.  So per K block of a 128 x 256 tile an
// SM has 512 cycles of MMA, and beside them 128 KB to read from TMEM and
// 32768 multiply-adds (256 cycles): two accumulators in TMEM, and the MMA of
// one block runs while the other is being added.
//
// Two kernels:
//   b128_pair_kernel    M > 64: CTA pairs (cta_group::2), 256 x 256 tiles,
//                       each CTA with 128 rows of A and 128 columns of B a
//                       K block: 32 KB of operands per 512 cycles and SM.
//                       Bound by the epilogue beside the MMAs: the MMA
//                       warp shares its issue slots with two epilogue warps, and
//                       a block's MMAs wait until its accumulator is read.
//                       8192 x 28672 x 8192 BF16: 1240 us (3.1 PFLOP/s, 0.81 of
//                       the measured 8-bit rate) in short runs at 2.07 GHz,
//                       1360-1450 us under the power limit (1.7 GHz).  K of the
//                       last tiles is cut for several pairs; the one that is done
//                       last adds their sums, in order, and nobody waits.
//   b128_skinny_kernel  M <= 64: transposed, 128 columns of B on the MMA's
//                       128-row side and the rows of A as its N, K split over
//                       a cluster; bound by reading B once: 16 x 8192 x 8192
//                       15.9 us (4.3 TB/s) with B in L2 and 23 us without, 16 x
//                       16384 x 16384 5.4 TB/s from DRAM.
//
// Waits are bounded as in the other kernels: one that runs out records
// MXGEMM_ERR_TIMEOUT, the roles drain and return, and loads that are on their way
// land first.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "tmem_util.cuh"

namespace mxg {

struct B128Params {
  int M, N, K;
  int kb;          // ceil(K / 128)
  const float *a_scale;  // M x kb
  const float *b_scale;
  int64_t bs_n, bs_k;  // entries of B_scale from one block of columns (of K) to the next
  int64_t bs_cols;     // blocks of columns
  void *C;
  int use_acc;
  uint32_t idesc_fmt;
  int *status;
  unsigned long long timeout_ns;
  int stall_producer;
  // pairs
  int m_tiles, n_tiles;
  // whole tiles [0, dp_tiles), a multiple of the grid's pairs, then the last
  // tail_items / split tiles with their K cut into `split` parts, one pair each
  int dp_tiles, split, tail_items;
  float *partials;     // tail item x CTA of the pair x epilogue warp: 32 x 128 sums
  unsigned *counters;  // tail tile x CTA of the pair x epilogue warp: parts that are there (0 between launches)
  int tma_store;  // C's rows are multiples of 16 bytes and nothing is added
  // skinny
  int nm;      // M rounded up to 16
  int splits;  // CTAs of a cluster that share a column block's K
};

// Instruction descriptor of kind::f8f6f4: FP32 accumulator, M x N; the
// operands' formats are OR-ed in, and the transpose bit of an operand whose
// M (N) dimension is the contiguous one.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 lanes x 32 columns as the fragments of an 8 x 8 grid: of each eight
// columns, thread (g, t) = (lane / 4, lane % 4) gets columns 2t, 2t + 1 of lanes
// g (r[4 i], r[4 i + 1]) and g + 8 (r[4 i + 2], r[4 i + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Four bytes from global to shared memory, and this thread's arrive on a
// barrier once its copies so far have landed.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

constexpr int kB128Bf16 = 1;    // BF16 output (else FP32)
constexpr int kB128KMajor = 2;  // B given N x K (else K x N)
constexpr int kB128Cols = 4;    // a scale of B for each column (else for 128)

template <int V>
struct PairCfg {
  static constexpr bool COLS = (V & kB128Cols) != 0;
  static constexpr int STAGES = 5;
  static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;  // per CTA
  static constexpr uint32_t STAGE_TX = 2 * (A_BYTES + B_BYTES);   // both CTAs
  static constexpr int EPI_WARPS = 8;
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
  static constexpr int OFF_STG = OFF_B + STAGES * B_BYTES;  // 4 KB for each epilogue warp: C on its way out
  // scales of eight K blocks, two slots: [K block][132] of the CTA's 128 rows,
  // and [K block][260] of the tile's 256 columns (or [K block][4] of its two
  // blocks); the odd pitches keep the transposing copies free of bank conflicts
  static constexpr int KB = 8;
  static constexpr int AS_PITCH = 132, BS_PITCH = COLS ? 260 : 4;
  static constexpr int SLOT_BYTES = KB * (AS_PITCH + BS_PITCH) * 4;
  static constexpr int OFF_SC = OFF_STG + EPI_WARPS * 4096;
  static constexpr int OFF_BAR = OFF_SC + 2 * SLOT_BYTES;  // (accumulators' pairs 16-byte aligned)
  // full, empty, acc_full[2], acc_empty[2], sc_full[2], sc_empty[2], final
  static constexpr int NUM_BARS = 2 * STAGES + 8 + 1;
  static_assert((OFF_BAR + 16 * STAGES) % 16 == 0, "barrier pairs");
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 32 * (4 + EPI_WARPS);
  // registers a thread: 168 at launch, then of the first four warps and of the
  // epilogue's eight (3 x 168 = 56 + 2 x 224: the block's own)
  static constexpr int REGS_MAIN = 56, REGS_EPI = 224;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(OFF_SC % 16 == 0 && SLOT_BYTES % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
};

// Work i of pair `unit`: a tile and its K blocks [kb, ke).  The tiles that do not
// fill the last wave (all of them where there are fewer than pairs) are cut
// along K, and the pair whose part is done last adds the parts' sums in order.
// A pair has one part at most: part `unit`.
struct PairWork {
  int tile, kb, ke, part, item;
};
__device__ __forceinline__ bool pair_work(const B128Params &p, int unit, int units, int i, PairWork &w) {
  const int t = unit + i * units;
  w.part = 0;
  w.kb = 0;
  w.ke = p.kb;
  w.tile = t;
  w.item = t - p.dp_tiles;
  if (w.item < 0) return true;
  if (w.item >= p.tail_items) return false;
  w.tile = p.dp_tiles + w.item / p.split;
  w.part = w.item % p.split;
  w.kb = static_cast<int>(static_cast<long long>(w.part) * p.kb / p.split);
  w.ke = static_cast<int>(static_cast<long long>(w.part + 1) * p.kb / p.split);
  return true;
}

// Warp roles (per CTA, 384 threads): warp 0 loads, warp 1 of the pair's first
// CTA issues the MMAs (and allocates TMEM in both), warp 2 brings the scales
// (with a scale for each column, those by warp 3), warps 4-11 are the
// epilogue: warp w has TMEM lanes 32 (w % 4) .. +31, rows of its CTA's half
// tile, and 128 of the tile's 256 columns, one row and 128 sums a thread.  The
// first four warps give registers to the others.
// Scales come through shared memory because a warp's load of its 32 rows'
// scales of one K block touches 32 lines: read by the epilogue warps
// themselves they held up every K block (8192 x 28672 x 8192: 1784 us; with
// one line for all rows, for comparison, 1533 us).
template <int V>
__global__ void __launch_bounds__(PairCfg<V>::THREADS, 1)
    b128_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const B128Params p) {
  using C = PairCfg<V>;
  constexpr bool kBF16 = (V & kB128Bf16) != 0, kKM = (V & kB128KMajor) != 0, kCols = (V & kB128Cols) != 0;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  const uint32_t bar_full = base + C::OFF_BAR;
  const uint32_t bar_empty = bar_full + 8 * C::STAGES;
  const uint32_t bar_acc_full = bar_empty + 8 * C::STAGES;
  const uint32_t bar_acc_empty = bar_acc_full + 16;
  const uint32_t bar_sc_full = bar_acc_empty + 16;
  const uint32_t bar_sc_empty = bar_sc_full + 16;
  const uint32_t bar_final = bar_sc_empty + 16;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::OFF_MISC + 4);
  volatile int *never = reinterpret_cast<volatile int *>(sm + C::OFF_MISC + 8);  // never raised
  volatile int *peer_fills = reinterpret_cast<volatile int *>(sm + C::OFF_MISC + 12);  // first CTA: the second's fills + 1

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc_full + 8 * b, 1);
      mbar_init(bar_acc_empty + 8 * b, 2 * C::EPI_WARPS);
      mbar_init(bar_sc_full + 8 * b, C::COLS ? 64 : 32);  // lanes of the warps that copy
      mbar_init(bar_sc_empty + 8 * b, C::EPI_WARPS);
    }
    mbar_init(bar_final, 1);
    *abort_flag = 0;
    *never = 0;
    *peer_fills = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_u32(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();  // the next kernel's set-up may begin
  griddep_wait();               // no global memory before the kernel before has ended
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};
  const WaitCtl wn{p.status, never, landing_limit(p.timeout_ns)};
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  const int kb = p.kb;

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_MAIN));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one() != 0;
    int st = 0;
    uint32_t ph = 0;
    long long issued = 0;
    bool ok = true;
    // (tests: no loads, or, of one CTA of each pair, two, or none of the first pair)
    const long long stop = p.stall_producer == 1 || (p.stall_producer == 4 && unit == 0) ? 0
                           : p.stall_producer == 2 + static_cast<int>(rank)              ? 2
                                                                                         : -1;
    PairWork w;
    for (int i = 0; ok && pair_work(p, unit, units, i, w); ++i) {
      int mt, nt;
      tile_coords(w.tile, p.m_tiles, p.n_tiles, mt, nt);
      const int row = mt * 256 + 128 * static_cast<int>(rank), col = nt * 256 + 128 * static_cast<int>(rank);
      for (int ks = w.kb; ks < w.ke; ++ks) {
        // (a producer that is stopped waits for a fill that it does not issue)
        if (!__all_sync(0xFFFFFFFFu, wait_phase<false>(issued == stop ? bar_full + 8 * st : bar_empty + 8 * st,
                                                       issued == stop ? ph : ph ^ 1u, wc, 0x01 | (st << 8)))) {
          ok = false;
          break;
        }
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * st, C::STAGE_TX);
          const uint32_t fb = mapa_shared(bar_full + 8 * st, 0);
          tma_load_2d_pair(base + C::OFF_A + st * C::A_BYTES, &tmA, ks * 128, row, fb);
          if constexpr (kKM) tma_load_2d_pair(base + C::OFF_B + st * C::B_BYTES, &tmB, ks * 128, col, fb);
          else tma_load_2d_pair(base + C::OFF_B + st * C::B_BYTES, &tmB, col, ks * 128, fb);
        }
        __syncwarp();
        ++issued;
        if (++st == C::STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    // Before the CTA may finish: every fill's MMA has released its stage.  Where
    // a wait gave up, the fills that are still on their way land: both CTAs'
    // loads count on the first one's full barriers, so it waits for all of them,
    // and the second one says how many it has issued.  A fill that only one of
    // them issued lacks the other's share: the barrier is told so.
    if (rank == 1 && leader)
      asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(base + C::OFF_MISC + 12, 0)),
                   "r"(static_cast<int>(issued < 0x7FFFFFFF ? issued + 1 : 0x7FFFFFFF))
                   : "memory");
    bool clean = ok;
    for (long long i = ring_pending(issued, C::STAGES); clean && i < issued; ++i) {
      const int s = static_cast<int>(i % C::STAGES);
      clean = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_empty + 8 * s, ring_parity(i, C::STAGES), wc, 0x11 | (s << 8)));
    }
    if (!clean && rank == 0 && leader) {
      // (the other producer's waits are bounded: it says so in time)
      const uint64_t t0 = globaltimer_ns();
      while (*peer_fills == 0 && globaltimer_ns() - t0 < 2 * wn.timeout_ns) {
      }
      const long long theirs = *peer_fills ? *peer_fills - 1 : issued, most = issued > theirs ? issued : theirs;
      for (long long i = ring_pending(most, C::STAGES); i < most; ++i) {
        const int s = static_cast<int>(i % C::STAGES);
        const uint32_t fb = bar_full + 8 * s;
        if (i >= issued) mbar_arrive_expect_tx(fb, C::STAGE_TX / 2);
        if (i >= theirs)
          asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(fb), "r"(C::STAGE_TX / 2) : "memory");
        wait_phase<false>(fb, ring_parity(i, C::STAGES), wn, 0x11 | (s << 8));
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // One thread runs the whole loop.  What comes between the epilogue's
    // release of an accumulator and the next MMA into it is on the critical
    // path of two accumulators (release, MMA 560 cycles, read, release), and
    // this warp shares its issue slots with two busy epilogue warps: so the
    // operands' barrier is waited for first, and the descriptors are ready.
    if (rank == 0) {
      if (elect_one()) {
        int st = 0;
        uint32_t ph = 0, it = 0;
        bool ok = true;
        const uint32_t idesc = idesc_f8(256, 256, false, !kKM) | p.idesc_fmt;
        // A (and a K-major B): 128-byte swizzle, 8-row groups 1 KB apart, 32
        // bytes per K = 32; an N-major B: 32 K rows (4 KB) per K = 32
        const uint64_t dA = smem_desc(base + C::OFF_A, 0, 1024, 2);
        const uint64_t dB = smem_desc(base + C::OFF_B, kKM ? 0 : 16384, 1024, 2);
        constexpr uint32_t kBStep = (kKM ? 32 : 4096) >> 4;
        PairWork w;
        for (int i = 0; ok && pair_work(p, unit, units, i, w); ++i) {
          for (int ks = w.kb; ks < w.ke; ++ks, ++it) {
            const uint32_t buf = it & 1u;
            ok = wait_phase<false>(bar_full + 8 * st, ph, wc, 0x03 | (st << 8));
            if (!ok) break;
            const uint64_t a = dA + static_cast<uint32_t>(st * (C::A_BYTES >> 4));
            const uint64_t b = dB + static_cast<uint32_t>(st * (C::B_BYTES >> 4));
            // only tcgen05.ld of the accumulator must come before: cluster-scope
            // acquire is not needed for that
            ok = wait_phase<false>(bar_acc_empty + 8 * buf, ((it >> 1) & 1u) ^ 1u, wc, 0x02);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f8<2>(tmem + 256 * buf, a + 2 * k, b + kBStep * k, idesc, k != 0);
            tc_commit_pair(bar_acc_full + 8 * buf, 0x3);
            tc_commit_pair(bar_empty + 8 * st, 0x3);
            if (++st == C::STAGES) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
        tc_commit_pair(bar_final, 0x3);
      }
      __syncwarp();
      wait_phase<false>(bar_final, 0, wn, 0x04);
    }
  } else if (warp == 2 || kCols) {
    // ------------------------------------------------------------ scales
    const bool cols = warp == 3;  // the columns' scales, else the rows'
    uint32_t n = 0;               // groups of eight K blocks so far
    bool ok = true;
    PairWork w;
    for (int i = 0; ok && pair_work(p, unit, units, i, w); ++i) {
      int mt, nt;
      tile_coords(w.tile, p.m_tiles, p.n_tiles, mt, nt);
      const int row0 = mt * 256 + 128 * static_cast<int>(rank);
      for (int k0 = w.kb; k0 < w.ke; k0 += C::KB, ++n) {
        const uint32_t slot = n & 1u;
        ok = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_sc_empty + 8 * slot, ((n >> 1) & 1u) ^ 1u, wc, 0x09));
        if (!ok) break;
        const uint32_t as = base + C::OFF_SC + slot * C::SLOT_BYTES, bs = as + C::KB * C::AS_PITCH * 4;
        // (rows, columns and K blocks past the edge repeat the last)
        if (!cols) {
          const int j = lane & 7, k = min(k0 + j, kb - 1);
#pragma unroll 8
          for (int i = 0; i < 32; ++i) {
            const int r = 4 * i + (lane >> 3);
            cp_async4(as + (j * C::AS_PITCH + r) * 4, p.a_scale + static_cast<int64_t>(min(row0 + r, p.M - 1)) * kb + k);
          }
          if (!kCols && lane < 16)
            cp_async4(bs + (j * C::BS_PITCH + (lane >> 3)) * 4,
                      p.b_scale + min(static_cast<int64_t>(2 * nt + (lane >> 3)), p.bs_cols - 1) * p.bs_n + k * p.bs_k);
        } else if constexpr (kKM) {
          const int j = lane & 7, k = min(k0 + j, kb - 1);
#pragma unroll 8
          for (int i = 0; i < 64; ++i) {
            const int c = 4 * i + (lane >> 3);
            cp_async4(bs + (j * C::BS_PITCH + c) * 4, p.b_scale + min(static_cast<int64_t>(nt * 256 + c), p.bs_cols - 1) * p.bs_n + k);
          }
        } else {
#pragma unroll 8
          for (int i = 0; i < 64; ++i) {
            const int j = i >> 3, k = min(k0 + j, kb - 1), c = 32 * (i & 7) + lane;
            cp_async4(bs + (j * C::BS_PITCH + c) * 4, p.b_scale + min(static_cast<int64_t>(nt * 256 + c), p.bs_cols - 1) + k * p.bs_k);
          }
        }
        cp_async_arrive(bar_sc_full + 8 * slot);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the last of what the commits signal in the second CTA (not before its own
    // work is nearly done: the wait's limit is not one for a whole call)
    if (rank == 1 && warp == 2) wait_phase<false>(bar_final, 0, wn, 0x04);
  }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_EPI));
    const int w = warp - 4, q = warp & 3, half = w >> 2;
    const uint32_t stg = base + C::OFF_STG + w * 4096;
    // accumulator and barrier of the block to come: the two of each alternate
    uint32_t acc_at = tmem + (static_cast<uint32_t>(32 * q) << 16) + 128 * half;
    uint32_t full_at = bar_acc_full, full_ph = 0;
    uint32_t empty_at = mapa_shared(bar_acc_empty, 0);  // of the pair's first CTA
    uint32_t n = 0;  // groups of eight K blocks so far
    // This warp's part of a tile whose K is cut is there: whether it is the last
    // one.  Nobody waits: the warp that arrives last adds, and leaves the counter
    // at zero for the next launch.
    auto arrive = [&](int item) -> bool {
      __threadfence();
      __syncwarp();
      unsigned before = 0;
      if (lane == 0) {
        unsigned *at = p.counters + (item / p.split * 2 + static_cast<int>(rank)) * C::EPI_WARPS + w;
        before = atomicAdd(at, 1u);
        if (before == static_cast<unsigned>(p.split) - 1u) *at = 0;
      }
      before = __shfl_sync(0xFFFFFFFFu, before, 0);
      __threadfence();
      return before == static_cast<unsigned>(p.split) - 1u;
    };
    bool ok = true, arrived = false;
    PairWork pw;
    for (int i = 0; ok && pair_work(p, unit, units, i, pw); ++i) {
      int mt, nt;
      tile_coords(pw.tile, p.m_tiles, p.n_tiles, mt, nt);
      const int row0 = mt * 256 + 128 * static_cast<int>(rank) + 32 * q;
      const int col0 = nt * 256 + 128 * half;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      // Scales of the block to come, read a block ahead.  With one scale of B
      // for 128 columns a thread has one row, and s its scale times theirs.
      // With a scale for each column a thread has a fragment, four rows (lane / 4
      // + 8 i, scales s) and 32 columns, so that it reads 32 columns' scales for
      // each block and not 128.
      constexpr int kRows = kCols ? 4 : 1;
      float s[kRows];
      const float *sc;
      auto scale_at = [&](int ks) {
        sc = reinterpret_cast<const float *>(sm + C::OFF_SC + (n & 1u) * C::SLOT_BYTES);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          s[i] = sc[(ks & (C::KB - 1)) * C::AS_PITCH + 32 * q + (kCols ? (lane >> 2) + 8 * i : lane)];
        sc += C::KB * C::AS_PITCH + (ks & (C::KB - 1)) * C::BS_PITCH;
        // (The product of the scales has to stay in FP32's normal range, which the
        // interface asks for: a test of it here, for each K block, with a loop in
        // two steps for the others, 110 -> 122 us at 2048 x 9728 x 8192; by the
        // warps that bring the scales, 139 us.)
        if constexpr (!kCols) s[0] *= sc[half];
      };
      ok = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_sc_full + 8 * (n & 1u), (n >> 1) & 1u, wc, 0x0A));
      if (!ok) break;
      scale_at(0);
      const int steps = pw.ke - pw.kb;
#pragma unroll 1
      for (int ks = 0; ks < steps; ++ks) {
        ok = warp_wait(full_at, full_ph, wc, 0x05);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[2][32];
        auto load = [&](int c, uint32_t (&r)[32]) {  // columns 32 c .. +31
          if constexpr (kCols) {
            tmem_ld_16x256b_x4(acc_at + 32 * c, r);
            tmem_ld_16x256b_x4(acc_at + 32 * c + (16u << 16), r + 16);
          } else {
            tmem_ld_32x32b_x32(acc_at + 32 * c, r);
          }
        };
        load(0, v[0]);
        tmem_ld_done(v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < 3) load(c + 1, v[(c + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 f = make_float2(1.f, 1.f);
            if constexpr (kCols) f = *reinterpret_cast<const float2 *>(sc + 128 * half + 32 * c + 8 * (i & 3) + 2 * (lane & 3));
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const float x = __uint_as_float(v[c & 1][4 * i + j]), y = __uint_as_float(v[c & 1][4 * i + j + 1]);
              float &a = acc[32 * c + 4 * i + j], &b = acc[32 * c + 4 * i + j + 1];
              if constexpr (kCols) {
                // two at a time: half the instructions of two FP32 operations a
                // value (137 -> 125 us); slower where there is one (1293 -> 1389 us)
                const float k = s[2 * (i >> 2) + (j >> 1)];
                const float2 r = fma2(mul2(make_float2(x, y), f), make_float2(k, k), make_float2(a, b));
                a = r.x;
                b = r.y;
              } else {
                a = fmaf(x, s[0], a);
                b = fmaf(y, s[0], b);
              }
            }
          }
          if (c < 3) tmem_ld_done(v[(c + 1) & 1]);
          if (c == 2) {  // the accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
              asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(empty_at) : "memory");
          }
        }
        // the other accumulator and its barriers
        acc_at ^= 256u;
        full_ph ^= (full_at >> 3) & 1u;
        full_at ^= 8u;
        empty_at ^= 8u;
        if (ks + 1 == steps || ((ks + 1) & (C::KB - 1)) == 0) {  // the group's scales have been read
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_sc_empty + 8 * (n & 1u));
          ++n;
          if (ks + 1 == steps) break;
          ok = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_sc_full + 8 * (n & 1u), (n >> 1) & 1u, wc, 0x0A));
          if (!ok) break;
        }
        scale_at(ks + 1);
      }
      if (!ok) break;
      if (p.split > 1 && pw.item >= 0) {
        // 16-byte pieces of a thread's sums, 32 lanes side by side
        auto slot = [&](int part) {
          return reinterpret_cast<float4 *>(p.partials) +
                 static_cast<int64_t>(((pw.item - pw.part + part) * 2 + static_cast<int>(rank)) * C::EPI_WARPS + w) * 1024 + lane;
        };
        float4 *to = slot(pw.part);
#pragma unroll
        for (int j = 0; j < 32; ++j) to[32 * j] = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        arrived = true;
        if (!arrive(pw.item)) continue;
        // The last of the tile's parts: all of their sums, in order.  Its own are
        // still here, but for the first two (a + b is b + a) they are read back.
        if (pw.part > 1) {
#pragma unroll
          for (int j = 0; j < 128; ++j) acc[j] = 0.f;
        }
#pragma unroll 1
        for (int r = 0; r < p.split; ++r) {
          if (r == pw.part && r <= 1) continue;
          const float4 *from = slot(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float4 x = __ldcg(from + 32 * j);
            acc[4 * j] += x.x;
            acc[4 * j + 1] += x.y;
            acc[4 * j + 2] += x.z;
            acc[4 * j + 3] += x.w;
          }
        }
      }
      // C: rows row0 .. +31, columns col0 .. +127, in pieces of 128 bytes a
      // row through this warp's 4 KB (16-byte units swizzled by the row)
      if (row0 >= p.M || col0 >= p.N) continue;
      // piece c: columns 32 c .. +31 in FP32, or 64 c .. +63 in BF16
      auto stage_f32 = [&](int c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float *a = acc + 32 * c + 4 * j;
          if constexpr (kCols) {
            // i = j: rows 16 (i / 4) + lane / 4 (+ 8), columns 8 (i % 4) + 2 (lane % 4), + 1
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = 16 * (j >> 2) + 8 * h + (lane >> 2), u = 2 * (j & 3) + ((lane >> 1) & 1);
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(stg + r * 128 + ((u ^ (r & 7)) << 4) + 8 * (lane & 1)),
                           "r"(__float_as_uint(a[2 * h])), "r"(__float_as_uint(a[2 * h + 1]))
                           : "memory");
            }
          } else {
            st_shared_v4(stg + lane * 128 + ((j ^ (lane & 7)) << 4), __float_as_uint(a[0]), __float_as_uint(a[1]),
                         __float_as_uint(a[2]), __float_as_uint(a[3]));
          }
        }
      };
      auto stage_bf16 = [&](int c) {
        auto two = [](float a, float b) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
          return *reinterpret_cast<const uint32_t *>(&h);
        };
        if constexpr (kCols) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float *a = acc + 64 * c + 4 * j;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = 16 * ((j >> 2) & 1) + 8 * h + (lane >> 2), u = 4 * (j >> 3) + (j & 3);
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(stg + r * 128 + ((u ^ (r & 7)) << 4) + 4 * (lane & 3)),
                           "r"(two(a[2 * h], a[2 * h + 1]))
                           : "memory");
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float *a = acc + 64 * c + 8 * j;
            st_shared_v4(stg + lane * 128 + ((j ^ (lane & 7)) << 4), two(a[0], a[1]), two(a[2], a[3]), two(a[4], a[5]),
                         two(a[6], a[7]));
          }
        }
      };
      if (p.tma_store) {
        constexpr int kCol = kBF16 ? 64 : 32;
#pragma unroll
        for (int c = 0; c < 128 / kCol; ++c) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
          if constexpr (kBF16) stage_bf16(c);
          else stage_f32(c);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && col0 + c * kCol < p.N) {
            tma_store_2d(&tmC, stg, col0 + c * kCol, row0);
            bulk_commit_group();
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          __syncwarp();
          stage_f32(c);
          __syncwarp();
          const int col = col0 + c * 32 + lane;
          const int rows = min(32, p.M - row0);
          const float *from = reinterpret_cast<const float *>(sm + (stg - base));
          if (col < p.N)
            for (int r = 0; r < rows; ++r) {
              float x = from[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
              const int64_t at = static_cast<int64_t>(row0 + r) * p.N + col;
              if constexpr (kBF16) {
                __nv_bfloat16 *cp = static_cast<__nv_bfloat16 *>(p.C) + at;
                if (p.use_acc) x += __bfloat162float(*cp);
                *cp = __float2bfloat16_rn(x);
              } else {
                float *cp = static_cast<float *>(p.C) + at;
                if (p.use_acc) x += *cp;
                *cp = x;
              }
            }
        }
      }
    }
    // (after a wait that gave up too: the counters belong to the next launch)
    if (p.split > 1 && !arrived && unit < p.tail_items) arrive(unit);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, 512);
}

// ---------------------------------------------------------------------------
// M <= 64: C^T[n, m] for 128 columns n of B and the rows m of A.
template <int NT>
struct SkinnyCfg {
  static constexpr int BT_BYTES = 128 * 128;  // 128 columns of B
  static constexpr int AT_BYTES = NT * 128;   // up to NT rows of A
  static constexpr int STAGES = NT <= 16 ? 11 : NT <= 32 ? 10 : 8;
  static constexpr int BUFS = 4;  // accumulators
  static constexpr int OFF_BT = 0;
  static constexpr int OFF_AT = OFF_BT + STAGES * BT_BYTES;
  // scales of A, for each epilogue warp [2 groups][4 K blocks][NT]
  static constexpr int OFF_CS = OFF_AT + STAGES * AT_BYTES;
  static constexpr int OFF_BAR = OFF_CS + 4 * 2 * 4 * NT * 4;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * BUFS + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr uint32_t TM_COLS = NT * BUFS < 32 ? 32 : NT * BUFS;
  static constexpr int THREADS = 6 * 32;
  // the cluster reduction reuses the ring: NT x 128 sums of each other CTA
  static constexpr int MAX_SPLITS = OFF_CS / (NT * 128 * 4) + 1 < 8 ? OFF_CS / (NT * 128 * 4) + 1 : 8;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(AT_BYTES % 1024 == 0 && OFF_CS % 16 == 0, "operand alignment");
};

template <int NT, int V>
__global__ void __launch_bounds__(SkinnyCfg<NT>::THREADS, 1)
    b128_skinny_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA,
                       const B128Params p) {
  using S = SkinnyCfg<NT>;
  constexpr bool kBF16 = (V & kB128Bf16) != 0, kKM = (V & kB128KMajor) != 0, kCols = (V & kB128Cols) != 0;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = p.splits;
  const int split = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int n0 = static_cast<int>(blockIdx.x) / splits * 128;
  const int k_beg = static_cast<int>(static_cast<long long>(split) * p.kb / splits);
  const int k_end = static_cast<int>(static_cast<long long>(split + 1) * p.kb / splits);

  const uint32_t bar_full = base + S::OFF_BAR;
  const uint32_t bar_empty = bar_full + 8 * S::STAGES;
  const uint32_t bar_acc_full = bar_empty + 8 * S::STAGES;
  const uint32_t bar_acc_empty = bar_acc_full + 8 * S::BUFS;
  const uint32_t bar_final = bar_acc_empty + 8 * S::BUFS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + S::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + S::OFF_MISC + 4);
  volatile int *never = reinterpret_cast<volatile int *>(sm + S::OFF_MISC + 8);  // never raised
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};
  const WaitCtl wn{p.status, never, landing_limit(p.timeout_ns)};

  auto load_step = [&](int st, int ks) {
    const uint32_t fb = bar_full + 8 * st;
    mbar_arrive_expect_tx(fb, S::BT_BYTES + p.nm * 128);
    if constexpr (kKM) tma_load_2d(base + S::OFF_BT + st * S::BT_BYTES, &tmB, ks * 128, n0, fb);
    else tma_load_2d(base + S::OFF_BT + st * S::BT_BYTES, &tmB, n0, ks * 128, fb);
    tma_load_2d(base + S::OFF_AT + st * S::AT_BYTES, &tmA, ks * 128, 0, fb);
  };
  // the first ring round goes out before the rest of the set-up
  const int n_early = p.stall_producer ? 0 : min(S::STAGES, k_end - k_beg);
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmB);
      tma_prefetch_desc(&tmA);
      for (int s = 0; s < S::STAGES; ++s) {
        mbar_init(bar_full + 8 * s, 1);
        mbar_init(bar_empty + 8 * s, 1);
      }
      for (int b = 0; b < S::BUFS; ++b) {
        mbar_init(bar_acc_full + 8 * b, 1);
        mbar_init(bar_acc_empty + 8 * b, 4);
      }
      mbar_init(bar_final, 1);
      *abort_flag = 0;
      *never = 0;
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
    griddep_launch_dependents();  // the next kernel's set-up may begin
    griddep_wait();               // no global memory before the kernel before has ended
    if (lane < n_early) load_step(lane, k_beg + lane);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_slot), S::TM_COLS);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  float acc[NT];  // epilogue: this lane's column of C, one sum per row
  bool have = false;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one() != 0;
    int st = n_early == S::STAGES ? 0 : n_early;
    uint32_t ph = n_early == S::STAGES ? 1u : 0u;
    int issued = n_early;
    for (int ks = k_beg + n_early; ks < k_end && !p.stall_producer; ++ks) {
      if (!__all_sync(0xFFFFFFFFu, wait_phase<false>(bar_empty + 8 * st, ph ^ 1u, wc, 0x01 | (st << 8)))) break;
      if (leader) load_step(st, ks);
      __syncwarp();
      ++issued;
      if (++st == S::STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }
    // every fill has been consumed (or, after a wait that gave up, has
    // landed) before the CTA may finish or reuse the ring
    bool clean = true;
    const int n = min(issued, S::STAGES);
    for (int i = 0; i < n; ++i) {
      const int s = (st + S::STAGES - n + i) % S::STAGES;
      const uint32_t par = s < st ? ph : ph ^ 1u;
      if (clean)
        clean = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_empty + 8 * s, par, wc, 0x11 | (s << 8)));
      if (!clean) wait_phase<false>(bar_full + 8 * s, par, wn, 0x11 | (s << 8));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one() != 0;
    const uint32_t idesc = idesc_f8(128, p.nm, !kKM, false) | p.idesc_fmt;
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < k_end - k_beg; ++i) {
      const int buf = i % S::BUFS;
      if (!__all_sync(0xFFFFFFFFu, wait_phase<false>(bar_acc_empty + 8 * buf, ((i / S::BUFS) & 1) ^ 1u, wc, 0x02)) ||
          !__all_sync(0xFFFFFFFFu, wait_phase<false>(bar_full + 8 * st, ph, wc, 0x03 | (st << 8))))
        break;
      tc_fence_after();
      if (leader) {
        const uint32_t sB = base + S::OFF_BT + st * S::BT_BYTES, sA = base + S::OFF_AT + st * S::AT_BYTES;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8<1>(tmem + NT * buf,
                    kKM ? smem_desc(sB + 32 * k, 0, 1024, 2) : smem_desc(sB + 4096 * k, 16384, 1024, 2),
                    smem_desc(sA + 32 * k, 0, 1024, 2), idesc, k != 0);
        tc_commit(bar_empty + 8 * st);
        tc_commit(bar_acc_full + 8 * buf);
      }
      __syncwarp();
      if (++st == S::STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (leader) tc_commit(bar_final);
    __syncwarp();
    wait_phase<false>(bar_final, 0, wn, 0x04);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int col = n0 + 32 * q + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float *cs = reinterpret_cast<float *>(sm + S::OFF_CS) + q * 8 * NT;
    const float *bs = p.b_scale + (kCols ? min(static_cast<int64_t>(col), p.bs_cols - 1)
                                         : static_cast<int64_t>(n0 >> 7)) * p.bs_n;
#pragma unroll
    for (int m = 0; m < NT; ++m) acc[m] = 0.f;
    // scales, a group of four K blocks ahead: B's of this lane (s, nb), and
    // A's 4 x NT, NT / 8 of them by each lane, through the warp's shared memory
    constexpr int kPer = NT / 8;
    float s[4], nb[4], na[kPer];
    auto fetch = [&](int g) {
#pragma unroll
      for (int j = 0; j < 4; ++j) nb[j] = __ldg(bs + min(k_beg + 4 * g + j, k_end - 1) * p.bs_k);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = lane + 32 * j, k = min(k_beg + 4 * g + i / NT, k_end - 1), m = i % NT;
        na[j] = m < p.M ? __ldg(p.a_scale + static_cast<int64_t>(m) * p.kb + k) : 0.f;
      }
    };
    fetch(0);
    have = true;
    for (int i = 0; i < k_end - k_beg; ++i) {
      if ((i & 3) == 0) {
        const int g = i >> 2;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = nb[j];
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          cs[(g & 1) * 4 * NT + lane + 32 * j] = na[j];
        __syncwarp();
        fetch(g + 1);
      }
      const int buf = i % S::BUFS;
      have = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_acc_full + 8 * buf, (i / S::BUFS) & 1, wc, 0x05));
      if (!have) break;
      tc_fence_after();
      const float sb = s[0];
      s[0] = s[1];
      s[1] = s[2];
      s[2] = s[3];
      const float4 *c4 = reinterpret_cast<const float4 *>(cs + ((i >> 2) & 1) * 4 * NT + (i & 3) * NT);
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(lane_addr + NT * buf + 16 * c, v);
        tmem_ld_done(v);
        if (c == NT / 16 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acc_empty + 8 * buf);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 f = c4[4 * c + e];
          acc[16 * c + 4 * e + 0] += __uint_as_float(v[4 * e + 0]) * (f.x * sb);
          acc[16 * c + 4 * e + 1] += __uint_as_float(v[4 * e + 1]) * (f.y * sb);
          acc[16 * c + 4 * e + 2] += __uint_as_float(v[4 * e + 2]) * (f.z * sb);
          acc[16 * c + 4 * e + 3] += __uint_as_float(v[4 * e + 3]) * (f.w * sb);
        }
      }
    }
  }

  // K split: the other CTAs of the cluster put their sums into the first one's
  // ring, which adds them in rank order.  (First barrier: all main loops are
  // done, the ring is free; second: the sums have been written.)
  const bool epi = warp >= 2;
  const int n = 32 * (warp & 3) + lane;
  if (splits > 1) {
    cluster_sync();
    if (epi && split > 0) {
      const uint32_t dst = mapa_shared(base, 0) + static_cast<uint32_t>(((split - 1) * (NT / 4)) * 128 + n) * 16;
#pragma unroll
      for (int j = 0; j < NT / 4; ++j)
        st_cluster_v4(dst + j * 2048, __float_as_uint(acc[4 * j]), __float_as_uint(acc[4 * j + 1]),
                      __float_as_uint(acc[4 * j + 2]), __float_as_uint(acc[4 * j + 3]));
    }
    cluster_sync();
    if (epi && split == 0 && have) {
      for (int r = 1; r < splits; ++r) {
        const uint32_t src = base + static_cast<uint32_t>(((r - 1) * (NT / 4)) * 128 + n) * 16;
#pragma unroll
        for (int j = 0; j < NT / 4; ++j) {
          const uint4 o = ld_shared_v4(src + j * 2048);
          acc[4 * j + 0] += __uint_as_float(o.x);
          acc[4 * j + 1] += __uint_as_float(o.y);
          acc[4 * j + 2] += __uint_as_float(o.z);
          acc[4 * j + 3] += __uint_as_float(o.w);
        }
      }
    }
  }
  // a row of C is 32 consecutive columns of a warp's lanes
  if (epi && split == 0 && have && n0 + n < p.N) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      if (m < p.M) {
        const int64_t at = static_cast<int64_t>(m) * p.N + n0 + n;
        float x = acc[m];
        if constexpr (kBF16) {
          __nv_bfloat16 *cp = static_cast<__nv_bfloat16 *>(p.C) + at;
          if (p.use_acc) x += __bfloat162float(*cp);
          *cp = __float2bfloat16_rn(x);
        } else {
          float *cp = static_cast<float *>(p.C) + at;
          if (p.use_acc) x += *cp;
          *cp = x;
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem, S::TM_COLS);
}

}  // namespace mxg
