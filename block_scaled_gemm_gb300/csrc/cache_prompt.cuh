// cache_prompt.cuh -- attention over the 8-bit key/value cache for many query
// rows (chunks of prompts), on the tensor cores.
//
// The mathematics is that of cache_attention.cuh: w_j = 2^(x_j log2 e +
// log2 vs - m + 7) meets the codes, o = (sum w_j V_j) / (2^7 sum 2^-7 w_j / vs_j).
//
// One CTA takes 256 query rows of a sequence and key/value head (row = token *
// group + head of the group, so that a group's heads share what is read) as
// two tiles of 128, and walks the keys in tiles of 128:
//   S_i = Q_i K^T    tcgen05.mma.kind::f16, Q (BF16 times its row's power of two,
//                    in FP16) and K (E4M3 converted to FP16, exact) in shared
//                    memory, S in TMEM
//   P_i              softmax warps, one thread a row: S from TMEM, P (FP16)
//                    back into S's columns
//   O_i += P_i V     P from TMEM, V (FP16) in shared memory, O in TMEM
// The tensor cores need 512 cycles for each of the four products of a key tile
// (D = 128); while they work on one Q tile, the other one's softmax runs.  The
// running maximum is moved, and O in TMEM rescaled, only when it grows by 2^8.
//
// Measured: 2 x 2048 tokens (the second 1741) over 8190 (5733) keys, 32/8 heads of
// 128: 315 us, 1.21 PFLOP/s, 0.63 of the measured FP16 rate (one of 1200 tokens over
// 16000 keys, a row tile an SM, 216 us, 0.73); a key tile takes 1.65 us, some 3200
// cycles, where the four products alone take 2048 and shared memory's traffic
// 2560.  A Q tile's chain (softmax, P V, the next Q K^T into the same columns)
// is what is left, and about 8 us before a row tile's first and after its last
// product.  Half steps of 64 keys with two S a Q tile shorten the chain but
// read Q twice (409 us); two threads a row with 16 softmax warps took 410 us;
// CTAs that stay for the next row tile took 338 us.
//
// Where the row tiles are fewer than the SMs, and for those past a multiple of
// them, each one's keys are cut into parts for several CTAs; they leave FP32
// partials in the workspace, and the one that arrives last adds them in order.
//
// Warps (512 threads): 0 TMA loads of the pages' codes, and the scales;
// 1 MMAs; 4-7 convert codes to FP16 in the MMA's layout (128-byte swizzle);
// 8-11 and 12-15 the softmax of the two Q tiles.
#pragma once
#include "cache_attention.cuh"
#include "tmem_util.cuh"

namespace mxg {

template <int D>
struct PromptCfg {
  static constexpr int ROWS = 256, KT = 128;
  static constexpr int CH = D / 64;            // 128-byte chunks of an FP16 row
  static constexpr int TILE16 = 128 * D * 2;   // 128 rows of FP16: [chunk][128 rows][128 bytes]
  static constexpr int TILE8 = 128 * D;
  static constexpr int OFF_Q = 0;              // two tiles
  static constexpr int OFF_K = OFF_Q + 2 * TILE16;  // two buffers
  static constexpr int OFF_V = OFF_K + 2 * TILE16;  // two buffers
  static constexpr int OFF_K8 = OFF_V + 2 * TILE16;
  static constexpr int OFF_V8 = OFF_K8 + TILE8;
  static constexpr int OFF_SC = OFF_V8 + TILE8;  // [4 tiles][ks, log2 vs, 2^-7/vs][8 groups of 16 keys]
  static constexpr int OFF_PG = OFF_SC + 4 * 3 * 8 * 4;  // [4 tiles] bit mask of the groups that are there
  static constexpr int OFF_BAR = OFF_PG + 16;
  static constexpr int NUM_BARS = 4 + 2 * 4 + 2 + 4 + 2 + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int PARTIAL = ROWS * (D + 2);  // floats of a partial: O by 4 d and row, m, l
  static constexpr int THREADS = 512;
  // registers a thread: 128 at launch, then of the four groups of four warps
  // (56 + 88 + 2 x 184 = 4 x 128: the block's own)
  static constexpr int REGS_MAIN = 56, REGS_CONV = 88, REGS_SOFT = 184;
  static constexpr uint32_t TM_S = 0, TM_O = 256;  // S_i at 128 i, O_i at 256 + 128 i
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Instruction descriptor of kind::f16: FP16 operands, FP32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The n lowest bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

// Least factor of S in an exponent: keeps a hidden key's -inf times it -inf
// where scale * ks underflows or is 0.
constexpr float kTinyFactor = 1.1754943508222875080e-38f;  // 2^-126

template <int D>
__global__ void __launch_bounds__(PromptCfg<D>::THREADS, 1)
    cache_prompt_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const AttnParams p) {
  using S = PromptCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_launch_dependents();
  griddep_wait();
  // ------------------------------------------------------------ this CTA's rows
  // Sequence b's row tiles are numbered from f(b) = floor(q_start group / 256) + b
  // (room for all of them); the last tiles, which see most keys, come first.
  const int beyond = static_cast<int>(blockIdx.x) - p.whole;  // among the CTAs of row tiles whose keys are cut
  const int item = beyond < 0 ? static_cast<int>(blockIdx.x) : p.whole + beyond / p.parts;
  const int h = static_cast<int>(item % p.c.kv_heads);
  const int64_t id = p.items / p.c.kv_heads - 1 - item / p.c.kv_heads;
  auto f = [&](int b) -> int64_t {
    const int64_t q = p.b.q_start ? p.b.q_start[b] : b;
    return q * p.group / S::ROWS + b;
  };
  const int b = warp_find(p.b.batch, f, id);
  const Sequence s = load_sequence(p.b, p.c, b);
  const int64_t row_first = (id - f(b)) * S::ROWS;
  const int64_t row_count = static_cast<int64_t>(s.n) * p.group;
  if (row_first < 0 || row_first >= row_count) return;
  const int row0 = static_cast<int>(row_first);
  const int rows = static_cast<int>(min(static_cast<int64_t>(S::ROWS), row_count - row_first));
  const int nq = rows > 128 ? 2 : 1;
  const int pos0 = s.len - s.n;
  // keys that any of the rows sees: tiles of first tokens, then from tile `lo`
  const int pos_first = pos0 + row0 / p.group, pos_last = pos0 + (row0 + rows - 1) / p.group;
  const int end = p.causal ? max(0, min(s.len, pos_last + 1)) : s.len;
  const int win_lo = p.window > 0 ? static_cast<int>(min(max(static_cast<int64_t>(0), pos_first - p.window + 1), static_cast<int64_t>(end))) : 0;
  const int lo = win_lo >> 7;
  const int ns = static_cast<int>(min((min(p.sinks, static_cast<int64_t>(win_lo)) + 127) >> 7, static_cast<int64_t>(lo)));
  const int all_tiles = max(1, ns + ((end + 127) >> 7) - lo);
  // this CTA's part of them: four at least
  const int parts = beyond < 0 ? 1 : min(p.parts, max(1, all_tiles >> 2)), part = beyond < 0 ? 0 : beyond % p.parts;
  if (part >= parts) return;
  const int tile0 = static_cast<int>(static_cast<int64_t>(part) * all_tiles / parts);
  const int tiles = static_cast<int>(static_cast<int64_t>(part + 1) * all_tiles / parts) - tile0;
  auto tile_key = [&](int j) { return (j + tile0 < ns ? j + tile0 : lo + j + tile0 - ns) * 128; };

  const uint32_t bars = base + S::OFF_BAR;
  const uint32_t k8_full = bars, v8_full = bars + 8, k8_empty = bars + 16, v8_empty = bars + 24;
  const uint32_t k_full = bars + 32, v_full = bars + 48, k_empty = bars + 64, v_empty = bars + 80;  // two each
  const uint32_t s_full = bars + 96, p_full = bars + 112;  // one and two (P's halves) for each Q tile
  const uint32_t o_done = bars + 144, q_full = bars + 160;  // one for each Q tile
  const uint32_t bar_final = bars + 176;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + S::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + S::OFF_MISC + 4);
  volatile int *never = reinterpret_cast<volatile int *>(sm + S::OFF_MISC + 8);  // never raised
  float *scales = reinterpret_cast<float *>(sm + S::OFF_SC);
  volatile uint32_t *groups = reinterpret_cast<volatile uint32_t *>(sm + S::OFF_PG);
  if (threadIdx.x == 0) {
    mbar_init(k8_full, 1);
    mbar_init(v8_full, 1);
    mbar_init(k8_empty, 4);
    mbar_init(v8_empty, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, 4);
      mbar_init(v_full + 8 * i, 4);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(p_full + 16 + 8 * i, 4);
      mbar_init(o_done + 8 * i, 1);
      mbar_init(q_full + 8 * i, 4);
    }
    mbar_init(bar_final, 1);
    *abort_flag = 0;
    *never = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_slot), 512);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{p.b.status, abort_flag, p.timeout_ns};
  const WaitCtl wn{p.b.status, never, landing_limit(p.timeout_ns)};
  auto wait = [&](uint32_t bar, uint32_t parity, int detail) {
    return __all_sync(0xFFFFFFFFu, wait_phase<false>(bar, parity, wc, detail));
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_MAIN));
    if (warp == 0) {
      // ---------------------------------------------------------- loads
      const int lg = p.c.page_log2, npg = 128 >> lg;  // pages of a tile
      bool ok = !p.stall_producer;
      int k_loads = 0, v_loads = 0;
      for (int j = 0; ok && j < tiles; ++j) {
        const int key0 = tile_key(j);
        // lane g < 8: the 16 keys of group g, unless none of the rows sees a key of
        // their page (a window may have passed it)
        int pg = -1;
        const int k0 = key0 + 16 * lane, page0 = k0 >> lg << lg;
        if (lane < 8 && k0 < end && (page0 + (1 << lg) > win_lo || page0 < p.sinks)) pg = load_page(p.b, p.c, b, k0 >> lg);
        float ks = 1.f, vs = 1.f;
        if (pg >= 0) {
          const int64_t cell = static_cast<int64_t>(pg) * p.c.kv_heads + h;
          ks = p.c.K_scale[cell];
          vs = fmaxf(p.c.V_scale[cell], kScaleFloor);
        }
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, pg >= 0);
        // lane i < npg: page i of the tile
        const int page = __shfl_sync(0xFFFFFFFFu, pg, (lane << (lg - 4)) & 7);
        const bool load = lane < npg && page >= 0;
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, load)) * static_cast<uint32_t>(D << lg);
        const int row = load ? (page * p.c.kv_heads + h) << lg : 0;
        // (the slot of tile j - 4, whose softmax is over: the converters are
        // past tile j - 2's, which waited for it)
        ok = wait(k8_empty, (j & 1) ^ 1, 0x41);
        if (!ok) break;
        if (lane < 8) {
          float *sc = scales + (j & 3) * 24 + lane;
          sc[0] = ks;
          const float lv = lg2(vs);
          sc[8] = lv;
          sc[16] = inverse_of_log2(lv) * kWeightDown;
        }
        if (lane == 0) groups[j & 3] = there;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(k8_full, bytes);
        __syncwarp();
        if (load) tma_load_2d(base + S::OFF_K8 + (lane << lg) * D, &tmK, 0, row, k8_full);
        ++k_loads;
        ok = wait(v8_empty, (j & 1) ^ 1, 0x42);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(v8_full, bytes);
        __syncwarp();
        if (load) tma_load_2d(base + S::OFF_V8 + (lane << lg) * D, &tmV, 0, row, v8_full);
        ++v_loads;
      }
      // The last loads land before the CTA ends, whoever gave up: the
      // converters may have left without waiting for them.
      if (k_loads > 0) wait_phase<false>(k8_full, ring_parity(k_loads - 1, 1), wn, 0x43);
      if (v_loads > 0) wait_phase<false>(v8_full, ring_parity(v_loads - 1, 1), wn, 0x43);
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMAs
      if (elect_one()) {
        auto w1 = [&](uint32_t bar, uint32_t parity, int detail) { return wait_phase<false>(bar, parity, wc, detail); };
        constexpr uint32_t kIdS = idesc_f16(128, 128, false), kIdO = idesc_f16(128, D, true);
        auto qk = [&](int i, int buf) {
          // both K-major: chunks of 64 d 16 KB apart, 32 bytes per K = 16
          const uint32_t a = base + S::OFF_Q + i * S::TILE16, k = base + S::OFF_K + buf * S::TILE16;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t off = (c >> 2) * 16384 + (c & 3) * 32;
            mma_f16_ss(tmem + S::TM_S + 128 * i, smem_desc(a + off, 0, 1024, 2), smem_desc(k + off, 0, 1024, 2), kIdS,
                       c != 0);
          }
          tc_commit(s_full + 8 * i);
        };
        bool ok = true;
        for (int i = 0; ok && i < nq; ++i) ok = w1(q_full + 8 * i, 0, 0x44);
        ok = ok && w1(k_full, 0, 0x45);
        if (ok) {
          tc_fence_after();
          for (int i = 0; i < nq; ++i) qk(i, 0);
          tc_commit(k_empty);
        }
        for (int j = 0; ok && j < tiles; ++j) {
          const int buf = j & 1;
          for (int i = 0; i < nq; ++i) {
            ok = i || w1(v_full + 8 * buf, (j >> 1) & 1, 0x46);
            // P: 8 columns per K = 16 keys; V: N-major, chunks of 64 d 16 KB
            // apart, 16 keys 2 KB apart
            const uint32_t v = base + S::OFF_V + buf * S::TILE16;
            for (int hf = 0; hf < 2; ++hf) {  // P of 64 keys, then of the others
              ok = ok && w1(p_full + 16 * i + 8 * hf, j & 1, 0x47);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < 4; ++c)
                mma_f16_ts(tmem + S::TM_O + 128 * i, tmem + S::TM_S + 128 * i + 32 * hf + 8 * c,
                           smem_desc(v + 8192 * hf + 2048 * c, 16384, 1024, 2), kIdO, j != 0 || hf != 0 || c != 0);
            }
            if (!ok) break;
            tc_commit(o_done + 8 * i);
            if (i == nq - 1) tc_commit(v_empty + 8 * buf);
            if (j + 1 < tiles) {
              // into the columns that P was read from: MMAs execute in order
              if (i == 0) {
                ok = w1(k_full + 8 * (buf ^ 1), ((j + 1) >> 1) & 1, 0x45);
                if (!ok) break;
                tc_fence_after();
              }
              qk(i, buf ^ 1);
              if (i == nq - 1) tc_commit(k_empty + 8 * (buf ^ 1));
            }
          }
        }
        tc_commit(bar_final);
        wait_phase<false>(bar_final, 0, wn, 0x48);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_CONV));
    const int tid = threadIdx.x - 128;
    constexpr int kCh8 = D / 16;            // 16-byte chunks of a row of codes
    constexpr int kIter = 128 * kCh8 / 128;  // chunks of a thread
    const int q = tid % kCh8, r0 = tid / kCh8;
    // a row's chunk q (16 codes) is units 2q, 2q + 1 of 16 bytes of its FP16 row
    const int first = D == 128 && q >= 4 ? 1 : 0;  // the order that keeps the stores free of bank conflicts
    for (int j = 0; j < tiles; ++j) {
      const int buf = j & 1, key0 = tile_key(j);
      bool ok = true;
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {  // K, then V
        const uint32_t full8 = v ? v8_full : k8_full, empty8 = v ? v8_empty : k8_empty;
        const uint32_t full = (v ? v_full : k_full) + 8 * buf, empty = (v ? v_empty : k_empty) + 8 * buf;
        ok = wait(full8, j & 1, 0x49 + 2 * v) && wait(empty, ((j >> 1) & 1) ^ 1, 0x4A + 2 * v);
        if (!ok) break;
        const uint32_t there = groups[j & 3];
        const uint32_t from = base + (v ? S::OFF_V8 : S::OFF_K8) + r0 * D + q * 16;
        const uint32_t to = base + (v ? S::OFF_V : S::OFF_K) + buf * S::TILE16 + (q >> 2) * 16384 + r0 * 128;
        // (rows 8 and more apart have one swizzle: 128 / kCh8 is 16 or 32)
        const int u = 2 * (q & 3);
        const uint32_t d0 = to + (((u + first) ^ (r0 & 7)) << 4), d1 = to + (((u + 1 - first) ^ (r0 & 7)) << 4);
        // V's codes of keys that no row sees may be anything: 0 * NaN is NaN
        const bool mask = v && (there != 0xFFu || key0 + 128 > end || (key0 < win_lo && key0 + 128 > p.sinks));
#pragma unroll 4
        for (int it = 0; it < kIter; ++it) {
          constexpr int kStep = 128 / kCh8;
          uint4 w = ld_shared_v4(from + it * kStep * D);
          if (mask) {
            const int r = r0 + it * kStep, key = key0 + r;
            if (!((there >> (r >> 4)) & 1u) || key >= end || (key < win_lo && key >= p.sinks)) w = make_uint4(0, 0, 0, 0);
          }
          if (first) {
            uint32_t x = w.x, y = w.y;
            w.x = w.z; w.y = w.w; w.z = x; w.w = y;
          }
          st_shared_v4(d0 + it * kStep * 128, e4m3_lo(w.x), e4m3_hi(w.x), e4m3_lo(w.y), e4m3_hi(w.y));
          st_shared_v4(d1 + it * kStep * 128, e4m3_lo(w.z), e4m3_hi(w.z), e4m3_lo(w.w), e4m3_hi(w.w));
        }
        fence_proxy_async_smem();  // the MMAs read what was written, and the next load overwrites what was read
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full);
          mbar_arrive(empty8);
        }
      }
      if (!ok) break;
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::REGS_SOFT));
    const int i = (warp - 8) >> 2, qd = warp & 3;  // Q tile, and quarter of its rows
    const int r = 128 * i + 32 * qd + lane;        // this thread's row of the CTA's
    if (i < nq) {
      const bool live = r < rows;
      const int tok = (row0 + (live ? r : 0)) / p.group, head = h * p.group + (row0 + (live ? r : 0)) % p.group;
      // Q times its row's power of two in FP16; rows past the last are zero
      float cq;
      {
        // whole rows side by side, kUnits lanes (16 bytes each) a row
        constexpr int kUnits = D / 8, kRows = 32 / kUnits;
        const int64_t mine = static_cast<int64_t>(s.first + tok) * p.q_pitch + static_cast<int64_t>(head) * D;
        const int unit = lane % kUnits, sub = lane / kUnits;
        uint4 x[32 / kRows];
#pragma unroll
        for (int n = 0; n < 32 / kRows; ++n) {
          const int from = kRows * n + sub;
          const int64_t at = __shfl_sync(0xFFFFFFFFu, mine, from);
          x[n] = 128 * i + 32 * qd + from < rows ? *reinterpret_cast<const uint4 *>(p.Q + at + 8 * unit) : make_uint4(0, 0, 0, 0);
        }
        float top = 0.f;  // of this thread's row
        const uint32_t dst = base + S::OFF_Q + i * S::TILE16 + (unit >> 3) * 16384;
#pragma unroll
        for (int n = 0; n < 32 / kRows; ++n) {
          const int rr = 32 * qd + kRows * n + sub;
          const uint32_t u[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
          float t = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            t = fmaxf(t, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xFFFF0000u))));
#pragma unroll
          for (int o = kUnits / 2; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
          const float own = __shfl_sync(0xFFFFFFFFu, t, (lane % kRows) * kUnits);
          if (lane / kRows == n) top = own;
          // (a negative scale's sign goes to Q: the exponents' factors are positive)
          const float up = copysignf(pow2(q_exponent(t)), p.scale);
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = half2_of(__uint_as_float(u[k] << 16) * up, __uint_as_float(u[k] & 0xFFFF0000u) * up);
          st_shared_v4(dst + rr * 128 + (((unit & 7) ^ (rr & 7)) << 4), y[0], y[1], y[2], y[3]);
        }
        cq = fabsf(p.scale) * 1.44269504088896340736f * pow2(-q_exponent(top));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + 8 * i);
      }
      const int pos = pos0 + tok;
      // this thread's row sees keys [row_from, row_to) and the first tokens; all
      // rows of the warp see [all_from, all_to)
      auto window_from = [&](int pos) {
        return p.window == 0 ? 0 : static_cast<int>(max(static_cast<int64_t>(0), pos - p.window + 1));
      };
      const int w0 = 128 * i + 32 * qd;
      const int row_to = p.causal ? min(end, pos + 1) : end, row_from = window_from(pos);
      const int all_to = p.causal ? min(end, pos0 + (row0 + min(w0, rows - 1)) / p.group + 1) : end;
      const int all_from = window_from(pos0 + (row0 + min(w0 + 31, rows - 1)) / p.group);
      const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
      const uint32_t ts = tmem + S::TM_S + 128 * i + lanes, to = tmem + S::TM_O + 128 * i + lanes;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < tiles; ++j) {
        const int key0 = tile_key(j);
        ok = warp_wait(s_full + 8 * i, j & 1, wc, 0x4D);
        if (!ok) break;
        tc_fence_after();
        const float *sc = scales + (j & 3) * 24;
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, v[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_done(v[c]);
        const uint32_t there = groups[j & 3];
        const int jlast = key0 + 127;
        const bool whole = there == 0xFFu && jlast < all_to && (key0 >= all_from || jlast < p.sinks);
        if (!whole) {
          // columns [from, upto) and [0, sink) of the tile are seen
          const int upto = row_to - key0, from = row_from - key0;
          const int sink = static_cast<int>(min(p.sinks, static_cast<int64_t>(end))) - key0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t seen = low_bits(upto - 32 * c) & (~low_bits(from - 32 * c) | low_bits(sink - 32 * c)) &
                                  (((there >> (2 * c)) & 1u ? 0xFFFFu : 0u) | ((there >> (2 * c + 1)) & 1u ? 0xFFFF0000u : 0u));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((seen >> e) & 1u)) v[c][e] = 0xFF800000u;  // -inf
          }
        }
        // exponents of group c: S * k + a, k > 0: their maximum is the one of S's
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t *x = v[c >> 1] + 16 * (c & 1);
          float g = __uint_as_float(x[0]);
#pragma unroll
          for (int e = 1; e < 15; e += 2) g = max3(g, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          g = fmaxf(g, __uint_as_float(x[15]));
          top = fmaxf(top, fmaf(g, fmaxf(cq * sc[c], kTinyFactor), sc[8 + c]));
        }
        const bool grow = top > m + 8.f;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float mn = grow ? top : m;
          const float k = mn == -INFINITY ? 1.f : ex2(m - mn);
          m = mn;
          l *= k;
          if (j > 0) {
            ok = wait(o_done + 8 * i, (j - 1) & 1, 0x4E);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(to + 16 * c, o);
              tmem_ld_done(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * k);
              tmem_st_x16(to + 16 * c, o);
            }
            tmem_st_wait();
          }
        }
        const float ms = m == -INFINITY ? 0.f : m - kWeightUp;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float k = fmaxf(cq * sc[2 * c + hf], kTinyFactor), a = sc[8 + 2 * c + hf] - ms;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 x = fma2(make_float2(__uint_as_float(v[c][16 * hf + 2 * e]), __uint_as_float(v[c][16 * hf + 2 * e + 1])),
                                    make_float2(k, k), make_float2(a, a));
              const float2 w = make_float2(ex2(x.x), ex2(x.y));
              sum = add2(sum, w);
              pk[8 * hf + e] = half2_of(w.x, w.y);
            }
            l = fmaf(sum.x + sum.y, sc[16 + 2 * c + hf], l);
          }
          tmem_st_x16(ts + 16 * c, pk);
          if (c & 1) {  // 64 keys: their MMAs may begin
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 16 * i + 8 * (c >> 1));
          }
        }
      }
      if (ok) ok = wait(o_done + 8 * i, (tiles - 1) & 1, 0x4F);
      if (ok) {
        tc_fence_after();
        const int at = (s.first + tok) * p.heads + head;
        if (parts > 1) {
          float *slot = p.partials + (static_cast<int64_t>(item - p.whole) * p.parts + part) * S::PARTIAL;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 32 * c, o);
            tmem_ld_done(o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4 *>(slot)[(8 * c + e) * S::ROWS + r] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          slot[S::ROWS * D + r] = m;
          slot[S::ROWS * D + S::ROWS + r] = l;
        } else {
          // through the rows of Q, whose products are done: a store of whole
          // lines, where a thread's own row would touch 32
          const float k = l == 0.f ? 0.f : kWeightDown / l;
          const uint32_t rr = 32 * qd + lane, q_row = base + S::OFF_Q + i * S::TILE16 + rr * 128;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 32 * c, o);
            tmem_ld_done(o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t x[4];
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * w]) * k,
                                                               __uint_as_float(o[8 * e + 2 * w + 1]) * k);
                x[w] = *reinterpret_cast<const uint32_t *>(&y);
              }
              st_shared_v4(q_row + (c >> 1) * 16384 + (((4 * (c & 1) + e) ^ (rr & 7)) << 4), x[0], x[1], x[2], x[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int from = 4 * j + (lane >> 3), q = lane & 7;
            const int64_t to_row = __shfl_sync(0xFFFFFFFFu, at, from);
            if (128 * i + 32 * qd + from < rows) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<uint4 *>(p.O + to_row * D + 64 * c + 8 * q) =
                    ld_shared_v4(q_row + (from - lane) * 128 + c * 16384 + ((q ^ (from & 7)) << 4));
            }
          }
          if (live && p.lse) p.lse[at] = log_sum(m, l);
        }
      }
    }
    if (parts > 1) {
      // (every softmax warp comes here: all their waits are bounded)
      __threadfence();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (threadIdx.x == 256) *tmem_slot = atomicAdd(p.counters + item - p.whole, 1u) == static_cast<unsigned>(parts - 1) ? 1u : 0u;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (*reinterpret_cast<volatile uint32_t *>(tmem_slot)) {
        if (threadIdx.x == 256) p.counters[item - p.whole] = 0;  // for the next launch
        __threadfence();
        const float *first = p.partials + static_cast<int64_t>(item - p.whole) * p.parts * S::PARTIAL;
        if (r < rows) {
          const int tok = (row0 + r) / p.group, head = h * p.group + (row0 + r) % p.group;
          float top = -INFINITY, sum = 0.f;
          for (int c = 0; c < parts; ++c) top = fmaxf(top, __ldcg(first + c * S::PARTIAL + S::ROWS * D + r));
          for (int c = 0; c < parts; ++c) {
            const float mc = __ldcg(first + c * S::PARTIAL + S::ROWS * D + r);
            sum = fmaf(__ldcg(first + c * S::PARTIAL + S::ROWS * D + S::ROWS + r), mc == -INFINITY ? 0.f : ex2(mc - top), sum);
          }
          const float k = sum == 0.f ? 0.f : kWeightDown / sum;
          __nv_bfloat16 *dst = p.O + (static_cast<int64_t>(s.first + tok) * p.heads + head) * D;
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            float4 a[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int c = 0; c < parts; ++c) {
              const float mc = __ldcg(first + c * S::PARTIAL + S::ROWS * D + r);
              const float f = mc == -INFINITY ? 0.f : ex2(mc - top) * k;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(first + c * S::PARTIAL) + (d / 4 + e) * S::ROWS + r);
                a[e].x = fmaf(x.x, f, a[e].x);
                a[e].y = fmaf(x.y, f, a[e].y);
                a[e].z = fmaf(x.z, f, a[e].z);
                a[e].w = fmaf(x.w, f, a[e].w);
              }
            }
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(a[e].x, a[e].y), z = __floats2bfloat162_rn(a[e].z, a[e].w);
              x[2 * e] = *reinterpret_cast<const uint32_t *>(&y);
              x[2 * e + 1] = *reinterpret_cast<const uint32_t *>(&z);
            }
            *reinterpret_cast<uint4 *>(dst + d) = make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4 *>(dst + d + 8) = make_uint4(x[4], x[5], x[6], x[7]);
          }
          if (p.lse)
            p.lse[static_cast<int64_t>(s.first + tok) * p.heads + head] = log_sum(top, sum);
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem, 512);
}

}  // namespace mxg
