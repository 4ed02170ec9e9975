// gated_skinny.cuh -- the gated pair of products for M <= 64 rows:
//
//   H[m,n] = act(sum_k A[m,k] G[n,k]) * (sum_k A[m,k] U[n,k]),  blocks of 128 scaled
//
// Bound by reading both weights once.  Transposed, as the single product's kernel
// for few rows: 128 columns of a weight on the MMA's 128-row side and the rows of A
// as its N.  A step of the ring is one K block of one column block: 16 KB of each
// weight and A's rows.  More column blocks than SMs: all their steps, laid end to end,
// are cut into equal ranges, one for each CTA, so that no SM waits for a last wave and
// the loads go on across column blocks.  Fewer: each is cut into whole CTAs' parts.  A
// CTA leaves its FP32 sums of a column block in the workspace, and the one that arrives
// last there adds them, in order, and finishes the block: nobody waits for another CTA.
// It does so from the workspace, also where
// the block is its own alone, with a warp for each row: sums lie in registers by
// columns, and the end of a block from there (64 rows: 32 values of each of two sums a
// thread, in code that runs once) took 5 us, a row's largest value a reduction each.
//
// Measured: 16 x 28672 x 8192 to codes 80.5 us on the same buffers again and again and
// 82 us with others each time (5.8 and 5.7 TB/s, 0.86 and 0.84 of the measured copy
// rate), 1 x 4096 x 4096 9.8 us with the weights in L2, 64 x 8192 x 8192 38 us.  The
// rest is the start (3-4 us before the first loads land) and, where column blocks are
// shared by several CTAs, their join (some 3 us: sums to L2 1, counted 1, read and
// added 1, and the rows).
//
// Waits are bounded as in the other kernels.  The epilogue's warps go on to the end
// after a wait that gave up, without waiting again: their barrier and the arrivals
// at shared column blocks stay whole, and the counters are left at zero.
#pragma once
#include "block128_kernel.cuh"

namespace mxg {

struct GatedSkinnyParams {
  B128Params b;
  int n_tiles;
  int64_t total;       // steps: column blocks x K blocks
  float *partials;     // two slots a CTA: [2][NT rows][128 columns]
  unsigned *counters;  // of the CTA with a shared column block's first step
  int h_type;          // mxgemm_out_dtype_t
};

template <int NT>
struct GatedSkinnyCfg {
  static constexpr int BT_BYTES = 128 * 128, AT_BYTES = NT * 128;
  static constexpr int STAGE = 2 * BT_BYTES + AT_BYTES;
  static constexpr int STAGES = NT <= 32 ? 6 : 5;
  static constexpr int BUFS = 4;  // accumulators, each of both products
  // Epilogue warps: four for the 128 columns, and from 32 rows on two sets of them
  // with half the rows each.
  static constexpr int SETS = NT >= 32 ? 2 : 1, ROWS = NT / SETS, EPI_WARPS = 4 * SETS;
  // scales of A, for each epilogue warp [2 groups][4 steps][ROWS]
  static constexpr int OFF_CS = STAGES * STAGE;
  static constexpr int OFF_BAR = OFF_CS + EPI_WARPS * 2 * 4 * ROWS * 4;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * BUFS + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr uint32_t TM_COLS = 2 * NT * BUFS;
  static constexpr int THREADS = (2 + EPI_WARPS) * 32;
  static constexpr int PARTIAL = 2 * NT * 128;  // floats
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(STAGE % 1024 == 0 && OFF_BAR % 8 == 0 && TM_COLS <= 512, "layout");
};

// The end of a column block: rows warp, warp + EPI_WARPS, ... by this warp, a lane four
// columns, from the parts of CTAs c0 .. c1.  Four rows' loads of two parts at a time.
template <int NT, typename Slot>
__device__ __forceinline__ void gated_skinny_rows(const GatedSkinnyParams &gp, Slot slot, int64_t c0, int64_t c1, int tile, int warp, int lane) {
  constexpr int kStep = GatedSkinnyCfg<NT>::EPI_WARPS, kRows = 4, kParts = 2;
  const B128Params &p = gp.b;
  const int col = tile * 128 + 4 * lane, there = p.N - col;  // columns from here on (0 or fewer: none)
  const bool whole = there >= 4 && p.N % 4 == 0;              // four, and aligned
#pragma unroll 1
  for (int r0 = warp; r0 < p.M; r0 += kRows * kStep) {
    float4 s[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i][0] = s[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int64_t c = c0; c <= c1; c += kParts) {
      float4 o[kParts][kRows][2];
#pragma unroll
      for (int n = 0; n < kParts; ++n)
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int r = r0 + i * kStep;
            o[n][i][w] = c + n <= c1 && r < p.M ? __ldcg(reinterpret_cast<const float4 *>(slot(c + n) + (w * NT + r) * 128) + lane)
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
      for (int n = 0; n < kParts; ++n)
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            s[i][w].x += o[n][i][w].x;
            s[i][w].y += o[n][i][w].y;
            s[i][w].z += o[n][i][w].z;
            s[i][w].w += o[n][i][w].w;
          }
    }
    auto pack = [](float a, float b) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      return *reinterpret_cast<const uint32_t *>(&h);
    };
    auto store_bf16 = [&](__nv_bfloat16 *to, float4 v) {
      if (whole) {
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack(v.x, v.y), pack(v.z, v.w));
      } else {
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < there) to[e] = __float2bfloat16_rn(x[e]);
      }
    };
    // (step by step for all rows together: one row after the other takes 0.32 us each)
    float4 h[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float4 g = s[i][0], u = s[i][1];
      h[i] = make_float4(gated(g.x, u.x, p.act), gated(g.y, u.y, p.act), gated(g.z, u.z, p.act), gated(g.w, u.w, p.act));
    }
    float top[kRows], inv[kRows];
    if (gp.h_type == 2) {  // MXGEMM_OUT_E4M3 (columns past the last are 0)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float most = fmaxf(fmaxf(fabsf(h[i].x), fabsf(h[i].y)), fmaxf(fabsf(h[i].z), fabsf(h[i].w)));
        // (NaN is passed over, as the quantizer does; four of them would win as bits)
        top[i] = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(most, kQ128Least))));
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) inv[i] = __fdiv_rn(448.0f, top[i]);
      if (lane < kRows && r0 + lane * kStep < p.M) {
        float mine = top[0];
#pragma unroll
        for (int i = 1; i < kRows; ++i) mine = lane == i ? top[i] : mine;
        p.h_scale[static_cast<int64_t>(r0 + lane * kStep) * p.bs_cols + tile] = __fdiv_rn(mine, 448.0f);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i * kStep;
      if (r >= p.M) continue;
      const int64_t at = static_cast<int64_t>(r) * p.N + col;
      if (p.gate) {
        store_bf16(p.gate + at, s[i][0]);
        store_bf16(p.up + at, s[i][1]);
      }
      if (gp.h_type == 2) {
        if (there > 0)
          *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.C) + at) =
              mx_e4m3x2(h[i].x * inv[i], h[i].y * inv[i]) | (mx_e4m3x2(h[i].z * inv[i], h[i].w * inv[i]) << 16);
      } else if (gp.h_type == 1) {
        store_bf16(static_cast<__nv_bfloat16 *>(p.C) + at, h[i]);
      } else if (whole) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + at) = h[i];
      } else {
        const float x[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < there) static_cast<float *>(p.C)[at + e] = x[e];
      }
    }
  }
}

template <int NT, bool kKM>
__global__ void __launch_bounds__(GatedSkinnyCfg<NT>::THREADS, 1)
    gated_skinny_kernel(const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmU,
                        const __grid_constant__ CUtensorMap tmA, const GatedSkinnyParams gp) {
  using S = GatedSkinnyCfg<NT>;
  const B128Params &p = gp.b;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kb = p.kb;
  const int64_t total = gp.total, ctas = gridDim.x;
  const int64_t u0 = blockIdx.x * total / ctas, u1 = (blockIdx.x + 1) * total / ctas;
  const int steps = static_cast<int>(u1 - u0);
  const int tile0 = static_cast<int>(u0 / kb), k0 = static_cast<int>(u0 - static_cast<int64_t>(tile0) * kb);

  const uint32_t bar_full = base + S::OFF_BAR;
  const uint32_t bar_empty = bar_full + 8 * S::STAGES;
  const uint32_t bar_acc_full = bar_empty + 8 * S::STAGES;
  const uint32_t bar_acc_empty = bar_acc_full + 8 * S::BUFS;
  const uint32_t bar_final = bar_acc_empty + 8 * S::BUFS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + S::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + S::OFF_MISC + 4);
  volatile int *never = reinterpret_cast<volatile int *>(sm + S::OFF_MISC + 8);  // never raised
  volatile int *last = reinterpret_cast<volatile int *>(sm + S::OFF_MISC + 12);
  const WaitCtl wc{p.status, abort_flag, p.timeout_ns};
  const WaitCtl wn{p.status, never, landing_limit(p.timeout_ns)};

  auto load_step = [&](int st, int i) {  // step i of this CTA's
    const int64_t u = u0 + i;
    const int tile = static_cast<int>(u / kb), ks = static_cast<int>(u - static_cast<int64_t>(tile) * kb);
    const uint32_t fb = bar_full + 8 * st, to = base + st * S::STAGE;
    mbar_arrive_expect_tx(fb, 2 * S::BT_BYTES + p.nm * 128);
    if constexpr (kKM) {
      tma_load_2d(to, &tmG, ks * 128, tile * 128, fb);
      tma_load_2d(to + S::BT_BYTES, &tmU, ks * 128, tile * 128, fb);
    } else {
      tma_load_2d(to, &tmG, tile * 128, ks * 128, fb);
      tma_load_2d(to + S::BT_BYTES, &tmU, tile * 128, ks * 128, fb);
    }
    tma_load_2d(to + 2 * S::BT_BYTES, &tmA, ks * 128, 0, fb);
  };
  // the first ring round goes out before the rest of the set-up
  const int n_early = p.stall_producer ? 0 : min(S::STAGES, steps);
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmG);
      tma_prefetch_desc(&tmU);
      tma_prefetch_desc(&tmA);
      for (int s = 0; s < S::STAGES; ++s) {
        mbar_init(bar_full + 8 * s, 1);
        mbar_init(bar_empty + 8 * s, 1);
      }
      for (int b = 0; b < S::BUFS; ++b) {
        mbar_init(bar_acc_full + 8 * b, 1);
        mbar_init(bar_acc_empty + 8 * b, S::EPI_WARPS);
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
    if (lane < n_early) load_step(lane, lane);
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

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one() != 0;
    int issued = n_early;
    for (; issued < steps && !p.stall_producer; ++issued) {
      const int st = issued % S::STAGES;
      if (!__all_sync(0xFFFFFFFFu, wait_phase<false>(bar_empty + 8 * st, ring_parity(issued, S::STAGES) ^ 1u, wc, 0x01 | (st << 8))))
        break;
      if (leader) load_step(st, issued);
      __syncwarp();
    }
    // every fill has been consumed (or, after a wait that gave up, has landed)
    // before the CTA may finish
    bool clean = true;
    for (int64_t i = ring_pending(issued, S::STAGES); i < issued; ++i) {
      const int s = static_cast<int>(i % S::STAGES);
      const uint32_t par = ring_parity(i, S::STAGES);
      if (clean) clean = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_empty + 8 * s, par, wc, 0x11 | (s << 8)));
      if (!clean) wait_phase<false>(bar_full + 8 * s, par, wn, 0x11 | (s << 8));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one() != 0;
    const uint32_t idesc = idesc_f8(128, p.nm, !kKM, false) | p.idesc_fmt;
    for (int i = 0; i < steps; ++i) {
      const int st = i % S::STAGES, buf = i % S::BUFS;
      if (!__all_sync(0xFFFFFFFFu, wait_phase<false>(bar_acc_empty + 8 * buf, ((i / S::BUFS) & 1) ^ 1u, wc, 0x02)) ||
          !__all_sync(0xFFFFFFFFu, wait_phase<false>(bar_full + 8 * st, ring_parity(i, S::STAGES), wc, 0x03 | (st << 8))))
        break;
      tc_fence_after();
      if (leader) {
        const uint32_t at = base + st * S::STAGE, sA = at + 2 * S::BT_BYTES;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t sB = at + w * S::BT_BYTES;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f8<1>(tmem + 2 * NT * buf + NT * w,
                      kKM ? smem_desc(sB + 32 * k, 0, 1024, 2) : smem_desc(sB + 4096 * k, 16384, 1024, 2),
                      smem_desc(sA + 32 * k, 0, 1024, 2), idesc, k != 0);
        }
        tc_commit(bar_empty + 8 * st);
        tc_commit(bar_acc_full + 8 * buf);
      }
      __syncwarp();
    }
    if (leader) tc_commit(bar_final);
    __syncwarp();
    wait_phase<false>(bar_final, 0, wn, 0x04);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int ROWS = S::ROWS;
    const int q = warp & 3, n = 32 * q + lane;                // this lane's column of the block
    const int set = (warp - 2) >> 2, row0 = set * ROWS;       // and its rows
    const int rows = min(ROWS, p.M - row0);                   // that there are (0 or fewer: none)
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16) + row0;
    float *cs = reinterpret_cast<float *>(sm + S::OFF_CS) + (warp - 2) * 8 * ROWS;
    auto all_warps = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * S::EPI_WARPS) : "memory"); };  // of the epilogue
    float acc[2][ROWS];
#pragma unroll
    for (int m = 0; m < ROWS; ++m) acc[0][m] = acc[1][m] = 0.f;
    // Scales, a group of four steps ahead: of the weights lane 2 j + w has step j's
    // of weight w, and A's 4 x ROWS, ROWS / 8 of them by each lane, go through the
    // warp's shared memory.  (gt, gk): the group's first column block and K block.
    constexpr int kPer = ROWS / 8;
    float nb = 0.f, sb = 0.f, na[kPer];
    int gt = tile0, gk = k0;
    auto step_at = [&](int j, int &t, int &k) {
      t = gt;
      k = gk + j;
      while (k >= kb) {
        k -= kb;
        ++t;
      }
      t = min(t, gp.n_tiles - 1);  // (past the last step: anything)
    };
    auto fetch = [&]() {
      int t, k;
      if (lane < 8) {
        step_at(lane >> 1, t, k);
        nb = __ldcg((lane & 1 ? p.u_scale : p.b_scale) + t * p.bs_n + k * p.bs_k);
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = lane + 32 * j, m = i % ROWS;
        step_at(i / ROWS, t, k);
        na[j] = m < rows ? __ldcg(p.a_scale + static_cast<int64_t>(row0 + m) * kb + k) : 0.f;
      }
      step_at(4, gt, gk);
    };
    fetch();
    bool have = true;
    int tile = tile0, k = k0, begin = k0;
    for (int i = 0; i < steps; ++i) {
      if ((i & 3) == 0) {
        sb = nb;
#pragma unroll
        for (int j = 0; j < kPer; ++j) cs[((i >> 2) & 1) * 4 * ROWS + lane + 32 * j] = na[j];
        __syncwarp();
        fetch();
      }
      const int buf = i % S::BUFS;
      if (have) have = __all_sync(0xFFFFFFFFu, wait_phase<false>(bar_acc_full + 8 * buf, (i / S::BUFS) & 1, wc, 0x05));
      tc_fence_after();
      const float4 *c4 = reinterpret_cast<const float4 *>(cs + ((i >> 2) & 1) * 4 * ROWS + (i & 3) * ROWS);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float sw = __shfl_sync(0xFFFFFFFFu, sb, 2 * (i & 3) + w);
        uint32_t v[ROWS / 16][16];
#pragma unroll
        for (int c = 0; c < ROWS / 16; ++c) tmem_ld_32x32b_x16(lane_addr + 2 * NT * buf + NT * w + 16 * c, v[c]);
#pragma unroll
        for (int c = 0; c < ROWS / 16; ++c) tmem_ld_done(v[c]);
        if (w == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acc_empty + 8 * buf);
        }
#pragma unroll
        for (int c = 0; c < ROWS / 16; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 f = c4[4 * c + e];
            float *a = acc[w] + 16 * c + 4 * e;
            a[0] = fmaf(__uint_as_float(v[c][4 * e + 0]), f.x * sw, a[0]);
            a[1] = fmaf(__uint_as_float(v[c][4 * e + 1]), f.y * sw, a[1]);
            a[2] = fmaf(__uint_as_float(v[c][4 * e + 2]), f.z * sw, a[2]);
            a[3] = fmaf(__uint_as_float(v[c][4 * e + 3]), f.w * sw, a[3]);
          }
      }
      if (++k < kb && i + 1 < steps) continue;
      // -------------------------------------------------------- the end of this
      // CTA's part [begin, k) of the column block
      const bool split = begin > 0 || k < kb;
      int64_t c0 = blockIdx.x, c1 = blockIdx.x;  // the CTAs that share the block
      if (split) {
        const int64_t first = static_cast<int64_t>(tile) * kb, end = first + kb;
        c0 = ((first + 1) * ctas - 1) / total;
        c1 = (end * ctas - 1) / total;
      }
      auto slot = [&](int64_t c) { return gp.partials + (2 * c + (c == c0)) * S::PARTIAL; };
      float *to = slot(blockIdx.x) + row0 * 128 + n;
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
          if (m < rows) to[(w * NT + m) * 128] = acc[w][m];
      if (split) __threadfence();
      all_warps();
      bool finish = true;
      if (split) {
        if (threadIdx.x == 64) {
          const bool mine = atomicAdd(gp.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
          if (mine) gp.counters[c0] = 0;  // for the next launch
          *last = mine;
        }
        all_warps();
        finish = *last != 0;
        if (finish) __threadfence();
      }
      if (finish && have) gated_skinny_rows<NT>(gp, slot, c0, c1, tile, warp - 2, lane);
      all_warps();  // the slot has been read
#pragma unroll
      for (int m = 0; m < ROWS; ++m) acc[0][m] = acc[1][m] = 0.f;
      ++tile;
      k = begin = 0;
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
