// cache_attention.cuh -- attention over the 8-bit key/value cache for few
// query rows (single tokens, short runs): bound by reading the codes once.
//
//   x_j = scale * q . k_j,  k_j = ks * K_j,  v_j = vs * V_j   (ks, vs per page)
//   o = sum_j e^(x_j) v_j / sum_j e^(x_j)
//
// A page's vs goes into the exponent: with w_j = 2^(x_j log2 e + log2 vs - m + 7),
// m the running maximum of that exponent,
//   o = (sum_j w_j V_j) / (2^7 sum_j 2^-7 w_j / vs_j):
// the weights that meet the codes in the tensor cores are at most 2^15 and the
// largest is near 2^7 whatever the pages' scales are, so FP16 holds them: with
// 11 bits down to 2^-21 of the largest, and to 2^-32 of it below, so that the many
// small weights of a long sequence count beside a large one.  FP16 also holds
// V's and K's codes, E4M3, exactly.  A row of Q is multiplied by a power of two
// that brings its largest value to 2^15 .. 2^16: its BF16 values are then exact in
// FP16 down to 2^-32 of that, and below they are off by 2^-40 of it at most.  Sums
// are FP32.
//
// Transposed: S^T = K Q^T and O^T = V^T P^T with mma.m16n8k16, so that 8
// query rows (the heads of a group) fill the MMA's narrow side and K and V,
// converted in registers, its 16-row side.  One warp takes tiles of 32 keys:
// TMA brings each page's rows, swizzled, into the warp's own ring of shared
// memory; no other warp waits for it.  Running maximum, sum and O stay in
// the warp until the end of its run.
//
// Measured: 64 sequences of 2048-8192 tokens, 64/8 heads of 128: 120 us (5.6
// TB/s, 0.83 of the measured copy rate); two of 91752 and 131071 tokens, 32/4 heads:
// 54 us (4.2 TB/s: some 50 CTAs' partials join for each item, about 8 us, and the
// first codes arrive 3 us after the start).  The warps' chains of dependent
// instructions bound it: issue slots are used to 46 %.
//
// Behind shared tokens (kOwnKeys) the ranges are of warps and not of CTAs, and what they
// leave is added by the launch that joins: 64 sequences of 100-982 own keys, 64/8 heads,
// 22-24 us where all keys by ranges of CTAs take 36, and 34 us on the 72 SMs that the
// launch over the shared keys leaves.
//
// Work: an item is one sequence, key/value head and ROWS query rows; all
// items' tiles, laid end to end, are cut into equal ranges, one per CTA, or,
// where items are few, each one's into parts for CTAs of its own.  An item
// that spans CTAs leaves FP32 partials in the workspace and the CTA that
// arrives last adds them, in order: the result does not depend on timing.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_common.cuh"
#include "ring.h"

namespace mxg {

struct AttnParams {
  CacheView c;
  BatchView b;
  const __nv_bfloat16 *Q;
  int64_t q_pitch;
  int heads, group;  // query heads, query heads per key/value head
  float scale;
  int causal;
  int64_t window, sinks;
  __nv_bfloat16 *O;
  float *lse;
  float *partials;     // of split items: two slots per CTA (prompts: one for each part)
  unsigned *counters;  // arrivals at split items, zero between launches
  int items, whole;    // prompts: row tiles (all heads'), and how many of them, the first, have one CTA each
  int parts;           // CTAs that each other one's keys may be cut for
  unsigned long long timeout_ns;
  int stall_producer;  // tests: nothing is loaded
  // attention behind shared tokens: keys [0, shared), a multiple of 32 and of the
  // pages, are one launch's, which leaves partials in `left`, `left_parts` of each row
  // tile, numbered as its CTAs; the others are another's, which leaves its sums of
  // each row (token x head) in `own` and `own_ml`, or in partials of several warps,
  // and in `own_at` (null: none is) which: the first one (-1: none), and 16 times how
  // many more there are plus the row in them; a third joins all
  int shared;
  float *left, *own;
  float2 *own_ml;
  int2 *own_at;
  int own_rows;  // of a partial
  int beside_blocks;     // CTAs of the second launch that work where there are few own keys:
  int64_t beside_tiles;  // `beside_tiles` tiles of 32 or fewer (-1: all always work)
  unsigned *begun;  // set by the first launch while the second runs
  int left_parts, left_tiles;  // parts of a row tile, row tiles of a key/value head
};

// Rows of a row tile of the kernel for prompts, and a partial of it: sums of O by
// 4 d and row, then maximum and sum of each row.
constexpr int kTileRows = 256;
template <int D>
constexpr int kTilePartial = kTileRows * (D + 2);

// What a launch computes: all keys; the shared ones for all tokens; the others.
constexpr int kAllKeys = 0, kSharedKeys = 1, kOwnKeys = 2;

// Before a launch reads global memory.  The one over the own keys comes behind the one
// over the shared keys, needs nothing of it and does not wait for it to end.  What came
// before both is in order for it by a word of the handle: a thread of the first launch,
// which has waited, sets it with a release, and every thread of this one reads it with
// an acquire, behind which no older line of the SM's is read; the fence carries that
// over to the codes' copies.  (The first launch sets it before it lets this one begin,
// but for its block's other warps: a wait of some ns, bounded as the others are.  The
// launch that joins clears it.)
template <int MODE>
__device__ __forceinline__ void start_after(const AttnParams &p) {
  if constexpr (MODE == kOwnKeys) {
    auto begun = [&]() {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p.begun) : "memory");
      return v != 0;
    };
    if (!begun()) {
      const uint64_t t0 = globaltimer_ns();
      while (!begun())
        if (globaltimer_ns() - t0 > p.timeout_ns) {
          if (atomicCAS(p.b.status, 0, 6) == 0) atomicExch(p.b.status + 1, 0x32);
          break;
        }
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");
    __syncwarp();
  } else {
    griddep_wait();
    if (MODE == kSharedKeys && blockIdx.x == 0 && threadIdx.x == 0)
      asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.begun), "r"(1u) : "memory");
  }
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two E4M3 codes (the low or the high half of w) as FP16.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async4_cache(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Exponent of the power of two for a row of Q whose largest magnitude is `top`
// (0 for a row of zeros; 2^126 is the largest, whose reciprocal is normal).
__device__ __forceinline__ int q_exponent(float top) {
  return top > 0.f ? min(142 - (__float_as_int(top) >> 23), 126) : 0;
}
__device__ __forceinline__ float pow2(int k) { return __int_as_float((127 + k) << 23); }

// 1 / vs from log2 vs as it went into the exponents, whose error (2^-22 of the
// logarithm) then drops out of the sums of weights.
__device__ __forceinline__ float inverse_of_log2(float lv) { return ex2(-lv); }
// The natural logarithm of a row's sum of weights, 2^m times `sum`; -inf where it saw
// no key.  The sum's power of two is taken apart: lg2's error is 2^-22 near 1, and 2^-22
// of the result elsewhere.
__device__ __forceinline__ float log_sum(float m, float sum) {
  const int k = min((__float_as_int(sum) >> 23) - 127, 126);
  return sum == 0.f ? -INFINITY : (m + static_cast<float>(k) + lg2(sum * pow2(-k))) * 0.69314718055994530942f;
}

constexpr float kWeightUp = 7.f, kWeightDown = 0.0078125f;  // weights carry 2^7, and sums give it back

constexpr float kScaleFloor = 7.8886090522101180541e-31f;  // 2^-100, for 1 / vs

// Which keys of a sequence any of its queries sees, as tiles of 32: `ns` tiles
// of first tokens from key 0, then the tiles from tile `lo` on, `tiles` in all
// (one at least, so that a sequence without keys still has its zeros written).
struct KeyTiles {
  int ns, lo, tiles;
  int end;       // keys >= end are seen by no query
  int win_lo;    // keys < win_lo are seen only as first tokens
};

template <int MODE>
__device__ __forceinline__ KeyTiles key_tiles(const AttnParams &p, const Sequence &s) {
  KeyTiles k;
  if constexpr (MODE == kOwnKeys) {
    k.end = s.n > 0 && s.len > p.shared ? s.len : 0;  // (a sequence that is within the shared tokens has none)
    k.win_lo = k.end ? p.shared : 0;
    k.lo = k.win_lo >> 5;
    k.ns = 0;
    k.tiles = max(1, ((k.end + 31) >> 5) - k.lo);
    return k;
  }
  const int64_t first = static_cast<int64_t>(s.len) - s.n;  // position of the first query
  k.end = s.n > 0 ? s.len : 0;  // (the last query stands at len - 1)
  int64_t lo = 0;
  if (p.window > 0) lo = max(static_cast<int64_t>(0), first - p.window + 1);
  k.win_lo = static_cast<int>(min(lo, static_cast<int64_t>(k.end)));
  k.lo = k.win_lo >> 5;
  k.ns = static_cast<int>(min((min(p.sinks, static_cast<int64_t>(k.win_lo)) + 31) >> 5, static_cast<int64_t>(k.lo)));
  k.tiles = max(1, k.ns + ((k.end + 31) >> 5) - k.lo);
  return k;
}

// Items of sequence s: row tiles x key/value heads.
__device__ __forceinline__ int64_t item_count(const AttnParams &p, const Sequence &s, int rows) {
  return ((static_cast<int64_t>(s.n) * p.group + rows - 1) >> (rows == 8 ? 3 : 4)) * p.c.kv_heads;
}

// a / b for a >= 0, b > 0: in 32 bits where both fit, as they mostly do.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Position in the flat order of tiles: a sequence, and in it an item.
template <int MODE>
struct Cursor {
  int b;
  Sequence s;
  KeyTiles k;
  int64_t beg;    // the item's first tile
  int64_t items;  // of the sequence
  int64_t item;
  int h;          // the item's key/value head

  // the item of tile x, in sequence b_ whose tiles begin at `base`
  __device__ void start(const AttnParams &p, int rows, int b_, int64_t base, int64_t x) {
    b = b_;
    enter(p, rows);
    item = quotient(x - base, k.tiles);
    beg = base + item * k.tiles;
    h = static_cast<int>(item - quotient(item, p.c.kv_heads) * p.c.kv_heads);
  }
  // forward to the item of tile x (below the total)
  __device__ void to(const AttnParams &p, int rows, int64_t x) {
    while (x >= beg + k.tiles) {
      beg += k.tiles;
      if (++item == items) {
        do {
          ++b;
          enter(p, rows);
        } while (items == 0);
        item = 0;
        h = 0;
      } else if (++h == p.c.kv_heads) {
        h = 0;
      }
    }
  }
  __device__ void enter(const AttnParams &p, int rows) {
    s = load_sequence<MODE == kOwnKeys>(p.b, p.c, b);
    k = key_tiles<MODE>(p, s);
    items = item_count(p, s, rows);
  }
  // first key of tile x of the item
  __device__ int key(int64_t x) const {
    const int tile = static_cast<int>(x - beg);
    return (tile < k.ns ? tile : k.lo + tile - k.ns) * 32;
  }
};

// Items of sequence b (none past the batch), and tiles of each.
template <int MODE>
__device__ __forceinline__ int64_t sequence_items(const AttnParams &p, int rows, int b, int &tiles) {
  tiles = 1;
  if (b >= p.b.batch) return 0;
  const Sequence s = load_sequence<MODE == kOwnKeys>(p.b, p.c, b);
  tiles = key_tiles<MODE>(p, s).tiles;
  return item_count(p, s, rows);
}
__device__ __forceinline__ int64_t warp_prefix(int64_t v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

template <int D, int NT>
struct DecodeCfg {
  static constexpr int ROWS = 8 * NT;  // query rows of an item
  static constexpr int WARPS = 4;
  static constexpr int TILE = 32;
  static constexpr int STAGE = 2 * TILE * D;              // K, then V
  // CTAs of an SM: three where the registers allow it (the warps' chains of
  // dependent instructions bound them, more warps hide them), with two tiles of
  // 8 KB in flight for each warp, else two with three
  static constexpr int CTAS = NT == 1 ? 3 : 2;
  static constexpr int STAGES = (CTAS == 3 ? 2 : 3) * 128 / D;
  static constexpr int OFF_MERGE = WARPS * STAGES * STAGE;  // [warp][8 rows][64] floats
  static constexpr int OFF_ML = OFF_MERGE + WARPS * 8 * 64 * 4;  // m and l: [2][warp][ROWS]
  static constexpr int OFF_SC = OFF_ML + 2 * WARPS * ROWS * 4;   // [warp][stage][K, V][2 pages] scales
  static constexpr int OFF_PG = OFF_SC + WARPS * STAGES * 16;    // [warp][stage][2] whether the page is there
  static constexpr int OFF_BAR = OFF_PG + WARPS * STAGES * 8;
  static constexpr int OFF_MISC = OFF_BAR + WARPS * STAGES * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 192 + 1024;
  static constexpr int PARTIAL = ROWS * (D + 2);  // floats of a partial: O, m, l
  static_assert(CTAS * (SMEM_BYTES + 1024) <= 233472, "CTAs per SM");
};

template <int D, int NT, int MODE>
__global__ void __launch_bounds__(128, DecodeCfg<D, NT>::CTAS)
    cache_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const AttnParams p) {
  using S = DecodeCfg<D, NT>;
  constexpr int ROWS = S::ROWS, STAGES = S::STAGES, KW = D / 16;  // 32-bit words of a K row per thread
  constexpr int MT = D / 16;                                      // 16-row tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = base + warp * STAGES * S::STAGE;
  const uint32_t bars = base + S::OFF_BAR + warp * STAGES * 8;
  float *sc = reinterpret_cast<float *>(sm + S::OFF_SC) + warp * STAGES * 4;
  int *pg_ok = reinterpret_cast<int *>(sm + S::OFF_PG) + warp * STAGES * 2;
  float *merge = reinterpret_cast<float *>(sm + S::OFF_MERGE);
  float *ml = reinterpret_cast<float *>(sm + S::OFF_ML);
  int *last_at = reinterpret_cast<int *>(sm + S::OFF_MISC);
  // Attention behind shared tokens: each warp is a unit of its own, whose sums go to
  // the workspace without a barrier (items of single tiles, 512 of them: 20 us with
  // units of a CTA, 4.5 us of them an item's end).  Else a unit is a CTA.
  constexpr bool kWarps = MODE == kOwnKeys;
  constexpr int kStep = kWarps ? 1 : 4;  // from a warp's tile to its next
  // (its last CTA does nothing but wait for the launch over the shared keys, so that
  // the launch that joins need not)
  if (MODE == kOwnKeys && blockIdx.x == gridDim.x - 1) {
    griddep_wait();
    return;
  }
  int64_t blocks = gridDim.x - (MODE == kOwnKeys ? 1 : 0);
  // how tiles are cut: all of them and the units that share them, or 0 and the
  // first and the last unit of this one's item; then the range's first tile
  // (kept here: registers are short)
  int64_t *cut = reinterpret_cast<int64_t *>(sm + S::OFF_MISC + 8) + (kWarps ? 4 * warp : 0);
  const bool cuts = kWarps ? lane == 0 : threadIdx.x == 0;

  if (lane == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 33);  // the bytes' arrive, and the lanes' copies
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  if (MODE != kOwnKeys) griddep_launch_dependents();  // (the launch that joins is kept away: see there)
  start_after<MODE>(p);
  // All tiles (each warp counts for itself, 32 sequences at a time), and this
  // CTA's range of them: ranges of four tiles at least.
  int mt;
  int64_t mi = sequence_items<MODE>(p, ROWS, lane, mt);
  int64_t mine = mi * mt, upto = warp_prefix(mine);  // the first 32 sequences
  int64_t total = __shfl_sync(0xFFFFFFFFu, upto, 31);
  unsigned all_items = __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(mi));
  for (int b = 32; b < p.b.batch; b += 32) {
    int tiles;
    const int64_t items = sequence_items<MODE>(p, ROWS, b + lane, tiles);
    total += __shfl_sync(0xFFFFFFFFu, warp_prefix(items * tiles), 31);
    all_items += __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(items));
  }
  // (no more keys than the SMs beside the launch over the shared keys take in its time:
  // by the CTAs that start there, and the others have none)
  if (MODE == kOwnKeys && total <= p.beside_tiles) {
    blocks = p.beside_blocks;
    if (blockIdx.x >= blocks) return;
  }
  const int64_t unit = kWarps ? warp * blocks + blockIdx.x : blockIdx.x;
  const int64_t units_most = kWarps ? 4 * blocks : blocks;
  // the sequence of the range's first tile, and where its tiles begin
  int b0 = 0;
  int64_t base_b = 0, x0, x1;
  auto next_sequences = [&]() {  // the next 32
    base_b += __shfl_sync(0xFFFFFFFFu, upto, 31);
    b0 += 32;
    mi = sequence_items<MODE>(p, ROWS, b0 + lane, mt);
    mine = mi * mt;
    upto = warp_prefix(mine);
  };
  const int64_t ctas = min(units_most, (total + kStep - 1) / kStep);
  // Few items: each one's tiles are cut for CTAs of its own, into parts of q tiles
  // at most, since a CTA that ends two items' parts ends late (17 tiles for
  // each of 8 heads: 16.5 -> 10.8 us).  And no more parts than pay: one costs
  // the join 0.12 us, four tiles more a CTA 2 us, which is least at parts of
  // sqrt(0.24 tiles) (one head of 20000 keys: 27.2 -> 18 us).
  const bool own = 4 * static_cast<int64_t>(all_items) <= units_most;
  if (own) {
    const int64_t room = units_most - all_items, q = max(static_cast<int64_t>(kWarps ? 2 : 4), quotient(total + room - 1, room));
    auto parts_of = [&](int tiles) {
      const int64_t n = max(q, static_cast<int64_t>(sqrtf(0.24f * tiles)));
      return quotient(tiles + n - 1, n);
    };
    int64_t base_u = 0, units, u;
    uint32_t past;
    for (;;) {
      units = mi * parts_of(mt);
      u = warp_prefix(units);
      past = __ballot_sync(0xFFFFFFFFu, base_u + u > unit);
      if (past) break;
      if (b0 + 32 >= p.b.batch) return;
      base_u += __shfl_sync(0xFFFFFFFFu, u, 31);
      next_sequences();
    }
    const int i = __ffs(past) - 1;
    base_u += __shfl_sync(0xFFFFFFFFu, u - units, i);
    base_b += __shfl_sync(0xFFFFFFFFu, upto - mine, i);
    b0 += i;
    const int tiles = __shfl_sync(0xFFFFFFFFu, mt, i);
    const int64_t parts = parts_of(tiles), rel = unit - base_u, item = quotient(rel, parts), part = rel - item * parts;
    x0 = base_b + item * tiles + quotient(part * tiles, parts);
    x1 = base_b + item * tiles + quotient((part + 1) * tiles, parts);
    if (cuts) {
      cut[0] = 0;
      cut[1] = unit - part;
      cut[2] = unit - part + parts - 1;
    }
  } else {
    if (unit >= ctas) return;
    auto first_tile = [&](int64_t u) { return quotient(u * total, ctas); };
    x0 = first_tile(unit);
    x1 = first_tile(unit + 1);
    uint32_t past;
    while (!(past = __ballot_sync(0xFFFFFFFFu, base_b + upto > x0))) next_sequences();
    const int i = __ffs(past) - 1;
    base_b += __shfl_sync(0xFFFFFFFFu, upto - mine, i);
    b0 += i;
    if (cuts) {
      cut[0] = total;
      cut[1] = ctas;
    }
  }

  if (cuts) cut[3] = x0;
  if (kWarps) __syncwarp();

  const int lg = p.c.page_log2, per = lg == 4 ? 2 : 1;  // pages of a tile
  const uint32_t box_bytes = (lg == 4 ? 16 : 32) * D;
  // ------------------------------------------------------------ loads
  Cursor<MODE> at, in;  // of the item being computed, and of the next tile to load
  at.start(p, ROWS, b0, base_b, x0);
  in = at;
  auto issue = [&](int64_t x, int st) {
    in.to(p, ROWS, x);
    const int h = in.h, key0 = in.key(x);
    int pg = -1;
    // (a page of which no query sees a key is left alone: a window may have passed it)
    const int k0 = key0 + 16 * lane;
    if (lane < per && k0 < in.k.end && (k0 + 32 / per > in.k.win_lo || k0 < p.sinks)) pg = load_page<MODE == kOwnKeys>(p.b, p.c, in.b, k0 >> lg);
    const uint32_t bar = bars + 8 * st;
    const uint32_t there = __ballot_sync(0xFFFFFFFFu, pg >= 0);
    if (lane < per) {
      pg_ok[2 * st + lane] = pg >= 0;
      const int64_t cell = static_cast<int64_t>(pg) * p.c.kv_heads + h;
      if (pg >= 0) {
        cp_async4_cache(smem_u32(sc + 4 * st + lane), p.c.K_scale + cell);
        cp_async4_cache(smem_u32(sc + 4 * st + 2 + lane), p.c.V_scale + cell);
      }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * box_bytes * __popc(there));
    __syncwarp();
    if (pg >= 0) {
      const int row = (pg * p.c.kv_heads + h) * p.c.page_size + (key0 & (p.c.page_size - 1));
      const uint32_t dst = ring + st * S::STAGE + lane * 16 * D;
      tma_load_2d(dst, &tmK, 0, row, bar);
      tma_load_2d(dst + 32 * D, &tmV, 0, row, bar);
    }
  };
  // Q of the item at `at`, as it lies: thread (g, t) has rows g of each 8,
  // d = (D/4) t .. + D/4 - 1; rows past the last are zero
  uint4 qraw[NT][D / 32];
  auto load_q = [&]() {
    const int row0 = static_cast<int>(quotient(at.item, p.c.kv_heads)) * ROWS;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + 8 * n + g;
      const bool live = r < at.s.n * p.group;
      const int tok = r / p.group, hd = at.h * p.group + r % p.group;
      const uint4 *src = reinterpret_cast<const uint4 *>(p.Q + static_cast<int64_t>(at.s.first + tok) * p.q_pitch +
                                                         static_cast<int64_t>(hd) * D + t * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) qraw[n][i] = live ? (MODE == kOwnKeys ? __ldcg(src + i) : __ldg(src + i)) : make_uint4(0, 0, 0, 0);
    }
  };
  load_q();
  // bounded wait (whole warp): the loads of this stage have landed
  auto wait_stage = [&](int st, uint32_t ph, unsigned long long limit) -> bool {
    bool ok = mbar_try_wait(bars + 8 * st, ph);
    if (!ok) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = 1; !(ok = mbar_try_wait(bars + 8 * st, ph)); ++i)
        if ((i & 31u) == 0 && globaltimer_ns() - t0 > limit) {
          if (atomicCAS(p.b.status, 0, 6) == 0) atomicExch(p.b.status + 1, 0x31);
          break;
        }
    }
    return __all_sync(0xFFFFFFFFu, ok);
  };
  const int mine_at = kWarps ? 0 : warp;
  int64_t px = x0 + mine_at;  // next tile to load
  int pst = 0;
  for (int i = 0; i < STAGES && px < x1 && !p.stall_producer; ++i, px += kStep) {
    issue(px, pst);
    pst = pst + 1 == STAGES ? 0 : pst + 1;
  }

  // ------------------------------------------------------------ items
  int64_t x = x0 + mine_at;  // this warp's next tile
  int st = 0;
  uint32_t ph = 0;
  bool alive = true;
  for (int64_t seg = x0; seg < x1;) {
    const int64_t item_beg = at.beg, item_end = item_beg + at.k.tiles;
    const int64_t seg_end = min(item_end, x1);
    const int h = at.h;
    const int row0 = static_cast<int>(quotient(at.item, p.c.kv_heads)) * ROWS;  // row = token * group + head of the group
    const int rows = min(ROWS, at.s.n * p.group - row0);
    const int pos0 = at.s.len - at.s.n;

    // Q in the order of K's words
    uint32_t q[NT][KW][2];
    float cq[NT][2];  // logits of this lane's columns 2t, 2t+1: S * cq
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 (&w)[D / 32] = qraw[n];
      const uint32_t *u = reinterpret_cast<const uint32_t *>(w);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[i] << 16)), fabsf(__uint_as_float(u[i] & 0xFFFF0000u))));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int e = q_exponent(top);
      const float up = pow2(e);
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t b = u[2 * i + c];
          q[n][i][c] = half2_of(__uint_as_float(b << 16) * up, __uint_as_float(b & 0xFFFF0000u) * up);
        }
      const float c = p.scale * 1.44269504088896340736f * pow2(-e);
      cq[n][0] = __shfl_sync(0xFFFFFFFFu, c, 8 * t);
      cq[n][1] = __shfl_sync(0xFFFFFFFFu, c, 8 * t + 4);
    }
    // positions of this lane's columns, and of all rows
    int pos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) pos[n][c] = pos0 + (row0 + min(8 * n + 2 * t + c, rows - 1)) / p.group;
    const int pos_lo = pos0 + row0 / p.group, pos_hi = pos0 + (row0 + rows - 1) / p.group;

    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    for (; x < seg_end; x += kStep) {
      const int key0 = at.key(x);
      if (alive) alive = wait_stage(st, ph, p.timeout_ns);
      const uint32_t kb = ring + st * S::STAGE, vb = kb + 32 * D;
      // S^T: keys 16 mt + g (+ 8) x rows; two sums for the halves of D, so that
      // chains of dependent MMAs are half as long
      float s[2][NT][4], s1[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][n][j] = s1[mt][n][j] = 0.f;
#pragma unroll
      for (int c = 0; c < KW / 4; ++c) {
        uint4 k0[2], k1[2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int ra = 16 * mt + g, rb = ra + 8, ch = (KW / 4) * t + c;  // 16-byte chunk of the row
          k0[mt] = ld_shared_v4(kb + ra * D + ((ch ^ (D == 128 ? ra & 7 : (ra >> 1) & 3)) << 4));
          k1[mt] = ld_shared_v4(kb + rb * D + ((ch ^ (D == 128 ? rb & 7 : (rb >> 1) & 3)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint32_t a = i == 0 ? k0[mt].x : i == 1 ? k0[mt].y : i == 2 ? k0[mt].z : k0[mt].w;
            const uint32_t b = i == 0 ? k1[mt].x : i == 1 ? k1[mt].y : i == 2 ? k1[mt].z : k1[mt].w;
            const uint32_t a0 = e4m3_lo(a), a1 = e4m3_lo(b), a2 = e4m3_hi(a), a3 = e4m3_hi(b);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_f16((i & 1) ? s1[mt][n] : s[mt][n], a0, a1, a2, a3, q[n][4 * c + i][0], q[n][4 * c + i][1]);
          }
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][n][j] += s1[mt][n][j];
      // exponents; ivs = 2^-7 / vs
      const bool ok0 = pg_ok[2 * st] != 0, ok1 = per == 2 ? pg_ok[2 * st + 1] != 0 : ok0;
      float ivs[2];
      const int jlast = key0 + 31;
      const bool whole = ok0 && ok1 && jlast < at.k.end && (!p.causal || jlast <= pos_lo) &&
                         (p.window == 0 || pos_hi - key0 < p.window || jlast < p.sinks);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float ks = sc[4 * st + (per == 2 ? mt : 0)], vs = sc[4 * st + 2 + (per == 2 ? mt : 0)];
        const float v1 = fmaxf(vs, kScaleFloor), lv = lg2(v1);
        ivs[mt] = inverse_of_log2(lv) * kWeightDown;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][n][j] = fmaf(s[mt][n][j], cq[n][j & 1] * ks, lv);
      }
      if (!whole) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key0 + 16 * mt + g + 8 * (j >> 1), ps = pos[n][j & 1];
              const bool seen = (mt ? ok1 : ok0) && key < at.k.end && (!p.causal || key <= ps) &&
                                (p.window == 0 || ps - key < p.window || key < p.sinks);
              if (!seen) s[mt][n][j] = -INFINITY;
            }
      }
      // running maximum, moved only when it grows by 2^8
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float top[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[c] = fmaxf(fmaxf(s[0][n][c], s[0][n][c + 2]), fmaxf(s[1][n][c], s[1][n][c + 2]));
          top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 4));
          top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 8));
          top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 16));
        }
        if (__any_sync(0xFFFFFFFFu, top[0] > m[n][0] + 8.f || top[1] > m[n][1] + 8.f)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float mn = fmaxf(m[n][c], top[c]);
            const float f = mn == -INFINITY ? 1.f : ex2(m[n][c] - mn);
            m[n][c] = mn;
            l[n][c] *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[n][i][c] *= f;
              o[n][i][c + 2] *= f;
            }
          }
        }
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - kWeightUp, m1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - kWeightUp;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const float w0 = ex2(s[mt][n][0] - m0), w1 = ex2(s[mt][n][1] - m1);
          const float w2 = ex2(s[mt][n][2] - m0), w3 = ex2(s[mt][n][3] - m1);
          l[n][0] = fmaf(w0 + w2, ivs[mt], l[n][0]);
          l[n][1] = fmaf(w1 + w3, ivs[mt], l[n][1]);
          pb[mt][n][0] = transpose8x8(half2_of(w0, w1));
          pb[mt][n][1] = transpose8x8(half2_of(w2, w3));
        }
      }
      // O^T += V^T P^T: thread (g, t) has keys 2t, 2t+1, 2t+8, 2t+9 of each 16 and
      // d = (D/8) g .. + D/8 - 1
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * mt + 2 * t + (i & 1) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 a = ld_shared_v4(vb + r * D + ((g ^ (r & 7)) << 4));
            v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
          } else {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(v[i][0]), "=r"(v[i][1])
                         : "r"(vb + r * D + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + 8 * (g & 1))
                         : "memory");
          }
          if (!whole) {
            // codes of keys that no row sees may be anything: 0 * NaN is NaN
            const int key = key0 + r;
            const bool used = (mt ? ok1 : ok0) && key < at.k.end && (key >= at.k.win_lo || key < p.sinks);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[i][w] = used ? v[i][w] : 0u;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t a = __byte_perm(v[0][w], v[1][w], 0x5140), b = __byte_perm(v[2][w], v[3][w], 0x5140);
          const uint32_t c = __byte_perm(v[0][w], v[1][w], 0x7362), d = __byte_perm(v[2][w], v[3][w], 0x7362);
          const uint32_t a0 = e4m3_lo(a), a1 = e4m3_hi(a), a2 = e4m3_lo(b), a3 = e4m3_hi(b);
          const uint32_t c0 = e4m3_lo(c), c1 = e4m3_hi(c), c2 = e4m3_lo(d), c3 = e4m3_hi(d);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(o[n][2 * w], a0, a1, a2, a3, pb[mt][n][0], pb[mt][n][1]);
            mma_f16(o[n][2 * w + 1], c0, c1, c2, c3, pb[mt][n][0], pb[mt][n][1]);
          }
        }
      }
      // this stage's reads come before the next load into it
      fence_proxy_async_smem();
      __syncwarp();
      if (alive && px < x1) {
        issue(px, st);
        px += kStep;
      }
      if (++st == STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }

    // ---------------------------------------------------------- the unit's result
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 4);
        l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 8);
        l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 16);
        if (!kWarps && g == 0) {
          ml[warp * ROWS + 8 * n + 2 * t + c] = m[n][c];
          ml[(4 + warp) * ROWS + 8 * n + 2 * t + c] = l[n][c];
        }
      }
    const bool split = item_beg < cut[3] || item_end > x1;
    // the CTAs that share the item
    int64_t u0 = 0, u1 = 0;
    if (split) {
      const int64_t all = cut[0], n = cut[1];
      u0 = all ? quotient((item_beg + 1) * n - 1, all) : n;
      u1 = all ? quotient(item_end * n - 1, all) : cut[2];
    }
    if constexpr (kWarps) {
      // thread (g, t) has rows 2t, 2t + 1 of each eight and d = (D/8) g .. + D/8 - 1
      constexpr int kQuads = D / 32;
      float *part = p.partials + (2 * unit + (unit == u0)) * S::PARTIAL;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = 8 * n + 2 * t + c;
          if (r >= rows) continue;
          const int64_t row = static_cast<int64_t>(at.s.first + (row0 + r) / p.group) * p.heads + h * p.group + (row0 + r) % p.group;
          float *to = (split ? part + r * D : p.own + row * D) + (D / 8) * g;
#pragma unroll
          for (int k = 0; k < kQuads; ++k)
            reinterpret_cast<float4 *>(to)[k] = make_float4(o[n][2 * k][c], o[n][2 * k][c + 2], o[n][2 * k + 1][c], o[n][2 * k + 1][c + 2]);
          if (g == 0) {
            if (split) {
              part[ROWS * D + r] = m[n][c];
              part[ROWS * D + ROWS + r] = l[n][c];
            } else {
              p.own_ml[row] = make_float2(m[n][c], l[n][c]);
            }
            if (!split || unit == u0) p.own_at[row] = split ? make_int2(static_cast<int>(u0), static_cast<int>(u1 - u0) * 16 + r) : make_int2(-1, 0);
          }
        }
    } else {
    __syncthreads();
    float *part = p.partials + (2 * static_cast<int64_t>(blockIdx.x) + (blockIdx.x == u0)) * S::PARTIAL;
    const int hr = threadIdx.x >> 4, hd = threadIdx.x & 15;  // output: row of 8, four of 64 d
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // this warp's sums over the maximum of the four
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n + 2 * t + c;
        const float top = fmaxf(fmaxf(ml[r], ml[ROWS + r]), fmaxf(ml[2 * ROWS + r], ml[3 * ROWS + r]));
        f[c] = m[n][c] == -INFINITY ? 0.f : ex2(m[n][c] - top);
      }
      const int r = 8 * n + hr;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w * ROWS + r]);
#pragma unroll
      for (int w = 0; w < 4; ++w)  // (a sum of NaN stays one, also where no weight gave a maximum)
        sum = fmaf(ml[(4 + w) * ROWS + r], ml[w * ROWS + r] == -INFINITY ? 0.f : ex2(ml[w * ROWS + r] - top), sum);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        __syncthreads();
        // d = (D/8) g + 2 i (+ 1): the lanes whose d lie in this 64
        if (D == 64 || (g >> 2) == e) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < MT; ++i)
              *reinterpret_cast<float2 *>(merge + (warp * 8 + 2 * t + c) * 64 + ((D / 8) * g + 2 * i) % 64) =
                  make_float2(o[n][i][c] * f[c], o[n][i][c + 2] * f[c]);
        }
        __syncthreads();
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 b = *reinterpret_cast<const float4 *>(merge + (w * 8 + hr) * 64 + 4 * hd);
          a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        const int d = 64 * e + 4 * hd;
        if (split) {
          *reinterpret_cast<float4 *>(part + r * D + d) = a;
        } else if (r < rows) {
          const float k = sum == 0.f ? 0.f : kWeightDown / sum;
          const int tok = at.s.first + (row0 + r) / p.group, head = h * p.group + (row0 + r) % p.group;
          const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * k, a.y * k), hi = __floats2bfloat162_rn(a.z * k, a.w * k);
          *reinterpret_cast<uint2 *>(p.O + (static_cast<int64_t>(tok) * p.heads + head) * D + d) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
      }
      if (hd == 0) {
        if (split) {
          part[ROWS * D + r] = top;
          part[ROWS * D + ROWS + r] = sum;
        } else if (r < rows && p.lse) {
          const int tok = at.s.first + (row0 + r) / p.group, head = h * p.group + (row0 + r) % p.group;
          p.lse[static_cast<int64_t>(tok) * p.heads + head] = log_sum(top, sum);
        }
      }
    }
    // ---------------------------------------------------------- split items
    if (split) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0)
        *last_at = atomicAdd(p.counters + u0, 1u) == static_cast<unsigned>(u1 - u0);
      __syncthreads();
      if (*last_at) {
        if (threadIdx.x == 0) p.counters[u0] = 0;  // for the next launch
        __threadfence();
        auto slot = [&](int64_t u) { return p.partials + (2 * u + (u == u0)) * S::PARTIAL; };
        // 16 threads a row; they take the contributors' m and l 16 at a time
        for (int rr = hr; rr < ROWS; rr += 8) {
          float top = -INFINITY, sum = 0.f;
          for (int64_t u = u0 + hd; u <= u1; u += 16) top = fmaxf(top, __ldcg(slot(u) + ROWS * D + rr));
#pragma unroll
          for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          float4 a[D / 64];
#pragma unroll
          for (int e = 0; e < D / 64; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int64_t v = u0; v <= u1; v += 16) {
            float kv = 0.f;
            if (v + hd <= u1) {
              const float mu = __ldcg(slot(v + hd) + ROWS * D + rr);
              kv = mu == -INFINITY ? 0.f : ex2(mu - top);
              sum = fmaf(__ldcg(slot(v + hd) + ROWS * D + ROWS + rr), kv, sum);
            }
#pragma unroll 8
            for (int i = 0; i < 16; ++i) {
              const float k = __shfl_sync(0xFFFFFFFFu, kv, (lane & 16) + i);
              const float *from = slot(min(v + i, u1)) + rr * D + 4 * hd;
#pragma unroll
              for (int e = 0; e < D / 64; ++e) {
                const float4 b = __ldcg(reinterpret_cast<const float4 *>(from + 64 * e));
                a[e].x = fmaf(b.x, k, a[e].x); a[e].y = fmaf(b.y, k, a[e].y);
                a[e].z = fmaf(b.z, k, a[e].z); a[e].w = fmaf(b.w, k, a[e].w);
              }
            }
          }
#pragma unroll
          for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
          if (rr >= rows) continue;
          const int tok = at.s.first + (row0 + rr) / p.group, head = h * p.group + (row0 + rr) % p.group;
          const float k = sum == 0.f ? 0.f : kWeightDown / sum;
#pragma unroll
          for (int e = 0; e < D / 64; ++e) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(a[e].x * k, a[e].y * k), hi = __floats2bfloat162_rn(a[e].z * k, a[e].w * k);
            *reinterpret_cast<uint2 *>(p.O + (static_cast<int64_t>(tok) * p.heads + head) * D + 64 * e + 4 * hd) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
          }
          if (hd == 0 && p.lse)
            p.lse[static_cast<int64_t>(tok) * p.heads + head] = log_sum(top, sum);
        }
      }
    }
    }
    seg = seg_end;
    if (seg < x1) {
      at.to(p, ROWS, seg);
      load_q();
    }
    if (!kWarps) __syncthreads();  // ml and merge are free for the next item
  }
  // after a wait that gave up: loads still on their way land first
  if (!alive) {
    const int64_t issued = (px - (cut[3] + mine_at)) / kStep;
    for (int64_t i = ring_pending(issued, STAGES); i < issued; ++i)
      wait_stage(static_cast<int>(i % STAGES), ring_parity(i, STAGES), landing_limit(p.timeout_ns));
  }
}

}  // namespace mxg
