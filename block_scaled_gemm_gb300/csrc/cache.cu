// cache.cu -- the 8-bit key/value cache: argument checks and launches of
// mxgemm_cache_append and mxgemm_cache_attention.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "cache_append.cuh"
#include "cache_attention.cuh"
#include "cache_join.cuh"
#include "cache_prompt.cuh"
#include "context.h"
#include "launch.h"
#include "mxgemm.h"

namespace {

using mxg::aligned;
using mxg::kLim;

// The checks that both entry points share; fills the kernels' views.
int cache_args(const mxg::HandleView &v, const mxgemm_cache_t *c, int64_t batch, const int32_t *table,
               int64_t table_pitch, const int32_t *kv_len, const int32_t *q_start, int64_t tokens,
               mxg::CacheView *cv, mxg::BatchView *bv) {
  if (!c || batch < 0 || batch >= (1 << 20) || tokens < 0 || tokens >= kLim || table_pitch < 0)
    return MXGEMM_ERR_INVALID_VALUE;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return MXGEMM_ERR_INVALID_VALUE;
  if (c->head_dim != 64 && c->head_dim != 128) return MXGEMM_ERR_INVALID_VALUE;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || c->num_pages < 0 || c->num_pages >= kLim)
    return MXGEMM_ERR_INVALID_VALUE;
  // (positions of whole tiles, and rows of query tokens x heads, stay below 2^31)
  if (table_pitch >= kLim || table_pitch * c->page_size > kLim / 2 ||
      c->num_pages * c->kv_heads >= kLim / c->page_size)
    return MXGEMM_ERR_INVALID_VALUE;
  if (!q_start && tokens != batch) return MXGEMM_ERR_INVALID_VALUE;
  if (batch == 0 || tokens == 0) return MXGEMM_OK;
  if (!kv_len || (table_pitch > 0 && !table)) return MXGEMM_ERR_INVALID_VALUE;
  if (c->num_pages > 0 && (!c->K || !c->V || !c->K_scale || !c->V_scale)) return MXGEMM_ERR_INVALID_VALUE;
  if (!aligned(c->K, 16) || !aligned(c->V, 16) || !aligned(c->K_scale, 4) || !aligned(c->V_scale, 4) ||
      !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(q_start, 4))
    return MXGEMM_ERR_MISALIGNED;
  for (const void *p : {static_cast<const void *>(c->K), static_cast<const void *>(c->V),
                        static_cast<const void *>(c->K_scale), static_cast<const void *>(c->V_scale),
                        static_cast<const void *>(table), static_cast<const void *>(kv_len),
                        static_cast<const void *>(q_start)})
    if (p && !mxg::pointer_on_device(p, v.device)) return MXGEMM_ERR_INVALID_VALUE;
  cv->K = static_cast<uint8_t *>(c->K);
  cv->V = static_cast<uint8_t *>(c->V);
  cv->K_scale = c->K_scale;
  cv->V_scale = c->V_scale;
  cv->num_pages = c->num_pages;
  cv->page_size = c->page_size;
  cv->page_log2 = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  cv->kv_heads = c->kv_heads;
  bv->batch = static_cast<int>(batch);
  bv->table = table;
  bv->table_pitch = table_pitch;
  bv->kv_len = kv_len;
  bv->q_start = q_start;
  bv->tokens = tokens;
  bv->status = v.status;
  return MXGEMM_OK;
}

// Passes over a page's rows: of 128 threads, eight values each.
template <typename T, int D, int LG>
int launch_append_page(const mxg::AppendParams &p, dim3 grid, cudaStream_t stream) {
  constexpr int kRows = 128 / (D / 8), kAll = ((1 << LG) + kRows - 1) / kRows;
  return mxg::launch(p.b.q_start ? mxg::cache_append_kernel<T, D, LG, kAll>
                                 : mxg::cache_append_kernel<T, D, LG, 1>,  // one token
                     grid, 128, 0, 1, stream, p);
}

template <typename T, int D>
int launch_append(const mxg::AppendParams &p, dim3 grid, cudaStream_t stream) {
  switch (p.c.page_log2) {
    case 4: return launch_append_page<T, D, 4>(p, grid, stream);
    case 5: return launch_append_page<T, D, 5>(p, grid, stream);
    case 6: return launch_append_page<T, D, 6>(p, grid, stream);
    default: return launch_append_page<T, D, 7>(p, grid, stream);
  }
}

// Tensor map of a cache's codes as rows of head_dim bytes, swizzled or not.
int encode_rows(const mxg::HandleView &v, CUtensorMap *tm, const void *base, int64_t rows, int d, int box_rows,
                bool swizzle) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return v.encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  !swizzle   ? CU_TENSOR_MAP_SWIZZLE_NONE
                  : d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                             : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MXGEMM_OK
             : MXGEMM_ERR_CUDA;
}

int encode_cache(const mxg::HandleView &v, const mxg::CacheView &c, int d, int box_rows, bool swizzle,
                 CUtensorMap *tK, CUtensorMap *tV) {
  // (a cache of no pages: the maps are not used)
  std::memset(tK, 0, sizeof(*tK));
  std::memset(tV, 0, sizeof(*tV));
  const int64_t rows = c.num_pages * c.kv_heads * c.page_size;
  if (rows > 0 && (encode_rows(v, tK, c.K, rows, d, box_rows, swizzle) ||
                   encode_rows(v, tV, c.V, rows, d, box_rows, swizzle)))
    return MXGEMM_ERR_CUDA;
  return MXGEMM_OK;
}

// Many query rows: one CTA for each 256 of a sequence and key/value head.  The
// row tiles that do not fill a round of the SMs, all of them where they are
// few, get up to 16 CTAs each (44 row tiles of 61102 keys: 816 -> 296 us; the
// last 24 of 480: 334 -> 328 us).  The grid has room for every split of the rows
// into sequences; the count of row tiles that decides is that of equal ones.
int64_t equal_row_tiles(const mxg::AttnParams &p) {
  constexpr int64_t kRows = mxg::PromptCfg<128>::ROWS;
  return (p.b.tokens * p.group / p.b.batch + kRows - 1) / kRows * p.b.batch * p.c.kv_heads;
}

// How row tiles and their keys are cut: fills in p, and gives the bytes of the
// partials, or -1 where there are too many.
template <int D>
int64_t plan_prompt(const mxg::HandleView &v, mxg::AttnParams &p) {
  using S = mxg::PromptCfg<D>;
  const int64_t rows = p.b.tokens * p.group;
  const int64_t items = (rows / S::ROWS + p.b.batch) * p.c.kv_heads;
  if (items >= kLim - 16 * mxg::kCounters) return -1;
  const int64_t tiles = equal_row_tiles(p), over = tiles % v.sm_count;
  p.items = p.whole = static_cast<int>(items);
  p.parts = over > 0 ? static_cast<int>(std::min<int64_t>(16, v.sm_count / over)) : 1;
  if (p.parts > 1) {
    if (tiles >= v.sm_count) p.whole -= static_cast<int>(std::min(items, over));
    else p.whole = 0;
    const int cut = p.items - p.whole;
    if (cut > mxg::kCounters) p.whole = p.items;
    else return static_cast<int64_t>(cut) * p.parts * S::PARTIAL * static_cast<int64_t>(sizeof(float));
  }
  return 0;
}

template <int D, int MODE>
int launch_prompt(const mxg::HandleView &v, mxg::AttnParams &p, cudaStream_t stream) {
  using S = mxg::PromptCfg<D>;
  // (behind shared tokens one CTA more waits for the launch over the shared keys)
  const int grid = p.whole + (p.items - p.whole) * p.parts + (MODE == mxg::kOwnKeys ? 1 : 0);
  CUtensorMap tK, tV;
  if (int st = encode_cache(v, p.c, D, p.c.page_size, false, &tK, &tV)) return st;
  return mxg::launch(mxg::cache_prompt_kernel<D, MODE>, dim3(static_cast<unsigned>(grid)), S::THREADS, S::SMEM_BYTES, 1, stream,
                     tK, tV, p);
}

template <int D, int NT>
int decode_grid(int sms) {
  return std::min(mxg::DecodeCfg<D, NT>::CTAS * sms, mxg::kCounters / 4);
}
template <int D, int NT>
int64_t decode_bytes(const mxg::AttnParams &p, int sms) {
  // two slots a CTA, or, behind shared tokens, a warp
  return static_cast<int64_t>(decode_grid<D, NT>(sms)) * (p.shared ? 8 : 2) * mxg::DecodeCfg<D, NT>::PARTIAL * sizeof(float);
}

template <int D, int NT, int MODE>
int launch_decode(const mxg::HandleView &v, mxg::AttnParams &p, int sms, cudaStream_t stream) {
  using S = mxg::DecodeCfg<D, NT>;
  CUtensorMap tK, tV;
  if (int st = encode_cache(v, p.c, D, std::min(p.c.page_size, 32), true, &tK, &tV)) return st;
  const int grid = decode_grid<D, NT>(sms) + (MODE == mxg::kOwnKeys ? 1 : 0);
  return mxg::launch(mxg::cache_decode_kernel<D, NT, MODE>, dim3(static_cast<unsigned>(grid)), 128, S::SMEM_BYTES, 1, stream, tK, tV, p);
}

// Rows (query tokens x heads of a group) of an ordinary sequence decide: many
// go to the tensor cores by 256, few to the kernel whose items are 8 or 16.
// At 64 rows both take the same time on 32 row tiles of 8192 keys (70 us); on
// 128 the first takes 106 us and the second 219, and with more than 16 rows
// the second reads the keys again; but it cuts them for all SMs where the
// first's row tiles times 16 do not fill half of them.
// (Behind shared tokens, whose own keys are mostly few: from 64 rows on.)
bool takes_prompt(const mxg::HandleView &v, const mxg::AttnParams &p) {
  const int64_t rows = p.b.tokens * p.group;
  if (p.shared) return rows >= 64 * p.b.batch;
  return rows >= 64 * p.b.batch || (rows > 16 * p.b.batch && equal_row_tiles(p) * 32 >= v.sm_count);
}
// (of the kernel for few rows: items of 16)
bool takes_two(const mxg::AttnParams &p) { return p.b.tokens * p.group > 8 * p.b.batch; }

// How an attention runs: by which kernel, on how many SMs (that for few rows), and the
// bytes of its partials (-1: too many row tiles).
struct AttnPlan {
  bool prompt, two;
  int sms;
  int64_t bytes;
};
template <int D>
AttnPlan plan_attention(const mxg::HandleView &v, mxg::AttnParams &p, int sms) {
  AttnPlan a{takes_prompt(v, p), takes_two(p), sms, 0};
  a.bytes = a.prompt ? plan_prompt<D>(v, p) : a.two ? decode_bytes<D, 2>(p, sms) : decode_bytes<D, 1>(p, sms);
  return a;
}
template <int D, int MODE>
int launch_attention(const mxg::HandleView &v, mxg::AttnParams &p, const AttnPlan &a, cudaStream_t stream) {
  if (a.prompt) return launch_prompt<D, MODE>(v, p, stream);
  return a.two ? launch_decode<D, 2, MODE>(v, p, a.sms, stream) : launch_decode<D, 1, MODE>(v, p, a.sms, stream);
}

template <int D>
int run_attention(mxgemm_handle_t h, const mxg::HandleView &v, mxg::AttnParams &p, cudaStream_t stream) {
  const AttnPlan a = plan_attention<D>(v, p, v.sm_count);
  if (a.bytes < 0) return MXGEMM_ERR_INVALID_VALUE;
  if (a.bytes > 0) {
    uint8_t *ws = nullptr;
    if (int st = mxg::handle_workspace(h, static_cast<size_t>(a.bytes), stream, &ws)) return st;
    p.partials = reinterpret_cast<float *>(ws);
  }
  return launch_attention<D, mxg::kAllKeys>(v, p, a, stream);
}

// Time (us) of an attention over `keys` keys of each sequence on `sms` SMs: start and
// end, and 1.65 us for a row tile's 128 keys, or the codes at the rate of an SM, once for
// each 8 or 16 rows.  Fitted to 2-128 sequences of 1-64 tokens, 512-65536 keys; the
// kernel for few rows without the join of its parts where only own keys are its.
struct AttnTime {
  double start, key, tile;  // key: on one SM; tile: 32 keys of an item of the kernel for few rows, on one SM
  double us(double keys, int sms) const { return start + key * keys / sms; }
};
AttnTime attention_time(const mxg::AttnParams &p, bool prompt, bool own, int d) {
  if (prompt) return AttnTime{13, 1.65 * static_cast<double>(equal_row_tiles(p)) / 128, 0};
  const int64_t rows = takes_two(p) ? 16 : 8, passes = (p.b.tokens * p.group + rows * p.b.batch - 1) / (rows * p.b.batch);
  // bytes a us (heads of 64: 1.4 times the keys)
  const double rate = (own ? (rows == 16 ? 30e3 : 36e3) : (rows == 16 ? 22e3 : 42e3)) * (d == 64 ? 0.72 : 1);
  return AttnTime{own ? 6.0 : 12.0, static_cast<double>(passes * p.b.batch * p.c.kv_heads * 2 * d) / rate, 64 * d / rate};
}

// How the shared keys and the sequences' own are computed apart: parts of the shared
// keys for each of `tiles` row tiles (a CTA each), the SMs for the own keys, and the time
// (us).  A key tile takes a CTA 1.65 us, its start and end as long as five or (more than
// 128 rows) seven, and the launch that joins 3 us and its reads.  Where the
// first launch leaves SMs, the second runs there beside it, in one wave: 64 tokens of
// 64/8 heads behind 8192 keys, 100-1000 of their own: 43.7 us with 5 parts and 72 SMs
// for the own keys (4 and 88: 48.7, 6 and 56: 49.6; two waves on 72 SMs 50), and one
// launch after the other with 8 parts 56.
// How many keys sequences have of their own is known to the device alone.  The host
// knows the table's room, of which three quarters are taken where tables are about as wide
// as the longest sequence needs, but no more than kOwnMost: a table for the greatest length
// there can be says nothing.  So the second launch has CTAs for all SMs, and on the device
// those beside the first one alone work where that takes no longer than 1.3 times the
// first (`beside_tiles`); else all, and those that find no place begin when the first one's end.
// The same 64 tokens with tables of 16384 to 131072: 44.7 us; by the table's room alone
// 59.7, and from 65536 on, where the own keys' two estimates differ by more than the
// shared keys cost, not apart at all, 162.  16 x 4 tokens behind 65536, 1000-2000 of
// their own: 79 (with a kOwnMost of 1024 84.5); 8 tokens behind 8192, 50-500 of their own:
// 20.2, and 22.3 with wider tables (of 2048: 23.6).
constexpr double kOwnMost = 1536;
struct SharedPlan {
  int parts, sms;        // sms: beside the first launch
  double us, keys;       // keys: of each sequence's own, as estimated
  int64_t beside_tiles;  // -1: the launches come one after the other
};
SharedPlan plan_shared(const mxg::HandleView &v, const mxg::AttnParams &p, int64_t tiles, int d) {
  const int64_t rows = p.b.tokens * p.group, key_tiles = (p.shared + 127) / 128, most = std::min<int64_t>(64, std::max<int64_t>(1, key_tiles / 4));
  auto shared_us = [&](int64_t n) {
    return 1.65 * static_cast<double>((tiles * n + v.sm_count - 1) / v.sm_count) * (static_cast<double>((key_tiles + n - 1) / n) + (rows > 128 ? 7 : 5));
  };
  double least = 1e300;
  for (int64_t n = 1; n <= most; ++n) least = std::min(least, shared_us(n));
  const bool prompt = takes_prompt(v, p);
  const AttnTime own = attention_time(p, prompt, true, d);
  const double keys = std::min(0.75 * static_cast<double>(p.b.table_pitch * p.c.page_size - p.shared), kOwnMost);
  SharedPlan best{1, v.sm_count, 1e300, keys, -1};
  for (int64_t n = 1; n <= most; ++n) {
    const double shared = shared_us(n), join = 3 + static_cast<double>(rows * p.c.kv_heads * (n + 2)) * 1e-4;
    const double after = shared + own.us(keys, v.sm_count) + join;
    if (after < best.us) best = SharedPlan{static_cast<int>(n), v.sm_count, after, keys, -1};
    // (a shared launch made longer than it need be has to pay whatever own keys there are)
    if (tiles * n < v.sm_count && shared <= 1.4 * least && !prompt) {
      const int busy = static_cast<int>(tiles * n), left = v.sm_count - busy;
      const double limit = 1.3 * shared, one = own.us(keys, left), all = own.us(keys, v.sm_count) + shared * busy / v.sm_count;
      const double beside = std::max(shared, one <= limit ? one : all) + join;
      if (beside < best.us) best = SharedPlan{static_cast<int>(n), left, beside, keys, static_cast<int64_t>((limit - own.start) * left / own.tile)};
    }
  }
  return best;
}

// The shared keys for all tokens, then each sequence's own, then both joined.
template <int D>
int run_shared(mxgemm_handle_t h, const mxg::HandleView &v, mxg::AttnParams &p, cudaStream_t stream) {
  using S = mxg::PromptCfg<D>;
  p.left_tiles = static_cast<int>((p.b.tokens * p.group + S::ROWS - 1) / S::ROWS);
  const int64_t items = static_cast<int64_t>(p.left_tiles) * p.c.kv_heads;
  const SharedPlan plan = plan_shared(v, p, items, D);
  mxg::AttnParams all = p;
  all.shared = 0;
  if (!v.shared_keys && plan.us > attention_time(all, takes_prompt(v, all), false, D).us(p.shared + plan.keys, v.sm_count)) {
    p.shared = 0;
    return run_attention<D>(h, v, p, stream);
  }
  p.left_parts = plan.parts;
  const int64_t left = items * p.left_parts * S::PARTIAL * static_cast<int64_t>(sizeof(float));
  const int64_t rows = p.b.tokens * p.heads, own = rows * (D + 4) * static_cast<int64_t>(sizeof(float));
  const int64_t blocks = (p.b.tokens * p.group + mxg::JoinCfg<D>::ROWS - 1) / mxg::JoinCfg<D>::ROWS;
  mxg::AttnParams first = p;
  const AttnPlan a = plan_attention<D>(v, p, plan.beside_tiles < 0 ? plan.sms : v.sm_count);
  p.beside_tiles = plan.beside_tiles;
  p.beside_blocks = a.two ? decode_grid<D, 2>(plan.sms) : decode_grid<D, 1>(plan.sms);
  if (items * p.left_parts >= kLim || a.bytes < 0) return MXGEMM_ERR_INVALID_VALUE;
  uint8_t *ws = nullptr;
  if (int st = mxg::handle_workspace(h, static_cast<size_t>(left + (own + 15) / 16 * 16 + a.bytes), stream, &ws)) return st;
  p.left = first.left = reinterpret_cast<float *>(ws);
  p.own = reinterpret_cast<float *>(ws + left);
  p.own_ml = reinterpret_cast<float2 *>(p.own + rows * D);
  p.own_at = a.prompt ? nullptr : reinterpret_cast<int2 *>(p.own_ml + rows);
  p.own_rows = a.two ? 16 : 8;
  p.partials = reinterpret_cast<float *>(ws + left + (own + 15) / 16 * 16);
  first.items = static_cast<int>(items);
  first.whole = 0;
  first.parts = first.left_parts;
  if (int st = launch_prompt<D, mxg::kSharedKeys>(v, first, stream)) return st;
  ++*v.launches;
  if (int st = launch_attention<D, mxg::kOwnKeys>(v, p, a, stream)) return st;
  ++*v.launches;
  return mxg::launch(mxg::cache_join_kernel<D>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(p.c.kv_heads)), 256, 0, 1, stream, p);
}

// The checks of an attention's arguments beyond the cache's; fills the kernels' view.
int attention_args(const mxg::HandleView &v, const mxgemm_cache_t *cache, int64_t batch, int64_t heads, int64_t tokens, const void *Q,
                   int64_t q_pitch, float scale, int causal, int64_t window, int64_t sinks, void *O, float *lse, mxg::AttnParams *p) {
  if (heads < 1 || heads >= (1 << 16) || heads % cache->kv_heads != 0 || tokens * heads >= kLim)
    return MXGEMM_ERR_INVALID_VALUE;
  if (q_pitch < heads * cache->head_dim || !std::isfinite(scale)) return MXGEMM_ERR_INVALID_VALUE;
  if ((causal != 0 && causal != 1) || window < 0 || sinks < 0) return MXGEMM_ERR_INVALID_VALUE;
  if (batch == 0 || tokens == 0) return MXGEMM_OK;
  if (!Q || !O) return MXGEMM_ERR_INVALID_VALUE;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(lse, 4) || q_pitch % 8 != 0)
    return MXGEMM_ERR_MISALIGNED;
  if (!mxg::pointer_on_device(Q, v.device) || !mxg::pointer_on_device(O, v.device) ||
      (lse && !mxg::pointer_on_device(lse, v.device)))
    return MXGEMM_ERR_INVALID_VALUE;
  p->Q = static_cast<const __nv_bfloat16 *>(Q);
  p->q_pitch = q_pitch;
  p->heads = static_cast<int>(heads);
  p->group = static_cast<int>(heads / cache->kv_heads);
  p->scale = scale;
  p->causal = causal;
  // (positions stay below 2^31: a longer window sees as much, and the kernels'
  // sums with these stay far from 64 bits' end)
  p->window = std::min(window, kLim);
  p->sinks = std::min(sinks, kLim);
  p->O = static_cast<__nv_bfloat16 *>(O);
  p->lse = lse;
  p->counters = v.counters;
  p->begun = v.counters + mxg::kCounters;
  p->timeout_ns = v.timeout_ns;
  p->stall_producer = v.stall_producer;
  p->shared = p->left_parts = p->left_tiles = 0;
  p->left = p->own = nullptr;
  p->own_ml = nullptr;
  p->own_at = nullptr;
  p->own_rows = p->beside_blocks = 0;
  p->beside_tiles = -1;
  return MXGEMM_OK;
}

}  // namespace

extern "C" int mxgemm_cache_append(mxgemm_handle_t h, const mxgemm_cache_t *cache, int64_t batch,
                                   const int32_t *page_table, int64_t table_pitch,
                                   const int32_t *kv_len, const int32_t *q_start, int64_t tokens,
                                   const void *new_K, const void *new_V, int64_t pitch, int x_dtype,
                                   mxgemm_stream_t stream_) {
  if (!h) return MXGEMM_ERR_INVALID_VALUE;
  const mxg::HandleView v = mxg::handle_view(h);
  mxg::CurrentDevice g(v.device);
  mxg::AppendParams p;
  if (int st = cache_args(v, cache, batch, page_table, table_pitch, kv_len, q_start, tokens, &p.c, &p.b))
    return st;
  if (x_dtype != MXGEMM_IN_F32 && x_dtype != MXGEMM_IN_BF16) return MXGEMM_ERR_INVALID_VALUE;
  if (pitch < static_cast<int64_t>(cache->kv_heads) * cache->head_dim) return MXGEMM_ERR_INVALID_VALUE;
  if (batch == 0 || tokens == 0) return MXGEMM_OK;
  if (!new_K || !new_V) return MXGEMM_ERR_INVALID_VALUE;
  const size_t al = x_dtype == MXGEMM_IN_F32 ? 32 : 16;
  if (!aligned(new_K, al) || !aligned(new_V, al) || pitch % 8 != 0) return MXGEMM_ERR_MISALIGNED;
  if (!mxg::pointer_on_device(new_K, v.device) || !mxg::pointer_on_device(new_V, v.device))
    return MXGEMM_ERR_INVALID_VALUE;
  p.newK = new_K;
  p.newV = new_V;
  p.pitch = pitch;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int64_t items = q_start ? (tokens >> p.c.page_log2) + 2 * batch : batch;
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>(cache->kv_heads), 2);
  const bool f32 = x_dtype == MXGEMM_IN_F32;
  const int st = cache->head_dim == 128
                     ? (f32 ? launch_append<float, 128>(p, grid, stream) : launch_append<__nv_bfloat16, 128>(p, grid, stream))
                     : (f32 ? launch_append<float, 64>(p, grid, stream) : launch_append<__nv_bfloat16, 64>(p, grid, stream));
  if (st != MXGEMM_OK) return st;
  ++*v.launches;
  return MXGEMM_OK;
}

extern "C" int mxgemm_cache_attention(mxgemm_handle_t h, const mxgemm_cache_t *cache, int64_t batch,
                                      int64_t heads, const int32_t *page_table, int64_t table_pitch,
                                      const int32_t *kv_len, const int32_t *q_start, int64_t tokens,
                                      const void *Q, int64_t q_pitch, float scale, int causal,
                                      int64_t window, int64_t sinks, void *O, float *lse,
                                      mxgemm_stream_t stream_) {
  if (!h) return MXGEMM_ERR_INVALID_VALUE;
  const mxg::HandleView v = mxg::handle_view(h);
  mxg::CurrentDevice g(v.device);
  mxg::AttnParams p;
  if (int st = cache_args(v, cache, batch, page_table, table_pitch, kv_len, q_start, tokens, &p.c, &p.b))
    return st;
  if (int st = attention_args(v, cache, batch, heads, tokens, Q, q_pitch, scale, causal, window, sinks, O, lse, &p)) return st;
  if (batch == 0 || tokens == 0) return MXGEMM_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int st = cache->head_dim == 128 ? run_attention<128>(h, v, p, stream) : run_attention<64>(h, v, p, stream);
  if (st != MXGEMM_OK) return st;
  ++*v.launches;
  return MXGEMM_OK;
}

extern "C" int mxgemm_cache_attention_shared(mxgemm_handle_t h, const mxgemm_cache_t *cache, int64_t batch, int64_t heads,
                                             const int32_t *page_table, int64_t table_pitch, const int32_t *kv_len,
                                             const int32_t *q_start, int64_t tokens, int64_t shared, const void *Q,
                                             int64_t q_pitch, float scale, int causal, void *O, float *lse,
                                             mxgemm_stream_t stream_) {
  if (!h) return MXGEMM_ERR_INVALID_VALUE;
  const mxg::HandleView v = mxg::handle_view(h);
  mxg::CurrentDevice g(v.device);
  mxg::AttnParams p;
  if (int st = cache_args(v, cache, batch, page_table, table_pitch, kv_len, q_start, tokens, &p.c, &p.b))
    return st;
  if (shared < 0) return MXGEMM_ERR_INVALID_VALUE;
  if (int st = attention_args(v, cache, batch, heads, tokens, Q, q_pitch, scale, causal, 0, 0, O, lse, &p)) return st;
  if (batch == 0 || tokens == 0) return MXGEMM_OK;
  // whole pages and whole tiles of the kernel for few rows; what is over is read as
  // each sequence's own.  (No sequence is longer than its table.)
  const int64_t unit = std::max(cache->page_size, 32);
  p.shared = static_cast<int>(std::min(shared, table_pitch * cache->page_size) / unit * unit);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const bool d128 = cache->head_dim == 128;
  const int st = p.shared == 0 ? (d128 ? run_attention<128>(h, v, p, stream) : run_attention<64>(h, v, p, stream))
                               : (d128 ? run_shared<128>(h, v, p, stream) : run_shared<64>(h, v, p, stream));
  if (st != MXGEMM_OK) return st;
  ++*v.launches;
  return MXGEMM_OK;
}
