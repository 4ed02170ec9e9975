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
#include "cache_prompt.cuh"
#include "context.h"
#include "launch.h"
#include "mxgemm.h"

namespace {

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kLim = int64_t(1) << 31;

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

template <int D>
int run_prompt(mxgemm_handle_t h, const mxg::HandleView &v, mxg::AttnParams &p, cudaStream_t stream) {
  using S = mxg::PromptCfg<D>;
  const int64_t rows = p.b.tokens * p.group;
  const int64_t items = (rows / S::ROWS + p.b.batch) * p.c.kv_heads;
  if (items >= kLim - 16 * mxg::kCounters) return MXGEMM_ERR_INVALID_VALUE;
  const int64_t tiles = equal_row_tiles(p), over = tiles % v.sm_count;
  p.items = p.whole = static_cast<int>(items);
  p.parts = over > 0 ? static_cast<int>(std::min<int64_t>(16, v.sm_count / over)) : 1;
  if (p.parts > 1) {
    if (tiles >= v.sm_count) p.whole -= static_cast<int>(std::min(items, over));
    else p.whole = 0;
    const int cut = p.items - p.whole;
    if (cut > mxg::kCounters) {
      p.whole = p.items;
    } else {
      uint8_t *ws = nullptr;
      if (int st = mxg::handle_workspace(h, static_cast<size_t>(cut) * p.parts * S::PARTIAL * sizeof(float), stream, &ws))
        return st;
      p.partials = reinterpret_cast<float *>(ws);
    }
  }
  const int grid = p.whole + (p.items - p.whole) * p.parts;
  CUtensorMap tK, tV;
  if (int st = encode_cache(v, p.c, D, p.c.page_size, false, &tK, &tV)) return st;
  return mxg::launch(mxg::cache_prompt_kernel<D>, dim3(static_cast<unsigned>(grid)), S::THREADS, S::SMEM_BYTES, 1, stream,
                     tK, tV, p);
}

template <int D, int NT>
int run_decode(mxgemm_handle_t h, const mxg::HandleView &v, mxg::AttnParams &p, cudaStream_t stream) {
  using S = mxg::DecodeCfg<D, NT>;
  const int grid = std::min(S::CTAS * v.sm_count, mxg::kCounters);
  uint8_t *ws = nullptr;
  if (int st = mxg::handle_workspace(h, static_cast<size_t>(grid) * 2 * S::PARTIAL * sizeof(float), stream, &ws))
    return st;
  p.partials = reinterpret_cast<float *>(ws);
  CUtensorMap tK, tV;
  if (int st = encode_cache(v, p.c, D, std::min(p.c.page_size, 32), true, &tK, &tV)) return st;
  return mxg::launch(mxg::cache_decode_kernel<D, NT>, dim3(static_cast<unsigned>(grid)), 128, S::SMEM_BYTES, 1, stream, tK,
                     tV, p);
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
  p.Q = static_cast<const __nv_bfloat16 *>(Q);
  p.q_pitch = q_pitch;
  p.heads = static_cast<int>(heads);
  p.group = static_cast<int>(heads / cache->kv_heads);
  p.scale = scale;
  p.causal = causal;
  // (positions stay below 2^31: a longer window sees as much, and the kernels'
  // sums with these stay far from 64 bits' end)
  p.window = std::min(window, kLim);
  p.sinks = std::min(sinks, kLim);
  p.O = static_cast<__nv_bfloat16 *>(O);
  p.lse = lse;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  p.counters = v.counters;
  p.timeout_ns = v.timeout_ns;
  p.stall_producer = v.stall_producer;
  // Rows (query tokens x heads of a group) of an ordinary sequence decide: many
  // go to the tensor cores by 256, few to the kernel whose items are 8 or 16.
  // At 64 rows both take the same time on 32 row tiles of 8192 keys (70 us); on
  // 128 the first takes 106 us and the second 219, and with more than 16 rows
  // the second reads the keys again; but it cuts them for all SMs where the
  // first's row tiles times 16 do not fill half of them.
  int st;
  const int64_t rows = tokens * p.group;
  if (rows >= 64 * batch || (rows > 16 * batch && equal_row_tiles(p) * 32 >= v.sm_count)) {
    st = cache->head_dim == 128 ? run_prompt<128>(h, v, p, stream) : run_prompt<64>(h, v, p, stream);
  } else {
    const bool two = tokens * p.group > 8 * batch;
    st = cache->head_dim == 128 ? (two ? run_decode<128, 2>(h, v, p, stream) : run_decode<128, 1>(h, v, p, stream))
                                : (two ? run_decode<64, 2>(h, v, p, stream) : run_decode<64, 1>(h, v, p, stream));
  }
  if (st != MXGEMM_OK) return st;
  ++*v.launches;
  return MXGEMM_OK;
}
