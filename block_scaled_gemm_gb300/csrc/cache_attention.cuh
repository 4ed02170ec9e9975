// cache_attention.cuh -- attention over the 8-bit key/value cache.
//
// One warp per (query token, head); the keys in order, with the running
// maximum and sum of the softmax.
#pragma once
#include <cuda_bf16.h>

#include "cache_common.cuh"

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
};

template <int D>
__global__ void __launch_bounds__(128) cache_attention_kernel(const AttnParams p) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= p.b.tokens * p.heads) return;
  const int64_t t = w / p.heads;
  const int h = static_cast<int>(w % p.heads), kv = h / p.group;
  auto f = [&](int b) -> int64_t { return p.b.q_start ? p.b.q_start[b] : b; };
  const int b = warp_find(p.b.batch, f, t);
  const Sequence s = load_sequence(p.b, p.c, b);
  const int64_t pos = static_cast<int64_t>(s.len) - s.n + (t - s.first);
  float q[kPer], o[kPer];
  for (int e = 0; e < kPer; ++e) {
    q[e] = __bfloat162float(p.Q[t * p.q_pitch + static_cast<int64_t>(h) * D + lane * kPer + e]) * p.scale;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t last = p.causal ? min(static_cast<int64_t>(s.len), pos + 1) : s.len;
  int page = -1, pg = -1;
  for (int64_t j = 0; j < last; ++j) {
    if (p.window > 0 && pos - j >= p.window && j >= p.sinks) continue;
    if (static_cast<int>(j >> p.c.page_log2) != page) {
      page = static_cast<int>(j >> p.c.page_log2);
      pg = load_page(p.b, p.c, b, page);
    }
    if (pg < 0) continue;
    const int64_t cell = static_cast<int64_t>(pg) * p.c.kv_heads + kv;
    const int64_t at = (cell * p.c.page_size + (j & (p.c.page_size - 1))) * D + lane * kPer;
    float x = 0.f;
    for (int e = 0; e < kPer; ++e)
      x += q[e] * __half2float(__half(__nv_cvt_fp8_to_halfraw(p.c.K[at + e], __NV_E4M3)));
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    x *= p.c.K_scale[cell];
    const float mn = fmaxf(m, x), c = __expf(m - mn), e0 = __expf(x - mn), vs = p.c.V_scale[cell];
    l = l * c + e0;
    for (int e = 0; e < kPer; ++e)
      o[e] = o[e] * c + e0 * vs * __half2float(__half(__nv_cvt_fp8_to_halfraw(p.c.V[at + e], __NV_E4M3)));
    m = mn;
  }
  for (int e = 0; e < kPer; ++e)
    p.O[(t * p.heads + h) * D + lane * kPer + e] = __float2bfloat16_rn(l > 0.f ? o[e] / l : 0.f);
  if (p.lse && lane == 0) p.lse[t * p.heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace mxg
