// cache_join.cuh -- attention behind shared tokens: the shared keys' partials and the
// sequences' own sums of each row joined and normalized.
//
//   top = max over parts of m,  o = sum 2^(m - top) o_part / (2^7 sum 2^(m - top) l_part)
//
// In a launch of its own, by all SMs: 64 tokens of 64 heads with nine parts each are
// 19 MB from L2, 4 us; the CTA that arrives last in the launch over the shared keys
// took 22 us for its row tile, and the launch over the own keys, at the end of each of
// its items, 30 us.
#pragma once
#include "cache_attention.cuh"

namespace mxg {

// 256 threads: ROWS rows of a key/value head, D / 4 threads a row.
template <int D>
struct JoinCfg {
  static constexpr int ROWS = 256 / (D / 4);
};

template <int D>
__global__ void __launch_bounds__(256) cache_join_kernel(const AttnParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int d4 = threadIdx.x / JoinCfg<D>::ROWS, h = blockIdx.y;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * JoinCfg<D>::ROWS + threadIdx.x % JoinCfg<D>::ROWS;  // token x head of the group
  if (row >= p.b.tokens * p.group) return;
  const int64_t tile = row / kTileRows;
  const float *left = p.left + ((p.left_tiles - 1 - tile) * p.c.kv_heads + h) * p.left_parts * kTilePartial<D>;
  const int r = static_cast<int>(row % kTileRows);
  auto top_of = [&](int v) { return __ldcg(left + static_cast<int64_t>(v) * kTilePartial<D> + kTileRows * D + r); };
  auto sum_of = [&](int v) { return __ldcg(left + static_cast<int64_t>(v) * kTilePartial<D> + kTileRows * (D + 1) + r); };
  if (sum_of(0) < 0.f) return;  // a row that is no sequence's
  const int64_t at = row / p.group * p.heads + h * p.group + row % p.group;
  const float2 own = __ldcg(p.own_ml + at);
  float4 a = __ldcg(reinterpret_cast<const float4 *>(p.own + at * D) + d4);
  float top = own.x;
#pragma unroll 8
  for (int v = 0; v < p.left_parts; ++v) top = fmaxf(top, top_of(v));
  const float f = own.x == -INFINITY ? 0.f : ex2(own.x - top);
  float sum = own.y * f;
  a = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
#pragma unroll 8
  for (int v = 0; v < p.left_parts; ++v) {
    const float m = top_of(v), k = m == -INFINITY ? 0.f : ex2(m - top);
    sum = fmaf(sum_of(v), k, sum);
    float4 b = __ldcg(reinterpret_cast<const float4 *>(left + static_cast<int64_t>(v) * kTilePartial<D>) + d4 * kTileRows + r);
    if (k == 0.f) b = make_float4(0.f, 0.f, 0.f, 0.f);  // (a part without keys holds anything)
    a = make_float4(fmaf(b.x, k, a.x), fmaf(b.y, k, a.y), fmaf(b.z, k, a.z), fmaf(b.w, k, a.w));
  }
  const float k = sum == 0.f ? 0.f : kWeightDown / sum;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * k, a.y * k), hi = __floats2bfloat162_rn(a.z * k, a.w * k);
  *reinterpret_cast<uint2 *>(p.O + at * D + 4 * d4) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  if (d4 == 0 && p.lse) p.lse[at] = log_sum(top, sum);
}

}  // namespace mxg
