// cache_join.cuh -- attention behind shared tokens: the shared keys' partials and the
// sequences' own sums of each row joined and normalized.
//
//   top = max over parts of m,  o = sum 2^(m - top) o_part / (2^7 sum 2^(m - top) l_part)
//
// In a launch of its own, by all SMs: 64 tokens of 64 heads behind 8192 shared ones
// are some 30 MB of partials from L2, 7 us.  Joined by the CTA that arrives last in the
// launch over the shared keys they took 22 us for its row tile, and by the launch over
// the own keys, at the end of each of its items, 30 us.
// It begins when the launch before it has ended, and lets the next one begin when it has
// ended itself: its blocks waiting on freed SMs slowed those that still computed
// (the own keys' last 44 -> 52 us), and a next launch that comes while some are left
// finds SMs in no order, the two launches' CTAs crowded together (50 -> 43.7 us in all).
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
  griddep_wait();
  if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) *p.begun = 0;  // for the next call
  const int d4 = threadIdx.x / JoinCfg<D>::ROWS, h = blockIdx.y;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * JoinCfg<D>::ROWS + threadIdx.x % JoinCfg<D>::ROWS;  // token x head of the group
  if (row >= p.b.tokens * p.group) return;
  const int64_t tile = row / kTileRows;
  const float *left = p.left + ((p.left_tiles - 1 - tile) * p.c.kv_heads + h) * p.left_parts * kTilePartial<D>;
  const int r = static_cast<int>(row % kTileRows);
  const int64_t at = row / p.group * p.heads + h * p.group + row % p.group;  // token x head
  // A row that is no sequence's (before the first one, behind the last one, of one whose
  // start was refused) has a negative sum in the first part, always, and nothing else of
  // it is set: `own_at` holds what the workspace held, and is not followed.
  const float whose = __ldcg(left + kTileRows * D + kTileRows + r);
  const int2 where = p.own_at ? __ldcg(p.own_at + at) : make_int2(-1, 0);
  if (whose < 0.f) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY, sum = 0.f;
  // the shared keys' parts, then the own keys' sums or parts: eight loads of each
  // kind at once, then their sums in order, over the maximum so far
  const int rows = p.own_rows, size = rows * (D + 2), rr = where.y & 15, parts = p.left_parts + (where.x < 0 ? 0 : where.y >> 4) + 1;
  for (int v = 0; v < parts; v += 8) {
    float m[8], l[8];
    float4 b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (v + i >= parts) continue;
      const float *ml, *o;  // maximum (the sum is `apart` behind it), and the four values
      int apart;
      if (v + i < p.left_parts) {
        const float *part = left + static_cast<int64_t>(v + i) * kTilePartial<D>;
        ml = part + kTileRows * D + r;
        o = part + (d4 * kTileRows + r) * 4;
        apart = kTileRows;
      } else if (where.x < 0) {
        ml = &p.own_ml[at].x;
        o = p.own + at * D + 4 * d4;
        apart = 1;
      } else {
        const int n = v + i - p.left_parts;
        const float *part = p.partials + (2 * static_cast<int64_t>(where.x + n) + (n == 0)) * size;
        ml = part + rows * D + rr;
        o = part + rr * D + 4 * d4;
        apart = rows;
      }
      m[i] = __ldcg(ml);
      l[i] = __ldcg(ml + apart);
      b[i] = __ldcg(reinterpret_cast<const float4 *>(o));
    }
    float most = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, m[i]);
    const float f = top == -INFINITY ? 0.f : ex2(top - most);
    sum *= f;
    a = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
    top = most;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float k = m[i] == -INFINITY ? 0.f : ex2(m[i] - top);
      sum = fmaf(l[i], k, sum);
      if (k == 0.f) continue;  // (a part without keys holds anything)
      a = make_float4(fmaf(b[i].x, k, a.x), fmaf(b[i].y, k, a.y), fmaf(b[i].z, k, a.z), fmaf(b[i].w, k, a.w));
    }
  }
  const float k = sum == 0.f ? 0.f : kWeightDown / sum;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * k, a.y * k), hi = __floats2bfloat162_rn(a.z * k, a.w * k);
  *reinterpret_cast<uint2 *>(p.O + at * D + 4 * d4) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  if (d4 == 0 && p.lse) p.lse[at] = log_sum(top, sum);
}

}  // namespace mxg
