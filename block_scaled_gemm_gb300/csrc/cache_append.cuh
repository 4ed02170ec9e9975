// cache_append.cuh -- new keys and values into the pages of the 8-bit cache.
//
// Of each page that new tokens touch, each head and each of K and V:
//   need  = max(2^-64, least power of two >= amax(new) / 448)
//   scale = the new tokens begin the page ? need : max(old, need)
//   codes = E4M3(clamp(x * (1 / scale))), and where the scale grew, the page's
//           earlier codes E4M3(code * (old / scale)).
// Powers of two: x * (1 / scale) is exact, and so is an earlier code's move to a
// larger scale unless it falls below E4M3's normal range.
//
// Bound by latency: five dependent loads (row starts, length, page number, scale
// and values) and the launch.  64 tokens x 8 heads x 128 4.4 us on the device, 8125
// tokens 12.7 us (4.2 TB/s); with two passes over the values instead of registers
// 19.3 us.
//
// One block of threads per (page, head, K or V).  The pages that a batch
// touches are numbered without a scan: sequence b's begin at
// f(b) = floor(q_start[b] / page_size) + 2 b, which leaves room for all of
// them (n tokens touch at most floor(n / page_size) + 2 pages), and a block
// whose number names no page ends at once.
#pragma once
#include "cache_common.cuh"
#include "quantize128.cuh"

namespace mxg {

constexpr float kCacheLeast = 5.4210108624275221700e-20f;  // 2^-64

struct AppendParams {
  CacheView c;
  BatchView b;
  const void *newK, *newV;
  int64_t pitch;
};

// Least power of two >= amax / 448, and 2^-64 at least.
__device__ __forceinline__ float cache_need(float amax) {
  return amax > 0.f ? fmaxf(__int_as_float(mx_scale_of(amax) << 23), kCacheLeast) : kCacheLeast;
}

template <typename T, int D, int LG, int PASSES>
__global__ void __launch_bounds__(128) cache_append_kernel(const AppendParams p) {
  // threads of a row, rows of a pass
  constexpr int lg = LG, ps = 1 << LG, kPer = D / 8, kRows = 128 / kPer;
  __shared__ float part[4];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t item = blockIdx.x;
  const int head = blockIdx.y;
  // (one token each: one page each)
  auto f = [&](int b) -> int64_t { return p.b.q_start ? (p.b.q_start[b] >> lg) + 2 * static_cast<int64_t>(b) : b; };
  const int b = p.b.q_start ? warp_find(p.b.batch, f, item) : static_cast<int>(item);
  const Sequence s = load_sequence(p.b, p.c, b);
  if (s.n == 0) return;
  const int start = s.len - s.n;  // position of the first new token
  if (start < 0) {
    if (s.len >= 0) cache_invalid(p.b, 0x24);
    return;
  }
  const int64_t slot = (start >> lg) + (item - f(b));
  if (item < f(b) || slot > ((s.len - 1) >> lg)) return;
  const int pg = load_page(p.b, p.c, b, slot);
  if (pg < 0) return;
  const int p0 = static_cast<int>(slot) << lg;
  const int lo = max(start - p0, 0), hi = min(s.len - p0, ps);  // the page's rows that are new

  const bool isV = blockIdx.z != 0;
  const int64_t cell = static_cast<int64_t>(pg) * p.c.kv_heads + head;
  uint8_t *codes = (isV ? p.c.V : p.c.K) + cell * ps * D;
  float *scale_at = (isV ? p.c.V_scale : p.c.K_scale) + cell;
  const T *x = static_cast<const T *>(isV ? p.newV : p.newK) +
               static_cast<int64_t>(s.first + p0 - start) * p.pitch + static_cast<int64_t>(head) * D;
  const int col = (threadIdx.x % kPer) * 8, row0 = threadIdx.x / kPer;  // new rows: lo + row0, + kRows, ...

  // all loads before the first use; the values stay in registers until the
  // scale is known
  Eight<T> v[PASSES];
  const float old = lo > 0 ? *scale_at : 0.f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = lo + row0 + i * kRows;
    if (r < hi) v[i].load(x + static_cast<int64_t>(r) * p.pitch + col);
    else v[i].zero();
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) amax = fmaxf(amax, v[i].top());
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) amax = fmaxf(amax, part[w]);
  const float scale = fmaxf(old, cache_need(amax));
  const float inv = __frcp_rn(scale);
  if (threadIdx.x == 0) *scale_at = scale;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = lo + row0 + i * kRows;
    if (r < hi) {
      *reinterpret_cast<uint2 *>(codes + r * D + col) = v[i].codes(inv);
    }
  }
  if (lo > 0 && scale > old) {
    const float ratio = __fdiv_rn(old, scale);
    for (int r = row0; r < lo; r += kRows) {
      uint2 *at = reinterpret_cast<uint2 *>(codes + r * D + col);
      const uint2 w = *at;
      uint32_t out[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t u = q ? w.y : w.x;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<uint8_t>(u >> (8 * e)), __NV_E4M3))) * ratio;
        out[q] = mx_e4m3x2(v[0], v[1]) | (mx_e4m3x2(v[2], v[3]) << 16);
      }
      *at = make_uint2(out[0], out[1]);
    }
  }
}

}  // namespace mxg
