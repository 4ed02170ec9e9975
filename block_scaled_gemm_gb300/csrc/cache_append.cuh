// cache_append.cuh -- new keys and values into the pages of the 8-bit cache.
//
// Of each page that new tokens touch, each head and each of K and V:
//   need  = max(2^-64, least power of two >= amax(new) / 448)
//   scale = the new tokens begin the page ? need : max(old, need)
//   codes = E4M3(clamp(x / scale)), and where the scale grew, the page's
//           earlier codes E4M3(code * (old / scale)).
// Powers of two: x / scale is exact, and so is an earlier code's move to a
// larger scale unless it falls below E4M3's normal range.
//
// One block of threads per (page, head, K or V).  The pages that a batch
// touches are numbered without a scan: sequence b's begin at
// f(b) = floor(q_start[b] / page_size) + 2 b, which leaves room for all of
// them (n tokens touch at most floor(n / page_size) + 2 pages), and a block
// whose number names no page ends at once.
#pragma once
#include "cache_common.cuh"

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

template <typename T, int D>
__global__ void __launch_bounds__(128) cache_append_kernel(const AppendParams p) {
  constexpr int kVec = 8, kPer = D / kVec, kRows = 128 / kPer;  // threads of a row, rows of a pass
  __shared__ float part[4];
  const int ps = p.c.page_size, lg = p.c.page_log2;
  const int64_t item = blockIdx.x;
  const int head = blockIdx.y;
  auto f = [&](int b) -> int64_t {
    const int64_t q = p.b.q_start ? p.b.q_start[b] : b;
    return (q >> lg) + 2 * static_cast<int64_t>(b);
  };
  const int b = warp_find(p.b.batch, f, item);
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
  const int col = (threadIdx.x % kPer) * kVec, row0 = threadIdx.x / kPer;

  auto load = [&](int r, float(&v)[8]) {
    const T *src = x + static_cast<int64_t>(r) * p.pitch + col;
    if constexpr (sizeof(T) == 4) {
      const float4 a = reinterpret_cast<const float4 *>(src)[0], c = reinterpret_cast<const float4 *>(src)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = c.x; v[5] = c.y; v[6] = c.z; v[7] = c.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4 *>(src);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
  };

  float amax = 0.f;
  for (int r = lo + row0; r < hi; r += kRows) {
    float v[8];
    load(r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  }
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  const float old = lo > 0 ? *scale_at : 0.f;
  __syncthreads();
  amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float need = cache_need(amax);
  const float scale = fmaxf(old, need);
  if (threadIdx.x == 0) *scale_at = scale;
  for (int r = lo + row0; r < hi; r += kRows) {
    float v[8];
    load(r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fdiv_rn(v[e], scale);
    *reinterpret_cast<uint2 *>(codes + r * D + col) =
        make_uint2(mx_e4m3x2(v[0], v[1]) | (mx_e4m3x2(v[2], v[3]) << 16),
                   mx_e4m3x2(v[4], v[5]) | (mx_e4m3x2(v[6], v[7]) << 16));
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
