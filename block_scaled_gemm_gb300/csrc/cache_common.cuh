// cache_common.cuh -- what the kernels of the 8-bit key/value cache share:
// the description of a cache and of a batch of sequences, and the checks that
// keep every access of device-side lengths and page numbers in bounds.
#pragma once
#include <cstdint>

#include "quantize.cuh"

namespace mxg {

struct CacheView {
  uint8_t *K, *V;          // num_pages x kv_heads x page_size x D codes
  float *K_scale, *V_scale;  // num_pages x kv_heads
  int64_t num_pages;
  int page_size, page_log2, kv_heads;
};

struct BatchView {
  int batch;
  const int32_t *table;  // batch rows of page numbers
  int64_t table_pitch;
  const int32_t *kv_len;   // lengths with the new tokens
  const int32_t *q_start;  // batch + 1, or null: one token each
  int64_t tokens;
  int *status;
};

constexpr int kStatusInvalid = 1;  // MXGEMM_ERR_INVALID_VALUE

__device__ __forceinline__ void cache_invalid(const BatchView &b, int detail) {
  if (atomicCAS(b.status, 0, kStatusInvalid) == 0) atomicExch(b.status + 1, detail);
}

struct Sequence {
  int len;    // tokens in the cache, new ones included
  int first;  // its first row among the new tokens (queries)
  int n;      // how many new tokens (queries)
};

// A load, from L2 where FRESH: by the launch that has not itself waited for the one that
// wrote the value (start_after puts it in order behind that).
template <bool FRESH, typename T>
__device__ __forceinline__ T load_value(const T *p) {
  if constexpr (FRESH) return __ldcg(p);
  else return *p;
}

// Sequence b with values that stay in bounds whatever the arrays hold: a
// length that does not fit the page table counts as 0, rows are clamped to
// [0, tokens].
template <bool FRESH = false>
__device__ __forceinline__ Sequence load_sequence(const BatchView &bv, const CacheView &c, int b) {
  Sequence s;
  s.len = load_value<FRESH>(bv.kv_len + b);
  if (s.len < 0 || s.len > bv.table_pitch * c.page_size) {
    cache_invalid(bv, 0x21);
    s.len = 0;
  }
  if (bv.q_start) {
    const int64_t s0 = load_value<FRESH>(bv.q_start + b), s1 = load_value<FRESH>(bv.q_start + b + 1);
    if (s0 < 0 || s1 < s0 || s1 > bv.tokens) {
      cache_invalid(bv, 0x22);
      s.first = s.n = 0;
    } else {
      s.first = static_cast<int>(s0);
      s.n = static_cast<int>(s1 - s0);
    }
  } else {
    s.first = b;
    s.n = 1;
  }
  return s;
}

// Page number of page slot `i` of sequence b, or -1 when it names none.
template <bool FRESH = false>
__device__ __forceinline__ int load_page(const BatchView &bv, const CacheView &c, int b, int64_t i) {
  const int pg = load_value<FRESH>(bv.table + b * bv.table_pitch + i);
  if (pg < 0 || pg >= c.num_pages) {
    cache_invalid(bv, 0x23);
    return -1;
  }
  return pg;
}

// Largest b in [0, batch) with f(b) <= x, where f ascends and f(0) <= x:
// a 32-way search by a whole warp (two rounds of loads for up to 1024
// sequences).
template <typename F>
__device__ __forceinline__ int warp_find(int batch, F f, int64_t x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && f(at) <= x;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, le);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace mxg
