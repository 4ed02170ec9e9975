// ring.h -- loads through a ring of stages with one barrier each, counted from
// 0: load i goes into stage i % stages.  Plain C++, compiled on the host too.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MXG_HOST_DEVICE __host__ __device__
#else
#define MXG_HOST_DEVICE
#endif

namespace mxg {

// Parity of the phase of its stage's barrier that load i completes.
MXG_HOST_DEVICE constexpr uint32_t ring_parity(int64_t i, int stages) {
  return static_cast<uint32_t>(i / stages) & 1u;
}

// After `issued` loads, the first that may be on its way: a stage is loaded
// anew only after its last load was waited for.
MXG_HOST_DEVICE constexpr int64_t ring_pending(int64_t issued, int stages) {
  return issued > stages ? issued - stages : 0;
}

// Limit (ns) of the waits at a kernel's end for what is on its way: loads and
// MMAs that were issued end by themselves, in microseconds, and they must have
// before the CTA does, however short the caller's limit for the other waits is.
MXG_HOST_DEVICE constexpr unsigned long long landing_limit(unsigned long long timeout_ns) {
  return timeout_ns > 2000000000ull ? timeout_ns : 2000000000ull;
}

}  // namespace mxg
