// context.h -- what the library's other translation units see of a handle
// (not part of the C interface; mxgemm.cu owns the handle).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "mxgemm.h"

namespace mxg {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kLim = int64_t(1) << 31;

struct HandleView {
  int device;
  int sm_count;
  int *status;  // device status word: [0] code, [1] detail
  unsigned long long timeout_ns;
  int stall_producer;
  int a_fmt, b_fmt;  // mxgemm_format_t
  int b_major;       // mxgemm_b_major_t
  int shared_keys;   // MXGEMM_OPT_SHARED_KEYS
  int64_t *launches;
  cudaEvent_t prof_before, prof_after;
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  unsigned *counters;  // kCounters words, zero between launches, and one more: AttnParams::begun
};

// Counters of a handle: the arrivals of work split over CTAs, each taken by
// at most one piece of work of a launch and left at zero by it, also where a
// wait of the launch gave up.
constexpr int kCounters = 4096;

HandleView handle_view(mxgemm_handle_t h);

// The handle's workspace, grown in stream order to at least `bytes`.
int handle_workspace(mxgemm_handle_t h, size_t bytes, cudaStream_t stream, uint8_t **ptr);

// Whether p is device (or managed) memory of `device`.
bool pointer_on_device(const void *p, int device);

struct CurrentDevice {
  int prev = -1;
  bool changed = false;
  explicit CurrentDevice(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) changed = cudaSetDevice(dev) == cudaSuccess;
  }
  ~CurrentDevice() {
    if (changed) cudaSetDevice(prev);
  }
};

}  // namespace mxg
