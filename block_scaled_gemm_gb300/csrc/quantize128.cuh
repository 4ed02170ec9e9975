// quantize128.cuh -- operands of the block-128 product: an FP32 or BF16
// matrix to E4M3 codes with one FP32 scale per block of 128 values (1 x 128,
// 128 x 1 stored transposed, or 128 x 128).
//
//   top = max(max |x|, 2^-100), scale = top / 448,
//   code = E4M3(clamp(x * (448 / top), +-448)), round to nearest even
//
// All in FP32 with IEEE division: 448 / top is finite for top >= 2^-100, and
// the saturating hardware conversion is the clamp.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "quantize.cuh"

namespace mxg {

constexpr float kQ128Least = 7.8886090522101180541e-31f;  // 2^-100

// One warp per block of 128 values of a row; lane l holds values
// 4 l .. 4 l + 3.
template <typename T>
__global__ void quantize128_rows_kernel(const T *__restrict__ X, int64_t R, int64_t C, int64_t kb,
                                        uint8_t *__restrict__ codes, float *__restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); b < R * kb;
       b += warps) {
    const int64_t r = b / kb, c = (b - r * kb) * 128 + lane * 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < C)
      for (int e = 0; e < 4; ++e) v[e] = mx_to_float<T>(X[r * C + c + e]);
    float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    top = fmaxf(top, kQ128Least);
    const float inv = __fdiv_rn(448.0f, top);
    if (c < C)
      *reinterpret_cast<uint32_t *>(codes + r * C + c) =
          mx_e4m3x2(v[0] * inv, v[1] * inv) | (mx_e4m3x2(v[2] * inv, v[3] * inv) << 16);
    if (lane == 0) scales[b] = __fdiv_rn(top, 448.0f);
  }
}

// One thread per column of a 128-row block, the codes written transposed.
template <typename T>
__global__ void quantize128_cols_kernel(const T *__restrict__ X, int64_t R, int64_t C, int64_t pitch,
                                        uint8_t *__restrict__ codes, float *__restrict__ scales) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t rb = blockIdx.y, r0 = rb * 128;
  if (c >= C) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(128), R - r0));
  const int np = static_cast<int>(min(static_cast<int64_t>(128), pitch - r0));
  float top = kQ128Least;
  for (int i = 0; i < n; ++i) top = fmaxf(top, fabsf(mx_to_float<T>(X[(r0 + i) * C + c])));
  const float inv = __fdiv_rn(448.0f, top);
  for (int i = 0; i < np; ++i)
    codes[c * pitch + r0 + i] =
        i < n ? static_cast<uint8_t>(mx_e4m3(mx_to_float<T>(X[(r0 + i) * C + c]) * inv)) : 0;
  scales[c * gridDim.y + rb] = __fdiv_rn(top, 448.0f);
}

// One block of threads per 128 x 128 tile.
template <typename T>
__global__ void quantize128_tiles_kernel(const T *__restrict__ X, int64_t R, int64_t C,
                                         uint8_t *__restrict__ codes, float *__restrict__ scales) {
  __shared__ float part[32];
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128, c0 = static_cast<int64_t>(blockIdx.x) * 128;
  const int c = threadIdx.x & 127;
  float top = 0.f;
  for (int r = threadIdx.x >> 7; r < 128; r += blockDim.x >> 7)
    if (r0 + r < R && c0 + c < C) top = fmaxf(top, fabsf(mx_to_float<T>(X[(r0 + r) * C + c0 + c])));
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = kQ128Least;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) top = fmaxf(top, part[w]);
  const float inv = __fdiv_rn(448.0f, top);
  for (int r = threadIdx.x >> 7; r < 128; r += blockDim.x >> 7)
    if (r0 + r < R && c0 + c < C)
      codes[(r0 + r) * C + c0 + c] =
          static_cast<uint8_t>(mx_e4m3(mx_to_float<T>(X[(r0 + r) * C + c0 + c]) * inv));
  if (threadIdx.x == 0) scales[blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x] = __fdiv_rn(top, 448.0f);
}

}  // namespace mxg
