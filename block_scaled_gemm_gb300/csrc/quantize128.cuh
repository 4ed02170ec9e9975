// quantize128.cuh -- operands of the block-128 product: an FP32 or BF16
// matrix to E4M3 codes with one FP32 scale per block of 128 values (1 x 128,
// 128 x 1 stored transposed, or 128 x 128).
//
//   top = max(max |x|, 2^-100), scale = top / 448,
//   code = E4M3(clamp(x * (448 / top), +-448)), round to nearest even
//
// Measured: 8192 x 8192 BF16 by rows 31.1 us (6.5 TB/s, 0.96 of the measured copy
// rate; with a warp for each block, two loads of 8 bytes a lane, 79 us), 5000 x 4096
// FP32 by columns 17.3 us (6.0 TB/s; reading X twice, one column a thread, 190 us).
//
// All in FP32 with IEEE division: 448 / top is finite for top >= 2^-100, and
// the saturating hardware conversion is the clamp.  HBM-bound: every kernel
// reads X once, keeps its block in registers until the maximum is known, and
// writes each code once.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "quantize.cuh"

namespace mxg {

constexpr float kQ128Least = 7.8886090522101180541e-31f;  // 2^-100

// Eight consecutive values of X (16-byte aligned), as they lie: two 16-byte
// words of FP32, or one of BF16 (the other is not used).
template <typename T>
struct Eight {
  uint4 w[sizeof(T) == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const T *src) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(w);
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    else return __uint_as_float((i & 1) ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
  }
  __device__ __forceinline__ float top() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf((*this)[i]));
    return m;
  }
  __device__ __forceinline__ uint2 codes(float inv) const {
    return make_uint2(mx_e4m3x2((*this)[0] * inv, (*this)[1] * inv) | (mx_e4m3x2((*this)[2] * inv, (*this)[3] * inv) << 16),
                      mx_e4m3x2((*this)[4] * inv, (*this)[5] * inv) | (mx_e4m3x2((*this)[6] * inv, (*this)[7] * inv) << 16));
  }
};

// 1 x 128.  Eight lanes a block, 16 values each; a warp takes UNROLL groups of
// four blocks at a time, all loads first.  RAGGED: C is no multiple of 128,
// so that blocks do not follow one another in memory.
template <typename T, bool RAGGED, int UNROLL>
__global__ void __launch_bounds__(256)
    quantize128_rows_kernel(const T *__restrict__ X, int64_t C, int64_t kb, int64_t blocks,
                            uint8_t *__restrict__ codes, float *__restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t first = warp * (4 * UNROLL) + (lane >> 3);
  Eight<T> v[UNROLL][2];
  int64_t at[UNROLL];
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    const int64_t b = first + 4 * i;
    at[i] = b < blocks ? b * 128 + sub * 16 : -1;
    if constexpr (RAGGED) {
      if (at[i] >= 0) {
        const int64_t r = b / kb, c = (b - r * kb) * 128 + sub * 16;
        at[i] = c < C ? r * C + c : -1;
      }
    }
    if (at[i] >= 0) {
      v[i][0].load(X + at[i]);
      v[i][1].load(X + at[i] + 8);
    } else {
      v[i][0].zero();
      v[i][1].zero();
    }
  }
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    float top = fmaxf(v[i][0].top(), v[i][1].top());
#pragma unroll
    for (int o = 4; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    top = fmaxf(top, kQ128Least);
    const float inv = __fdiv_rn(448.0f, top);
    if (at[i] >= 0) {
      const uint2 a = v[i][0].codes(inv), b = v[i][1].codes(inv);
      *reinterpret_cast<uint4 *>(codes + at[i]) = make_uint4(a.x, a.y, b.x, b.y);
    }
    if (sub == 0 && first + 4 * i < blocks) scales[first + 4 * i] = __fdiv_rn(top, 448.0f);
  }
}

// 128 x 1, stored transposed: 256 threads take 128 rows x 64 columns.  Thread
// (ty, tx) has rows 4 ty .. +3 of columns 8 tx .. +7: a warp's load is four
// rows of 64 columns, and the four rows' codes of a column are one 32-bit
// word of the transposed tile.
template <typename T>
__global__ void __launch_bounds__(256)
    quantize128_cols_kernel(const T *__restrict__ X, int64_t R, int64_t C, int64_t pitch, int64_t row0, int64_t rb_count,
                            uint8_t *__restrict__ codes, float *__restrict__ scales) {
  constexpr int kPitch = 33;  // words of a column (odd: the transposing accesses are spread over the banks)
  __shared__ float tops[8][64];
  __shared__ uint32_t tile[64 * kPitch];
  griddep_launch_dependents();
  griddep_wait();
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  Eight<T> v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * ty + i, c = c0 + 8 * tx;
    if (r < R && c < C) v[i].load(X + r * C + c);
    else v[i].zero();
  }
  float top[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top[e] = fmaxf(fmaxf(fabsf(v[0][e]), fabsf(v[1][e])), fmaxf(fabsf(v[2][e]), fabsf(v[3][e])));
    top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 8));
    top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], 16));
  }
  if ((threadIdx.x & 31) < 8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) tops[warp][8 * tx + e] = top[e];
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    float m = kQ128Least;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, tops[w][threadIdx.x]);
    tops[0][threadIdx.x] = __fdiv_rn(448.0f, m);
    if (c0 + threadIdx.x < C) scales[(c0 + threadIdx.x) * rb_count + blockIdx.y] = __fdiv_rn(m, 448.0f);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float inv = tops[0][8 * tx + e];
    tile[(8 * tx + e) * kPitch + ty] =
        mx_e4m3x2(v[0][e] * inv, v[1][e] * inv) | (mx_e4m3x2(v[2][e] * inv, v[3][e] * inv) << 16);
  }
  __syncthreads();
  // 16 codes of a column at a time (X's first row is row `row0` of the whole
  // matrix); past the last row up to the pitch are the zeros that were put there
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = (threadIdx.x >> 3) + 32 * i, part = threadIdx.x & 7;
    const uint32_t *w = tile + c * kPitch + 4 * part;
    if (c0 + c < C && row0 + r0 + 16 * part < pitch)
      *reinterpret_cast<uint4 *>(codes + (c0 + c) * pitch + row0 + r0 + 16 * part) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 128 x 128: 512 threads a tile; thread (ty, tx) has columns 8 tx .. +7 of
// rows ty, ty + 32, ty + 64, ty + 96.
template <typename T>
__global__ void __launch_bounds__(512)
    quantize128_tiles_kernel(const T *__restrict__ X, int64_t R, int64_t C, uint8_t *__restrict__ codes,
                             float *__restrict__ scales) {
  __shared__ float part[16];
  griddep_launch_dependents();
  griddep_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128 + ty, c = static_cast<int64_t>(blockIdx.x) * 128 + 8 * tx;
  Eight<T> v[4];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (r0 + 32 * i < R && c < C) v[i].load(X + (r0 + 32 * i) * C + c);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, v[i].top());
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  top = kQ128Least;
#pragma unroll
  for (int w = 0; w < 16; ++w) top = fmaxf(top, part[w]);
  const float inv = __fdiv_rn(448.0f, top);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + 32 * i < R && c < C) *reinterpret_cast<uint2 *>(codes + (r0 + 32 * i) * C + c) = v[i].codes(inv);
  if (threadIdx.x == 0) scales[blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x] = __fdiv_rn(top, 448.0f);
}

}  // namespace mxg
