// block128_kernel.cuh -- C (+)= sum over K blocks of 128 of
// A_scale * B_scale * (A block . B block), the products of a block summed
// unscaled in FP32 and the scaled blocks added in FP32.
//
// 64 x 64 tiles, 256 threads of 4 x 4 results, operands decoded to FP32 in
// shared memory 16 K values at a time.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>

namespace mxg {

struct B128Params {
  int64_t M, N, K, kb;
  const uint8_t *A, *B;
  const float *a_scale, *b_scale;
  void *C;
  int64_t b_pitch_k, b_pitch_n;    // elements of B from one k (n) to the next
  int64_t bs_pitch_k, bs_pitch_n;  // entries of B_scale
  int b_block;
  int use_acc, out_bf16;
  int a_e5m2, b_e5m2;
};

__device__ __forceinline__ float fp8_value(uint8_t c, int e5m2) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, e5m2 ? __NV_E5M2 : __NV_E4M3)));
}

__global__ void __launch_bounds__(256) block128_kernel(const B128Params p) {
  __shared__ float sa[16][65], sb[16][65];
  const int64_t tiles_n = (p.N + 63) / 64;
  const int64_t m0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t b = 0; b < p.kb; ++b) {
    float part[4][4] = {};
    const int64_t ke = min(p.K, (b + 1) * 128);
    for (int64_t k0 = b * 128; k0 < ke; k0 += 16) {
      __syncthreads();
      for (int i = threadIdx.x; i < 1024; i += 256) {
        const int r = i >> 4, k = i & 15;
        sa[k][r] = m0 + r < p.M ? fp8_value(p.A[(m0 + r) * p.K + k0 + k], p.a_e5m2) : 0.f;
        sb[k][r] = n0 + r < p.N ? fp8_value(p.B[(n0 + r) * p.b_pitch_n + (k0 + k) * p.b_pitch_k], p.b_e5m2) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < 16; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) part[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < p.M && n < p.N)
          acc[i][j] += part[i][j] * (p.a_scale[m * p.kb + b] *
                                     p.b_scale[n / p.b_block * p.bs_pitch_n + b * p.bs_pitch_k]);
      }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      if (p.out_bf16) {
        __nv_bfloat16 *c = static_cast<__nv_bfloat16 *>(p.C) + m * p.N + n;
        *c = __float2bfloat16_rn(acc[i][j] + (p.use_acc ? __bfloat162float(*c) : 0.f));
      } else {
        float *c = static_cast<float *>(p.C) + m * p.N + n;
        *c = acc[i][j] + (p.use_acc ? *c : 0.f);
      }
    }
}

}  // namespace mxg
