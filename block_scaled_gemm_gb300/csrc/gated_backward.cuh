// gated_backward.cuh -- the gradient of a gated feed-forward block's middle:
//
//   h = act(g) u,  dgate = dH u act'(g),  dup = dH act(g)
//
// as the operands of the products that come next: dgate and dup quantized by rows
// (for the gradient of the input) and by columns (of the two weights), h by columns
// (of the down-projection's weight), or dgate and dup in BF16.
//
// Bound by HBM: six bytes of a value are read (BF16) and five written, where BF16
// gradients that are quantized by calls of their own move 22.  A block takes a tile
// of 128 x 128, computes the three values once, keeps them in registers until its
// rows' and its columns' largest are known, and stores the columns' codes through
// shared memory.
#pragma once
#include "gated_math.cuh"
#include "quantize128.cuh"

namespace mxg {

struct Blocks128 {
  uint8_t *codes;  // or null
  float *scales;
};

struct GatedGradParams {
  const __nv_bfloat16 *gate, *up;
  const void *dH;
  int64_t R, C, pitch, rb, cb;  // pitch: of the columns' codes; blocks of rows, of columns
  int act;
  __nv_bfloat16 *dgate, *dup;  // or null
  Blocks128 rows[2];           // dgate, dup
  Blocks128 cols[3];           // dgate, dup, h
};

// BF16 gradients alone: eight values a thread.
template <typename T>
__global__ void __launch_bounds__(256) gated_grad_flat_kernel(const GatedGradParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t all = p.R * p.C, at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  const T *dh = static_cast<const T *>(p.dH);
  if (at + 8 <= all) {
    Eight<__nv_bfloat16> g, u;
    Eight<T> d;
    g.load(p.gate + at);
    u.load(p.up + at);
    d.load(dh + at);
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const GatedGrad x = gated_grad(g[2 * i], u[2 * i], d[2 * i], p.act), y = gated_grad(g[2 * i + 1], u[2 * i + 1], d[2 * i + 1], p.act);
      const __nv_bfloat162 e = __floats2bfloat162_rn(x.dg, y.dg), f = __floats2bfloat162_rn(x.du, y.du);
      a[i] = *reinterpret_cast<const uint32_t *>(&e);
      b[i] = *reinterpret_cast<const uint32_t *>(&f);
    }
    if (p.dgate) *reinterpret_cast<uint4 *>(p.dgate + at) = make_uint4(a[0], a[1], a[2], a[3]);
    if (p.dup) *reinterpret_cast<uint4 *>(p.dup + at) = make_uint4(b[0], b[1], b[2], b[3]);
  } else {
    for (int64_t i = at; i < all; ++i) {
      const GatedGrad x = gated_grad(__bfloat162float(p.gate[i]), __bfloat162float(p.up[i]), static_cast<float>(dh[i]), p.act);
      if (p.dgate) p.dgate[i] = __float2bfloat16_rn(x.dg);
      if (p.dup) p.dup[i] = __float2bfloat16_rn(x.du);
    }
  }
}

struct GatedGradCfg {
  static constexpr int OFF_TOP = 0;                          // [3][16 warps][128 columns], then [3][128] reciprocals
  static constexpr int OFF_TILE = OFF_TOP + 3 * 16 * 128 * 4;  // [3][128 columns][32 words]
  static constexpr int SMEM_BYTES = OFF_TILE + 3 * 128 * 32 * 4;
};

// 512 threads: thread (ty, tx) has rows 4 ty .. +3 of columns 8 tx .. +7, so that
// the four rows' codes of a column are one word of the transposed tile.
template <typename T>
__global__ void __launch_bounds__(512, 1) gated_grad_tile_kernel(const GatedGradParams p) {
  using S = GatedGradCfg;
  extern __shared__ __align__(16) uint8_t smem[];
  float *tops = reinterpret_cast<float *>(smem + S::OFF_TOP);
  uint32_t *tile = reinterpret_cast<uint32_t *>(smem + S::OFF_TILE);
  griddep_launch_dependents();
  griddep_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t cblock = blockIdx.x % p.cb, rblock = blockIdx.x / p.cb;
  const int64_t r0 = rblock * 128 + 4 * ty, c0 = cblock * 128 + 8 * tx;
  const bool in = c0 < p.C;
  float v[3][4][8];  // dgate, dup, h
  {
    Eight<__nv_bfloat16> g[4], u[4];
    Eight<T> d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = (r0 + i) * p.C + c0;
      if (in && r0 + i < p.R) {
        g[i].load(p.gate + at);
        u[i].load(p.up + at);
        d[i].load(static_cast<const T *>(p.dH) + at);
      } else {
        g[i].zero();
        u[i].zero();
        d[i].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const GatedGrad x = gated_grad(g[i][e], u[i][e], d[i][e], p.act);
        v[0][i][e] = x.dg;
        v[1][i][e] = x.du;
        v[2][i][e] = x.h;
      }
  }
  // columns' largest: of this thread's rows, of the warp's eight, then of all warps
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    if (!p.cols[m].codes) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float t = fmaxf(fmaxf(fabsf(v[m][0][e]), fabsf(v[m][1][e])), fmaxf(fabsf(v[m][2][e]), fabsf(v[m][3][e])));
      t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
      if ((threadIdx.x & 16) == 0) tops[(m * 16 + warp) * 128 + 8 * tx + e] = t;
    }
  }
  __syncthreads();
  // rows: a row's 128 values are 16 lanes'
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    __nv_bfloat16 *plain = m ? p.dup : p.dgate;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool there = in && r0 + i < p.R;
      const int64_t at = (r0 + i) * p.C + c0;
      if (plain && there) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[m][i][2 * e], v[m][i][2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(plain + at) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (!p.rows[m].codes) continue;
      float t = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) t = fmaxf(t, fabsf(v[m][i][e]));
#pragma unroll
      for (int o = 8; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
      t = fmaxf(t, kQ128Least);
      const float inv = __fdiv_rn(448.0f, t);
      if (there) {
        uint32_t w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[e] = mx_e4m3x2(v[m][i][4 * e] * inv, v[m][i][4 * e + 1] * inv) |
                 (mx_e4m3x2(v[m][i][4 * e + 2] * inv, v[m][i][4 * e + 3] * inv) << 16);
        *reinterpret_cast<uint2 *>(p.rows[m].codes + at) = make_uint2(w[0], w[1]);
        if (tx == 0) p.rows[m].scales[(r0 + i) * p.cb + cblock] = __fdiv_rn(t, 448.0f);
      }
    }
  }
  // the columns' reciprocals, in the place of the first warp's largest
  if (threadIdx.x < 384) {
    const int m = threadIdx.x >> 7, c = threadIdx.x & 127;
    if (p.cols[m].codes) {
      float t = kQ128Least;
#pragma unroll
      for (int w = 0; w < 16; ++w) t = fmaxf(t, tops[(m * 16 + w) * 128 + c]);
      tops[m * 16 * 128 + c] = __fdiv_rn(448.0f, t);
      if (cblock * 128 + c < p.C) p.cols[m].scales[(cblock * 128 + c) * p.rb + rblock] = __fdiv_rn(t, 448.0f);
    }
  }
  __syncthreads();
  // word ty of column c is at ty ^ 2 (c / 8): neither the stores nor the 16-byte
  // loads meet in a bank
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    if (!p.cols[m].codes) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float inv = tops[m * 16 * 128 + 8 * tx + e];
      tile[(m * 128 + 8 * tx + e) * 32 + (ty ^ (2 * tx))] =
          mx_e4m3x2(v[m][0][e] * inv, v[m][1][e] * inv) | (mx_e4m3x2(v[m][2][e] * inv, v[m][3][e] * inv) << 16);
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    if (!p.cols[m].codes) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = (threadIdx.x >> 3) + 64 * i, part = threadIdx.x & 7, x = c >> 3;
      uint4 w = *reinterpret_cast<const uint4 *>(tile + (m * 128 + c) * 32 + 4 * (part ^ (x >> 1)));
      if (x & 1) w = make_uint4(w.z, w.w, w.x, w.y);
      const int64_t col = cblock * 128 + c, row = rblock * 128 + 16 * part;
      if (col < p.C && row < p.pitch) *reinterpret_cast<uint4 *>(p.cols[m].codes + col * p.pitch + row) = w;
    }
  }
}

}  // namespace mxg
