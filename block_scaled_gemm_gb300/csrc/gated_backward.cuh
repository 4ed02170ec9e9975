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
  __nv_bfloat16 *dgate, *dup;  // or null
  Blocks128 rows[2];           // dgate, dup
  Blocks128 cols[3];           // dgate, dup, h
};

// Values 2 i, 2 i + 1 of eight.
template <typename T>
__device__ __forceinline__ float2 two_of(const Eight<T> &v, int i) {
  return make_float2(v[2 * i], v[2 * i + 1]);
}

// BF16 gradients alone: eight values a thread.
template <typename T, int ACT>
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
      const GatedGrad2 x = gated_grad<ACT>(two_of(g, i), two_of(u, i), two_of(d, i));
      const __nv_bfloat162 e = __float22bfloat162_rn(x.dg), f = __float22bfloat162_rn(x.du);
      a[i] = *reinterpret_cast<const uint32_t *>(&e);
      b[i] = *reinterpret_cast<const uint32_t *>(&f);
    }
    if (p.dgate) *reinterpret_cast<uint4 *>(p.dgate + at) = make_uint4(a[0], a[1], a[2], a[3]);
    if (p.dup) *reinterpret_cast<uint4 *>(p.dup + at) = make_uint4(b[0], b[1], b[2], b[3]);
  } else {
    for (int64_t i = at; i < all; ++i) {
      const GatedGrad2 x = gated_grad<ACT>(make_float2(__bfloat162float(p.gate[i]), 0.f), make_float2(__bfloat162float(p.up[i]), 0.f),
                                           make_float2(static_cast<float>(dh[i]), 0.f));
      if (p.dgate) p.dgate[i] = __float2bfloat16_rn(x.dg.x);
      if (p.dup) p.dup[i] = __float2bfloat16_rn(x.du.x);
    }
  }
}

template <typename T>
struct GatedGradCfg {
  static constexpr int WORDS = 2 + sizeof(T) / 2;  // 16-byte words of eight values of gate, up and dH
  static constexpr int OFF_TOP = 0;                            // [3][16 warps][128 columns], then [3][128] reciprocals
  static constexpr int OFF_TILE = OFF_TOP + 3 * 16 * 128 * 4;  // [3][128 columns][32 words]
  static constexpr int OFF_IN = OFF_TILE + 3 * 128 * 32 * 4;   // the next tile: [4 rows][WORDS][512 threads] words
  static constexpr int SMEM_BYTES = OFF_IN + 4 * WORDS * 512 * 16;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// 16 bytes to shared memory, zeros where `there` is false.
__device__ __forceinline__ void grad_copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// One block of 512 threads an SM, which goes from tile to tile and copies the next
// one's values to shared memory while it stores this one's codes (each thread copies
// what it will read itself).  Thread (ty, tx) has rows 4 ty .. +3 of columns 8 tx ..
// +7, so that the four rows' codes of a column are one word of the transposed tile.
template <typename T, int ACT>
__global__ void __launch_bounds__(512, 1) gated_grad_tile_kernel(const GatedGradParams p) {
  using S = GatedGradCfg<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  float *tops = reinterpret_cast<float *>(smem + S::OFF_TOP);
  uint32_t *tile = reinterpret_cast<uint32_t *>(smem + S::OFF_TILE);
  griddep_launch_dependents();
  griddep_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const uint32_t in = smem_u32(smem + S::OFF_IN) + threadIdx.x * 16;
  const int64_t tiles = p.rb * p.cb;
  auto load = [&](int64_t t) {
    const int64_t r0 = t / p.cb * 128 + 4 * ty, c0 = t % p.cb * 128 + 8 * tx;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool there = t < tiles && c0 < p.C && r0 + i < p.R;
      const int64_t at = there ? (r0 + i) * p.C + c0 : 0;
      const uint32_t to = in + i * S::WORDS * 8192;
      grad_copy16(to, p.gate + at, there);
      grad_copy16(to + 8192, p.up + at, there);
#pragma unroll
      for (int w = 0; w < S::WORDS - 2; ++w)
        grad_copy16(to + (2 + w) * 8192, reinterpret_cast<const uint4 *>(static_cast<const T *>(p.dH) + at) + w, there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  load(blockIdx.x);
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t rblock = t / p.cb, cblock = t % p.cb;
    const int64_t r0 = rblock * 128 + 4 * ty, c0 = cblock * 128 + 8 * tx;
    const bool inside = c0 < p.C;
    float v[3][4][8];  // dgate, dup, h
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Eight<__nv_bfloat16> g, u;
      Eight<T> d;
      const uint32_t from = in + i * S::WORDS * 8192;
      g.w[0] = ld_shared_v4(from);
      u.w[0] = ld_shared_v4(from + 8192);
#pragma unroll
      for (int w = 0; w < S::WORDS - 2; ++w) d.w[w] = ld_shared_v4(from + (2 + w) * 8192);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const GatedGrad2 x = gated_grad<ACT>(two_of(g, e), two_of(u, e), two_of(d, e));
        v[0][i][2 * e] = x.dg.x;
        v[0][i][2 * e + 1] = x.dg.y;
        v[1][i][2 * e] = x.du.x;
        v[1][i][2 * e + 1] = x.du.y;
        v[2][i][2 * e] = x.h.x;
        v[2][i][2 * e + 1] = x.h.y;
      }
    }
    // columns' largest: of this thread's rows, of the warp's eight, then of all warps
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      if (!p.cols[m].codes) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float top = fmaxf(fmaxf(fabsf(v[m][0][e]), fabsf(v[m][1][e])), fmaxf(fabsf(v[m][2][e]), fabsf(v[m][3][e])));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
        if ((threadIdx.x & 16) == 0) tops[(m * 16 + warp) * 128 + 8 * tx + e] = top;
      }
    }
    __syncthreads();
    load(t + gridDim.x);
    // rows: a row's 128 values are 16 lanes'
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      __nv_bfloat16 *plain = m ? p.dup : p.dgate;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool there = inside && r0 + i < p.R;
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
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[m][i][e]));
#pragma unroll
        for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        top = fmaxf(top, kQ128Least);
        const float inv = __fdiv_rn(448.0f, top);
        if (there) {
          uint32_t w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            w[e] = mx_e4m3x2(v[m][i][4 * e] * inv, v[m][i][4 * e + 1] * inv) |
                   (mx_e4m3x2(v[m][i][4 * e + 2] * inv, v[m][i][4 * e + 3] * inv) << 16);
          *reinterpret_cast<uint2 *>(p.rows[m].codes + at) = make_uint2(w[0], w[1]);
          if (tx == 0) p.rows[m].scales[(r0 + i) * p.cb + cblock] = __fdiv_rn(top, 448.0f);
        }
      }
    }
    // the columns' reciprocals, in the place of the first warp's largest
    if (threadIdx.x < 384) {
      const int m = threadIdx.x >> 7, c = threadIdx.x & 127;
      if (p.cols[m].codes) {
        float top = kQ128Least;
#pragma unroll
        for (int w = 0; w < 16; ++w) top = fmaxf(top, tops[(m * 16 + w) * 128 + c]);
        tops[m * 16 * 128 + c] = __fdiv_rn(448.0f, top);
        if (cblock * 128 + c < p.C) p.cols[m].scales[(cblock * 128 + c) * p.rb + rblock] = __fdiv_rn(top, 448.0f);
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
    // (the next tile's largest are written after every thread has passed the second
    // barrier, and its words after two more)
  }
}

}  // namespace mxg
