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
//
// Measured: 4096 x 28672, BF16 dH, to five quantized operands 226 us (5.8 TB/s, 0.86 of
// the measured copy rate; with one tile a block and its loads in registers 501 us, with
// scalar operations and a division for each row by all lanes 321 us, with the next
// tile's loads after the first barrier 240 us): issue slots are used to half.  4096 x
// 14336, FP32 dH, 124 us (6.2 TB/s; with each thread copying its own 32 bytes 146).
// 1741 x 7000, FP32 dH, to BF16 17.9 us with inputs in L2.
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
  static constexpr int OFF_TOP = 0;                            // [3][32 ty][128 columns] largest values
  static constexpr int OFF_INV = OFF_TOP + 3 * 32 * 128 * 4;   // [3][128 columns] reciprocals
  static constexpr int OFF_TILE = OFF_INV + 3 * 128 * 4;       // [3][128 columns][32 words]
  static constexpr int OFF_IN = OFF_TILE + 3 * 128 * 32 * 4;   // the next tile: [4 rows][WORDS][512 threads] words
  static constexpr int SMEM_BYTES = OFF_IN + 4 * WORDS * 512 * 16;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// 16 bytes to shared memory, zeros where `there` is false.
__device__ __forceinline__ void grad_copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ float abs_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return mx_e4m3x2(a, b) | (mx_e4m3x2(c, d) << 16); }

// One block of 512 threads an SM, which goes from tile to tile and copies the next
// one's values to shared memory, a row as soon as this tile's has been read from there
// (each thread copies what it, or a lane beside it, will read).  Thread (ty, tx) has rows 4 ty .. +3 of columns 8 tx ..
// +7, so that the four rows' codes of a column are one word of the transposed tile.
// Issue slots are as short as bandwidth: operations go in pairs, and a row's largest
// values are exchanged so that each lane ends with one of them and divides once.
template <typename T, int ACT>
__global__ void __launch_bounds__(512, 1) gated_grad_tile_kernel(const GatedGradParams p) {
  using S = GatedGradCfg<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  float *tops = reinterpret_cast<float *>(smem + S::OFF_TOP);
  float *invs = reinterpret_cast<float *>(smem + S::OFF_INV);
  uint32_t *tile = reinterpret_cast<uint32_t *>(smem + S::OFF_TILE);
  griddep_launch_dependents();
  griddep_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const uint32_t in = smem_u32(smem + S::OFF_IN) + threadIdx.x * 16;
  const uint32_t tiles = static_cast<uint32_t>(p.rb * p.cb), cb = static_cast<uint32_t>(p.cb);
  // a tile's place in the matrices, for this thread: how many of its rows are there, and
  // columns of the tile
  struct Place {
    int64_t at;
    int rows, cols;
  };
  auto place = [&](uint32_t t) {
    const uint32_t rblock = t / cb, cblock = t - rblock * cb;
    const int64_t r0 = static_cast<int64_t>(rblock) * 128 + 4 * ty, c0 = static_cast<int64_t>(cblock) * 128;
    return Place{r0 * p.C + c0 + 8 * tx, t < tiles ? static_cast<int>(min(static_cast<int64_t>(4), p.R - r0)) : 0,
                 static_cast<int>(min(static_cast<int64_t>(128), p.C - c0))};
  };
  // Row i of a tile.  A row's FP32 dH is 32 copies by 16 lanes: lane tx takes those of
  // columns 4 tx and 64 + 4 tx, so that copies lie side by side, and reads 8 tx and
  // 8 tx + 4, copies of its neighbours (the warp meets before it reads, and before the
  // next copies).
  auto load = [&](int i, const Place &a) {
    const bool row = i < a.rows, there = row && 8 * tx < a.cols;
    const int64_t from = there ? a.at + i * p.C : 0;
    const uint32_t to = in + i * S::WORDS * 8192;
    grad_copy16(to, p.gate + from, there);
    grad_copy16(to + 8192, p.up + from, there);
    if constexpr (sizeof(T) == 4) {
      __syncwarp();
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const bool four = row && 64 * w + 4 * tx < a.cols;
        grad_copy16(to + (2 + w) * 8192, static_cast<const T *>(p.dH) + (four ? a.at + i * p.C + 64 * w - 4 * tx : 0), four);
      }
    } else {
      grad_copy16(to + 16384, static_cast<const T *>(p.dH) + from, there);
    }
  };
  {
    const Place first = place(blockIdx.x);
#pragma unroll
    for (int i = 0; i < 4; ++i) load(i, first);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const uint32_t rblock = t / cb, cblock = t - rblock * cb;
    const int64_t r0 = static_cast<int64_t>(rblock) * 128 + 4 * ty, c0 = static_cast<int64_t>(cblock) * 128 + 8 * tx;
    const int rows = c0 < p.C ? static_cast<int>(min(static_cast<int64_t>(4), p.R - r0)) : 0;
    float2 v[3][4][4];  // dgate, dup, h: [row][columns 2 e, + 1]
    const Place next = place(t + gridDim.x);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (sizeof(T) == 4) __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Eight<__nv_bfloat16> g, u;
      Eight<T> d;
      const uint32_t from = in + i * S::WORDS * 8192;
      g.w[0] = ld_shared_v4(from);
      u.w[0] = ld_shared_v4(from + 8192);
      if constexpr (sizeof(T) == 4) {
        const uint32_t two = from + 16384 + (tx >> 3) * 8192 + (((2 * tx) & 15) - tx) * 16;
        d.w[0] = ld_shared_v4(two);
        d.w[1] = ld_shared_v4(two + 16);
      } else {
        d.w[0] = ld_shared_v4(from + 16384);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const GatedGrad2 x = gated_grad<ACT>(two_of(g, e), two_of(u, e), two_of(d, e));
        v[0][i][e] = x.dg;
        v[1][i][e] = x.du;
        v[2][i][e] = x.h;
      }
      load(i, next);  // into what has just been read
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // columns' largest of this thread's rows
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      float c[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[2 * e] = abs_max3(fmaxf(fabsf(v[m][0][e].x), fabsf(v[m][1][e].x)), v[m][2][e].x, v[m][3][e].x);
        c[2 * e + 1] = abs_max3(fmaxf(fabsf(v[m][0][e].y), fabsf(v[m][1][e].y)), v[m][2][e].y, v[m][3][e].y);
      }
      float4 *to = reinterpret_cast<float4 *>(tops + (m * 32 + ty) * 128 + 8 * tx);
      to[0] = make_float4(c[0], c[1], c[2], c[3]);
      to[1] = make_float4(c[4], c[5], c[6], c[7]);
    }
    __syncthreads();
    // the columns' reciprocals and scales
    if (threadIdx.x < 384) {
      const int m = threadIdx.x >> 7, c = threadIdx.x & 127;
      float top = kQ128Least;
      const float *from = tops + m * 32 * 128 + c;
#pragma unroll
      for (int w = 0; w < 32; w += 2) top = abs_max3(top, from[w * 128], from[(w + 1) * 128]);
      invs[threadIdx.x] = __fdiv_rn(448.0f, top);
      const int64_t col = static_cast<int64_t>(cblock) * 128 + c;
      if (p.cols[m].codes && col < p.C) p.cols[m].scales[col * p.rb + rblock] = __fdiv_rn(top, 448.0f);
    }
    // rows: a row's 128 values are 16 lanes'.  Of the eight rows of both matrices,
    // lane tx comes to hold the largest value of row (tx / 2) % 4 of matrix tx / 8.
    float inv;
    {
      float a[8], b[4], c[2];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2(&x)[4] = v[k >> 2][k & 3];
        a[k] = abs_max3(abs_max3(abs_max3(fmaxf(fabsf(x[0].x), fabsf(x[0].y)), x[1].x, x[1].y), x[2].x, x[2].y), x[3].x, x[3].y);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        b[k] = fmaxf(tx & 8 ? a[k + 4] : a[k], __shfl_xor_sync(0xFFFFFFFFu, tx & 8 ? a[k] : a[k + 4], 8));
#pragma unroll
      for (int k = 0; k < 2; ++k)
        c[k] = fmaxf(tx & 4 ? b[k + 2] : b[k], __shfl_xor_sync(0xFFFFFFFFu, tx & 4 ? b[k] : b[k + 2], 4));
      float top = fmaxf(tx & 2 ? c[1] : c[0], __shfl_xor_sync(0xFFFFFFFFu, tx & 2 ? c[0] : c[1], 2));
      top = fmaxf(fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1)), kQ128Least);
      inv = __fdiv_rn(448.0f, top);
      const Blocks128 &to = p.rows[tx >> 3];
      const int64_t row = r0 + ((tx >> 1) & 3);
      if ((tx & 1) == 0 && to.codes && row < p.R) to.scales[row * p.cb + cblock] = __fdiv_rn(top, 448.0f);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      int64_t at = r0 * p.C + c0;
      __nv_bfloat16 *plain = m ? p.dup : p.dgate;
      uint8_t *codes = p.rows[m].codes;
#pragma unroll
      for (int i = 0; i < 4; ++i, at += p.C) {
        const float2(&x)[4] = v[m][i];
        if (plain && i < rows) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __float22bfloat162_rn(x[e]);
            w[e] = *reinterpret_cast<const uint32_t *>(&b);
          }
          *reinterpret_cast<uint4 *>(plain + at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (!codes) continue;
        const float k = __shfl_sync(0xFFFFFFFFu, inv, (threadIdx.x & 16) | (8 * m + 2 * i));
        float2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = mul2(x[e], make_float2(k, k));
        if (i < rows)
          *reinterpret_cast<uint2 *>(codes + at) = make_uint2(e4m3x4(y[0].x, y[0].y, y[1].x, y[1].y), e4m3x4(y[2].x, y[2].y, y[3].x, y[3].y));
      }
    }
    __syncthreads();
    // word ty of column c is at ty ^ 2 (c / 8): neither the stores nor the 16-byte
    // loads meet in a bank
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      if (!p.cols[m].codes) continue;
      const float4 ka = *reinterpret_cast<const float4 *>(invs + m * 128 + 8 * tx), kb = *reinterpret_cast<const float4 *>(invs + m * 128 + 8 * tx + 4);
      const float2 k[4] = {make_float2(ka.x, ka.y), make_float2(ka.z, ka.w), make_float2(kb.x, kb.y), make_float2(kb.z, kb.w)};
      uint32_t *to = tile + (m * 128 + 8 * tx) * 32 + (ty ^ (2 * tx));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(v[m][i][e], k[e]);
        to[2 * e * 32] = e4m3x4(y[0].x, y[1].x, y[2].x, y[3].x);
        to[(2 * e + 1) * 32] = e4m3x4(y[0].y, y[1].y, y[2].y, y[3].y);
      }
    }
    __syncthreads();
    const int part = threadIdx.x & 7, c = threadIdx.x >> 3;
    const int64_t col = static_cast<int64_t>(cblock) * 128 + c, row = static_cast<int64_t>(rblock) * 128 + 16 * part;
    const int64_t to = col * p.pitch + row;
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      if (!p.cols[m].codes) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = (c >> 3) + 8 * i;
        uint4 w = *reinterpret_cast<const uint4 *>(tile + (m * 128 + c + 64 * i) * 32 + 4 * (part ^ (x >> 1)));
        if (x & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        if (col + 64 * i < p.C && row < p.pitch) *reinterpret_cast<uint4 *>(p.cols[m].codes + to + 64 * i * p.pitch) = w;
      }
    }
    // (the next tile's largest are written after every thread has passed the second
    // barrier, its reciprocals after the third, and its words after two more)
  }
}

}  // namespace mxg
