// rope.cuh -- norms of queries and keys for each head with the rotation by
// positions in the same pass, and the gradient.
//
//   r = 1 / sqrt(mean x^2 + eps),  n = r x w,  y = factor R(pos) n
//   dn = factor R(pos)^T dy,  dw = sum dn r x,
//   dx = r (dn w - r x mean(dn w r x))
//
// R turns the pairs of a head's first `rot` values, pair j by the angle pos f_j;
// the others pass.  The angle of a far position has to be reduced to one turn
// before it is rounded to FP32: f_j / (2 pi) is held as a fixed-point fraction of
// a turn in 64 bits, and its product with the position, modulo 2^64, is the
// angle's fraction of a turn, exact but for the fraction's own 2^-53.  An integer
// product where FP64 would be far slower on this GPU.
//
// Bound by HBM: each value is read once and written once, and everything between
// happens in registers.  A head is D / 16 lanes, each with two runs of eight
// values that hold whole pairs in either layout (run s of the first half of the
// rotated values and run s of the second), so that a rotation needs no exchange
// between lanes.  Cosines and sines are computed once for a block's tokens and
// shared through shared memory by all heads.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace mxg {

struct RopeTensor {
  const void *x, *dy;
  void *out;  // y, or dx
  int64_t x_pitch, dy_pitch, out_pitch;
  const void *w;  // or null: no norm
  float *dw;
  int heads;
  int chunks;     // blocks along a token's heads (forward)
  int blocks;     // blocks of this tensor (backward)
};

struct RopeParams {
  RopeTensor t[2];  // queries, keys (no heads where there are none)
  int64_t tokens;
  int w_bf16;
  float eps, factor;
  const int32_t *positions;
  const double *freqs;
  int rot, interleaved;
  float *partials;     // backward: a row of D for each block, then one for each group of blocks
  unsigned *counters;  // backward: groups of queries, groups of keys, then one for each tensor
};

// Eight consecutive values (16-byte aligned) in FP32.
struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 load8(const float *p) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ F8 load8(const __nv_bfloat16 *p) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(u[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
  return r;
}
__device__ __forceinline__ void store8(float *p, const F8 &a) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(a.v[4], a.v[5], a.v[6], a.v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const F8 &a) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a.v[2 * i], a.v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ F8 load_weight8(const void *w, int at, int bf16) {
  return bf16 ? load8(static_cast<const __nv_bfloat16 *>(w) + at) : load8(static_cast<const float *>(w) + at);
}

// A frequency (radians a position) as a fraction of a turn, times 2^64.
__device__ __forceinline__ uint64_t turn_of(double freq) {
  const double t = freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}
// Cosine and sine of the angle at a position, times the factor.
__device__ __forceinline__ float2 angle_at(uint64_t turn, int pos, float factor) {
  const uint64_t a = turn * static_cast<uint64_t>(static_cast<int64_t>(pos));
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
  return make_float2(c * factor, s * factor);
}

template <int D>
struct RopeCfg {
  static constexpr int LANES = D / 16, HEADS = 32 / LANES;  // lanes of a head, heads of a warp
};

// The two runs of a head's lane, and whether they are rotated.
struct Runs {
  int a, b;
  bool turned;
};
__device__ __forceinline__ Runs runs_of(int sub, int rot) {
  const int n = rot >> 4;
  if (sub < n) return Runs{8 * sub, (rot >> 1) + 8 * sub, true};
  const int at = rot + 16 * (sub - n);
  return Runs{at, at + 8, false};
}

// The lane's eight angles of a token: cs holds its rot / 2.
__device__ __forceinline__ void lane_angles(const float2 *cs, int sub, int rot, int interleaved, bool turned, float2 (&k)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int j = !interleaved ? 8 * sub + e : e < 4 ? 4 * sub + e : (rot >> 2) + 4 * sub + e - 4;
    k[e] = turned ? cs[j] : make_float2(1.f, 0.f);
  }
}

// Pairs turned forward (BACK = false) or back.
template <bool BACK>
__device__ __forceinline__ void turn(F8 &a, F8 &b, const float2 (&k)[8], int interleaved) {
  auto one = [](float &x, float &y, float2 cs) {
    const float s = BACK ? -cs.y : cs.y, u = x, v = y;
    x = u * cs.x - v * s;
    y = v * cs.x + u * s;
  };
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      one(a.v[2 * e], a.v[2 * e + 1], k[e]);
      one(b.v[2 * e], b.v[2 * e + 1], k[4 + e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) one(a.v[e], b.v[e], k[e]);
  }
}

template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Angles of TT tokens from the block's first into cs.
template <int D, int TT>
__device__ __forceinline__ void block_angles(const RopeParams &p, int64_t first, float2 (*cs)[D / 2]) {
  const int half = p.rot >> 1;
  for (int i = threadIdx.x; i < TT * half; i += 256) {
    const int t = i / half, j = i - t * half;
    if (first + t < p.tokens) cs[t][j] = angle_at(turn_of(p.freqs[j]), p.positions[first + t], p.factor);
  }
}

// 256 threads: TT tokens, 8 / TT warps each; a warp takes HEADS heads at a time.
template <typename T, int D, int TT>
__global__ void __launch_bounds__(256) norm_rope_kernel(const RopeParams p) {
  using C = RopeCfg<D>;
  constexpr int WARPS = 8 / TT, STEP = WARPS * C::HEADS;  // warps of a token, heads of a pass
  __shared__ float2 cs[TT][D / 2];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % C::LANES;
  const int y = blockIdx.y;
  const RopeTensor &t = p.t[y < p.t[0].chunks ? 0 : 1];
  const int chunk = y < p.t[0].chunks ? y : y - p.t[0].chunks;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * TT, token = first + warp / WARPS;
  const int per = (t.heads + t.chunks * STEP - 1) / (t.chunks * STEP) * STEP;  // heads of a chunk
  const int h_end = min(t.heads, (chunk + 1) * per);
  const Runs r = runs_of(sub, p.rot);
  if (p.rot) {
    block_angles<D, TT>(p, first, cs);
    __syncthreads();
  }
  if (token >= p.tokens) return;
  float2 k[8];
  lane_angles(cs[warp / WARPS], sub, p.rot, p.interleaved, r.turned, k);
  F8 wa, wb;
  if (t.w) {
    wa = load_weight8(t.w, r.a, p.w_bf16);
    wb = load_weight8(t.w, r.b, p.w_bf16);
  }
  const T *x = static_cast<const T *>(t.x) + token * t.x_pitch;
  T *out = static_cast<T *>(t.out) + token * t.out_pitch;
#pragma unroll 2
  for (int h0 = chunk * per + (warp % WARPS) * C::HEADS; h0 < h_end; h0 += STEP) {
    const int h = h0 + lane / C::LANES;
    F8 a{}, b{};
    if (h < h_end) {
      a = load8(x + h * D + r.a);
      b = load8(x + h * D + r.b);
    }
    if (t.w) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(a.v[e], a.v[e], fmaf(b.v[e], b.v[e], sum));
      const float inv = 1.f / sqrtf(fmaf(head_sum<C::LANES>(sum), 1.f / D, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a.v[e] *= inv * wa.v[e];
        b.v[e] *= inv * wb.v[e];
      }
    }
    if (r.turned) turn<false>(a, b, k, p.interleaved);
    if (h < h_end) {
      store8(out + h * D + r.a, a);
      store8(out + h * D + r.b, b);
    }
  }
}

// Sum of `rows` rows of D partials by 256 threads into `to`, in a fixed order.
template <int D>
__device__ __forceinline__ void sum_rows(const float *from, int rows, float *to, float *part) {
  constexpr int PARTS = 256 / D;
  const int col = threadIdx.x % D, first = threadIdx.x / D;
  float s = 0.f;
#pragma unroll 8
  for (int i = first; i < rows; i += PARTS) s += __ldcg(from + static_cast<int64_t>(i) * D + col);
  part[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < D) {
    s = part[threadIdx.x];
#pragma unroll
    for (int i = 1; i < PARTS; ++i) s += part[threadIdx.x + i * D];
    to[threadIdx.x] = s;
  }
}

// Blocks of a tensor whose partials of dw are added together first.
__host__ __device__ constexpr int rope_group(int blocks) {
  int g = 1;
  while (g * g < blocks) ++g;
  return g;
}

// The gradient: 256 threads, a token a warp and HEADS heads at a time, blocks that
// stay for further tokens.  dw is summed in registers over a thread's tokens and
// heads, then over the block, and the blocks' sums are added by the block that
// arrives last, first in groups and then over the groups: no float atomics, so that
// equal calls give equal bits, and 25 rows to add at most where 608 would take one
// block longer than the rest of the call.
template <typename T, int D>
__global__ void __launch_bounds__(256) norm_rope_backward_kernel(const RopeParams p) {
  using C = RopeCfg<D>;
  __shared__ float2 cs[8][D / 2];
  __shared__ float sums[8][D];
  __shared__ int last;
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % C::LANES;
  const int which = static_cast<int>(blockIdx.x) < p.t[0].blocks ? 0 : 1;
  const RopeTensor &t = p.t[which];
  const int block = blockIdx.x - (which ? p.t[0].blocks : 0);
  const Runs r = runs_of(sub, p.rot);
  F8 wa, wb, da{}, db{};
  if (t.w) {
    wa = load_weight8(t.w, r.a, p.w_bf16);
    wb = load_weight8(t.w, r.b, p.w_bf16);
  }
  for (int64_t first = static_cast<int64_t>(block) * 8; first < p.tokens; first += static_cast<int64_t>(t.blocks) * 8) {
    if (p.rot) {
      __syncthreads();  // the angles before have been read
      block_angles<D, 8>(p, first, cs);
      __syncthreads();
    }
    const int64_t token = first + warp;
    if (token >= p.tokens) continue;
    float2 k[8];
    lane_angles(cs[warp], sub, p.rot, p.interleaved, r.turned, k);
    const T *dy = static_cast<const T *>(t.dy) + token * t.dy_pitch;
    const T *x = static_cast<const T *>(t.x) + token * t.x_pitch;
    T *dx = static_cast<T *>(t.out) + token * t.out_pitch;
    for (int h0 = 0; h0 < t.heads; h0 += C::HEADS) {
      const int h = h0 + lane / C::LANES;
      F8 ga{}, gb{}, xa{}, xb{};
      if (h < t.heads) {
        ga = load8(dy + h * D + r.a);
        gb = load8(dy + h * D + r.b);
        if (t.w) {
          xa = load8(x + h * D + r.a);
          xb = load8(x + h * D + r.b);
        }
      }
      if (r.turned) turn<true>(ga, gb, k, p.interleaved);
      if (t.w) {
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(xa.v[e], xa.v[e], fmaf(xb.v[e], xb.v[e], ss));
          sd = fmaf(ga.v[e] * wa.v[e], xa.v[e], fmaf(gb.v[e] * wb.v[e], xb.v[e], sd));
        }
        const float inv = 1.f / sqrtf(fmaf(head_sum<C::LANES>(ss), 1.f / D, p.eps));
        const float m = head_sum<C::LANES>(sd) * (1.f / D) * inv * inv;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          da.v[e] = fmaf(ga.v[e], xa.v[e] * inv, da.v[e]);
          db.v[e] = fmaf(gb.v[e], xb.v[e] * inv, db.v[e]);
          ga.v[e] = inv * (ga.v[e] * wa.v[e] - xa.v[e] * m);
          gb.v[e] = inv * (gb.v[e] * wb.v[e] - xb.v[e] * m);
        }
      }
      if (h < t.heads) {
        store8(dx + h * D + r.a, ga);
        store8(dx + h * D + r.b, gb);
      }
    }
  }
  if (!t.dw) return;
  // this block's row of dw: its warps' heads, then its warps
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = C::LANES; o < 32; o <<= 1) {
      da.v[e] += __shfl_xor_sync(0xFFFFFFFFu, da.v[e], o);
      db.v[e] += __shfl_xor_sync(0xFFFFFFFFu, db.v[e], o);
    }
    if (lane < C::LANES) {
      sums[warp][r.a + e] = da.v[e];
      sums[warp][r.b + e] = db.v[e];
    }
  }
  __syncthreads();
  float *rows = p.partials + static_cast<int64_t>(which ? p.t[0].blocks : 0) * D;
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][threadIdx.x];
    rows[static_cast<int64_t>(block) * D + threadIdx.x] = s;
  }
  // the last block of a group adds its rows, and the last group of the tensor the groups'
  const int g = rope_group(t.blocks), groups = (t.blocks + g - 1) / g, group = block / g;
  const int g0 = rope_group(p.t[0].blocks), groups0 = (p.t[0].blocks + g0 - 1) / g0;
  auto arrive = [&](unsigned *at, int all) -> bool {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      last = atomicAdd(at, 1u) == static_cast<unsigned>(all) - 1u;
      if (last) *at = 0;  // for the next launch
    }
    __syncthreads();
    __threadfence();
    return last != 0;
  };
  float *group_rows = p.partials + static_cast<int64_t>(p.t[0].blocks + p.t[1].blocks + (which ? groups0 : 0)) * D;
  float *part = &sums[0][0];
  if (!arrive(p.counters + 2 + (which ? groups0 : 0) + group, min(g, t.blocks - group * g))) return;
  sum_rows<D>(rows + static_cast<int64_t>(group) * g * D, min(g, t.blocks - group * g), group_rows + static_cast<int64_t>(group) * D, part);
  if (!arrive(p.counters + which, groups)) return;
  sum_rows<D>(group_rows, groups, t.dw, part);
}

}  // namespace mxg
