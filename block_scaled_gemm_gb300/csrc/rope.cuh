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
// a turn in 64 bits, rounded once (the quotient by 2 pi is formed as a sum of two
// doubles), and its product with the position, modulo 2^64, is the angle's fraction of a
// turn, off by 2^-64 a position: 2^-33 of a turn at position 2^31, whatever the frequency
// is.  An integer product where FP64 would be far slower on this GPU.
//
// Bound by HBM: each value is read once and written once, and everything between
// happens in registers.  A lane has two runs of 16 bytes of a head (eight values in
// BF16, four in FP32) that hold whole pairs in either layout (run s of the first half of
// the rotated values and run s of the second), so that a rotation needs no exchange
// between lanes.  All tokens' heads, as many at a time as a warp has lanes for, are cut
// into equal ranges for the warps, each of which works by itself: its lanes copy what they will
// read themselves into a ring in shared memory, some steps ahead (cp.async: what is
// on its way takes no registers), and it computes a token's cosines and sines once
// for all of that token's heads in its range.
//
// Measured: 8192 tokens, 32/8 heads of 128 in BF16, half of each rotated: 29.3 us (5.7
// TB/s, 0.84 of the measured copy rate; with blocks of tokens and their loads in
// registers 40 us, ranges of a tensor's parity 46, halves of sectors where values
// pass 35); 64 tokens 3.7 us.  The gradient, all of each head rotated: 53 us (4.7 TB/s;
// 105 us with loads in registers), bound by dependent instructions at the 16 warps an SM
// that its registers allow, with issue slots used to 51 % (runs of four values
// and 24 warps: 59 us).  In FP32 4112 tokens, all of each head rotated: 28.7 us (5.9
// TB/s; with runs of eight values, of which a copy takes every other 16 bytes,
// 40.6), the gradient 51.8 (69.6), whose 90 registers a thread leave 16 warps an SM too.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"
#include "tmem_util.cuh"

namespace mxg {

struct RopeTensor {
  const void *x, *dy;
  void *out;  // y, or dx
  int64_t x_pitch, dy_pitch, out_pitch;
  const void *w;  // or null: no norm
  float *dw;
  int heads;
  int steps;   // of a token: the heads that a warp takes at a time
  int blocks;  // of this tensor (backward)
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
  unsigned *counters;  // backward: one for each tensor, then groups of queries, groups of keys
};

// R consecutive values (a run: 16 bytes as they lie) in FP32, in pairs.
template <int R>
struct Run {
  float2 v[R / 2];
};
__device__ __forceinline__ Run<4> floats_of(uint4 w, float) {
  return Run<4>{{make_float2(__uint_as_float(w.x), __uint_as_float(w.y)), make_float2(__uint_as_float(w.z), __uint_as_float(w.w))}};
}
__device__ __forceinline__ Run<8> floats_of(uint4 w, __nv_bfloat16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  Run<8> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  return r;
}
__device__ __forceinline__ void store_run(float *p, const Run<4> &a) {
  *reinterpret_cast<float4 *>(p) = make_float4(a.v[0].x, a.v[0].y, a.v[1].x, a.v[1].y);
}
__device__ __forceinline__ void store_run(__nv_bfloat16 *p, const Run<8> &a) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __float22bfloat162_rn(a.v[i]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
// A lane's R values of a table in shared memory whose values 4 k .. + 3 are at
// [k][lane of the head]: 16-byte loads of a head's lanes lie side by side.
template <int R, int LANES>
__device__ __forceinline__ Run<R> shared_run(uint32_t at, int sub) {
  at += sub * 16;
  Run<R> r;
#pragma unroll
  for (int k = 0; k < R / 4; ++k) {
    const Run<4> four = floats_of(ld_shared_v4(at + k * LANES * 16), 0.f);
    r.v[2 * k] = four.v[0];
    r.v[2 * k + 1] = four.v[1];
  }
  return r;
}

// A frequency (radians a position, below 2^50) as a fraction of a turn, times 2^64.
// 1 / (2 pi) is two doubles, and the product's own rounding is added to the smaller part:
// one double alone would be off by 2^-53 of itself, more than FP32's angle from a product
// with the position of some 2^28 on.
__device__ __forceinline__ uint64_t turn_of(double freq) {
  constexpr double kHigh = 0.15915494309189533577, kLow = -9.839338337591243e-18;
  const double t = freq * kHigh, rest = fma(freq, kLow, fma(freq, kHigh, -t));
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0) + static_cast<uint64_t>(__double2ll_rn(rest * 18446744073709551616.0));
}
// Cosine and sine of the angle at a position, times the factor.
__device__ __forceinline__ float2 angle_at(uint64_t turn, int pos, float factor) {
  const uint64_t a = turn * static_cast<uint64_t>(static_cast<int64_t>(pos));
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
  return make_float2(c * factor, s * factor);
}

template <typename T, int D, bool BACK>
struct RopeCfg {
  static constexpr int RUN = 16 / sizeof(T);                       // values of a run
  static constexpr int LANES = D / (2 * RUN), HEADS = 32 / LANES;  // lanes of a head, heads of a warp
  static constexpr int PIECES = BACK ? 4 : 2;                      // runs of a lane: dy and x, or x
  // Warps of a block, blocks of an SM, and loads of a warp on their way plus one.  The
  // gradient's registers in BF16 allow 16 warps without spills: 8192 tokens, 32/8 heads, 53
  // us so, 56 with four stages, 62 with two, 60 with 20 warps, 63 with 8.
  static constexpr int WARPS = 8, BLOCKS = BACK ? 2 : 4, STAGES = BACK ? 3 : 4;
  static constexpr int OFF_TURN = 0;                        // [D / 2] turns a position
  static constexpr int OFF_W = OFF_TURN + D / 2 * 8;        // [2][runs a, b][D / 2] weights
  static constexpr int OFF_CS = OFF_W + 2 * D * 4;          // [warps][cosines, sines][D / 2]
  static constexpr int OFF_POS = OFF_CS + WARPS * D / 2 * 8;  // [warps][STAGES] positions
  static constexpr int OFF_RING = (OFF_POS + WARPS * STAGES * 4 + 15) / 16 * 16;  // [warps][STAGES][PIECES][32 lanes] runs
  static constexpr int SMEM_BYTES = OFF_RING + WARPS * STAGES * PIECES * 512;
  static_assert(OFF_RING % 16 == 0, "alignment");
};

// The two runs of a head's lane, and whether they are rotated.
struct Runs {
  int a, b;
  bool turned;
};
// (the lanes' first runs lie side by side, and so do the second)
template <int D, int R>
__device__ __forceinline__ Runs runs_of(int sub, int rot) {
  const int n = rot / (2 * R);
  if (sub < n) return Runs{R * sub, (rot >> 1) + R * sub, true};
  const int at = rot + R * (sub - n);
  return Runs{at, at + ((D - rot) >> 1), false};
}

// Where pair j of a token's rot / 2 is in such a table of cosines (or sines).
template <int R, int LANES>
__device__ __forceinline__ int pair_place(int j, int rot, int interleaved) {
  int sub = j / R, e = j % R;
  if (interleaved) {  // a lane has R / 2 pairs in each run
    const bool second = j >= rot >> 2;
    if (second) j -= rot >> 2;
    sub = j / (R / 2);
    e = j % (R / 2) + (second ? R / 2 : 0);
  }
  return ((e >> 2) * LANES + sub) * 4 + (e & 3);
}
__device__ __forceinline__ uint32_t rope_shared_word(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void rope_store_word(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
// A lane's pairs turned forward, or back, by its cosines and sines.
template <bool BACK, int R>
__device__ __forceinline__ void turn(Run<R> &a, Run<R> &b, const Run<R> &c, const Run<R> &s, int interleaved) {
  if (interleaved) {  // (x, y) -> (x, y) c + (y, x) (-s, s)
#pragma unroll
    for (int e = 0; e < R; ++e) {
      float2 &x = e < R / 2 ? a.v[e] : b.v[e - R / 2];
      const float cc = e & 1 ? c.v[e >> 1].y : c.v[e >> 1].x, ss = e & 1 ? s.v[e >> 1].y : s.v[e >> 1].x, t = BACK ? -ss : ss;
      x = fma2(make_float2(x.y, x.x), make_float2(-t, t), mul2(x, make_float2(cc, cc)));
    }
  } else {
#pragma unroll
    for (int e = 0; e < R / 2; ++e) {
      const float2 t = BACK ? make_float2(-s.v[e].x, -s.v[e].y) : s.v[e], u = a.v[e], v = b.v[e];
      a.v[e] = fma2(v, make_float2(-t.x, -t.y), mul2(u, c.v[e]));
      b.v[e] = fma2(u, t, mul2(v, c.v[e]));
    }
  }
}

template <int LANES>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

__device__ __forceinline__ void rope_copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void rope_copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Where a warp is: a token, step j of it (the queries' steps, then the keys'), and
// this lane's head there.  Pointers and the head move on by additions; what depends on
// the tensor and the token is found anew where those change.
template <typename T>
struct RopeAt {
  int token, j, left;  // left: steps of the warp's range
  int h;
  T *a, *b;  // the head's first run in one or two matrices
};

// One warp's walk over its range of the steps of all tokens: the ring of loads that
// is ahead of it, and the angles of the token that it has reached.  Its state is kept
// small: the registers decide how many blocks an SM holds.
template <typename T, int D, bool BACK>
struct RopeWalk {
  using C = RopeCfg<T, D, BACK>;
  using F = Run<C::RUN>;
  const RopeParams &p;
  const int only;  // backward: the one tensor
  uint32_t sm;     // the block's shared memory
  int sub, apart;  // lane of the head; from its first run to its second
  RopeAt<T> at, ahead;  // at: a is the result; ahead: a is dy (backward), and b, or a, x
  int stage, filled;
  int angles_of;  // the token whose angles are there

  // warp `w` of `warps`
  __device__ RopeWalk(const RopeParams &p_, uint32_t sm_, int64_t w, int64_t warps, int which)
      : p(p_), only(which), sm(sm_), sub(threadIdx.x % C::LANES), stage(0), filled(0), angles_of(-1) {
    const Runs r = runs_of<D, C::RUN>(sub, p.rot);
    apart = r.b - r.a;
    const int64_t all = p.tokens * of_token(), u0 = w * all / warps;
    at.token = static_cast<int>(u0 / of_token());
    at.j = static_cast<int>(u0 - static_cast<int64_t>(at.token) * of_token());
    at.left = static_cast<int>((w + 1) * all / warps - u0);
    at.h = 0;
    at.a = at.b = nullptr;
    ahead = at;
    enter<false>(at);
    enter<true>(ahead);
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) load();
  }
  __device__ int first() const { return p.t[BACK ? only : 0].steps; }  // steps of a token before the keys'
  __device__ int of_token() const { return BACK ? first() : first() + p.t[1].steps; }
  __device__ int which(const RopeAt<T> &a) const { return BACK ? only : a.j >= first(); }
  __device__ uint32_t ring(int st) const {
    return sm + C::OFF_RING + (((threadIdx.x >> 5) * C::STAGES + st) * C::PIECES * 32 + (threadIdx.x & 31)) * 16;
  }
  __device__ uint32_t position(int st) const { return sm + C::OFF_POS + ((threadIdx.x >> 5) * C::STAGES + st) * 4; }
  __device__ uint32_t angles() const { return sm + C::OFF_CS + (threadIdx.x >> 5) * (D * 4); }
  template <bool LOADS>
  __device__ void enter(RopeAt<T> &a) const {
    const RopeTensor &t = p.t[which(a)];
    a.h = (a.j - (!BACK && which(a) ? first() : 0)) * C::HEADS + (threadIdx.x & 31) / C::LANES;
    const int64_t in_row = static_cast<int64_t>(a.h) * D + runs_of<D, C::RUN>(sub, p.rot).a, token = a.token;
    if (LOADS) {
      a.a = static_cast<T *>(const_cast<void *>(BACK ? t.dy : t.x)) + token * (BACK ? t.dy_pitch : t.x_pitch) + in_row;
      if (BACK) a.b = static_cast<T *>(const_cast<void *>(t.x)) + token * t.x_pitch + in_row;
    } else {
      a.a = static_cast<T *>(t.out) + token * t.out_pitch + in_row;
    }
  }
  template <bool LOADS>
  __device__ void next(RopeAt<T> &a) const {
    --a.left;
    ++a.j;
    if (a.j == first() || (!BACK && a.j == of_token())) {
      if (BACK || a.j == of_token()) {
        a.j = 0;
        ++a.token;
      }
      enter<LOADS>(a);
    } else {
      a.h += C::HEADS;
      a.a += C::HEADS * D;
      if (BACK && LOADS) a.b += C::HEADS * D;
    }
  }
  __device__ bool more() const { return at.left > 0; }
  __device__ bool live() const { return at.h < p.t[which(at)].heads; }
  __device__ bool norm() const { return p.t[which(at)].w != nullptr; }
  // The loads of the place that is ahead, into the next stage (an empty group past the end).
  __device__ void load() {
    if (ahead.left > 0) {
      if (ahead.h < p.t[which(ahead)].heads) {
        const uint32_t to = ring(filled);
#pragma unroll
        for (int k = 0; k < (BACK ? 2 : 1); ++k) {  // dy, then x
          if (k == 1 && !p.t[only].w) continue;
          const T *from = k ? ahead.b : ahead.a;
          rope_copy16(to + k * 1024, from);
          rope_copy16(to + k * 1024 + 512, from + apart);
        }
      }
      if ((threadIdx.x & 31) == 0 && p.rot) rope_copy4(position(filled), p.positions + ahead.token);
      next<true>(ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    filled = filled + 1 == C::STAGES ? 0 : filled + 1;
  }
  // Waits for the place that has been reached, and its token's angles.
  __device__ void arrive() {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::STAGES - 2) : "memory");
    __syncwarp();
    if (p.rot && at.token != angles_of) {
      angles_of = at.token;
      const int pos = static_cast<int>(rope_shared_word(position(stage)));
      for (int j = threadIdx.x & 31; j < p.rot >> 1; j += 32) {
        uint64_t turns;
        asm volatile("ld.shared.b64 %0, [%1];" : "=l"(turns) : "r"(sm + C::OFF_TURN + j * 8) : "memory");
        const float2 a = angle_at(turns, pos, p.factor);
        const uint32_t to = angles() + pair_place<C::RUN, C::LANES>(j, p.rot, p.interleaved) * 4;
        rope_store_word(to, __float_as_uint(a.x));
        rope_store_word(to + D * 2, __float_as_uint(a.y));
      }
      __syncwarp();
    }
  }
  template <bool BACKWARD>
  __device__ void turned(F &a, F &b) const {
    if (sub < p.rot / (2 * C::RUN))
      turn<BACKWARD>(a, b, shared_run<C::RUN, C::LANES>(angles(), sub), shared_run<C::RUN, C::LANES>(angles() + D * 2, sub), p.interleaved);
  }
  // This lane's weights of the tensor's run `i`.
  __device__ F weights(int i) const { return shared_run<C::RUN, C::LANES>(sm + C::OFF_W + (2 * which(at) + i) * (D * 2), sub); }
  // Run `i` (0, 1) of tensor k (0: dy where there is one, 1: then x).
  __device__ F run(int k, int i) const {
    return floats_of(ld_shared_v4(ring(stage) + (k * 2 + i) * 512), T{});
  }
  __device__ void store(const F &a, const F &b) const {
    if (live()) {
      store_run(at.a, a);
      store_run(at.a + apart, b);
    }
  }
  // Past this place: its stage has been read by this lane (and, positions, by the warp).
  __device__ void advance() {
    __syncwarp();
    load();
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;
    next<false>(at);
  }
};

// Turns a position and weights of both tensors into shared memory.
template <typename T, int D, bool BACK>
__device__ __forceinline__ void rope_tables(const RopeParams &p, uint8_t *sm) {
  using C = RopeCfg<T, D, BACK>;
  for (int j = threadIdx.x; j < p.rot >> 1; j += 32 * C::WARPS) reinterpret_cast<uint64_t *>(sm + C::OFF_TURN)[j] = turn_of(p.freqs[j]);
  for (int i = threadIdx.x; i < 2 * D; i += 32 * C::WARPS) {
    // value e of run `run` of lane `sub`, of tensor i / D
    const int run = i / C::RUN % 2, sub = i % D / (2 * C::RUN), e = i % C::RUN;
    const Runs r = runs_of<D, C::RUN>(sub, p.rot);
    const int from = (run ? r.b : r.a) + e;
    const void *w = p.t[i / D].w;
    if (w)
      reinterpret_cast<float *>(sm + C::OFF_W)[(i / D * 2 + run) * (D / 2) + ((e >> 2) * C::LANES + sub) * 4 + (e & 3)] =
          p.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[from]) : static_cast<const float *>(w)[from];
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * RopeCfg<T, D, false>::WARPS, RopeCfg<T, D, false>::BLOCKS) norm_rope_kernel(const RopeParams p) {
  using C = RopeCfg<T, D, false>;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  griddep_launch_dependents();
  griddep_wait();
  RopeWalk<T, D, false> walk(p, smem_u32(rope_smem), static_cast<int64_t>(blockIdx.x) * C::WARPS + (threadIdx.x >> 5),
                                static_cast<int64_t>(gridDim.x) * C::WARPS, 0);
  rope_tables<T, D, false>(p, rope_smem);
  __syncthreads();
  for (; walk.more(); walk.advance()) {
    walk.arrive();
    Run<C::RUN> a = walk.run(0, 0), b = walk.run(0, 1);
    if (walk.norm()) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < C::RUN / 2; ++e) sum = fma2(a.v[e], a.v[e], fma2(b.v[e], b.v[e], sum));
      const float inv = rsqrtf(fmaf(head_sum<C::LANES>(sum.x + sum.y), 1.f / D, p.eps));
      const Run<C::RUN> wa = walk.weights(0), wb = walk.weights(1);
#pragma unroll
      for (int e = 0; e < C::RUN / 2; ++e) {
        a.v[e] = mul2(mul2(a.v[e], make_float2(inv, inv)), wa.v[e]);
        b.v[e] = mul2(mul2(b.v[e], make_float2(inv, inv)), wb.v[e]);
      }
    }
    walk.template turned<false>(a, b);
    walk.store(a, b);
  }
}

// Sum of `rows` rows of D partials by a block's first 256 threads into `to`, in a fixed order.
template <int D>
__device__ __forceinline__ void sum_rows(const float *from, int rows, float *to, float *part) {
  constexpr int PARTS = 256 / D;
  const int col = threadIdx.x % D, first = threadIdx.x / D;
  float s = 0.f;
#pragma unroll 8
  for (int i = first; i < rows && first < PARTS; i += PARTS) s += __ldcg(from + static_cast<int64_t>(i) * D + col);
  if (first < PARTS) part[threadIdx.x] = s;
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

// The gradient: blocks that stay for further tokens.  dw is summed in registers over a thread's tokens and
// heads, then over the block, and the blocks' sums are added by the block that
// arrives last, first in groups and then over the groups: no float atomics, so that
// equal calls give equal bits, and 25 rows to add at most where 608 would take one
// block longer than the rest of the call.
template <typename T, int D>
__global__ void __launch_bounds__(32 * RopeCfg<T, D, true>::WARPS, RopeCfg<T, D, true>::BLOCKS) norm_rope_backward_kernel(const RopeParams p) {
  using C = RopeCfg<T, D, true>;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  __shared__ float sums[C::WARPS][D];
  __shared__ int last;
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int which = static_cast<int>(blockIdx.x) < p.t[0].blocks ? 0 : 1;
  const RopeTensor &t = p.t[which];
  const int block = blockIdx.x - (which ? p.t[0].blocks : 0);
  RopeWalk<T, D, true> walk(p, smem_u32(rope_smem), static_cast<int64_t>(block) * C::WARPS + warp, static_cast<int64_t>(t.blocks) * C::WARPS,
                               which);
  rope_tables<T, D, true>(p, rope_smem);
  __syncthreads();
  using F = Run<C::RUN>;
  F da{}, db{};
  for (; walk.more(); walk.advance()) {
    walk.arrive();
    F ga = walk.run(0, 0), gb = walk.run(0, 1);
    walk.template turned<true>(ga, gb);
    if (t.w) {
      // (values and weights are read twice from shared memory, not held)
      float2 ss = make_float2(0.f, 0.f), sd = ss;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const F &g = i ? gb : ga, x = walk.run(1, i), w = walk.weights(i);
#pragma unroll
        for (int e = 0; e < C::RUN / 2; ++e) {
          ss = fma2(x.v[e], x.v[e], ss);
          sd = fma2(mul2(g.v[e], w.v[e]), x.v[e], sd);
        }
      }
      const float inv = rsqrtf(fmaf(head_sum<C::LANES>(ss.x + ss.y), 1.f / D, p.eps));
      const float m = -head_sum<C::LANES>(sd.x + sd.y) * (1.f / D) * inv * inv * inv;
      // (a stage that nothing was copied to holds anything)
      const bool live = walk.live();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        F &g = i ? gb : ga, &d = i ? db : da;
        const F x = walk.run(1, i), w = walk.weights(i);
#pragma unroll
        for (int e = 0; e < C::RUN / 2; ++e) {
          const float2 r = mul2(g.v[e], make_float2(inv, inv));
          if (live) d.v[e] = fma2(r, x.v[e], d.v[e]);
          g.v[e] = fma2(r, w.v[e], mul2(x.v[e], make_float2(m, m)));
        }
      }
    }
    walk.store(ga, gb);
  }
  if (!t.dw) return;
  // this block's row of dw: its warps' heads, then its warps
  const Runs r = runs_of<D, C::RUN>(lane % C::LANES, p.rot);
#pragma unroll
  for (int e = 0; e < C::RUN; ++e) {
    float a = e & 1 ? da.v[e >> 1].y : da.v[e >> 1].x, b = e & 1 ? db.v[e >> 1].y : db.v[e >> 1].x;
#pragma unroll
    for (int o = C::LANES; o < 32; o <<= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (lane < C::LANES) {
      sums[warp][r.a + e] = a;
      sums[warp][r.b + e] = b;
    }
  }
  __syncthreads();
  float *rows = p.partials + static_cast<int64_t>(which ? p.t[0].blocks : 0) * D;
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) s += sums[w][threadIdx.x];
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
