// rope.cu -- norms of queries and keys with the rotation by positions: argument
// checks and launches of mxgemm_norm_rope and mxgemm_norm_rope_backward, and the
// frequencies of mxgemm_rope_frequencies.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "context.h"
#include "launch.h"
#include "mxgemm.h"
#include "rope.cuh"

namespace {

using mxg::aligned;
using mxg::cdiv;
using mxg::kLim;

// One tensor's checks but for its pointers' device, and the kernels' view of it.
int tensor_args(const mxgemm_heads_t *a, int64_t tokens, int64_t head_dim, int w_dtype, bool back, mxg::RopeTensor *t) {
  std::memset(t, 0, sizeof(*t));
  if (!a || a->heads == 0) return MXGEMM_OK;
  if (a->heads < 0 || a->heads >= (1 << 16) || tokens * a->heads >= kLim) return MXGEMM_ERR_INVALID_VALUE;
  const int64_t row = a->heads * head_dim;
  const bool need_x = !back || a->weight;
  if ((need_x && a->x_pitch < row) || a->out_pitch < row || (back && a->dy_pitch < row)) return MXGEMM_ERR_INVALID_VALUE;
  if (a->dweight && (!back || !a->weight)) return MXGEMM_ERR_INVALID_VALUE;
  t->heads = static_cast<int>(a->heads);
  if (tokens == 0) return MXGEMM_OK;
  if ((need_x && !a->x) || !a->out || (back && !a->dy)) return MXGEMM_ERR_INVALID_VALUE;
  const size_t w_al = w_dtype == MXGEMM_IN_F32 ? 4 : 2;
  if ((need_x && (!aligned(a->x, 16) || a->x_pitch % 8 != 0)) || !aligned(a->out, 16) || a->out_pitch % 8 != 0 ||
      (back && (!aligned(a->dy, 16) || a->dy_pitch % 8 != 0)) || (a->weight && !aligned(a->weight, w_al)) ||
      !aligned(a->dweight, 4))
    return MXGEMM_ERR_MISALIGNED;
  t->x = need_x ? a->x : nullptr;
  t->dy = back ? a->dy : nullptr;
  t->out = a->out;
  t->x_pitch = a->x_pitch;
  t->dy_pitch = a->dy_pitch;
  t->out_pitch = a->out_pitch;
  t->w = a->weight;
  t->dw = a->dweight;
  return MXGEMM_OK;
}

int rope_args(int device, const mxgemm_heads_t *q, const mxgemm_heads_t *k, int64_t tokens, int64_t head_dim,
              int x_dtype, int w_dtype, float eps, const mxgemm_rope_t *rope, bool back, mxg::RopeParams *p) {
  if (tokens < 0 || tokens >= kLim || (head_dim != 64 && head_dim != 128)) return MXGEMM_ERR_INVALID_VALUE;
  if ((x_dtype != MXGEMM_IN_F32 && x_dtype != MXGEMM_IN_BF16) || (w_dtype != MXGEMM_IN_F32 && w_dtype != MXGEMM_IN_BF16))
    return MXGEMM_ERR_INVALID_VALUE;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return MXGEMM_ERR_INVALID_VALUE;
  std::memset(p, 0, sizeof(*p));
  p->factor = 1.f;
  if (rope && rope->rot != 0) {
    if (rope->rot < 0 || rope->rot > head_dim || rope->rot % 16 != 0 || (rope->interleaved != 0 && rope->interleaved != 1) ||
        !std::isfinite(rope->factor))
      return MXGEMM_ERR_INVALID_VALUE;
    if (tokens > 0) {
      if (!rope->positions || !rope->freqs) return MXGEMM_ERR_INVALID_VALUE;
      if (!aligned(rope->positions, 4) || !aligned(rope->freqs, 8)) return MXGEMM_ERR_MISALIGNED;
    }
    p->positions = rope->positions;
    p->freqs = rope->freqs;
    p->rot = rope->rot;
    p->interleaved = rope->interleaved;
    p->factor = rope->factor;
  }
  p->tokens = tokens;
  p->w_bf16 = w_dtype == MXGEMM_IN_BF16;
  p->eps = eps;
  if (int st = tensor_args(q, tokens, head_dim, w_dtype, back, &p->t[0])) return st;
  if (int st = tensor_args(k, tokens, head_dim, w_dtype, back, &p->t[1])) return st;
  if (tokens == 0 || p->t[0].heads + p->t[1].heads == 0) return MXGEMM_OK;
  for (const void *x : {static_cast<const void *>(p->positions), static_cast<const void *>(p->freqs)})
    if (x && !mxg::pointer_on_device(x, device)) return MXGEMM_ERR_INVALID_VALUE;
  for (const mxg::RopeTensor &t : p->t)
    for (const void *x : {t.x, t.dy, static_cast<const void *>(t.out), t.w, static_cast<const void *>(t.dw)})
      if (x && !mxg::pointer_on_device(x, device)) return MXGEMM_ERR_INVALID_VALUE;
  return MXGEMM_OK;
}

// Steps of a token: a warp's heads at a time.
template <typename C>
int64_t count_steps(mxg::RopeParams &p) {
  int64_t steps = 0;
  for (mxg::RopeTensor &t : p.t) steps += t.steps = static_cast<int>(cdiv(t.heads, C::HEADS));
  return steps;
}

template <typename T, int D>
int run_forward(mxg::RopeParams &p, int device, cudaStream_t stream) {
  // as many blocks as the SMs hold, no more warps than steps
  using C = mxg::RopeCfg<T, D, false>;
  int sms = 1;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  const int64_t grid = std::min<int64_t>(cdiv(p.tokens * count_steps<C>(p), C::WARPS), static_cast<int64_t>(C::BLOCKS) * sms);
  return mxg::launch(mxg::norm_rope_kernel<T, D>, dim3(static_cast<unsigned>(grid)), 32 * C::WARPS, C::SMEM_BYTES, 1, stream, p);
}

template <typename T, int D>
int run_backward(mxgemm_handle_t h, const mxg::HandleView &v, mxg::RopeParams &p, cudaStream_t stream) {
  // as many blocks as the SMs hold, shared out by the tensors' steps
  using C = mxg::RopeCfg<T, D, true>;
  const int64_t all = count_steps<C>(p);
  int blocks = 0, rows = 0;
  for (mxg::RopeTensor &t : p.t) {
    t.blocks = t.heads ? static_cast<int>(std::min(cdiv(p.tokens * t.steps, C::WARPS), std::max<int64_t>(1, C::BLOCKS * v.sm_count * t.steps / all))) : 0;
    const int g = mxg::rope_group(t.blocks);
    blocks += t.blocks;
    rows += t.blocks + (t.blocks + g - 1) / g;
  }
  if (p.t[0].dw || p.t[1].dw) {
    uint8_t *ws = nullptr;
    if (int st = mxg::handle_workspace(h, static_cast<size_t>(rows) * D * sizeof(float), stream, &ws)) return st;
    p.partials = reinterpret_cast<float *>(ws);
    p.counters = v.counters;
  }
  return mxg::launch(mxg::norm_rope_backward_kernel<T, D>, dim3(blocks), 32 * C::WARPS, C::SMEM_BYTES, 1, stream, p);
}

}  // namespace

extern "C" int mxgemm_norm_rope(const mxgemm_heads_t *q, const mxgemm_heads_t *k, int64_t tokens, int64_t head_dim, int x_dtype,
                                int w_dtype, float eps, const mxgemm_rope_t *rope, mxgemm_stream_t stream_) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    device = -1;  // (no pointer is on it)
  }
  mxg::RopeParams p;
  if (int st = rope_args(device, q, k, tokens, head_dim, x_dtype, w_dtype, eps, rope, false, &p)) return st;
  if (tokens == 0 || p.t[0].heads + p.t[1].heads == 0) return MXGEMM_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const bool f32 = x_dtype == MXGEMM_IN_F32;
  return head_dim == 128 ? (f32 ? run_forward<float, 128>(p, device, stream) : run_forward<__nv_bfloat16, 128>(p, device, stream))
                         : (f32 ? run_forward<float, 64>(p, device, stream) : run_forward<__nv_bfloat16, 64>(p, device, stream));
}

extern "C" int mxgemm_norm_rope_backward(mxgemm_handle_t h, const mxgemm_heads_t *q, const mxgemm_heads_t *k, int64_t tokens,
                                         int64_t head_dim, int x_dtype, int w_dtype, float eps, const mxgemm_rope_t *rope,
                                         mxgemm_stream_t stream_) {
  if (!h) return MXGEMM_ERR_INVALID_VALUE;
  const mxg::HandleView v = mxg::handle_view(h);
  mxg::CurrentDevice g(v.device);
  mxg::RopeParams p;
  if (int st = rope_args(v.device, q, k, tokens, head_dim, x_dtype, w_dtype, eps, rope, true, &p)) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (tokens == 0) {  // sums of nothing
    for (const mxgemm_heads_t *a : {q, k})
      if (a && a->heads > 0 && a->dweight) {
        if (!aligned(a->dweight, 4)) return MXGEMM_ERR_MISALIGNED;
        if (!mxg::pointer_on_device(a->dweight, v.device)) return MXGEMM_ERR_INVALID_VALUE;
      }
    for (const mxgemm_heads_t *a : {q, k})
      if (a && a->heads > 0 && a->dweight &&
          cudaMemsetAsync(a->dweight, 0, static_cast<size_t>(head_dim) * sizeof(float), stream) != cudaSuccess) {
        cudaGetLastError();
        return MXGEMM_ERR_CUDA;
      }
    return MXGEMM_OK;
  }
  if (p.t[0].heads + p.t[1].heads == 0) return MXGEMM_OK;
  const bool f32 = x_dtype == MXGEMM_IN_F32;
  const int st = head_dim == 128
                     ? (f32 ? run_backward<float, 128>(h, v, p, stream) : run_backward<__nv_bfloat16, 128>(h, v, p, stream))
                     : (f32 ? run_backward<float, 64>(h, v, p, stream) : run_backward<__nv_bfloat16, 64>(h, v, p, stream));
  if (st != MXGEMM_OK) return st;
  ++*v.launches;
  return MXGEMM_OK;
}

extern "C" int mxgemm_rope_frequencies(int64_t rot, double base, int scaling, double scale, double trained, double slow,
                                       double fast, double *freqs) {
  if (rot < 0 || rot % 2 != 0 || rot >= kLim || (rot > 0 && !freqs)) return MXGEMM_ERR_INVALID_VALUE;
  if (!(base > 0) || !std::isfinite(base)) return MXGEMM_ERR_INVALID_VALUE;
  if (scaling < MXGEMM_ROPE_PLAIN || scaling > MXGEMM_ROPE_BY_PARTS) return MXGEMM_ERR_INVALID_VALUE;
  if (scaling != MXGEMM_ROPE_PLAIN && (!(scale >= 1) || !std::isfinite(scale))) return MXGEMM_ERR_INVALID_VALUE;
  if (scaling == MXGEMM_ROPE_BASE && rot == 2 && scale != 1) return MXGEMM_ERR_INVALID_VALUE;
  if (scaling == MXGEMM_ROPE_BY_PARTS &&
      (!(trained > 0) || !std::isfinite(trained) || !(slow > 0) || !(fast > slow) || !std::isfinite(fast)))
    return MXGEMM_ERR_INVALID_VALUE;
  if (scaling == MXGEMM_ROPE_BASE && rot > 2)
    base *= std::pow(scale, static_cast<double>(rot) / static_cast<double>(rot - 2));
  if (!std::isfinite(base)) return MXGEMM_ERR_INVALID_VALUE;
  for (int64_t j = 0; j < rot / 2; ++j) {
    double f = std::pow(base, -2.0 * static_cast<double>(j) / static_cast<double>(rot));
    if (scaling == MXGEMM_ROPE_LINEAR) f /= scale;
    if (scaling == MXGEMM_ROPE_BY_PARTS) {
      const double turns = trained * f / 6.283185307179586477;
      const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
      f = f / scale * (1 - keep) + f * keep;
    }
    freqs[j] = f;
  }
  return MXGEMM_OK;
}
