// gated.cu -- the gated pair of products with block-128 scales and its gradient:
// argument checks and launches of mxgemm_run_gated_block128 and
// mxgemm_gated_backward.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "block128_host.h"
#include "block128_kernel.cuh"
#include "context.h"
#include "gated_backward.cuh"
#include "gated_skinny.cuh"
#include "launch.h"
#include "mxgemm.h"

namespace {

using mxg::aligned;
using mxg::cdiv;
using mxg::encode;
using mxg::kLim;

// CTAs for each column block where those are fewer than the SMs.  What their number
// changes, in us: a K block takes 0.3 with up to 16 rows, 0.41 with up to 32 and 0.55
// with 64, a join 1 and 0.25 for each part, or 0.8 with 32 rows a warp.  Some 10 us of start
// and end, whatever the number, are left out.  Measured with each number of parts: 8 x
// 1024 x 8192 30.4 us with one, 12.9 with four, 10.8 with eight (the choice), 12.7 with 19;
// 64 x 1024 x 8192 45.8, 21.9, 20.5 (the choice), 28.4.
int block_parts(int64_t blocks, int64_t kb, int64_t sms, double k_block, double part) {
  int best = 1;
  double least = k_block * static_cast<double>(kb);
  for (int64_t n = 2; n * blocks <= sms && n <= kb; ++n) {
    const double us = k_block * static_cast<double>(cdiv(kb, n)) + 1 + part * static_cast<double>(n);
    if (us < least) {
      least = us;
      best = static_cast<int>(n);
    }
  }
  return best;
}

// M <= 64 by one CTA an SM at most.  Fewer column blocks than SMs: each is cut into
// whole CTAs' parts, so that no CTA ends two blocks' parts (30 x 4096 x 4096 19.5 -> 14
// us with 128 CTAs of eight K blocks and not 152 of six or seven).  More: all K blocks
// are cut into equal ranges (224 blocks on 152 SMs would take two rounds).
template <int NT, bool KM>
int run_skinny(mxgemm_handle_t h, const mxg::HandleView &v, mxg::GatedSkinnyParams &gp, const void *A, const void *G, const void *U,
               cudaStream_t stream) {
  using S = mxg::GatedSkinnyCfg<NT>;
  mxg::B128Params &p = gp.b;
  p.nm = (p.M + 15) / 16 * 16;
  // the MMA's A operand is a weight and its B operand A
  p.idesc_fmt = mxg::fmt_bits(v.b_fmt, v.a_fmt);
  gp.n_tiles = static_cast<int>(cdiv(p.N, 128));
  gp.total = static_cast<int64_t>(gp.n_tiles) * p.kb;
  const int sms = std::min(v.sm_count, mxg::kCounters);
  const int grid = gp.n_tiles <= sms ? gp.n_tiles * block_parts(gp.n_tiles, p.kb, sms, NT == 16 ? 0.3 : NT == 32 ? 0.41 : 0.55, S::ROWS >= 32 ? 0.8 : 0.25) : sms;
  uint8_t *ws = nullptr;
  if (int st = mxg::handle_workspace(h, static_cast<size_t>(grid) * 2 * S::PARTIAL * sizeof(float), stream, &ws)) return st;
  gp.partials = reinterpret_cast<float *>(ws);
  gp.counters = v.counters;
  CUtensorMap tG, tU, tA;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  auto weight = [&](CUtensorMap *tm, const void *w) {
    return KM ? encode(v, tm, u8, w, p.K, p.N, p.K, 128, 128) : encode(v, tm, u8, w, p.N, p.K, p.N, 128, 128);
  };
  if (encode(v, &tA, u8, A, p.K, p.M, p.K, 128, static_cast<uint32_t>(p.nm)) || weight(&tG, G) || weight(&tU, U))
    return MXGEMM_ERR_CUDA;
  return mxg::launch(mxg::gated_skinny_kernel<NT, KM>, dim3(grid), S::THREADS, S::SMEM_BYTES, 1, stream, tG, tU, tA, gp);
}

template <bool KM>
int run_skinny(mxgemm_handle_t h, const mxg::HandleView &v, mxg::GatedSkinnyParams &gp, const void *A, const void *G, const void *U,
               cudaStream_t stream) {
  if (gp.b.M <= 16) return run_skinny<16, KM>(h, v, gp, A, G, U, stream);
  if (gp.b.M <= 32) return run_skinny<32, KM>(h, v, gp, A, G, U, stream);
  return run_skinny<64, KM>(h, v, gp, A, G, U, stream);
}

// M > 64: CTA pairs, 256 rows and 128 columns of H a tile.
int run_pair(mxgemm_handle_t h, const mxg::HandleView &v, mxg::B128Params &p, const void *A, const void *G, const void *U, bool nk,
             int h_type, cudaStream_t stream) {
  mxg::PairMaps<true> tm;
  std::memset(&tm, 0, sizeof(tm));
  p.idesc_fmt = mxg::fmt_bits(v.a_fmt, v.b_fmt);
  if (int st = mxg::pair_plan(h, v, p, 128, stream)) return st;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int eb = h_type == MXGEMM_OUT_F32 ? 4 : h_type == MXGEMM_OUT_BF16 ? 2 : 1;
  p.tma_store = static_cast<int64_t>(p.N) * eb % 16 == 0;
  p.tma_keep = p.gate && p.N % 8 == 0;
  auto weight = [&](CUtensorMap *m, const void *w) {
    return nk ? encode(v, m, u8, w, p.K, p.N, p.K, 128, 128) : encode(v, m, u8, w, p.N, p.K, p.N, 128, 128);
  };
  if (encode(v, &tm.A, u8, A, p.K, p.M, p.K, 128, 128) || weight(&tm.B, G) || weight(&tm.U, U)) return MXGEMM_ERR_CUDA;
  if (h_type == MXGEMM_OUT_E4M3) {
    if (encode(v, &tm.C, u8, p.C, p.N, p.M, p.N, 64, 32, CU_TENSOR_MAP_SWIZZLE_64B)) return MXGEMM_ERR_CUDA;
  } else if (p.tma_store) {
    if (encode(v, &tm.C, eb == 2 ? bf : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.C, p.N, p.M, static_cast<int64_t>(p.N) * eb, eb == 2 ? 64 : 32, 32))
      return MXGEMM_ERR_CUDA;
  }
  if (p.tma_keep && (encode(v, &tm.gate, bf, p.gate, p.N, p.M, static_cast<int64_t>(p.N) * 2, 64, 32) ||
                     encode(v, &tm.up, bf, p.up, p.N, p.M, static_cast<int64_t>(p.N) * 2, 64, 32)))
    return MXGEMM_ERR_CUDA;
  const int variant = mxg::kB128Gated | (nk ? mxg::kB128KMajor : 0) |
                      (h_type == MXGEMM_OUT_E4M3 ? mxg::kB128Codes : h_type == MXGEMM_OUT_BF16 ? mxg::kB128Bf16 : 0);
  const int grid = mxg::pair_grid(v, p);
  switch (variant) {
#define MXG_PAIR(V)                                                                                     \
  case V:                                                                                               \
    return mxg::launch(mxg::b128_pair_kernel<V>, dim3(grid), mxg::PairCfg<V>::THREADS,                  \
                       mxg::PairCfg<V>::SMEM_BYTES, 2, stream, tm, p);
    MXG_PAIR(8)
    MXG_PAIR(9)
    MXG_PAIR(10)
    MXG_PAIR(11)
    MXG_PAIR(24)
    MXG_PAIR(26)
#undef MXG_PAIR
    default:
      return MXGEMM_ERR_INVALID_VALUE;
  }
}

template <typename T, int ACT>
int launch_grad(const mxg::GatedGradParams &p, bool tiles, int sms, cudaStream_t stream) {
  if (tiles) {
    if (p.rb * p.cb >= kLim - sms) return MXGEMM_ERR_INVALID_VALUE;
    const int64_t grid = std::min<int64_t>(p.rb * p.cb, sms);
    return mxg::launch(mxg::gated_grad_tile_kernel<T, ACT>, dim3(static_cast<unsigned>(grid)), 512, mxg::GatedGradCfg<T>::SMEM_BYTES, 1,
                       stream, p);
  }
  const int64_t grid = cdiv(p.R * p.C, 2048);
  if (grid >= kLim) return MXGEMM_ERR_INVALID_VALUE;
  return mxg::launch(mxg::gated_grad_flat_kernel<T, ACT>, dim3(static_cast<unsigned>(grid)), 256, 0, 1, stream, p);
}

template <typename T>
int launch_grad(const mxg::GatedGradParams &p, int act, bool tiles, int sms, cudaStream_t stream) {
  return act == MXGEMM_ACT_SILU ? launch_grad<T, mxg::kActSilu>(p, tiles, sms, stream)
                                : launch_grad<T, mxg::kActGeluTanh>(p, tiles, sms, stream);
}

}  // namespace

extern "C" int mxgemm_run_gated_block128(mxgemm_handle_t h, int64_t M, int64_t N, int64_t K, const void *A, const float *A_scale,
                                         const void *G, const float *G_scale, const void *U, const float *U_scale, int act,
                                         void *H, float *H_scale, int h_dtype, void *gate, void *up, mxgemm_stream_t stream_) {
  if (!h) return MXGEMM_ERR_INVALID_VALUE;
  const mxg::HandleView v = mxg::handle_view(h);
  const bool nk = v.b_major == MXGEMM_B_N_BY_K, codes = h_dtype == MXGEMM_OUT_E4M3;
  // (sizes rounded up to whole tiles stay below 2^31)
  if (M < 0 || N < 0 || K < 16 || M > kLim - 512 || N > kLim - 512 || K > kLim - 512) return MXGEMM_ERR_INVALID_VALUE;
  if (K % 16 != 0 || ((!nk || codes) && N % 16 != 0)) return MXGEMM_ERR_INVALID_VALUE;
  if (act != MXGEMM_ACT_SILU && act != MXGEMM_ACT_GELU_TANH) return MXGEMM_ERR_INVALID_VALUE;
  if (h_dtype != MXGEMM_OUT_F32 && h_dtype != MXGEMM_OUT_BF16 && !codes) return MXGEMM_ERR_INVALID_VALUE;
  if (v.a_fmt > MXGEMM_FMT_E5M2 || v.b_fmt > MXGEMM_FMT_E5M2) return MXGEMM_ERR_INVALID_VALUE;
  if (!gate != !up || (H_scale && !codes)) return MXGEMM_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) return MXGEMM_OK;
  if (!A || !A_scale || !G || !G_scale || !U || !U_scale || !H || (codes && !H_scale)) return MXGEMM_ERR_INVALID_VALUE;
  for (const void *x : {A, G, U, static_cast<const void *>(H), static_cast<const void *>(gate), static_cast<const void *>(up)})
    if (!aligned(x, 16)) return MXGEMM_ERR_MISALIGNED;
  for (const float *x : {A_scale, G_scale, U_scale, static_cast<const float *>(H_scale)})
    if (!aligned(x, 4)) return MXGEMM_ERR_MISALIGNED;
  mxg::CurrentDevice g(v.device);
  const void *const all[] = {A, A_scale, G, G_scale, U, U_scale, H, H_scale, gate, up};
  for (const void *x : all)
    if (x && !mxg::pointer_on_device(x, v.device)) return MXGEMM_ERR_INVALID_VALUE;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);

  mxg::GatedSkinnyParams gp;
  std::memset(&gp, 0, sizeof(gp));
  mxg::B128Params &p = gp.b;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.kb = static_cast<int>(cdiv(K, 128));
  p.a_scale = A_scale;
  p.b_scale = G_scale;
  p.u_scale = U_scale;
  p.bs_cols = cdiv(N, 128);
  p.bs_n = nk ? p.kb : 1;
  p.bs_k = nk ? 1 : p.bs_cols;
  p.C = H;
  p.h_scale = H_scale;
  p.gate = static_cast<__nv_bfloat16 *>(gate);
  p.up = static_cast<__nv_bfloat16 *>(up);
  p.act = act;
  p.status = v.status;
  p.timeout_ns = v.timeout_ns;
  p.stall_producer = v.stall_producer;
  gp.h_type = h_dtype;
  if (v.prof_before && cudaEventRecord(v.prof_before, stream) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  const int st = M > 64 ? run_pair(h, v, p, A, G, U, nk, h_dtype, stream)
                 : nk   ? run_skinny<true>(h, v, gp, A, G, U, stream)
                        : run_skinny<false>(h, v, gp, A, G, U, stream);
  if (st != MXGEMM_OK) return st;
  ++*v.launches;
  if (v.prof_after && cudaEventRecord(v.prof_after, stream) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  return MXGEMM_OK;
}

extern "C" int mxgemm_gated_backward(const void *gate, const void *up, const void *dH, int dh_dtype, int64_t R, int64_t C, int act,
                                     const mxgemm_gated_grads_t *out, mxgemm_stream_t stream_) {
  if (R < 0 || C < 0 || R >= kLim - 128 || C >= kLim - 128 || !out) return MXGEMM_ERR_INVALID_VALUE;
  if (dh_dtype != MXGEMM_IN_F32 && dh_dtype != MXGEMM_IN_BF16) return MXGEMM_ERR_INVALID_VALUE;
  if (act != MXGEMM_ACT_SILU && act != MXGEMM_ACT_GELU_TANH) return MXGEMM_ERR_INVALID_VALUE;
  const mxgemm_block128_t *const blocks[5] = {&out->dgate_rows, &out->dup_rows, &out->dgate_cols, &out->dup_cols, &out->hidden_cols};
  bool tiles = false;
  for (const mxgemm_block128_t *b : blocks) {
    if (!b->codes != !b->scales) return MXGEMM_ERR_INVALID_VALUE;
    tiles |= b->codes != nullptr;
  }
  if (tiles && C % 16 != 0) return MXGEMM_ERR_INVALID_VALUE;
  if (R == 0 || C == 0) return MXGEMM_OK;
  if (!gate || !up || !dH || (!tiles && !out->dgate && !out->dup)) return MXGEMM_ERR_INVALID_VALUE;
  for (const void *x : {gate, up, dH, static_cast<const void *>(out->dgate), static_cast<const void *>(out->dup)})
    if (!aligned(x, 16)) return MXGEMM_ERR_MISALIGNED;
  for (const mxgemm_block128_t *b : blocks)
    if (!aligned(b->codes, 16) || !aligned(b->scales, 4)) return MXGEMM_ERR_MISALIGNED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  for (const void *x : {gate, up, dH, static_cast<const void *>(out->dgate), static_cast<const void *>(out->dup)})
    if (x && !mxg::pointer_on_device(x, dev)) return MXGEMM_ERR_INVALID_VALUE;
  for (const mxgemm_block128_t *b : blocks)
    if (b->codes && (!mxg::pointer_on_device(b->codes, dev) || !mxg::pointer_on_device(b->scales, dev))) return MXGEMM_ERR_INVALID_VALUE;
  mxg::GatedGradParams p;
  p.gate = static_cast<const __nv_bfloat16 *>(gate);
  p.up = static_cast<const __nv_bfloat16 *>(up);
  p.dH = dH;
  p.R = R;
  p.C = C;
  p.pitch = cdiv(R, 16) * 16;
  p.rb = cdiv(R, 128);
  p.cb = cdiv(C, 128);
  p.dgate = static_cast<__nv_bfloat16 *>(out->dgate);
  p.dup = static_cast<__nv_bfloat16 *>(out->dup);
  for (int i = 0; i < 5; ++i)
    (i < 2 ? p.rows[i] : p.cols[i - 2]) = mxg::Blocks128{static_cast<uint8_t *>(blocks[i]->codes), blocks[i]->scales};
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int sms = 1;
  if (tiles && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  return dh_dtype == MXGEMM_IN_F32 ? launch_grad<float>(p, act, tiles, sms, stream)
                                   : launch_grad<__nv_bfloat16>(p, act, tiles, sms, stream);
}
