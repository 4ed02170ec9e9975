// block128.cu -- the product with one FP32 scale per block of 128 and the
// quantizer that makes its operands: argument checks and launches of
// mxgemm_run_block128 and mxgemm_quantize_block128.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "block128_host.h"
#include "block128_kernel.cuh"
#include "context.h"
#include "launch.h"
#include "mxgemm.h"
#include "quantize128.cuh"

namespace {

using mxg::aligned;
using mxg::cdiv;
using mxg::encode;
using mxg::kLim;

// Row (tile) blocks past a grid's y limit go to further launches.
constexpr int64_t kGridY = 65535;

template <typename T>
int launch_quantize128(const T *x, int64_t R, int64_t C, int block, uint8_t *cd, float *sc, cudaStream_t stream) {
  const int64_t kb = cdiv(C, 128), rb = cdiv(R, 128);
  if (block == MXGEMM_BLOCK_ROWS) {
    const int64_t blocks = R * kb;
    // four groups of blocks a warp: FP32 holds twice BF16's registers
    constexpr int kUnroll = sizeof(T) == 4 ? 2 : 4;
    const int64_t grid = cdiv(blocks, 8 * 4 * kUnroll);
    if (grid >= kLim) return MXGEMM_ERR_INVALID_VALUE;
    return mxg::launch(C % 128 == 0 ? mxg::quantize128_rows_kernel<T, false, kUnroll>
                                    : mxg::quantize128_rows_kernel<T, true, kUnroll>,
                       dim3(static_cast<unsigned>(grid)), 256, 0, 1, stream, x, C, kb, blocks, cd, sc);
  }
  const int64_t pitch = cdiv(R, 16) * 16;
  for (int64_t y = 0; y < rb; y += kGridY) {
    const unsigned gy = static_cast<unsigned>(std::min(kGridY, rb - y));
    const T *xr = x + y * 128 * C;
    const int st =
        block == MXGEMM_BLOCK_COLS
            ? mxg::launch(mxg::quantize128_cols_kernel<T>, dim3(static_cast<unsigned>(cdiv(C, 64)), gy), 256, 0, 1,
                          stream, xr, R - y * 128, C, pitch, y * 128, rb, cd, sc + y)
            : mxg::launch(mxg::quantize128_tiles_kernel<T>, dim3(static_cast<unsigned>(kb), gy), 512, 0, 1, stream, xr,
                          R - y * 128, C, cd + y * 128 * C, sc + y * kb);
    if (st != MXGEMM_OK) return st;
  }
  return MXGEMM_OK;
}

// Parts of K for each of `rem` tiles on `pairs` pairs, in K blocks' time: a part
// costs its own blocks; splitting, about eight more (sums written, counted and
// read) and four for each part whose sums the last one adds (with half of that,
// 512 x 4096 x 2048 takes 13.8 us instead of 11.2).  Whole against split, in a
// graph: 256 x 4096 x 8192 28.9 and 21.6 us, 128 x 8192 x 8192 29.5 and 24.5,
// 5000 x 4112 x 8192 (B K x N) 146 and 139.5, 4096 x 4096 x 5008 75.7 and 74.9,
// with a scale for each column 108.6 and 102.6.
int tail_split(int64_t rem, int64_t pairs, int64_t kb) {
  int best = 1;
  int64_t cost = kb;
  for (int64_t s = 2; s * rem <= pairs && s <= kb; ++s) {
    const int64_t c = cdiv(kb, s) + 4 + 4 * s;
    if (c < cost) {
      cost = c;
      best = static_cast<int>(s);
    }
  }
  return best;
}

}  // namespace

namespace mxg {

int pair_plan(mxgemm_handle_t h, const HandleView &v, B128Params &p, int tile_n, cudaStream_t stream) {
  p.m_tiles = static_cast<int>(cdiv(p.M, 256));
  p.n_tiles = static_cast<int>(cdiv(p.N, tile_n));
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  if (tiles >= kLim - 65536) return MXGEMM_ERR_INVALID_VALUE;
  const int64_t pairs = v.sm_count / 2, rem = tiles % pairs;
  p.dp_tiles = static_cast<int>(tiles - rem);
  using P = PairCfg<0>;
  p.split = rem && rem * 2 * P::EPI_WARPS <= kCounters ? tail_split(rem, pairs, p.kb) : 1;
  p.tail_items = static_cast<int>(rem) * p.split;
  if (p.split > 1) {
    uint8_t *ws = nullptr;
    if (int st = handle_workspace(h, static_cast<size_t>(p.tail_items) * 2 * P::EPI_WARPS * 32 * 128 * sizeof(float),
                                  stream, &ws))
      return st;
    p.partials = reinterpret_cast<float *>(ws);
    p.counters = v.counters;
  }
  return MXGEMM_OK;
}

}  // namespace mxg

namespace {

// M > 64: CTA pairs on 256 x 256 tiles, one pair per two SMs.
int run_pair(mxgemm_handle_t h, const mxg::HandleView &v, mxg::B128Params &p, const void *A, const void *B, bool nk, bool bf16,
             int variant, cudaStream_t stream) {
  mxg::PairMaps<false> tm;
  std::memset(&tm, 0, sizeof(tm));
  const int eb = bf16 ? 2 : 4;
  p.idesc_fmt = mxg::fmt_bits(v.a_fmt, v.b_fmt);
  if (int st = mxg::pair_plan(h, v, p, 256, stream)) return st;
  p.tma_store = !p.use_acc && static_cast<int64_t>(p.N) * eb % 16 == 0;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (encode(v, &tm.A, u8, A, p.K, p.M, p.K, 128, 128) ||
      (nk ? encode(v, &tm.B, u8, B, p.K, p.N, p.K, 128, 128) : encode(v, &tm.B, u8, B, p.N, p.K, p.N, 128, 128)) ||
      (p.tma_store && encode(v, &tm.C, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                             p.C, p.N, p.M, static_cast<int64_t>(p.N) * eb, bf16 ? 64 : 32, 32)))
    return MXGEMM_ERR_CUDA;
  const int grid = mxg::pair_grid(v, p);
  switch (variant) {
#define MXG_PAIR(V)                                                                                     \
  case V:                                                                                               \
    return mxg::launch(mxg::b128_pair_kernel<V>, dim3(grid), mxg::PairCfg<V>::THREADS,                  \
                       mxg::PairCfg<V>::SMEM_BYTES, 2, stream, tm, p);
    MXG_PAIR(0)
    MXG_PAIR(1)
    MXG_PAIR(2)
    MXG_PAIR(3)
    MXG_PAIR(4)
    MXG_PAIR(5)
    MXG_PAIR(6)
    MXG_PAIR(7)
#undef MXG_PAIR
    default:
      return MXGEMM_ERR_INVALID_VALUE;
  }
}

template <int NT>
int run_skinny_nt(const mxg::HandleView &v, mxg::B128Params &p, const void *A, const void *B, bool nk, int variant,
                  cudaStream_t stream) {
  using S = mxg::SkinnyCfg<NT>;
  p.nm = (p.M + 15) / 16 * 16;
  // the MMA's A operand is B and its B operand A
  p.idesc_fmt = mxg::fmt_bits(v.b_fmt, v.a_fmt);
  // enough CTAs for the SMs where the column blocks alone are too few, within
  // one cluster, four K blocks each at least
  const int64_t blocks = cdiv(p.N, 128);
  int64_t splits = std::max<int64_t>(1, v.sm_count / blocks);
  splits = std::min<int64_t>(splits, S::MAX_SPLITS);
  splits = std::min<int64_t>(splits, std::max(1, p.kb / 4));
  p.splits = static_cast<int>(splits);
  CUtensorMap tA, tB;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (encode(v, &tA, u8, A, p.K, p.M, p.K, 128, static_cast<uint32_t>(p.nm)) ||
      (nk ? encode(v, &tB, u8, B, p.K, p.N, p.K, 128, 128) : encode(v, &tB, u8, B, p.N, p.K, p.N, 128, 128)))
    return MXGEMM_ERR_CUDA;
  const int grid = static_cast<int>(blocks * splits);
  switch (variant) {
#define MXG_SKINNY(V)                                                                              \
  case V:                                                                                          \
    return mxg::launch(mxg::b128_skinny_kernel<NT, V>, dim3(grid), S::THREADS, S::SMEM_BYTES,      \
                       p.splits, stream, tB, tA, p);
    MXG_SKINNY(0)
    MXG_SKINNY(1)
    MXG_SKINNY(2)
    MXG_SKINNY(3)
    MXG_SKINNY(4)
    MXG_SKINNY(5)
    MXG_SKINNY(6)
    MXG_SKINNY(7)
#undef MXG_SKINNY
    default:
      return MXGEMM_ERR_INVALID_VALUE;
  }
}

// M <= 64: transposed, the kernel for M rounded up to 16, 32 or 64.  (N = K =
// 8192, B in L2: 16 rows 16 us, 64 rows 21-22 us; 128 rows took 33 us so, and
// 24 us on the pairs, whose time is the same for 65 to 256 rows.)
int run_skinny(const mxg::HandleView &v, mxg::B128Params &p, const void *A, const void *B, bool nk, int variant,
               cudaStream_t stream) {
  if (p.M <= 16) return run_skinny_nt<16>(v, p, A, B, nk, variant, stream);
  if (p.M <= 32) return run_skinny_nt<32>(v, p, A, B, nk, variant, stream);
  return run_skinny_nt<64>(v, p, A, B, nk, variant, stream);
}

}  // namespace

extern "C" int mxgemm_quantize_block128(const void *X, int x_dtype, int64_t R, int64_t C, int block,
                                        void *codes, float *scales, mxgemm_stream_t stream_) {
  if (R < 0 || C < 0 || R >= kLim || C >= kLim || C % 16 != 0) return MXGEMM_ERR_INVALID_VALUE;
  if (x_dtype != MXGEMM_IN_F32 && x_dtype != MXGEMM_IN_BF16) return MXGEMM_ERR_INVALID_VALUE;
  if (block != MXGEMM_BLOCK_ROWS && block != MXGEMM_BLOCK_COLS && block != MXGEMM_BLOCK_TILES)
    return MXGEMM_ERR_INVALID_VALUE;
  if (R == 0 || C == 0) return MXGEMM_OK;
  if (!X || !codes || !scales) return MXGEMM_ERR_INVALID_VALUE;
  if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MXGEMM_ERR_MISALIGNED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  if (!mxg::pointer_on_device(X, dev) || !mxg::pointer_on_device(codes, dev) ||
      !mxg::pointer_on_device(scales, dev))
    return MXGEMM_ERR_INVALID_VALUE;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  uint8_t *cd = static_cast<uint8_t *>(codes);
  if (x_dtype == MXGEMM_IN_F32)
    return launch_quantize128(static_cast<const float *>(X), R, C, block, cd, scales, stream);
  return launch_quantize128(static_cast<const __nv_bfloat16 *>(X), R, C, block, cd, scales, stream);
}

extern "C" int mxgemm_run_block128(mxgemm_handle_t h, int64_t M, int64_t N, int64_t K, const void *A,
                                   const float *A_scale, const void *B, const float *B_scale,
                                   int b_block, void *C, int use_acc, int out_dtype,
                                   mxgemm_stream_t stream_) {
  if (!h) return MXGEMM_ERR_INVALID_VALUE;
  const mxg::HandleView v = mxg::handle_view(h);
  const bool nk = v.b_major == MXGEMM_B_N_BY_K;
  // (sizes rounded up to whole tiles stay below 2^31)
  if (M < 0 || N < 0 || K < 0 || M > kLim - 512 || N > kLim - 512 || K > kLim - 512) return MXGEMM_ERR_INVALID_VALUE;
  if (K % 16 != 0 || (!nk && N % 16 != 0)) return MXGEMM_ERR_INVALID_VALUE;
  if (b_block != 1 && b_block != 128) return MXGEMM_ERR_INVALID_VALUE;
  if (out_dtype != MXGEMM_OUT_F32 && out_dtype != MXGEMM_OUT_BF16) return MXGEMM_ERR_INVALID_VALUE;
  if (use_acc != 0 && use_acc != 1) return MXGEMM_ERR_INVALID_VALUE;
  if (v.a_fmt > MXGEMM_FMT_E5M2 || v.b_fmt > MXGEMM_FMT_E5M2) return MXGEMM_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) return MXGEMM_OK;
  if (!C) return MXGEMM_ERR_INVALID_VALUE;
  if (!aligned(C, 16)) return MXGEMM_ERR_MISALIGNED;
  mxg::CurrentDevice g(v.device);
  if (!mxg::pointer_on_device(C, v.device)) return MXGEMM_ERR_INVALID_VALUE;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (K == 0) {
    if (!use_acc && cudaMemsetAsync(C, 0, static_cast<size_t>(M) * N * (out_dtype == MXGEMM_OUT_F32 ? 4 : 2),
                                    stream) != cudaSuccess) {
      cudaGetLastError();
      return MXGEMM_ERR_CUDA;
    }
    return MXGEMM_OK;
  }
  if (!A || !A_scale || !B || !B_scale) return MXGEMM_ERR_INVALID_VALUE;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(A_scale, 4) || !aligned(B_scale, 4))
    return MXGEMM_ERR_MISALIGNED;
  if (!mxg::pointer_on_device(A, v.device) || !mxg::pointer_on_device(B, v.device) ||
      !mxg::pointer_on_device(A_scale, v.device) || !mxg::pointer_on_device(B_scale, v.device))
    return MXGEMM_ERR_INVALID_VALUE;

  mxg::B128Params p;
  std::memset(&p, 0, sizeof(p));
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.kb = static_cast<int>(cdiv(K, 128));
  p.a_scale = A_scale;
  p.b_scale = B_scale;
  p.bs_cols = cdiv(N, b_block);
  p.bs_n = nk ? p.kb : 1;
  p.bs_k = nk ? 1 : p.bs_cols;
  p.C = C;
  p.use_acc = use_acc;
  p.status = v.status;
  p.timeout_ns = v.timeout_ns;
  p.stall_producer = v.stall_producer;
  const bool bf16 = out_dtype == MXGEMM_OUT_BF16;
  const int variant = (bf16 ? mxg::kB128Bf16 : 0) | (nk ? mxg::kB128KMajor : 0) | (b_block == 1 ? mxg::kB128Cols : 0);
  if (v.prof_before && cudaEventRecord(v.prof_before, stream) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  const int st = M <= 64 ? run_skinny(v, p, A, B, nk, variant, stream)
                          : run_pair(h, v, p, A, B, nk, bf16, variant, stream);
  if (st != MXGEMM_OK) return st;
  ++*v.launches;
  if (v.prof_after && cudaEventRecord(v.prof_after, stream) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  return MXGEMM_OK;
}
