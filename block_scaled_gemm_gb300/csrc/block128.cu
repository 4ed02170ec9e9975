// block128.cu -- the product with one FP32 scale per block of 128 and the
// quantizer that makes its operands: argument checks and launches of
// mxgemm_run_block128 and mxgemm_quantize_block128.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "block128_kernel.cuh"
#include "context.h"
#include "mxgemm.h"
#include "quantize128.cuh"

namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kLim = int64_t(1) << 31;

template <typename T>
int launch_quantize128(const T *x, int64_t R, int64_t C, int block, uint8_t *cd, float *sc, int sms,
                       cudaStream_t stream) {
  if (block == MXGEMM_BLOCK_ROWS) {
    const int64_t kb = cdiv(C, 128);
    const int grid = static_cast<int>(std::min<int64_t>(cdiv(R * kb, 8), int64_t(sms) * 8));
    mxg::quantize128_rows_kernel<T><<<grid, 256, 0, stream>>>(x, R, C, kb, cd, sc);
  } else if (block == MXGEMM_BLOCK_COLS) {
    const dim3 grid(static_cast<unsigned>(cdiv(C, 128)), static_cast<unsigned>(cdiv(R, 128)));
    mxg::quantize128_cols_kernel<T><<<grid, 128, 0, stream>>>(x, R, C, cdiv(R, 16) * 16, cd, sc);
  } else {
    const dim3 grid(static_cast<unsigned>(cdiv(C, 128)), static_cast<unsigned>(cdiv(R, 128)));
    mxg::quantize128_tiles_kernel<T><<<grid, 512, 0, stream>>>(x, R, C, cd, sc);
  }
  return cudaGetLastError() == cudaSuccess ? MXGEMM_OK : MXGEMM_ERR_CUDA;
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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  if (!mxg::pointer_on_device(X, dev) || !mxg::pointer_on_device(codes, dev) ||
      !mxg::pointer_on_device(scales, dev))
    return MXGEMM_ERR_INVALID_VALUE;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  uint8_t *cd = static_cast<uint8_t *>(codes);
  if (x_dtype == MXGEMM_IN_F32)
    return launch_quantize128(static_cast<const float *>(X), R, C, block, cd, scales, sms, stream);
  return launch_quantize128(static_cast<const __nv_bfloat16 *>(X), R, C, block, cd, scales, sms, stream);
}

extern "C" int mxgemm_run_block128(mxgemm_handle_t h, int64_t M, int64_t N, int64_t K, const void *A,
                                   const float *A_scale, const void *B, const float *B_scale,
                                   int b_block, void *C, int use_acc, int out_dtype,
                                   mxgemm_stream_t stream_) {
  if (!h) return MXGEMM_ERR_INVALID_VALUE;
  const mxg::HandleView v = mxg::handle_view(h);
  const bool nk = v.b_major == MXGEMM_B_N_BY_K;
  if (M < 0 || N < 0 || K < 0 || M >= kLim || N >= kLim || K >= kLim) return MXGEMM_ERR_INVALID_VALUE;
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
  p.M = M;
  p.N = N;
  p.K = K;
  p.kb = cdiv(K, 128);
  p.A = static_cast<const uint8_t *>(A);
  p.B = static_cast<const uint8_t *>(B);
  p.a_scale = A_scale;
  p.b_scale = B_scale;
  p.C = C;
  p.b_pitch_k = nk ? 1 : N;
  p.b_pitch_n = nk ? K : 1;
  p.bs_pitch_k = nk ? 1 : cdiv(N, b_block);
  p.bs_pitch_n = nk ? p.kb : 1;
  p.b_block = b_block;
  p.use_acc = use_acc;
  p.out_bf16 = out_dtype == MXGEMM_OUT_BF16;
  p.a_e5m2 = v.a_fmt == MXGEMM_FMT_E5M2;
  p.b_e5m2 = v.b_fmt == MXGEMM_FMT_E5M2;
  if (v.prof_before && cudaEventRecord(v.prof_before, stream) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  const int64_t mt = cdiv(M, 64), nt = cdiv(N, 64);
  mxg::block128_kernel<<<static_cast<unsigned>(mt * nt), 256, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return MXGEMM_ERR_CUDA;
  ++*v.launches;
  if (v.prof_after && cudaEventRecord(v.prof_after, stream) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  return MXGEMM_OK;
}
