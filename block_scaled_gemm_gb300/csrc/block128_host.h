// block128_host.h -- host side that the block-128 products share: tensor maps, and
// the plan of tiles for CTA pairs.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "block128_kernel.cuh"
#include "context.h"

namespace mxg {

// 2-D tensor map of bytes (or of C's elements): dims {inner, outer}, row pitch in
// bytes, box.
inline int encode(const HandleView &v, CUtensorMap *tm, CUtensorMapDataType dt, const void *base, int64_t inner, int64_t outer,
                  int64_t pitch, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return v.encode(tm, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MXGEMM_OK
             : MXGEMM_ERR_CUDA;
}

// Tiles of 256 rows and tile_n columns for CTA pairs: whole ones, and the last
// with their K cut (block128.cu).  Takes the workspace that the cut ones need.
int pair_plan(mxgemm_handle_t h, const HandleView &v, B128Params &p, int tile_n, cudaStream_t stream);

// CTAs of a planned launch.
inline int pair_grid(const HandleView &v, const B128Params &p) { return 2 * (p.dp_tiles > 0 ? v.sm_count / 2 : p.tail_items); }

}  // namespace mxg
