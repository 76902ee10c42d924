// Host-side construction of TMA tensor maps. The driver entry point
// cuTensorMapEncodeTiled is fetched through the runtime, so the library does
// not link libcuda directly and loads on machines without a GPU driver.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

namespace attn {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Map over a bf16 tensor viewed as [outer][rows][cols] (cols contiguous),
// box = (64 cols = 128 bytes, box_rows, 1), 128-byte swizzle. Reads outside
// the tensor (rows >= `rows`) are filled with zeros.
inline bool make_map_bf16_3d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
                             uint64_t outer, uint32_t box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, outer};
  const cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map over a float32 tensor viewed as [outer][rows][cols] (cols contiguous),
// box = (box_cols, box_rows, 1), no swizzle: the shared-memory side of a copy
// is the plain row-major box. Used for bulk reductions into an accumulator;
// rows >= `rows` of a box are left untouched.
inline bool make_map_f32_3d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
                            uint64_t outer, uint32_t box_cols, uint32_t box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, outer};
  const cuuint64_t strides[2] = {cols * 4, rows * cols * 4};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map over a bf16 tensor [outer][rows][cols] (cols 64 or 128, contiguous,
// rows a multiple of 8) for copies that take whole rows: viewed as
// [outer][row / 8][64-column half][row % 8][64], boxes of box_rows rows (a
// multiple of 8), 128-byte swizzle. A box lands as 1024-byte pieces of 8 rows
// x 64 columns, the halves of 8 rows next to each other.
inline bool make_map_bf16_joined(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
                                 uint64_t outer, uint32_t box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[5] = {64, 8, cols / 64, rows / 8, outer};
  const cuuint64_t strides[4] = {cols * 2, 128, cols * 16, rows * cols * 2};
  const cuuint32_t box[5] = {64, 8, cuuint32_t(cols / 64), box_rows / 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map over a bf16 tensor viewed as [rows][cols] (cols contiguous) for
// row gathers (tile::gather4): box = (cols, 1), no swizzle, so four gathered
// rows land as a plain row-major block. cols * 2 bytes must be a multiple of
// 16 and at most 512.
inline bool make_map_bf16_rows(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * 2};
  const cuuint32_t box[2] = {cuuint32_t(cols), 1};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
