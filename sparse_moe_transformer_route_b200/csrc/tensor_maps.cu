// TMA descriptors over three dimensions and over packed 4-bit codes.
#include <cudaTypedefs.h>

#include "moe_internal.h"

namespace moe {

PFN_cuTensorMapEncodeTiled_v12000 get_encode();

namespace {
bool encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box,
           CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto enc = get_encode();
  if (enc == nullptr) return false;
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

bool make_map_3d(CUtensorMap* m, const void* base, uint64_t mats, uint64_t rows, uint64_t cols, uint32_t box_cols,
                 uint32_t box_rows) {
  const cuuint64_t dims[3] = {cols, rows, mats};
  const cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box);
}

bool make_map_bytes(CUtensorMap* m, const void* base, uint64_t mats, uint64_t rows, uint64_t row_bytes,
                    uint32_t box_rows) {
  const cuuint64_t dims[3] = {row_bytes, rows, mats};
  const cuuint64_t strides[2] = {row_bytes, rows * row_bytes};
  const cuuint32_t box[3] = {128, box_rows, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box);
}

bool make_map_scales(CUtensorMap* m, const void* base, uint64_t mats, uint64_t rows, uint64_t row_bytes,
                     uint32_t box_rows) {
  const cuuint64_t dims[3] = {row_bytes, rows, mats};
  const cuuint64_t strides[2] = {row_bytes, rows * row_bytes};
  const cuuint32_t box[3] = {32, box_rows, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_32B);
}

}  // namespace moe
