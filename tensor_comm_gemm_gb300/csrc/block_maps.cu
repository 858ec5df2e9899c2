// Tensor maps of the block operators' matrix operands (host).

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "block_dev.h"

namespace tpo {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
}  // namespace

bool load_encode() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) ==
            cudaSuccess && r == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

bool encode(CUtensorMap* map, const void* base, bool fp8, int64_t inner, int64_t outer, int64_t ld, int box_inner,
            int box_outer, CUtensorMapSwizzle sw) {
  const int elem = fp8 ? 1 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * elem};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  return g_encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_operand(CUtensorMap* map, const Operand& o, bool fp8, int64_t rows, int64_t K, int box_rows) {
  if (o.mn_major) return encode(map, o.p, fp8, rows, K, o.ld, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  return encode(map, o.p, fp8, K, rows, o.ld, fp8 ? KB : KB / 2, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace tpo
