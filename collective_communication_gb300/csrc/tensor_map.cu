// tensor_map.cu -- TMA descriptors, made on the host for each call.
#include "tensor_core.cuh"

namespace rar {
namespace {

cudaError_t encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
  // the driver's function by way of the runtime: the library does not link the driver
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* found = nullptr;
    cudaDriverEntryPointQueryResult result;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &found, 12000, cudaEnableDefault, &result) != cudaSuccess ||
        result != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      found = nullptr;
    }
    return (PFN_cuTensorMapEncodeTiled_v12000)found;
  }();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box,
                        steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t make_map(CUtensorMap* map, const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t stride1_bytes,
                     int64_t stride2_bytes, int rows, int planes) {
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  // a single row's or plane's stride means nothing: any valid one will do
  const cuuint64_t row = (cuuint64_t)(d1 > 1 ? stride1_bytes : d0 * 2);
  const cuuint64_t strides[2] = {row, d2 > 1 ? (cuuint64_t)stride2_bytes : row};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, (cuuint32_t)planes};
  return encode(map, base, 3, dims, strides, box);
}

cudaError_t make_grouped_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int groups) {
  const cuuint64_t dims[4] = {64, 8, (cuuint64_t)(width / 64), (cuuint64_t)(rows / 8)};
  const cuuint64_t strides[3] = {(cuuint64_t)(width * 2), 128, (cuuint64_t)(8 * width * 2)};
  const cuuint32_t box[4] = {64, 8, (cuuint32_t)(width / 64), (cuuint32_t)groups};
  return encode(map, base, 4, dims, strides, box);
}

}  // namespace rar
