// TMA maps of the sliding-window kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "window.h"

namespace dash {

bool window_map(CUtensorMap* map, const View& v, int dtype, int64_t B, int64_t S, int64_t H, int D, int box_h,
                int box_s, bool narrow) {
  static const auto encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return false;
  const int64_t es = 2;
  const cuuint64_t extent[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
  const cuuint64_t stride[3] = {(cuuint64_t)(v.sh * es), (cuuint64_t)(v.ss * es), (cuuint64_t)(v.sb * es)};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_h, (cuuint32_t)box_s, 1}, step[4] = {1, 1, 1, 1};
  const auto type = dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto fetch = narrow ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  auto make = [&] {
    return encode(map, type, 4, const_cast<void*>(v.data), extent, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (make()) return true;
  // a driver call: it fails in a thread whose first CUDA work this is (an
  // autograd thread), where the runtime has not made the device's context
  // current yet
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && make();
}

}  // namespace dash
