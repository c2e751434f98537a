// ss_block_fill.hip -- fills and copies of the recurrent block's operators.
#include "ss_block.h"

namespace ss {
namespace {

template <class T>
__global__ __launch_bounds__(256) void fill_kernel(T* dst, const T* src, int64_t n) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll)
    dst[i] = src ? src[i] : T(0);
}

template <class T>
hipError_t fill(T* dst, const T* src, int64_t n, hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  const int64_t g = (n + 255) / 256;
  hipLaunchKernelGGL(fill_kernel<T>, dim3(static_cast<unsigned>(g < 4096 ? g : 4096)), dim3(256),
                     0, stream, dst, src, n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_zero(float* p, int64_t n, hipStream_t stream) {
  return fill<float>(p, nullptr, n, stream);
}
hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t stream) {
  return fill<uint8_t>(static_cast<uint8_t*>(p), nullptr, bytes, stream);
}
hipError_t launch_copy(float* dst, const float* src, int64_t n, hipStream_t stream) {
  return fill<float>(dst, src, n, stream);
}

}  // namespace ss
