// ss_block_util.hip -- fills, copies and column sums of the recurrent block's operators.
#include "ss_block.h"

namespace ss {
namespace {

template <class T>
__global__ __launch_bounds__(256) void fill_kernel(T* dst, const T* src, int64_t n) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll)
    dst[i] = src ? src[i] : T{};
}

template <class T>
hipError_t fill(T* dst, const T* src, int64_t n, hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  const int64_t g = (n + 255) / 256;
  hipLaunchKernelGGL(fill_kernel<T>, dim3(static_cast<unsigned>(g < 4096 ? g : 4096)), dim3(256),
                     0, stream, dst, src, n);
  return hipGetLastError();
}

// One workgroup sums 32 columns of one job: 32 strands of lines, eight lines in flight each, then
// the strands in order.  The order of the additions depends on the number of lines alone.  (With 16
// strands and one line in flight 1024 lines of 2 x 2560 took 24 us, with these 7.5.)
constexpr int kCols = 32, kStrands = 32, kAhead = 8;
__global__ __launch_bounds__(kCols * kStrands) void column_sums_kernel(ColumnSums p) {
  __shared__ float lds[kStrands][kCols + 1];
  const ColumnSums::Job job = p.job[blockIdx.y];
  const int x = threadIdx.x % kCols, y = threadIdx.x / kCols;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kCols + x;
  float acc = 0.0f;
  if (c < p.cols) {
    const float* src = job.src + c;
    for (int64_t r = y; r < p.lines; r += kStrands * kAhead) {
      float v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t at = r + k * kStrands;
        v[k] = at < p.lines ? src[at * p.stride] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) acc += v[k];
    }
  }
  lds[y][x] = acc;
  __syncthreads();
  if (y == 0 && c < p.cols) {
    float s = lds[0][x];
    for (int k = 1; k < kStrands; ++k) s += lds[k][x];
    job.out[c * job.out_stride] = s;
  }
}

}  // namespace

hipError_t launch_zero(float* p, int64_t n, hipStream_t stream) {
  return fill<float>(p, nullptr, n, stream);
}
hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t stream) {
  if (bytes % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0)
    return fill<uint4>(static_cast<uint4*>(p), nullptr, bytes / 16, stream);
  return fill<uint8_t>(static_cast<uint8_t*>(p), nullptr, bytes, stream);
}
hipError_t launch_copy(float* dst, const float* src, int64_t n, hipStream_t stream) {
  return fill<float>(dst, src, n, stream);
}

hipError_t launch_column_sums(const ColumnSums& p, hipStream_t stream) {
  if (p.jobs == 0) return hipSuccess;
  hipLaunchKernelGGL(column_sums_kernel,
                     dim3(static_cast<unsigned>((p.cols + kCols - 1) / kCols),
                          static_cast<unsigned>(p.jobs)),
                     dim3(kCols * kStrands), 0, stream, p);
  return hipGetLastError();
}

}  // namespace ss
