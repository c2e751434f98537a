// ss_dropout.hip -- dropout of a (rows, dim) array by the mask of ss_philox.h; its gradient is the
// same call on the upstream gradient.  Memory and the generator bind it alike: 16384 x 2560 bf16, 168
// MB, in 30.3 us (5.5 TB/s); the generator's multiplies alone would take about 25.
#include "ss_head.h"
#include "ss_octs.h"
#include "ss_philox.h"
#include "ss_rows.h"

namespace ss {
namespace {

// One lane per oct of a row; the launch walks the octs of all rows, `drow` rows and `doct` octs a
// stride (so that no division stands in the loop).
struct DropWalk {
  int64_t rows, dim, octs, drow, doct;
};

template <class IO>
__global__ __launch_bounds__(256) void dropout_kernel(const typename IO::elem* x,
                                                      typename IO::elem* out, DropArgs d,
                                                      DropWalk w) {
  const PhiloxKey key = philox_key(d.rng);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  int64_t row = first / w.octs, oct = first - row * w.octs;
  while (row < w.rows) {
    const int64_t at = row * w.dim + oct * 8, left = w.dim - oct * 8;
    const int n = left < 8 ? static_cast<int>(left) : 8;
    float v[8];
    load8<IO>(x + at, n, v);
    drop8(v, keep8(key, static_cast<uint32_t>(oct), static_cast<uint32_t>(row), d.cut), d.up);
    store8<IO>(out + at, n, v);
    row += w.drow;
    oct += w.doct;
    if (oct >= w.octs) {
      oct -= w.octs;
      ++row;
    }
  }
}

}  // namespace

hipError_t launch_dropout(const void* x, void* out, const DropArgs& d, int64_t rows, int64_t dim,
                          bool bf16, hipStream_t stream) {
  DropWalk w{rows, dim, (dim + 7) / 8, 0, 0};
  int64_t blocks = (rows * w.octs + 255) / 256;
  if (blocks > 8192) blocks = 8192;
  w.drow = blocks * 256 / w.octs;
  w.doct = blocks * 256 - w.drow * w.octs;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (bf16)
    hipLaunchKernelGGL(dropout_kernel<BF16>, grid, dim3(256), 0, stream,
                       static_cast<const uint16_t*>(x), static_cast<uint16_t*>(out), d, w);
  else
    hipLaunchKernelGGL(dropout_kernel<F32>, grid, dim3(256), 0, stream,
                       static_cast<const float*>(x), static_cast<float*>(out), d, w);
  return hipGetLastError();
}

}  // namespace ss
