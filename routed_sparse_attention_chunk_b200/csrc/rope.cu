// Rotary positions of the query path: the first rd dimensions of every head
// rotated by its token's position, in the pair layouts (x_i, x_{i + rd/2}) and
// (x_{2i}, x_{2i+1}); the gradient is the same kernel with the transposed
// rotation.  With (c, s) the table row of the position and pair (a, b):
//   y = (a c - b s, a s + b c)     transposed: (a c + b s, b c - a s)
// in fp32, rounded once on the store; the dimensions past rd are copied.
//
// Bound by memory (3 flop per 8 bytes): every 16-byte vector of x is read and
// written once, and a token's table row is read by its heads through L1.  A
// thread takes one unit: two vectors rd/2 apart (half layout), or one vector
// holding whole pairs (interleaved, and the copied tail).
#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace msa {
namespace {

// Launched as a programmatic dependent: it may start while the previous kernel of the stream
// drains, and reads nothing that kernel writes before this wait.
template <typename T>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a, int units, int64_t total) {
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < total; u += step) {
    const int64_t row = u / units;  // token * H + head
    const int unit = (int)(u - row * units);
    const int64_t n = row / a.H;
    const int h = (int)(row - n * a.H);
    const int pos = __ldg(a.pos + n);
    if (pos < 0 || pos >= a.max_len) {
      if (unit == 0 && h == 0) raise_flag(a.err_flag, MSA_FLAG_INDEX_OOB);
      continue;
    }
    const T* x = reinterpret_cast<const T*>(a.x) + n * a.x_ts + h * a.x_hs;
    T* y = reinterpret_cast<T*>(a.out) + n * a.out_ts + h * a.out_hs;
    rotate_unit<T>(x, y, unit, a.rd, a.interleaved, a.transpose, a.cs + (int64_t)pos * a.rd);
  }
}

template <typename T>
cudaError_t rope_t(const RopeArgs& a, cudaStream_t s) {
  const int units = rope_units<T>(a.d, a.rd, a.interleaved);
  const int64_t total = a.N * a.H * units;
  const int64_t blocks = (total + 255) / 256;
  // grid x holds 2^31 - 1 blocks; the kernel strides over the rest
  const unsigned grid = (unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
  count_launch();
  return launch_pdl(rope_kernel<T>, dim3(grid), dim3(256), 0, s, a, units, total);
}

}  // namespace

cudaError_t launch_rope(msa_dtype dt, const RopeArgs& a, cudaStream_t s) {
  return dt == MSA_F32 ? rope_t<float>(a, s) : rope_t<__nv_bfloat16>(a, s);
}

}  // namespace msa
