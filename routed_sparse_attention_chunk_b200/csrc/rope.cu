// Rotary positions of the query path: the first rd dimensions of every head
// rotated by its token's position, in the pair layouts (x_i, x_{i + rd/2}) and
// (x_{2i}, x_{2i+1}); the gradient is the same kernel with the transposed
// rotation.  With (c, s) the table row of the position and pair (a, b):
//   y = (a c - b s, a s + b c)     transposed: (a c + b s, b c - a s)
// in fp32, rounded once on the store; the dimensions past rd are copied.
//
// Bound by memory (3 flop per 8 bytes): every vector of x is read and written
// once.  A thread takes one unit (two vectors) of two heads of a token, so the
// table's pairs are read once for both and four loads are in flight.
#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace msa {
namespace {

// A programmatic dependent: it may start while the previous kernel of the stream
// drains, and reads nothing that kernel writes before the wait.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, int units, int groups, int64_t total) {
  pdl_wait();
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= total) return;
  const uint32_t per = (uint32_t)(units * groups);
  const int64_t n = total < 0xffffffffll ? (int64_t)((uint32_t)id / per) : id / per;
  const uint32_t r = (uint32_t)(id - n * per), hg = r / (uint32_t)units, u = r - hg * (uint32_t)units;
  const int pos = __ldg(a.pos + n);
  const RopeUnit<T> unit((int)u, a.rd, kInter);
  const T* x = reinterpret_cast<const T*>(a.x) + n * a.x_ts;
  T* y = reinterpret_cast<T*>(a.out) + n * a.out_ts;
  uint4 p[kRopeHeads], q[kRopeHeads];
#pragma unroll
  for (int j = 0; j < kRopeHeads; ++j) {
    const int h = (int)hg + j * groups;
    if (h < a.H) {
      const T* src = x + h * a.x_hs;
      p[j] = load_stream(src + unit.at0);
      q[j] = load_stream(src + unit.at1);
    }
  }
  if (pos < 0 || pos >= a.max_len) {
    if (r == 0) raise_flag(a.err_flag, MSA_FLAG_INDEX_OOB);
    return;
  }
  RopeTurn<T> turn;
  if (unit.rotated) turn.load(a.cs + (int64_t)pos * a.rd, (int)u, a.transpose ? -1.f : 1.f);
#pragma unroll
  for (int j = 0; j < kRopeHeads; ++j) {
    const int h = (int)hg + j * groups;
    if (h < a.H) {
      if (unit.rotated) turn.apply(p[j], q[j], kInter);
      T* dst = y + h * a.out_hs;
      store_stream(dst + unit.at0, p[j]);
      store_stream(dst + unit.at1, q[j]);
    }
  }
}

template <typename T>
cudaError_t rope_t(const RopeArgs& a, cudaStream_t s) {
  const int units = RopeUnit<T>::per_head(a.d), groups = (a.H + kRopeHeads - 1) / kRopeHeads;
  const int64_t total = a.N * units * groups;
  const int64_t blocks = (total + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;  // grid x
  count_launch();
  return launch_pdl(a.interleaved ? rope_kernel<T, true> : rope_kernel<T, false>, dim3((unsigned)blocks), dim3(kRopeThreads), 0,
                    s, a, units, groups, total);
}

}  // namespace

cudaError_t launch_rope(msa_dtype dt, const RopeArgs& a, cudaStream_t s) {
  return dt == MSA_F32 ? rope_t<float>(a, s) : rope_t<__nv_bfloat16>(a, s);
}

}  // namespace msa
