// The rotation of one head, in 16-byte units (rope.cu, paged_append.cu).
#pragma once

#include "common.cuh"

namespace msa {

// Units of one head of d dimensions of which rd are rotated (rd and d multiples of
// 2 * Vec<T>::N): half layout: a unit is the vectors at i and i + rd / 2; interleaved: a
// unit is one vector of whole pairs; past rd one vector, copied.
template <typename T>
__host__ __device__ __forceinline__ int rope_units(int d, int rd, bool interleaved) {
  const int rot = interleaved ? rd / Vec<T>::N : rd / 2 / Vec<T>::N;
  return rot + (d - rd) / Vec<T>::N;
}

template <typename T>
__device__ __forceinline__ void rotate_unit(const T* x, T* y, int unit, int rd, bool interleaved, bool transpose,
                                            const float* cs) {
  constexpr int N = Vec<T>::N;
  const int rot = interleaved ? rd / N : rd / 2 / N;
  if (unit >= rot) {  // past the rotated part
    const int at = rd + (unit - rot) * N;
    if (x != y) *reinterpret_cast<uint4*>(y + at) = *reinterpret_cast<const uint4*>(x + at);
    return;
  }
  const float sg = transpose ? -1.f : 1.f;
  if (interleaved) {
    const int at = unit * N;
    float v[N];
    unpack(*reinterpret_cast<const uint4*>(x + at), v);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 t = __ldg(reinterpret_cast<const float2*>(cs + at + i));  // pair (at + i) / 2
      const float a = v[i], b = v[i + 1], sn = sg * t.y;
      v[i] = a * t.x - b * sn;
      v[i + 1] = a * sn + b * t.x;
    }
    *reinterpret_cast<uint4*>(y + at) = pack(v);
  } else {
    const int at = unit * N, half = rd / 2;
    float v[N], w[N];
    unpack(*reinterpret_cast<const uint4*>(x + at), v);
    unpack(*reinterpret_cast<const uint4*>(x + at + half), w);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(cs + 2 * (at + i)));  // pairs at + i, at + i + 1
      const float a0 = v[i], b0 = w[i], s0 = sg * t.y;
      const float a1 = v[i + 1], b1 = w[i + 1], s1 = sg * t.w;
      v[i] = a0 * t.x - b0 * s0;
      w[i] = a0 * s0 + b0 * t.x;
      v[i + 1] = a1 * t.z - b1 * s1;
      w[i + 1] = a1 * s1 + b1 * t.z;
    }
    *reinterpret_cast<uint4*>(y + at) = pack(v);
    *reinterpret_cast<uint4*>(y + at + half) = pack(w);
  }
}

}  // namespace msa
