// The rotation of heads in units of two 16-byte vectors (rope.cu, paged_append.cu).
#pragma once

#include "common.cuh"

namespace msa {

// Unit u of a head of d dimensions, rd of them rotated (both multiples of 16): N =
// Vec<T>::N pairs u N .. u N + N - 1 of the rotation, or 2 N of the dimensions past it.
// Its two vectors lie rd / 2 apart in the half layout, side by side otherwise.
template <typename T>
struct RopeUnit {
  static constexpr int N = Vec<T>::N;
  int at0, at1;
  bool rotated;
  __device__ __forceinline__ RopeUnit(int u, int rd, bool interleaved) {
    rotated = u * 2 * N < rd;
    const bool half = rotated && !interleaved;
    at0 = half ? u * N : u * 2 * N;
    at1 = half ? at0 + rd / 2 : at0 + N;
  }
  static __host__ __device__ __forceinline__ int per_head(int d) { return d / (2 * N); }
};

// (cos, sin) of the unit's N pairs; the transposed rotation turns the other way.
template <typename T>
struct RopeTurn {
  static constexpr int N = Vec<T>::N;
  float c[N], s[N];
  __device__ __forceinline__ void load(const float* cs, int u, float sign) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(cs + 2 * (u * N + i)));
      c[i] = t.x;
      s[i] = sign * t.y;
      c[i + 1] = t.z;
      s[i + 1] = sign * t.w;
    }
  }
  __device__ __forceinline__ void turn(float& a, float& b, int i) const {
    const float x = a * c[i] - b * s[i];
    b = a * s[i] + b * c[i];
    a = x;
  }
  __device__ __forceinline__ void apply(uint4& p, uint4& q, bool interleaved) const {
    float v[N], w[N];
    unpack(p, v);
    unpack(q, w);
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        turn(v[i], v[i + 1], i / 2);
        turn(w[i], w[i + 1], N / 2 + i / 2);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) turn(v[i], w[i], i);
    }
    p = pack(v);
    q = pack(w);
  }
};

// Heads a thread takes, all of their loads in flight at once, and threads of a block.  Small blocks
// with streaming loads and stores came nearest to the copy rate (4096 tokens x 40 heads, bf16: 4
// heads and 256 threads 16.5 us, 2 and 128 16.0, and with streaming accesses 14.9).
constexpr int kRopeHeads = 2, kRopeThreads = 128;
__device__ __forceinline__ uint4 load_stream(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void store_stream(void* p, uint4 v) { __stcs(reinterpret_cast<uint4*>(p), v); }

}  // namespace msa
