// New tokens' keys and values into the pages of a cache, with the rotation of the
// keys (and of the queries, into q_out) on the way: token i of sequence b has
// cache position pos = seq_len[b] - n_b + i and goes to row pos % page of page
// block_table[b][pos / page]; its key and query are rotated by its rotary
// position (the cache position unless one is given).
//
// Bound by memory: q, k and v are read once, q_out and the cache rows written
// once, all in 16-byte vectors; a thread takes one unit of the rotation (two
// vectors) or one vector of v.  The token's place (its sequence by a warp-free
// binary search over the offsets, one block-table entry) costs a few dependent
// loads that overlap across the CTAs.
#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace msa {
namespace {

template <typename T>
__global__ void __launch_bounds__(256) paged_append_kernel(PagedAppendArgs a, int uq, int uk, int per_token,
                                                           int64_t total) {
  pdl_wait();  // the offsets, lengths and projections may come from the previous kernel
  const PagedBatch& p = a.p;
  const int Hkv = p.Hkv;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < total; u += step) {
    const int64_t n = u / per_token;
    int e = (int)(u - n * per_token);
    const bool report = e == 0;
    // the last sequence whose offset is at or before n
    int64_t lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (__ldg(p.q_off + mid) <= n) lo = mid; else hi = mid;
    }
    const int64_t q0 = __ldg(p.q_off + lo), q1 = __ldg(p.q_off + lo + 1);
    if (n < q0 || n >= q1) {  // a row behind the last sequence, or offsets that do not ascend from 0
      if (report && n < q0) raise_flag(p.err_flag, MSA_FLAG_OFFSETS);
      continue;
    }
    const int64_t len = __ldg(p.seq_len + lo);
    const int64_t at = len - (q1 - n);  // cache position
    if (q1 > p.N || at < 0) {
      if (report) raise_flag(p.err_flag, MSA_FLAG_OFFSETS);
      continue;
    }
    const int64_t pi = at / p.page;
    const int row = (int)(at - pi * p.page);
    const int64_t page = pi < p.max_pages ? __ldg(p.table + lo * p.max_pages + pi) : -1;
    const int64_t rp = a.pos ? __ldg(a.pos + n) : at;  // rotary position
    if (page < 0 || page >= p.num_pages || (a.cs && (rp < 0 || rp >= a.max_len))) {
      if (report) raise_flag(p.err_flag, MSA_FLAG_INDEX_OOB);
      continue;
    }
    const float* cs = a.cs ? a.cs + rp * a.rd : nullptr;
    const int rd = a.cs ? a.rd : 0;
    const int64_t base = page * a.page_stride + row * a.row_stride;
    if (e < Hkv * uk) {
      const int h = e / uk;
      rotate_unit<T>(reinterpret_cast<const T*>(a.k) + n * a.k_ts + h * a.d,
                     reinterpret_cast<T*>(a.K) + base + h * a.head_stride, e - h * uk, rd, a.interleaved, false, cs);
      continue;
    }
    e -= Hkv * uk;
    const int uv = a.d / Vec<T>::N;
    if (e < Hkv * uv) {
      const int h = e / uv, c = (e - h * uv) * Vec<T>::N;
      *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.V) + base + h * a.head_stride + c) =
          *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.v) + n * a.v_ts + h * a.d + c);
      continue;
    }
    e -= Hkv * uv;
    const int h = e / uq;
    rotate_unit<T>(reinterpret_cast<const T*>(a.q) + n * a.q_ts + h * a.d,
                   reinterpret_cast<T*>(a.q_out) + n * a.qo_ts + h * a.d, e - h * uq, rd, a.interleaved, false, cs);
  }
}

template <typename T>
cudaError_t append_t(const PagedAppendArgs& a, cudaStream_t s) {
  const int unit = rope_units<T>(a.d, a.cs ? a.rd : 0, a.interleaved);
  const int per_token = a.p.Hkv * (unit + a.d / Vec<T>::N) + (a.q ? a.Hq * unit : 0);
  const int64_t total = a.p.N * per_token;
  const int64_t blocks = (total + 255) / 256;
  const unsigned grid = (unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
  count_launch();
  return launch_pdl(paged_append_kernel<T>, dim3(grid), dim3(256), 0, s, a, unit, unit, per_token, total);
}

}  // namespace

cudaError_t launch_paged_append(msa_dtype dt, const PagedAppendArgs& a, cudaStream_t s) {
  return dt == MSA_F32 ? append_t<float>(a, s) : append_t<__nv_bfloat16>(a, s);
}

}  // namespace msa
