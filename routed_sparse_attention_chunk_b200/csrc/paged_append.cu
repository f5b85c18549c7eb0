// New tokens' keys and values into the pages of a cache, with the rotation of the
// keys (and of the queries, into q_out) on the way: token i of sequence b has
// cache position pos = seq_len[b] - n_b + i and goes to row pos % page of page
// block_table[b][pos / page]; its key and query are rotated by its rotary
// position (the cache position unless one is given).
//
// Bound by memory: q, k and v are read once, q_out and the cache rows written
// once.  A thread takes one unit (two 16-byte vectors) of two of the
// token's heads (queries, keys, values in that order): their loads go out first,
// and the token's place (its sequence, its block-table entry, the table's pairs: a
// chain of dependent loads) is found while they are in flight.
#include "common.cuh"
#include "internal.h"
#include "paged_seq.cuh"
#include "rope.cuh"

namespace msa {
namespace {

template <typename T, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) paged_append_kernel(PagedAppendArgs a, int units, int groups, int64_t total) {
  pdl_wait();  // the offsets, lengths and projections may come from the previous kernel
  const PagedBatch& p = a.p;
  const int Hkv = p.Hkv, Hq = a.q ? a.Hq : 0, heads = Hq + 2 * Hkv;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (blockIdx.x == 0 && p.err_flag)  // offsets and lengths that do not fit the arguments
    for (int64_t b = threadIdx.x; b < p.B; b += blockDim.x) paged::load_seq(p, b, p.err_flag);
  if (id >= total) return;
  const uint32_t per = (uint32_t)(units * groups);
  const int64_t n = total < 0xffffffffll ? (int64_t)((uint32_t)id / per) : id / per;
  const uint32_t r = (uint32_t)(id - n * per), hg = r / (uint32_t)units, u = r - hg * (uint32_t)units;
  const bool report = r == 0;
  const int rd = a.cs ? a.rd : 0;
  const RopeUnit<T> rot((int)u, rd, kInter);  // of queries and keys
  const int at1v = (int)u * 2 * Vec<T>::N + Vec<T>::N;
  uint4 v0[kRopeHeads], v1[kRopeHeads];
#pragma unroll
  for (int j = 0; j < kRopeHeads; ++j) {
    const int h = (int)hg + j * groups;
    if (h < heads) {
      const T* src;
      if (h < Hq) src = reinterpret_cast<const T*>(a.q) + n * a.q_ts + h * a.d;
      else if (h < Hq + Hkv) src = reinterpret_cast<const T*>(a.k) + n * a.k_ts + (h - Hq) * a.d;
      else src = reinterpret_cast<const T*>(a.v) + n * a.v_ts + (h - Hq - Hkv) * a.d;
      const bool val = h >= Hq + Hkv;
      v0[j] = load_stream(src + (val ? at1v - Vec<T>::N : rot.at0));
      v1[j] = load_stream(src + (val ? at1v : rot.at1));
    }
  }
  // the last sequence whose offset is at or before n; the proportional guess is right for one
  // token a sequence
  int64_t lo = p.N < 0x7fffffff && p.B * n < 0x7fffffff ? (int64_t)((uint32_t)(p.B * n) / (uint32_t)p.N) : 0;
  if (!(__ldg(p.q_off + lo) <= n && n < __ldg(p.q_off + lo + 1))) {
    int64_t hi = p.B;
    lo = 0;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (__ldg(p.q_off + mid) <= n) lo = mid; else hi = mid;
    }
  }
  const int64_t q0 = __ldg(p.q_off + lo), q1 = __ldg(p.q_off + lo + 1);
  if (n < q0 || n >= q1) return;  // a row outside every sequence
  const int64_t at = (int64_t)__ldg(p.seq_len + lo) - (q1 - n);  // cache position
  if (q0 < 0 || q1 > p.N || at < 0) {
    if (report) raise_flag(p.err_flag, MSA_FLAG_OFFSETS);
    return;
  }
  const uint32_t pi = (uint32_t)at / (uint32_t)p.page, row = (uint32_t)at - pi * (uint32_t)p.page;
  const int64_t page = (int64_t)pi < p.max_pages ? __ldg(p.table + lo * p.max_pages + pi) : -1;
  const int64_t rp = a.pos ? __ldg(a.pos + n) : at;  // rotary position
  if (page < 0 || page >= p.num_pages || (a.cs && (rp < 0 || rp >= a.max_len))) {
    if (report) raise_flag(p.err_flag, MSA_FLAG_INDEX_OOB);
    return;
  }
  RopeTurn<T> turn;
  if (rot.rotated) turn.load(a.cs + rp * rd, (int)u, 1.f);
  const int64_t base = page * a.page_stride + row * a.row_stride;
#pragma unroll
  for (int j = 0; j < kRopeHeads; ++j) {
    const int h = (int)hg + j * groups;
    if (h < heads) {
      const bool val = h >= Hq + Hkv;
      T* dst;
      if (h < Hq) dst = reinterpret_cast<T*>(a.q_out) + n * a.qo_ts + h * a.d;
      else if (!val) dst = reinterpret_cast<T*>(a.K) + base + (h - Hq) * a.head_stride;
      else dst = reinterpret_cast<T*>(a.V) + base + (h - Hq - Hkv) * a.head_stride;
      if (rot.rotated && !val) turn.apply(v0[j], v1[j], kInter);
      store_stream(dst + (val ? at1v - Vec<T>::N : rot.at0), v0[j]);
      store_stream(dst + (val ? at1v : rot.at1), v1[j]);
    }
  }
}

template <typename T>
cudaError_t append_t(const PagedAppendArgs& a, cudaStream_t s) {
  const int units = RopeUnit<T>::per_head(a.d);
  const int groups = ((a.q ? a.Hq : 0) + 2 * a.p.Hkv + kRopeHeads - 1) / kRopeHeads;
  const int64_t total = a.p.N * units * groups;
  const int64_t blocks = (total + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;  // grid x
  count_launch();
  return launch_pdl(a.interleaved ? paged_append_kernel<T, true> : paged_append_kernel<T, false>,
                    dim3((unsigned)blocks), dim3(kRopeThreads), 0, s, a, units, groups, total);
}

}  // namespace

cudaError_t launch_paged_append(msa_dtype dt, const PagedAppendArgs& a, cudaStream_t s) {
  return dt == MSA_F32 ? append_t<float>(a, s) : append_t<__nv_bfloat16>(a, s);
}

}  // namespace msa
