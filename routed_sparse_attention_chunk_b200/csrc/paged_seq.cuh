// One sequence of a ragged batch over a paged cache, as the kernels read it.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace msa {
namespace paged {

constexpr int kKeys = 128;  // keys per tile
constexpr int kTileSegs = kKeys / kSegRows;  // segments of the plan per memory tile

// One sequence as the kernels see it: query rows [q0, q0 + nq), `len` cached
// tokens, `nm` memory tiles.  Offsets or lengths that do not fit the arguments
// leave an empty sequence (nq = 0) or a clamped length; the caller that passes
// `flag` raises the matching MSA_FLAG bits.
struct Seq {
  int64_t q0;
  int nq, len, nm;
};
__device__ __forceinline__ Seq load_seq(const PagedBatch& p, int64_t b, int32_t* flag = nullptr) {
  Seq s;
  const int64_t q0 = __ldg(p.q_off + b), q1 = __ldg(p.q_off + b + 1);
  const int64_t cap = (int64_t)p.max_pages * p.page;
  const int len = __ldg(p.seq_len + b);
  const int ns = p.nseg ? __ldg(p.nseg + b) : 0;
  const bool bad_off = q0 < 0 || q1 < q0 || q1 > p.N || q1 - q0 > p.max_q;
  s.q0 = bad_off ? 0 : q0;
  s.nq = bad_off ? 0 : (int)(q1 - q0);
  s.len = len < 0 ? 0 : (int)min((int64_t)len, cap);
  s.nm = (min(max(ns, 0), p.Smax) + kTileSegs - 1) / kTileSegs;
  if (flag) {
    if (bad_off) raise_flag(flag, MSA_FLAG_OFFSETS);
    if (len < 0 || len > cap) raise_flag(flag, MSA_FLAG_INDEX_OOB);
  }
  return s;
}

}  // namespace paged
}  // namespace msa
