// Work split of the attention over a paged cache (paged_attn.cu, paged_decode.cu,
// paged_prefill.cu), computed by every CTA for itself from the sequences' lengths.
//
// An item is one block of TB query tokens of one sequence for one KV head; its
// keys are a list of 128-key tiles: the memory tiles of the sequence's segment
// plan first, then the local tiles up to the block's last causal position.
// All tiles of all items form one sequence f = 0 .. Ttot-1 (KV head outermost,
// then sequence, block, tile), and CTA c takes the contiguous share
// [c * per, (c + 1) * per), so every CTA streams the same number of tiles
// whatever the lengths are.  A stretch of the share inside one item is a
// segment.  An item inside one CTA is finished there; an item cut by a share's
// border leaves (row maxima, row sums, unnormalised rows) of each segment in
// the workspace, merged by a second kernel in the order of the CTAs (no atomics:
// the result does not depend on timing).  Only a CTA's first and last
// segments can be cut, so two slots per CTA hold every partial result.
#pragma once

#include <stdint.h>

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

// Tiles of block i: the memory tiles and the local tiles up to the block's last
// token's position; at least one, so that a block without a visible key is
// still an item (its rows are written as zeros).
__device__ __forceinline__ int block_tiles(const Seq& s, int TB, int i) {
  const int64_t e = (int64_t)s.len - s.nq + min((int64_t)(i + 1) * TB, (int64_t)s.nq);  // visible local keys
  const int lt = e > 0 ? (int)((e + kKeys - 1) / kKeys) : 0;
  return max(1, s.nm + lt);
}

// sum over 0 <= i < n of floor((a i + b) / m), for a, b >= 0 and m > 0, by the
// Euclidean reduction of (a, m) (the lattice points under a line).
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t ans = 0;
  while (n > 0) {
    ans += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t t = a;
    a = m;
    m = t;
  }
  return ans;
}

// Tiles of blocks [0, n) of a sequence.
__device__ __forceinline__ int64_t tiles_before(const Seq& s, int TB, int n) {
  const int nb = (s.nq + TB - 1) / TB;
  if (nb == 0 || n <= 0) return 0;
  const bool all = n >= nb;
  const int64_t m = all ? nb - 1 : n;  // blocks of TB whole tokens
  const int64_t hist = (int64_t)s.len - s.nq;
  int64_t i0 = hist >= 0 ? 0 : -hist / TB;  // blocks that end at or before position 0 see no local key
  if (i0 > m) i0 = m;
  int64_t t = i0 * max(1, s.nm);
  if (m > i0) t += (m - i0) * s.nm + floor_sum(m - i0, kKeys, TB, hist + (i0 + 1) * TB + kKeys - 1);
  return all ? t + block_tiles(s, TB, nb - 1) : t;
}

struct Start {            // where a CTA's share begins
  int64_t per, f0, f1;    // tiles per CTA, the share
  int64_t b;              // sequence, KV head, block and tile of f0
  int g, i, t;
  int any;                // the share is not empty
  int64_t sums[32];       // scan scratch (one per warp)
};

// All threads of the CTA call it (blockDim.x a multiple of 32, at most 1024);
// on return st (shared memory) holds share c of `grid` shares.
__device__ __forceinline__ void find_start(const PagedBatch& p, int TB, int64_t c, int64_t grid, bool report,
                                           Start* st) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int64_t chunk = (p.B + nt - 1) / nt;
  const int64_t b0 = min(p.B, tid * chunk), b1 = min(p.B, b0 + chunk);
  int64_t mine = 0;
  for (int64_t b = b0; b < b1; ++b) {
    const Seq s = load_seq(p, b, report ? p.err_flag : nullptr);
    mine += tiles_before(s, TB, 0x7fffffff);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) st->sums[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < (nt >> 5); ++w) {
    if (w < warp) before += st->sums[w];
    total += st->sums[w];
  }
  incl += before;
  const int64_t Ttot = total * p.Hkv;
  const int64_t per = max((int64_t)1, (Ttot + grid - 1) / grid);
  const int64_t f0 = c * per, f1 = min(f0 + per, Ttot);
  if (tid == 0) {
    st->per = per;
    st->f0 = f0;
    st->f1 = f1;
    st->any = f0 < f1;
  }
  if (f0 < f1) {
    const int64_t g = f0 / total, w = f0 - g * total;
    if (w >= incl - mine && w < incl) {  // exactly one thread
      int64_t rest = w - (incl - mine), b = b0;
      Seq s = load_seq(p, b);
      for (;;) {
        const int64_t n = tiles_before(s, TB, 0x7fffffff);
        if (rest < n) break;
        rest -= n;
        s = load_seq(p, ++b);
      }
      int lo = 0, hi = (s.nq + TB - 1) / TB;  // the block holding tile `rest`: tiles_before(lo) <= rest
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles_before(s, TB, mid) <= rest) lo = mid; else hi = mid;
      }
      st->b = b;
      st->g = (int)g;
      st->i = lo;
      st->t = (int)(rest - tiles_before(s, TB, lo));
    }
  }
  __syncthreads();
}

// Walks a CTA's share segment by segment.
struct Walk {
  int64_t f, f1, b;
  int g, i, t0, T, n;  // item, first tile of the segment, tiles of the item, tiles of the segment
  Seq s;
  __device__ __forceinline__ void span(int TB) {
    T = block_tiles(s, TB, i);
    n = (int)min((int64_t)(T - t0), f1 - f);
  }
  __device__ __forceinline__ Walk(const PagedBatch& p, int TB, const Start* st)
      : f(st->f0), f1(st->f1), b(st->b), g(st->g), i(st->i), t0(st->t) {
    s = load_seq(p, b);
    span(TB);
  }
  __device__ __forceinline__ bool more() const { return f < f1; }
  __device__ __forceinline__ bool whole() const { return n == T; }
  // Call only while more(); afterwards the item fields hold the next segment if more().
  __device__ __forceinline__ void next(const PagedBatch& p, int TB) {
    f += n;
    if (f >= f1) return;
    t0 = 0;
    if ((int64_t)++i * TB >= s.nq) {
      i = 0;
      do {
        if (++b == p.B) {
          b = 0;
          ++g;
        }
        s = load_seq(p, b);
      } while (s.nq == 0);
    }
    span(TB);
  }
};

// What a CTA leaves in the workspace for the merging kernel: where its share begins.
struct Mark {
  int64_t per, f0, b;
  int32_t g, i, t, any;
};
__device__ __forceinline__ void leave_mark(const Start* st, Mark* m) {
  Mark v;
  v.per = st->per;
  v.f0 = st->f0;
  v.b = st->b;
  v.g = st->g;
  v.i = st->i;
  v.t = st->t;
  v.any = st->any;
  *m = v;
}

// Workspace: one Mark per CTA, then two partial results per CTA.  A partial result of `rows`
// rows is rows x DH unnormalised output values and rows x (row maximum, row sum), as floats.
__host__ __device__ inline size_t marks_bytes(int grid) { return ((size_t)grid * sizeof(Mark) + 255) / 256 * 256; }
__host__ __device__ inline size_t slot_floats(int rows, int dh) {
  return ((size_t)rows * (dh + 2) + 3) / 4 * 4;
}
// The slot of segment `f` of CTA c's share that begins at f0 (only its first and its last
// segments can belong to cut items).
__device__ __forceinline__ int64_t slot_of(int64_t c, int64_t f, int64_t f0) { return 2 * c + (f == f0 ? 0 : 1); }

// The merging kernel (paged_attn.cu): one item per border that is the first to cut it.
struct MergeArgs {
  PagedBatch p;
  const Mark* marks;
  const float* slots;
  int rows, TB, G, Hq;
  float unit_log2;  // row maxima times this are in the log2 domain
  void* O;
  float* lse;
};
// quads: values (row, x) of a slot at (x / 4) * rows * 4 + row * 4 + x % 4 (a row per thread
// writes them coalesced), else at row * DH + x.
cudaError_t launch_merge(msa_dtype dt, int d, bool quads, const MergeArgs& a, int grid, cudaStream_t s);

}  // namespace paged
}  // namespace msa
