// Work split of the attention over a paged cache (paged_attn.cu, paged_decode.cu,
// paged_prefill.cu), computed by every CTA for itself from the sequences' lengths.
//
// An item is one block of TB query tokens of one sequence for one KV head; its
// keys are a list of 128-key tiles: the memory tiles of the sequence's segment
// plan first, then the local tiles up to the block's last causal position.
// An item weighs its tiles plus `cost`, the tiles that its start and end take the
// time of.  All items in a row (KV head outermost, then sequence, block) form one
// sequence f = 0 .. Ttot-1 of such units, and CTA c takes the contiguous share
// [c * per, (c + 1) * per), so every CTA streams the same number of tiles
// whatever the lengths are; or, where there are no more items than CTAs and the
// longest is at most `slack` tiles longer than that share, CTA c takes item c.  A stretch of the share inside one item is a
// segment.  An item inside one CTA is finished there; an item cut by a share's
// border leaves (row maxima, row sums, unnormalised rows) of each segment in
// the workspace, merged by a second kernel in the order of the CTAs (no atomics:
// the result does not depend on timing).  Only a CTA's first and last
// segments can be cut, so two slots per CTA hold every partial result.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "paged_seq.cuh"

namespace msa {
namespace paged {

__device__ __forceinline__ int blocks_of(const Seq& s, int TB) {
  return (int)(((uint32_t)s.nq + TB - 1) / (uint32_t)TB);
}
// Tiles of block i: the memory tiles and the local tiles up to the block's last
// token's position; at least one, so that a block without a visible key is
// still an item (its rows are written as zeros).
__device__ __forceinline__ int block_tiles(const Seq& s, int TB, int i) {
  const int64_t e = (int64_t)s.len - s.nq + min((int64_t)(i + 1) * TB, (int64_t)s.nq);  // visible local keys
  const int lt = e > 0 ? (int)((e + kKeys - 1) / kKeys) : 0;
  return max(1, s.nm + lt);
}

// sum over 0 <= i < n of floor((a i + b) / 128), a >= 1, b >= 0, a n + b < 2^32.
// For a power of two a <= 128 the quotients repeat c = 128 / a times each; else
// by the Euclidean reduction of (a, 128) (the lattice points under a line).
__device__ __forceinline__ int64_t sum_div_keys(uint32_t n, uint32_t a, uint32_t b) {
  static_assert(kKeys == 128, "shifts by 7");
  if ((a & (a - 1)) == 0 && a <= 128u) {
    const int sh = 7 - (31 - __clz(a));  // log2(128 / a)
    auto upto = [&](uint32_t x) {        // sum over j < x of j >> sh
      const int64_t q = x >> sh, r = x & ((1u << sh) - 1);
      return ((q * (q - 1)) >> 1 << sh) + q * r;
    };
    const uint32_t x0 = b / a;
    return upto(x0 + n) - upto(x0);
  }
  int64_t ans = 0;
  uint32_t m = 128;
  while (n > 0) {
    ans += (int64_t)n * (n - 1) / 2 * (a / m) + (int64_t)n * (b / m);
    a %= m;
    b %= m;
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = a;
    a = m;
    m = t;
  }
  return ans;
}

// Tiles of blocks [0, n) of a sequence, n at most the number of its blocks of TB whole tokens.
__device__ __forceinline__ int64_t tiles_before(const Seq& s, int TB, int n) {
  if (n <= 0) return 0;
  const int hist = s.len - s.nq;
  // blocks that end at or before position 0 see no local key
  const int i0 = hist >= 0 ? 0 : min(n, -hist / TB);
  int64_t t = (int64_t)i0 * max(1, s.nm);
  if (n > i0)
    t += (int64_t)(n - i0) * s.nm + sum_div_keys(n - i0, TB, (uint32_t)hist + (uint32_t)((i0 + 1) * TB) + kKeys - 1);
  return t;
}

// What a kernel's work looks like to the split.
struct Split {
  int TB;     // tokens of a block
  int cost;   // an item's start and end, in tiles
  int slack;  // tiles that not merging cut items is worth
};

struct Start {            // where a CTA's share begins
  int64_t per, f0, f1;    // units per CTA, the share
  int64_t b;              // sequence, KV head, block of f0
  Seq s;
  int g, i;
  int o;                  // units of that item before f0
  int any;                // the share has a tile
  int64_t rest;           // scratch: unit (or block) of the sequence
};

struct ScanScratch {  // shared memory, free again after find_start
  int64_t sums[16];   // per warp
  int counts[16], tops[16];
};

// All threads of the CTA call it (blockDim.x a multiple of 32, at most 512); on return st (shared
// memory) holds share c of `grid` shares.  kOneBlock: sp.TB covers every sequence.  Up to 32
// sequences take one warp's shuffles and one barrier (a kernel over a short cache spends a good
// part of its time before its first load).  The tile counts appear twice in the code only: the
// kernels' loops run slower the more of it lies around them (decoding 12 rows over 1.13 GB took
// 193 us with seven copies, 183 with two).
template <bool kOneBlock>
__device__ __forceinline__ void find_start(const PagedBatch& p, const Split& sp, int64_t c, int64_t grid,
                                           bool report, Start* st, ScanScratch* sc) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int TB = sp.TB;
  const bool one_warp = p.B <= 32;
  const int chunk = (int)(((uint32_t)p.B + nt - 1) / (uint32_t)nt);  // B < 2^31
  const int64_t b0 = min(p.B, (int64_t)tid * chunk), b1 = min(p.B, b0 + chunk);
  int64_t mine = 0;         // units of this thread's sequences
  int items = 0, most = 0;  // their blocks (no count above 2^20 is needed, and offsets out of order could
                            // bring more than 32 bits hold), the tiles of the largest
  int64_t per = 1, f0 = 0, rest = 0, b = b0;
  bool one = false, any = false, owner = false;
  int g = 0;
  Seq s{0, 0, 0, 0};
  for (int pass = 0;; ++pass) {
    // pass 0 sums this thread's sequences; pass 1, of the thread that has the share's start among
    // them, stops at its sequence
    for (b = b0; b < b1; ++b) {
      s = load_seq(p, b, report && pass == 0 ? p.err_flag : nullptr);
      const int nb = kOneBlock ? (s.nq > 0) : blocks_of(s, TB);
      const int last = nb > 0 ? block_tiles(s, TB, nb - 1) : 0;  // no block has more keys than the last
      const int64_t units = (kOneBlock ? 0 : tiles_before(s, TB, nb - 1)) + last + (int64_t)nb * sp.cost;
      if (pass == 0) {
        mine += units;
        items = (int)min((uint32_t)items + (uint32_t)nb, 1u << 20);
        most = max(most, last);
      } else {
        const int64_t n = one ? nb : units;
        if (rest < n) break;
        rest -= n;
      }
    }
    if (pass == 1) break;
    if (one_warp && warp > 0) break;
    int64_t incl = mine;
    int icl = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      const int u = __shfl_up_sync(0xffffffffu, icl, o);
      if (lane >= o) {
        incl += v;
        icl += u;
      }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    int n_items = __shfl_sync(0xffffffffu, icl, 31);
    if (!one_warp) {
      if (lane == 31) {
        sc->sums[warp] = incl;
        sc->counts[warp] = icl;
        sc->tops[warp] = most;
      }
      __syncthreads();
      total = 0;
      n_items = 0;
      most = 0;
      for (int w = 0; w < (nt >> 5); ++w) {
        if (w == warp) {
          incl += total;
          icl += n_items;
        }
        total += sc->sums[w];
        n_items += sc->counts[w];
        most = max(most, sc->tops[w]);
      }
    }
    const int64_t Ttot = total * p.Hkv;
    // 32-bit divisions where the numbers allow (64-bit ones cost about a microsecond together)
    const bool small = Ttot + grid < 0x7fffffff;
    per = max((int64_t)1, small ? (int64_t)((uint32_t)(Ttot + grid - 1) / (uint32_t)grid) : (Ttot + grid - 1) / grid);
    // an item per CTA, if there are no more and none is too long
    one = (int64_t)n_items * p.Hkv <= grid && most + sp.cost <= per + sp.slack;
    f0 = c * per;
    any = one ? c < (int64_t)n_items * p.Hkv : f0 < Ttot;
    // KV head, and the unit (or block) of that head where the share begins
    const int64_t div = one ? n_items : total, at = one ? c : f0;
    g = !any ? 0 : (int)(small ? (int64_t)((uint32_t)at / (uint32_t)div) : at / div);
    const int64_t w = at - g * div, lo_w = one ? icl - items : incl - mine, hi_w = one ? icl : incl;
    owner = any && w >= lo_w && w < hi_w;  // exactly one thread
    rest = w - lo_w;
    if (tid == 0) {
      st->per = per;
      st->f0 = one ? 0 : f0;
      st->f1 = min(f0 + per, Ttot);
      st->g = g;
      if (!any) st->any = 0;
    }
    if (!owner) break;
  }
  if (owner) {
    st->b = b;
    st->s = s;
    st->rest = rest;
  }
  if (one_warp) __syncwarp();
  else __syncthreads();
  if (any && warp == 0) {
    const Seq q = st->s;
    const int64_t at = st->rest;
    int lo = one ? (int)at : 0;
    int64_t before = 0;  // units of the blocks before `lo`
    if (!kOneBlock && !one) {
      // the block holding unit `at`: the last one with no more units before it, 32 probes at a time
      int n = blocks_of(q, TB);  // answer in [lo, lo + n)
      while (n > 1) {
        const int step = (n + 31) >> 5;
        const int probe = lo + min(lane * step, n - 1);
        const int64_t units = tiles_before(q, TB, probe) + (int64_t)probe * sp.cost;
        const unsigned hit = __ballot_sync(0xffffffffu, lane * step < n && units <= at);
        const int last = 31 - __clz(hit);  // lane 0 always hits
        before = __shfl_sync(0xffffffffu, units, last);
        lo += last * step;
        n = min(step, n - last * step);
      }
    }
    if (lane == 0) {
      const int o = one ? 0 : (int)(at - before);
      const int T = block_tiles(q, TB, lo);
      if (one) st->f1 = sp.cost + T;
      st->i = lo;
      st->o = o;
      // a share may hold nothing but the start of an item that the next one takes
      st->any = min((int64_t)T, o + (st->f1 - st->f0) - sp.cost) > max(0, o - sp.cost);
    }
  }
  __syncthreads();
}

// Walks a CTA's share segment by segment (only if the share has a tile).
template <bool kOneBlock>
struct WalkT {
  int64_t f, f1, b;
  int g, i, o, t0, T, n;  // item, units of it before f, first tile of the segment, tiles of item and segment
  Seq s;
  __device__ __forceinline__ void span(const Split& sp) {
    T = block_tiles(s, sp.TB, i);
    t0 = max(0, o - sp.cost);
    n = (int)min((int64_t)T, f1 - f + o - sp.cost) - t0;
    if (n <= 0) f = f1;  // the share ends before the item's first tile
  }
  __device__ __forceinline__ WalkT(const Split& sp, const Start* st)
      : f(st->f0), f1(st->f1), b(st->b), g(st->g), i(st->i), o(st->o), s(st->s) {
    span(sp);
  }
  __device__ __forceinline__ bool more() const { return f < f1; }
  __device__ __forceinline__ bool whole() const { return n == T; }
  // Whether next() will find a segment: the share goes on past this segment and the next item's start.
  __device__ __forceinline__ bool another(const Split& sp) const {
    return f + n + sp.cost + max(0, sp.cost - o) < f1;
  }
  // Call only while more(); afterwards the item fields hold the next segment if more().
  __device__ __forceinline__ void next(const PagedBatch& p, const Split& sp) {
    f += sp.cost + T - o;
    if (f >= f1) return;
    o = 0;
    if (kOneBlock || (int64_t)++i * sp.TB >= s.nq) {
      i = 0;
      do {
        if (++b == p.B) {
          b = 0;
          ++g;
        }
        s = load_seq(p, b);
      } while (s.nq == 0);
    }
    span(sp);
  }
};

// What CTA c leaves in the workspace for the merging kernel: the item that the border at the
// start of its share is the first to cut (tokens = 0: none).
struct Mark {
  int64_t row;     // packed row of the item's first token
  int32_t b;       // sequence
  int32_t c0;      // CTA of its first segment
  int32_t n;       // segments, in CTAs c0 .. c0 + n - 1
  int32_t late;    // the first segment is its CTA's last one, not its first
  int32_t tokens;  // of the item
  int32_t g;       // KV head
};
__device__ __forceinline__ void leave_mark(const Start* st, const Split& sp, int64_t c, Mark* m) {
  Mark v = {};
  const int t = st->o - sp.cost;  // tiles of the item before the border
  if (st->any && t > 0 && t <= st->per) {  // not cut at an earlier border already
    const int64_t end = st->f0 - t + block_tiles(st->s, sp.TB, st->i);
    v.row = st->s.q0 + (int64_t)st->i * sp.TB;
    v.b = (int32_t)st->b;
    v.c0 = (int32_t)(c - 1);
    v.late = st->o < st->per;
    v.n = 2;
    for (int64_t at = st->f1; at < end; at += st->per) ++v.n;
    v.tokens = min(sp.TB, st->s.nq - st->i * sp.TB);
    v.g = st->g;
  }
  *m = v;
}

// Workspace: one Mark per CTA, one byte per CTA (whether it left out values that are not finite, of
// keys that only some rows see: paged_tma.cuh), then two partial results per CTA.  A partial result of `rows`
// rows is rows x DH unnormalised output values and rows x (row maximum, row sum), as floats.
__host__ __device__ inline size_t marks_bytes(int grid) {
  return ((size_t)grid * (sizeof(Mark) + 1) + 16 + 255) / 256 * 256;
}
static_assert(sizeof(Mark) % 16 == 0, "the bytes after the marks are read 16 at a time");
// One thread of CTA c; the bytes up to the next multiple of 16 are cleared by the last CTA.
__device__ __forceinline__ void say_odd(Mark* marks, int grid, int c, int odd) {
  uint8_t* w = reinterpret_cast<uint8_t*>(marks + grid);
  w[c] = odd != 0;
  if (c == grid - 1)
    for (int i = grid; i & 15; ++i) w[i] = 0;
}
// One warp, after the kernel that left them: whether any of at most 512 is set.
__device__ __forceinline__ bool any_odd(const Mark* marks, int grid) {
  const uint4* w = reinterpret_cast<const uint4*>(marks + grid);
  const int lane = threadIdx.x & 31;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (lane * 16 < grid) v = w[lane];
  return __any_sync(0xffffffffu, (v.x | v.y | v.z | v.w) != 0);
}
__host__ __device__ inline size_t slot_floats(int rows, int dh) {
  return ((size_t)rows * (dh + 2) + 3) / 4 * 4;
}
// The slot of segment `f` of CTA c's share that begins at f0 (only its first and its last
// segments can belong to cut items).
__device__ __forceinline__ int64_t slot_of(int64_t c, int64_t f, int64_t f0) { return 2 * c + (f == f0 ? 0 : 1); }

// The merging kernel (paged_attn.cu): O and lse of the items the marks name; and of all items, the
// values that were left out of the products if a CTA says so.
struct MergeArgs {
  PagedAttnArgs a;
  Mark* marks;
  const float* slots;
  int grid, rows;   // CTAs that left marks, rows of a slot
  int TB;           // tokens of a block
  float unit_log2;  // row maxima times this are in the log2 domain
};
// quads: values (row, x) of a slot at (x / 4) * rows * 4 + row * 4 + x % 4 (a row per thread
// writes them coalesced), else at row * DH + x.
cudaError_t launch_merge(msa_dtype dt, bool quads, const MergeArgs& m, cudaStream_t s);

}  // namespace paged
}  // namespace msa
