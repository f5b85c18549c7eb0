// Tile loads of the bf16 kernels over a paged cache (paged_decode.cu, paged_prefill.cu).
//
// A K or V tile of 128 rows x DH in shared memory is 16 groups of 8 rows, each
// group DH / 64 blocks of 8 rows x 128 bytes (64 columns, 128-byte swizzle): groups
// kGroup bytes apart, a group's blocks 1024 apart.  In this order one TMA box holds
// all columns of a page's rows whatever the page size (each box costs its lane about
// 65 cycles to issue, so a box per 64 columns cost a warp 2,400 cycles a tile with
// pages of 16), and the matrix descriptors reach every group with one stride.
//
// The box is (64 columns, 8 rows, DH / 64 blocks, groups), which takes rank 5 with
// the pages, so the heads have to share a dimension with the blocks (heads next to
// one another in a row) or with the groups (a page's rows of one head together).
// Other strides take boxes of a single group.
#pragma once

#include "internal.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace msa {
namespace paged {

template <int DH>
struct Tile {
  static constexpr int kBlocks = DH / 64;
  static constexpr int kGroup = 1024 * kBlocks;
  static constexpr int kBytes = 16 * kGroup;
};

// Where (head g, row of a page, page) lies in the map: coordinate 1 is row * r1, 2 is
// g * h2, 3 is g * h3 + (row / 8) * r3.
struct PageMap {
  int box_rows;  // rows of one box
  int page_shift;
  int r1, h2, h3, r3;
};

// The tensor maps of K and V pages and of the bank's rows (copies of the pages' where there is none).
struct TileMaps {
  CUtensorMap k, v, kbar, vbar;
};
template <int DH>
inline bool make_tile_maps(const PagedAttnArgs& a, TileMaps* m, PageMap* pm) {
  constexpr int kBlocks = DH / 64;
  const int64_t page = a.p.page, heads = a.p.Hkv, rs = a.row_stride;
  pm->page_shift = __builtin_ctz((unsigned)page);
  pm->box_rows = page < 128 ? (int)page : 128;
  pm->r1 = pm->h2 = pm->h3 = pm->r3 = 0;
  int64_t dims[5] = {64, 8, 0, 0, a.p.num_pages}, st[4] = {rs, 64, 8 * rs, a.page_stride};
  int box[5] = {64, 8, kBlocks, pm->box_rows / 8, 1};
  if (heads == 1 || a.head_stride == DH) {  // heads among the blocks
    dims[2] = kBlocks * heads;
    dims[3] = page / 8;
    pm->h2 = kBlocks;
    pm->r3 = 1;
  } else if (a.head_stride == page * rs) {  // heads among the groups
    dims[2] = kBlocks;
    dims[3] = heads * (page / 8);
    pm->h3 = (int)(page / 8);
    pm->r3 = 1;
  } else {
    dims[1] = page;
    dims[2] = kBlocks;
    dims[3] = heads;
    st[2] = a.head_stride;
    box[3] = 1;
    pm->box_rows = 8;
    pm->r1 = 1;
    pm->h3 = 1;
  }
  if (!make_tmap_bf16(&m->k, a.K, 5, dims, st, box) || !make_tmap_bf16(&m->v, a.V, 5, dims, st, box)) return false;
  m->kbar = m->k;  // never read without a plan
  m->vbar = m->v;
  if (!a.Kbar) return true;
  const int64_t bd[3] = {64, a.C, kBlocks * heads}, bs[2] = {heads * DH, 64};
  const int bb[3] = {64, kSegRows, kBlocks};
  return make_tmap_bf16(&m->kbar, a.Kbar, 3, bd, bs, bb) && make_tmap_bf16(&m->vbar, a.Vbar, 3, bd, bs, bb);
}

// One lane's box of a tile.
struct Box {
  bool mine;
  int at, in_page;  // bank row, or page and row inside it
};
__device__ __forceinline__ Box locate_box(const PagedBatch& p, const PageMap& pm, const int32_t* seg_row, int64_t b,
                                          int nm, int len, int tile, int lane) {
  Box x{false, 0, 0};
  if (tile < nm) {
    x.mine = lane < 16;
    if (x.mine) x.at = __ldg(seg_row + b * p.Smax + tile * 16 + lane);
  } else {
    const int k = (tile - nm) * 128 + lane * pm.box_rows;
    x.mine = lane * pm.box_rows < 128 && k < len;
    if (x.mine) {
      const int pi = k >> pm.page_shift;
      x.in_page = k - (pi << pm.page_shift);
      x.at = __ldg(p.table + b * p.max_pages + pi);
    }
  }
  return x;
}
// A page outside the pool is flagged and read as zeros (a page past the last).
__device__ __forceinline__ void check_box(const PagedBatch& p, bool mem, Box* x) {
  if (!mem && x->mine && (x->at < 0 || x->at >= p.num_pages)) {
    raise_flag(p.err_flag, MSA_FLAG_INDEX_OOB);
    x->at = (int)p.num_pages;
  }
}
template <int DH>
__device__ __forceinline__ void load_box(uint8_t* tile, const CUtensorMap* pages, const CUtensorMap* bank,
                                         const PageMap& pm, bool mem, const Box& x, int g, int lane, uint64_t* bar) {
  if (mem)
    sm100::tma_load_3d(tile + lane * Tile<DH>::kGroup, bank, 0, x.at, g * Tile<DH>::kBlocks, bar);
  else
    sm100::tma_load_5d(tile + lane * (pm.box_rows * 128 * Tile<DH>::kBlocks), pages, 0, x.in_page * pm.r1, g * pm.h2,
                       g * pm.h3 + (x.in_page >> 3) * pm.r3, x.at, bar);
}

// Rows of a V tile that some query row must not see although its weight is 0 there: 0 x NaN and
// 0 x infinity are NaN.  A row that nobody sees (past the sequence's end, where a page holds
// anything, or padding of a bank run) is set to zeros before the product.  In a row that some see
// and others do not (a later token's of the same block), the values that are not finite are set to
// zeros; a finite weight above 0 times such a value is that value, whatever the weight, so they are
// added to the outputs that see them by the merging kernel.  Every other output keeps its bits.
template <int DH>
__device__ __forceinline__ uint8_t* tile_row(uint8_t* tile, int r) {
  return tile + (r >> 3) * Tile<DH>::kGroup + (r & 7) * 128;
}
template <int DH>
__device__ __forceinline__ void zero_row(uint8_t* tile, int r) {
  uint8_t* v = tile_row<DH>(tile, r);
#pragma unroll
  for (int c = 0; c < 8 * Tile<DH>::kBlocks; ++c)
    *reinterpret_cast<uint4*>(v + (c >> 3) * 1024 + ((c ^ r) & 7) * 16) = make_uint4(0, 0, 0, 0);
}
template <int DH>
__device__ __forceinline__ bool row_not_finite(uint8_t* tile, int r) {
  const uint8_t* v = tile_row<DH>(tile, r);
  uint32_t top = 0;  // bit 15 or 31: an exponent of ones carried out
#pragma unroll
  for (int c = 0; c < 8 * Tile<DH>::kBlocks; ++c) {
    const uint4 u = *reinterpret_cast<const uint4*>(v + (c >> 3) * 1024 + ((c ^ r) & 7) * 16);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) top |= (w[i] & 0x7f807f80u) + 0x00800080u;
  }
  return (top & 0x80008000u) != 0;
}
// Values of the row that are not finite become 0.  A call, not inlined: a rare path inside the tile
// loops, which run slower the more code lies in them (23 requests with heads of 64: 119 us without
// it, 120.6 with the call, 122.8 inlined and rolled, 130 unrolled by four).
template <int DH>
__device__ __noinline__ void drop_not_finite(uint8_t* tile, int r) {
  uint8_t* v = tile_row<DH>(tile, r);
#pragma unroll 1
  for (int c = 0; c < 32 * Tile<DH>::kBlocks; ++c) {
    uint32_t* w = reinterpret_cast<uint32_t*>(v + (c >> 5) * 1024 + (c & 31) * 4);
    const uint32_t u = *w, odd = (((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u) >> 15;
    *w = u & ~(odd * 0xffffu);
  }
}
}  // namespace paged
}  // namespace msa
