// Attention over a paged cache on the tensor cores for whole blocks of query rows
// (paged_attn.cu): bf16, d = 64 or 128, any GQA group of up to 64 heads.
//
// A block is up to 128 rows: TB = 128 / G tokens x the G query heads of one KV
// head, so one K/V tile serves every head of the group.  Per 128-key tile:
//   S = Q K^T by tcgen05.mma into one of two TMEM buffers (Q copied into tensor
//   memory once per item, K from its TMA tile);
//   P = 2^(scale log2(e) S - m), one row per thread, rounded to bf16 over its own
//   S buffer (2^-9 per weight, averaged over the keys; the row sum is taken from
//   the fp32 values);
//   O += P V (P from tensor memory, V MN-major from its tile).
// S and PV have their own issuing threads; K and V of a tile share one of three
// stages and one barrier.  The running maximum moves (and O is rescaled in TMEM)
// only when it grows by more than 2^8; the sum uses the same maximum, so the
// result is exact.  A row that has seen no key yet keeps the maximum -inf and
// weights of 0.
// A tile's K and V arrive as one box per page, straight from the block table's
// pages, or per run of bank rows of the segment plan.  Rows past the sequence's
// end are masked, and their V rows zeroed in shared memory before the product
// (0 x NaN is NaN, and a page's tail holds anything).
// Persistent: one CTA per SM walks its equal share of all (item, tile) pairs
// (paged_sched.cuh).  The pipeline runs through item borders: the next item's Q
// rows are copied to shared memory during the current item and into the other of
// two TMEM buffers behind its last tile, so the next S runs while the current
// item's output is written.
// Warp roles (224 threads): warp 0 TMA producer, warp 1 TMEM owner + S issuer,
// warps 2..5 softmax / output (one row per thread), warp 6 PV issuer.  Every
// wait is bounded and ends the CTA with MSA_FLAG_TIMEOUT on expiry.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged_sched.cuh"
#include "sm100.cuh"
#include "tma_host.h"

namespace msa {
namespace {

using namespace sm100;
using namespace paged;

constexpr int kRows = 128;     // MMA M: query rows per block
constexpr int kThreads = 224;  // producer, S issuer, four softmax warps, PV issuer
constexpr uint32_t kWaitPolls = 1u << 24;
constexpr float kRescaleLog2 = 8.0f;  // move the running max only when it grows by more than this

struct PreParams {
  PagedBatch p;
  const __nv_bfloat16* Q;
  int64_t q_ts;
  const int32_t* seg_row;
  const uint8_t* seg_cnt;
  int Hq, G, TB;
  int box_rows;  // rows of one box: min(page, 128)
  __nv_bfloat16* O;
  float* lse;
  Mark* marks;
  float* slots;
  float scale_log2;  // softmax scale * log2(e)
};

template <int DH>
struct Layout {
  static constexpr int kKV = 3;                // K + V stages
  static constexpr int kBoxes = DH / 64;
  static constexpr int kQ = kRows * DH * 2;    // the next item's query rows on their way to tensor memory
  static constexpr int kK = kKeys * DH * 2;    // one K (or V) tile
  static constexpr int kBar = 8 * 24;
  static constexpr int kSmem = 1024 + kQ + 2 * kKV * kK + kBar + (int)sizeof(Start);
  static constexpr uint32_t kTmemCols = 512;   // S0, S1 (128 each), O (DH), Q0, Q1 (DH / 2 each)
  static_assert(2 * kKeys + 2 * DH <= (int)kTmemCols, "tensor memory columns");
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 bytes from global to shared memory without passing registers; completes at cp_async_wait.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Packed pairs of fp32 (sm_100 f32x2 arithmetic: one instruction for two values).
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// max of three (exact, like any max; no NaN reaches it)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 2^x for a pair of arguments on the FMA and integer pipes, leaving the
// transcendental unit (whose ex2 throughput bounds the softmax) to the other
// keys: x = j + f with j = round(x) (read from the mantissa of x + 1.5 * 2^23)
// and f in [-1/2, 1/2]; 2^f by a cubic whose coefficients are a weighted
// least-squares fit of 2^f on [-1/2, 1/2] at Chebyshev nodes refined by Lawson
// iterations toward equal relative error (max relative error 7.5e-5, far below
// the bf16 rounding of P); 2^j is added to the exponent field.  Arguments below
// -126 are clamped there (weights below 2^-126 instead of 0; masked keys give
// 2^-126 * 2^f, which vanishes in the bf16 P and in the row sum's fp32).
__device__ __forceinline__ void exp2_poly2(float x0, float x1, float& e0, float& e1) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
  const uint64_t x = f2_pack(fmaxf(x0, -126.0f), fmaxf(x1, -126.0f));
  const uint64_t t = f2_add(x, f2_pack(kMagic, kMagic));         // round(x) in the low mantissa bits
  const uint64_t jf = f2_add(t, f2_pack(-kMagic, -kMagic));      // round(x) as a float
  const uint64_t f = f2_fma(jf, f2_pack(-1.0f, -1.0f), x);        // x - round(x)
  uint64_t q = f2_fma(f, f2_pack(0.0551716648f, 0.0551716648f), f2_pack(0.2426111251f, 0.2426111251f));
  q = f2_fma(q, f, f2_pack(0.6932609677f, 0.6932609677f));
  q = f2_fma(q, f, f2_pack(0.9999280572f, 0.9999280572f));
  float q0, q1, t0, t1;
  f2_unpack(q, q0, q1);
  f2_unpack(t, t0, t1);
  // the low bits of t hold round(x); shifted by 23 they add it to the exponent
  e0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
  e1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
}

// Of each 16 key pairs of a 32-key store, this many take exp2_poly2 (spread
// evenly); the rest take the transcendental unit's ex2.
constexpr int kPolyPairs = 6;
__host__ __device__ constexpr bool poly_pair(int i) { return (i * kPolyPairs) / 16 != ((i + 1) * kPolyPairs) / 16; }


template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefill_kernel(const __grid_constant__ CUtensorMap tmKm, const __grid_constant__ CUtensorMap tmVm,
                     const __grid_constant__ CUtensorMap tmKl, const __grid_constant__ CUtensorMap tmVl, PreParams a) {
  using L = Layout<DH>;
  constexpr int kKV = L::kKV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* Ks = smem;                // [kKV] K tiles
  uint8_t* Vs = Ks + kKV * L::kK;    // [kKV] V tiles
  uint8_t* Qs = Vs + kKV * L::kK;
  uint64_t* bars = reinterpret_cast<uint64_t*>(Qs + L::kQ);
  uint64_t* kv_full = bars;                // [kKV] K and V of a tile landed
  uint64_t* kv_empty = kv_full + kKV;      // [kKV] its PV is done
  uint64_t* s_full = kv_empty + kKV;       // [2] S done -> softmax
  uint64_t* p_full = s_full + 2;           // [2] P written over S -> PV
  uint64_t* p_free = p_full + 2;           // [2] PV done (O up to date, S buffer free)
  uint64_t* q_tmem = p_free + 2;           // an item's Q is in tensor memory
  uint64_t* drain_s = q_tmem + 1;
  uint64_t* drain_pv = drain_s + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_pv + 1);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Start* start = reinterpret_cast<Start*>(bars + 24);

  const PagedBatch& p = a.p;
  const int TB = a.TB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKV; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&p_free[i], 1);
    }
    mbar_init(q_tmem, 128);
    mbar_init(drain_s, 1);
    mbar_init(drain_pv, 1);
    *abort_s = 0;
    fence_mbar_init();
  }
  // a programmatic dependent: nothing an earlier kernel writes is read before this wait
  pdl_wait();
  find_start(p, TB, blockIdx.x, gridDim.x, blockIdx.x == 0, start);
  if (threadIdx.x == 0) leave_mark(start, TB, blockIdx.x, a.marks + blockIdx.x);
  pdl_trigger();
  if (!start->any) return;
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S0, S1 (128 each), O (DH), Q0, Q1 as the S MMAs' A operand (DH / 2: bf16 pairs)
  const uint32_t tS0 = tmem, tO = tmem + 2 * kKeys, tQ0 = tmem + 2 * kKeys + DH;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_or_stop(bar, parity, kWaitPolls, abort_s); };

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    // Lane 0 waits and arms the barriers.  A tile is up to 16 boxes per 64-column
    // half of K and of V, one lane each: the plan's segments of kSegRows bank rows,
    // or the pages (parts of pages) that hold cached tokens.  Each lands on a 1 KB
    // swizzle atom, so the tile's layout is that of one 128-row box.
    uint32_t it = 0;
    bool stop = false;
    for (Walk w(TB, start); w.more() && !stop; w.next(p, TB)) {
      for (int t = w.t0; t < w.t0 + w.n; ++t, ++it) {
        const uint32_t st = it % kKV, round = it / kKV;
        const bool mem = t < w.s.nm;
        const int key0 = mem ? 0 : (t - w.s.nm) * kKeys;
        const int rows = mem ? kSegRows : a.box_rows;
        bool mine;
        int at = 0, in_page = 0;  // bank row, or page and row inside it
        if (mem) {
          mine = lane < kTileSegs;
          if (mine) at = __ldg(a.seg_row + w.b * p.Smax + t * kTileSegs + lane);
        } else {
          const int k = key0 + lane * rows;
          mine = lane * rows < kKeys && k < w.s.len;
          if (mine) {
            const int pi = k / p.page;
            in_page = k - pi * p.page;
            at = __ldg(p.table + w.b * p.max_pages + pi);
            if (at < 0 || at >= p.num_pages) {  // read as zeros (a page past the last)
              raise_flag(p.err_flag, MSA_FLAG_INDEX_OOB);
              at = (int)p.num_pages;
            }
          }
        }
        const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
        int ok = 1;
        if (lane == 0) {
          ok = wait(&kv_empty[st], (round & 1) ^ 1);
          if (ok) mbar_arrive_expect_tx(&kv_full[st], (uint32_t)(boxes * rows * DH * 2 * 2));
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          stop = true;
          break;
        }
        if (mine) {
          uint8_t* dk = Ks + st * L::kK + lane * (rows * 128);
          uint8_t* dv = Vs + st * L::kK + lane * (rows * 128);
#pragma unroll
          for (int dc = 0; dc < L::kBoxes; ++dc) {
            if (mem) {
              tma_load_2d(dk + dc * (kKeys * 128), &tmKm, w.g * DH + dc * 64, at, &kv_full[st]);
              tma_load_2d(dv + dc * (kKeys * 128), &tmVm, w.g * DH + dc * 64, at, &kv_full[st]);
            } else {
              tma_load_4d(dk + dc * (kKeys * 128), &tmKl, dc * 64, w.g, in_page, at, &kv_full[st]);
              tma_load_4d(dv + dc * (kKeys * 128), &tmVl, dc * 64, w.g, in_page, at, &kv_full[st]);
            }
          }
        }
      }
    }
    if (lane == 0) {
      // the copies in flight land before the CTA leaves its shared memory
      for (uint32_t st = 0; st < (uint32_t)kKV && st < it; ++st)
        if (!mbar_wait(&kv_full[st], ((it - 1 - st) / kKV) & 1, kWaitPolls)) *abort_s = 1;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(kRows, kKeys);
      // descriptors of the operand bases; a k-step adds its byte offset / 16 to
      // the 14-bit start-address field (shared addresses stay below 256 KB, so
      // the field never carries)
      const uint64_t dk0 = desc_k_sw128(smem_u32(Ks));
      uint32_t g = 0, nseg = 0;
      bool ok = true;
      for (Walk w(TB, start); ok && w.more(); w.next(p, TB), ++nseg) {
        const uint32_t tQ = tQ0 + (nseg & 1) * (DH / 2);
        ok = wait(q_tmem, nseg & 1);
        for (int j = 0; ok && j < w.n; ++j, ++g) {
          // S goes into buffer g & 1 once the PV of tile g - 2 has read P from it
          if (g >= 2 && !(ok = wait(&p_free[g & 1], ((g - 2) >> 1) & 1))) break;
          const uint32_t ks = g % kKV;
          if (!(ok = wait(&kv_full[ks], (g / kKV) & 1))) break;
          tc_fence_after();
          const uint64_t dk = dk0 + (uint64_t)((ks * L::kK) >> 4);
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            // A = Q from TMEM (16 elements of bf16 per step are 8 columns), B = K from its tile
            const int box = k >> 2, kk = k & 3;
            mma_bf16_ts(tS0 + (g & 1) * kKeys, tQ + k * 8, dk + (uint64_t)((box * kKeys * 128 + kk * 32) >> 4), idS,
                        k > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[g & 1]);
        }
      }
      mma_commit(drain_s);
      if (!mbar_wait(drain_s, 0, kWaitPolls)) *abort_s = 1;
    }
  } else if (warp == 6) {
    // ---------------------------------------------------------------- PV issuer
    if (lane == 0) {
      constexpr uint32_t idO = idesc_bf16_f32(kRows, DH, /*b_mn_major=*/true);
      const uint64_t dv0 = desc_mn_sw128(smem_u32(Vs), kKeys * 128);
      uint32_t g = 0;
      bool ok = true;
      for (Walk w(TB, start); ok && w.more(); w.next(p, TB)) {
        for (int j = 0; ok && j < w.n; ++j, ++g) {
          const uint32_t st = g & 1, vs = g % kKV;
          // P written over S; V landed with K
          if (!(ok = wait(&p_full[st], (g >> 1) & 1)) || !(ok = wait(&kv_full[vs], (g / kKV) & 1))) break;
          tc_fence_after();
          const uint64_t dv = dv0 + (uint64_t)((vs * L::kK) >> 4);
          // A = P from TMEM: 16 keys of bf16 per step are 8 columns
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_bf16_ts(tO, tS0 + st * kKeys + k * 8, dv + (uint64_t)((k * 16 * 128) >> 4), idO,
                        (j > 0 || k > 0) ? 1u : 0u);
          mma_commit(&p_free[st]);
          mma_commit(&kv_empty[vs]);
        }
      }
      mma_commit(drain_pv);
      if (!mbar_wait(drain_pv, 0, kWaitPolls)) *abort_s = 1;
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int q = warp & 3;
    const int r = q * 32 + lane;                      // this thread's row (TMEM lane)
    const int tl = r / a.G, hh = r - tl * a.G;        // token of the block and head of the group
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    const float sl2 = a.scale_log2;
    uint8_t* qrow = Qs + r * (DH * 2);
    // this row of an item's queries into shared memory (zeros for a row that does not exist); the
    // 16-byte pieces swizzled by the row so that a warp's reads spread over the banks
    auto fetch_q = [&](const Walk& w) {
      const int t = w.i * TB + tl;
      const bool have = tl < TB && t < w.s.nq;
      const __nv_bfloat16* src = a.Q + (w.s.q0 + t) * a.q_ts + (w.g * a.G + hh) * DH;
#pragma unroll
      for (int c = 0; c < DH / 8; ++c) {
        uint8_t* dst = qrow + ((c ^ (r & 7)) << 4);
        if (have) cp_async16(dst, src + c * 8);
        else *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
      }
    };
    // ... and from there into a Q buffer of tensor memory, the S MMAs' A operand
    auto place_q = [&](uint32_t tQ) {
      cp_async_wait();
      __syncwarp();
#pragma unroll
      for (int c0 = 0; c0 < DH / 8; c0 += 4) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(qrow + (((c0 + c) ^ (r & 7)) << 4));
          w[c * 4 + 0] = v.x;
          w[c * 4 + 1] = v.y;
          w[c * 4 + 2] = v.z;
          w[c * 4 + 3] = v.w;
        }
        tmem_st16(tQ + lane_off + c0 * 4, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(q_tmem);
    };
    Walk w(TB, start);
    fetch_q(w);
    place_q(tQ0);
    uint32_t g = 0, nseg = 0;
    bool ok = true;
    while (ok && w.more()) {
      Walk wn = w;
      wn.next(p, TB);
      const bool more = wn.more();
      if (more) fetch_q(wn);
      const int t = w.i * TB + tl;
      const bool rvalid = tl < TB && t < w.s.nq;
      // local keys [0, seen) are visible to this row (rows that do not exist follow the last one)
      const int seen = w.s.len - w.s.nq + (rvalid ? t : min(w.i * TB + TB, w.s.nq) - 1) + 1;
      float m_run = -INFINITY, l_run = 0.f;  // running max in the scaled log2 domain
      for (int j = 0; j < w.n; ++j, ++g) {
        const int st = g & 1, tile = w.t0 + j;
        const bool mem = tile < w.s.nm;
        // a memory tile's segment counts (one byte per segment), loaded before the wait
        uint4 segc = make_uint4(0u, 0u, 0u, 0u);
        if (mem) segc = __ldg(reinterpret_cast<const uint4*>(a.seg_cnt + w.b * p.Smax + tile * kTileSegs));
        // waits are decided warp-wide so the warp-collective tcgen05 ops are never split
        if (!__all_sync(0xffffffffu, wait(&s_full[st], (g >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 16) tmem_ld16(tmem + lane_off + st * kKeys + c, *reinterpret_cast<float(*)[16]>(&s[c]));
        tmem_ld_wait();
        bool masked = false;  // some key of the tile is not visible to some row of the warp
        if (mem) {
          // key c of the tile is row c % kSegRows of segment c / kSegRows
          static_assert(kTileSegs == 16 && kSegRows == 8, "four segment counts per word");
          const uint32_t full8 = 0x08080808u;
          masked = !(segc.x == full8 && segc.y == full8 && segc.z == full8 && segc.w == full8);
          if (masked) {
            const uint32_t cw[4] = {segc.x, segc.y, segc.z, segc.w};
#pragma unroll
            for (int c = 0; c < kKeys; ++c) {
              const uint32_t n = (cw[c >> 5] >> (((c >> 3) & 3) * 8)) & 0xffu;
              s[c] = (uint32_t)(c & 7) < n ? s[c] : -INFINITY;
            }
          }
        } else {
          const int base = (tile - w.s.nm) * kKeys;
          const int lim = seen - base;
          masked = __any_sync(0xffffffffu, lim < kKeys);
          if (masked) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c) s[c] = c < lim ? s[c] : -INFINITY;
          }
          // Rows of V past the sequence's end: zeros.  The copy that filled the stage has landed
          // (S read the same barrier's K); this wait makes it visible to this thread.
          const int end = w.s.len - base;
          if (end < kKeys) {
            const uint32_t vs = g % kKV;
            if (!__all_sync(0xffffffffu, wait(&kv_full[vs], (g / kKV) & 1))) {
              ok = false;
              break;
            }
            if (r >= end) {
              uint8_t* v = Vs + vs * L::kK + r * 128;
#pragma unroll
              for (int c = 0; c < 8 * L::kBoxes; ++c)
                *reinterpret_cast<uint4*>(v + (c >> 3) * (kKeys * 128) + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
          }
        }
        // eight independent chains of three-input maxima (max is exact in any order)
        static_assert(kKeys == 128, "the chains cover 128 keys");
        float m8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m8[i] = fmax3(s[i], s[i + 8], s[i + 16]);
#pragma unroll
        for (int c = 24; c < 120; c += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = fmax3(m8[i], s[c + i], s[c + 8 + i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) m8[i] = fmaxf(m8[i], s[120 + i]);
        const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
        // move the max (and rescale O) only when it grows by more than 2^8
        const float mt = mx * sl2;
        const bool grow = mt > m_run + kRescaleLog2;
        float corr = 1.f;
        if (grow) {
          corr = m_run == -INFINITY ? 0.f : fast_exp2(m_run - mt);
          m_run = mt;
        }
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          // O must hold every earlier PV before it is rescaled
          if (!__all_sync(0xffffffffu, wait(&p_free[(g - 1) & 1], ((g - 1) >> 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < DH; c += 16) {
            float o[16];
            tmem_ld16(tO + lane_off + c, o);
            tmem_ld_wait();
            uint32_t wv[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) wv[i] = __float_as_uint(o[i] * corr);
            tmem_st16(tO + lane_off + c, wv);
          }
          tmem_st_wait();
        }
        l_run *= corr;
        const float nm = m_run == -INFINITY ? 0.f : -m_run;  // no key seen yet: 2^(-inf) below is 0
        // P over S: 32 keys (16 columns of bf16 pairs) per store; the scaled arguments and the row
        // sums in packed pairs (one f32x2 instruction for two keys).  Tiles with masked keys take
        // ex2 throughout, which gives masked keys exactly 0.
        const uint64_t sl2x2 = f2_pack(sl2, sl2), nmx2 = f2_pack(nm, nm);
        uint64_t lsa2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        auto weights = [&](auto poly) {
#pragma unroll
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            uint32_t wv[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1, e0, e1;
              f2_unpack(f2_fma(f2_pack(s[c0 + 2 * i], s[c0 + 2 * i + 1]), sl2x2, nmx2), x0, x1);
              if (poly.value && poly_pair(i)) {
                exp2_poly2(x0, x1, e0, e1);
              } else {
                e0 = fast_exp2(x0);
                e1 = fast_exp2(x1);
              }
              lsa2[i & 1] = f2_add(lsa2[i & 1], f2_pack(e0, e1));
              wv[i] = pack_bf16x2(e0, e1);
            }
            tmem_st16(tmem + lane_off + st * kKeys + c0 / 2, wv);
          }
        };
        if (masked) weights(std::false_type{});
        else weights(std::true_type{});
        float lsa[4];
        f2_unpack(lsa2[0], lsa[0], lsa[1]);
        f2_unpack(lsa2[1], lsa[2], lsa[3]);
        l_run += (lsa[0] + lsa[1]) + (lsa[2] + lsa[3]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[st]);
      }
      if (!ok) break;
      // the next item's Q, so that its first S runs beside this item's output; its buffer was last
      // read by the S MMAs of the item before this one
      if (more) place_q(tQ0 + ((nseg + 1) & 1) * (DH / 2));
      const uint32_t gl = g - 1;
      if (!__all_sync(0xffffffffu, wait(&p_free[gl & 1], (gl >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool whole = w.whole();
      // O / l, lse = (m + log2 l) ln 2; the sum is 0 only for a row that saw no key: O = 0, lse = -inf
      const bool none = l_run == 0.f;
      const float inv = none ? 0.f : 1.f / l_run;
      const int64_t row = w.s.q0 + t;
      const int h = w.g * a.G + hh;
      __nv_bfloat16* orow = a.O + (row * a.Hq + h) * DH;
      float* slot = a.slots + slot_of(blockIdx.x, w.f, start->f0) * slot_floats(kRows, DH);
#pragma unroll
      for (int c = 0; c < DH; c += 16) {
        float o[16];
        tmem_ld16(tO + lane_off + c, o);
        tmem_ld_wait();
        if (rvalid && whole) {
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            float f[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = none ? 0.f : o[i + x] * inv;
            *reinterpret_cast<uint4*>(orow + c + i) = pack(f);
          }
        } else if (rvalid) {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(slot + (((c + i) >> 2) * kRows + r) * 4) =
                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
        __syncwarp();
      }
      if (rvalid) {
        if (!whole) *reinterpret_cast<float2*>(slot + kRows * DH + 2 * r) = make_float2(m_run, l_run);
        else if (a.lse) a.lse[(int64_t)h * p.N + row] = none ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
      }
      ++nseg;
      w = wn;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_s) raise_flag(p.err_flag, MSA_FLAG_TIMEOUT);
}

template <int DH>
cudaError_t prefill_t(const PagedAttnArgs& a, cudaStream_t s) {
  using L = Layout<DH>;
  CUtensorMap tkm, tvm, tkl, tvl;
  const int box = a.p.page < kKeys ? a.p.page : kKeys;
  if (!make_tmap_pages_bf16(&tkl, a.K, DH, a.p.Hkv, a.p.page, a.p.num_pages, a.head_stride, a.row_stride,
                            a.page_stride, box) ||
      !make_tmap_pages_bf16(&tvl, a.V, DH, a.p.Hkv, a.p.page, a.p.num_pages, a.head_stride, a.row_stride,
                            a.page_stride, box))
    return cudaErrorInvalidValue;
  tkm = tkl;  // never read without a plan
  tvm = tvl;
  if (a.Kbar) {
    const uint64_t rowkv = (uint64_t)a.p.Hkv * DH * 2;
    if (!make_tmap_2d_bf16(&tkm, a.Kbar, (uint64_t)a.p.Hkv * DH, (uint64_t)a.C, rowkv, 64, kSegRows) ||
        !make_tmap_2d_bf16(&tvm, a.Vbar, (uint64_t)a.p.Hkv * DH, (uint64_t)a.C, rowkv, 64, kSegRows))
      return cudaErrorInvalidValue;
  }
  const int grid = sm_count(), G = a.Hq / a.p.Hkv;
  PreParams d;
  d.p = a.p;
  d.Q = reinterpret_cast<const __nv_bfloat16*>(a.Q);
  d.q_ts = a.q_ts;
  d.seg_row = a.seg_row;
  d.seg_cnt = a.seg_cnt;
  d.Hq = a.Hq;
  d.G = G;
  d.TB = kRows / G;
  d.box_rows = box;
  d.O = reinterpret_cast<__nv_bfloat16*>(a.O);
  d.lse = a.lse;
  d.marks = reinterpret_cast<Mark*>(a.part);
  d.slots = reinterpret_cast<float*>(reinterpret_cast<char*>(a.part) + marks_bytes(grid));
  d.scale_log2 = a.scale * 1.4426950408889634f;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(paged_prefill_kernel<DH>, L::kSmem, done);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_pdl(paged_prefill_kernel<DH>, dim3((unsigned)grid), dim3(kThreads), (size_t)L::kSmem, s, tkm, tvm, tkl,
                 tvl, d);
  if (e != cudaSuccess) return e;
  MergeArgs m{d.marks, d.slots, a.p.N, kRows, G, a.Hq, 1.f, a.O, a.lse};
  return launch_merge(MSA_BF16, DH, true, m, grid, s);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, cudaStream_t s) {
  return a.d == 64 ? prefill_t<64>(a, s) : prefill_t<128>(a, s);
}

}  // namespace msa
