// Attention over a paged cache on the tensor cores for whole blocks of query rows
// (paged_attn.cu): bf16, d = 64 or 128, any GQA group of up to 64 heads.
//
// A block is up to 128 rows: TB = 128 / G tokens x the G query heads of one KV
// head, so one K/V tile serves every head of the group.  Per 128-key tile:
//   S = Q K^T by tcgen05.mma into one of two TMEM buffers (Q copied into tensor
//   memory once per item, K from its TMA tile);
//   P = 2^(scale log2(e) S - m), one row per thread, rounded to bf16 (2^-9 per
//   weight on average less, over many keys; the row sum is taken from the fp32
//   values), into tensor memory;
//   O += P V (P from tensor memory, V MN-major from its tile).
// Two softmax warpgroups take the tiles in turn, so that one's exponentials run
// beside the other's loads, maxima and hand-offs (a single one was latency-bound at
// 2,700 cycles a tile against 1,030 of tensor-core work).  Each keeps a reference
// maximum of its own per row, a whole number in the log2 domain that moves only
// when a score passes it by 2^8; a tile's P is brought to O's reference when it is
// stored, which happens in the tiles' order, and O (in TMEM) is rescaled only when
// that reference has to grow.  All these factors are powers of two, and the sums of
// the two are added under O's reference at the item's end, so the result is exact.
// A row that has seen no key yet keeps the reference -inf and weights of 0.
// A tile's K and V arrive as one box per page, straight from the block table's
// pages, or per run of bank rows of the segment plan (paged_tma.cuh), K and V from a
// warp each, in rings of three.  Rows past the sequence's end are masked, and their
// V rows zeroed in shared memory before the product; what a query row does not see
// never reaches it, whatever it holds (paged_tma.cuh).
// Persistent: one CTA per SM walks its equal share of all (item, tile) pairs
// (paged_sched.cuh).  The pipeline runs through item borders: the next item's Q
// rows wait in shared memory, and move to tensor memory as soon as the current
// item's last S is done; the warpgroup without the last tile goes on to the next
// item while the other writes the output.
// Warp roles (384 threads): warp 0 K producer, warp 1 TMEM owner + S issuer, warp 2
// PV issuer, warp 3 V producer, warps 4..7 and 8..11 softmax / output
// (one row per thread), which take registers from the first four.  Every wait is
// bounded; after the first that runs out the softmax warps go on without data, the
// others stop, and MSA_FLAG_TIMEOUT is raised.
#include "common.cuh"
#include "internal.h"
#include "paged_sched.cuh"
#include "paged_tma.cuh"
#include "sm100.cuh"
#include "tma_host.h"

namespace msa {
namespace {

using namespace sm100;
using namespace paged;

constexpr int kRows = 128;     // MMA M: query rows per block
constexpr int kThreads = 384;  // K producer, S issuer, PV issuer, V producer, 2 x 4 softmax warps
constexpr int kSoftRegs = 208, kOtherRegs = 88;  // 256 x 208 + 128 x 88 = 384 x 168, the launch's registers
constexpr int kItemCost = 4, kSlack = 8;  // see Split
constexpr uint32_t kWaitPolls = 1u << 24;
constexpr float kRescaleLog2 = 8.0f;  // move the running max only when it grows by more than this

using Walk = WalkT<false>;

struct PreParams {
  PagedBatch p;
  const __nv_bfloat16* Q;
  int64_t q_ts;
  const int32_t* seg_row;
  const uint8_t* seg_cnt;
  int Hq, G, TB;
  PageMap pm;
  __nv_bfloat16* O;
  float* lse;
  Mark* marks;
  float* slots;
  float scale_log2;  // softmax scale * log2(e)
};

template <int DH>
struct Layout {
  static constexpr int kKV = 3;                // stages of the K ring and of the V ring
  static constexpr int kQ = kRows * DH * 2;    // the next item's query rows on their way to tensor memory
  static constexpr int kK = Tile<DH>::kBytes;  // one K (or V) tile
  static constexpr int kBars = 31;  // and tensor memory's address, the stop flag, the odd flag
  static constexpr int kRowState = kRows * 4 + kRows * 8;  // O's references; one warpgroup's (reference, sum)
  static constexpr int kSmem = 1024 + kQ + 2 * kKV * kK + 8 * kBars + kRowState + (int)sizeof(Start);
  static constexpr uint32_t kTmemCols = 512;   // S0, S1 (128 each), O (DH), P (64), Q (DH / 2)
  static_assert(2 * kKeys + DH + kKeys / 2 + DH / 2 <= (int)kTmemCols, "tensor memory columns");
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 bytes from global to shared memory without passing registers (zeros if !have).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(have ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// max of three (exact, like any max; it leaves NaN out, which then reaches the row by its weight)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefill_kernel(const __grid_constant__ TileMaps maps, PreParams a) {
  using L = Layout<DH>;
  constexpr int kKV = L::kKV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* Ks = smem;                // [kKV] K tiles
  uint8_t* Vs = Ks + kKV * L::kK;    // [kKV] V tiles
  uint8_t* Qs = Vs + kKV * L::kK;
  uint64_t* bars = reinterpret_cast<uint64_t*>(Qs + L::kQ);
  uint64_t* k_full = bars;                 // [kKV] K of a tile landed
  uint64_t* k_empty = k_full + kKV;        // [kKV] its S is done
  uint64_t* v_full = k_empty + kKV;        // [kKV]
  uint64_t* v_empty = v_full + kKV;        // [kKV] its PV is done
  uint64_t* s_full = v_empty + kKV;        // [2] S done -> softmax
  uint64_t* s_free = s_full + 2;           // [2] S read into registers
  uint64_t* p_full = s_free + 2;           // P in tensor memory -> PV
  uint64_t* p_free = p_full + 1;           // [2] PV of an even / odd tile done (O up to date, P free)
  uint64_t* q_tmem = p_free + 2;           // an item's Q is in tensor memory
  uint64_t* o_read = q_tmem + 1;           // an item's O and sums have been read
  uint64_t* l_ready = o_read + 1;          // [4 warps] the sums of the warpgroup without the last tile
  uint64_t* drain_s = l_ready + 4;
  uint64_t* drain_pv = drain_s + 1;
  static_assert(4 * kKV + 4 + 3 + 8 <= L::kBars - 2, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::kBars - 2);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* odd_s = abort_s + 1;  // values were left out of a product (drop_not_finite)
  float* m_s = reinterpret_cast<float*>(bars + L::kBars);     // [kRows] O's references, log2 domain
  float2* ml_s = reinterpret_cast<float2*>(m_s + kRows);      // [kRows] (reference, sum)
  Start* start = reinterpret_cast<Start*>(ml_s + kRows);

  const PagedBatch& p = a.p;
  const int TB = a.TB;
  const Split sp{TB, kItemCost, kSlack};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKV; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
      mbar_init(&p_free[i], 1);
    }
    mbar_init(p_full, 128);
    mbar_init(q_tmem, 128);
    mbar_init(o_read, 128);
    for (int i = 0; i < 4; ++i) mbar_init(&l_ready[i], 32);
    mbar_init(drain_s, 1);
    mbar_init(drain_pv, 1);
    *abort_s = 0;
    *odd_s = 0;
    fence_mbar_init();
  }
  // a programmatic dependent: nothing an earlier kernel writes is read before this wait
  pdl_wait();
  find_start<false>(p, sp, blockIdx.x, gridDim.x, blockIdx.x == 0, start, reinterpret_cast<ScanScratch*>(m_s));
  if (threadIdx.x == 0) leave_mark(start, sp, blockIdx.x, a.marks + blockIdx.x);
  pdl_trigger();
  if (!start->any) {
    if (threadIdx.x == 0) say_odd(a.marks, gridDim.x, blockIdx.x, 0);
    return;
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S0, S1 (128 each), O (DH), P (64: bf16 pairs), Q as the S MMAs' A operand (DH / 2)
  const uint32_t tS0 = tmem, tO = tmem + 2 * kKeys, tP = tO + DH, tQ = tP + kKeys / 2;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_or_stop(bar, parity, kWaitPolls, abort_s); };

  if (warp < 4) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == 0 || warp == 3) {
      // -------------------------------------------------------------- K and V producers
      // Lane 0 waits and arms the barriers.  A tile is up to 16 boxes, one lane each: the
      // plan's segments of kSegRows bank rows, or the pages (parts of pages) that hold
      // cached tokens.  A lane's place in the block table is looked up one tile ahead.
      const bool isK = warp == 0;
      uint8_t* ring = isK ? Ks : Vs;
      uint64_t* full = isK ? k_full : v_full;
      uint64_t* empty = isK ? k_empty : v_empty;
      const CUtensorMap* pages = isK ? &maps.k : &maps.v;
      const CUtensorMap* bank = isK ? &maps.kbar : &maps.vbar;
      auto locate = [&](const Walk& w, int t) {
        return locate_box(p, a.pm, a.seg_row, w.b, w.s.nm, w.s.len, t, lane);
      };
      uint32_t it = 0;
      bool stop = false;
      for (Walk w(sp, start); w.more() && !stop; w.next(p, sp)) {
        Box x = locate(w, w.t0);
        for (int t = w.t0; t < w.t0 + w.n; ++t, ++it) {
          const uint32_t st = it % kKV;
          const bool mem = t < w.s.nm;
          const int rows = mem ? kSegRows : a.pm.box_rows;
          check_box(p, mem, &x);
          Box nx{false, 0, 0};
          if (t + 1 < w.t0 + w.n) nx = locate(w, t + 1);
          const int boxes = __popc(__ballot_sync(0xffffffffu, x.mine));
          int ok = 1;
          if (lane == 0) {
            ok = wait(&empty[st], ((it / kKV) & 1) ^ 1);
            if (ok) mbar_arrive_expect_tx(&full[st], (uint32_t)(boxes * rows * DH * 2));
          }
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            stop = true;
            break;
          }
          if (x.mine) load_box<DH>(ring + st * L::kK, pages, bank, a.pm, mem, x, w.g, lane, &full[st]);
          x = nx;
        }
      }
      // the copies in flight land before the CTA leaves its shared memory
      if (lane == 0) {
        for (uint32_t st = 0; st < (uint32_t)kKV && st < it; ++st)
          if (!mbar_wait(&full[st], ((it - 1 - st) / kKV) & 1, kWaitPolls)) *abort_s = 1;
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- S issuer
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16_f32(kRows, kKeys);
        // descriptors of the operand bases; a k-step adds its byte offset / 16 to
        // the 14-bit start-address field (shared addresses stay below 256 KB, so
        // the field never carries)
        const uint64_t dk0 = desc_k_sw128_sbo(smem_u32(Ks), Tile<DH>::kGroup);
        uint32_t g = 0, nseg = 0;
        bool ok = true;
        for (Walk w(sp, start); ok && w.more(); w.next(p, sp), ++nseg) {
          ok = wait(q_tmem, nseg & 1);
          for (int j = 0; ok && j < w.n; ++j, ++g) {
            const uint32_t ks = g % kKV;
            // S goes into buffer g & 1 once the softmax has read tile g - 2 from it
            if (!(ok = wait(&s_free[g & 1], ((g >> 1) & 1) ^ 1)) || !(ok = wait(&k_full[ks], (g / kKV) & 1))) break;
            tc_fence_after();
            const uint64_t dk = dk0 + (uint64_t)((ks * L::kK) >> 4);
#pragma unroll
            for (int k = 0; k < DH / 16; ++k) {
              // A = Q from TMEM (16 elements of bf16 per step are 8 columns), B = K from its tile
              const int box = k >> 2, kk = k & 3;
              mma_bf16_ts(tS0 + (g & 1) * kKeys, tQ + k * 8, dk + (uint64_t)((box * 1024 + kk * 32) >> 4), idS,
                          k > 0 ? 1u : 0u);
            }
            mma_commit(&s_full[g & 1]);
            mma_commit(&k_empty[ks]);
          }
        }
        mma_commit(drain_s);
        if (!mbar_wait(drain_s, 0, kWaitPolls)) *abort_s = 1;
      }
    } else {
      // -------------------------------------------------------------- PV issuer
      if (lane == 0) {
        constexpr uint32_t idO = idesc_bf16_f32(kRows, DH, /*b_mn_major=*/true);
        const uint64_t dv0 = desc_mn_sw128_sbo(smem_u32(Vs), 1024, Tile<DH>::kGroup);
        uint32_t g = 0, nseg = 0;
        bool ok = true;
        for (Walk w(sp, start); ok && w.more(); w.next(p, sp), ++nseg) {
          // the first PV of an item overwrites O once the last one has been read
          if (nseg > 0) ok = wait(o_read, (nseg - 1) & 1);
          for (int j = 0; ok && j < w.n; ++j, ++g) {
            const uint32_t vs = g % kKV;
            if (!(ok = wait(&v_full[vs], (g / kKV) & 1)) || !(ok = wait(p_full, g & 1))) break;
            tc_fence_after();
            const uint64_t dv = dv0 + (uint64_t)((vs * L::kK) >> 4);
            // A = P from TMEM: 16 keys of bf16 per step are 8 columns
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_bf16_ts(tO, tP + k * 8, dv + (uint64_t)((k * 2 * Tile<DH>::kGroup) >> 4), idO, (j > 0 || k > 0) ? 1u : 0u);
            mma_commit(&p_free[g & 1]);
            mma_commit(&v_empty[vs]);
          }
        }
        mma_commit(drain_pv);
        if (!mbar_wait(drain_pv, 0, kWaitPolls)) *abort_s = 1;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    setmaxnreg_inc<kSoftRegs>();
    const int wg = (warp >> 2) - 1;                   // takes the tiles with g & 1 == wg
    const int q = warp & 3;
    const int r = q * 32 + lane;                      // this thread's row (TMEM lane)
    const int tl = r / a.G, hh = r - tl * a.G;        // token of the block and head of the group
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    const float sl2 = a.scale_log2;
    // A wait that runs out stops the waiting, not the loops: a warp goes on (without data) to the
    // end of its share, so that no tcgen05 operation is split among its lanes.
    auto hold = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_test(bar, parity) && !*abort_s) mbar_wait_or_stop(bar, parity, kWaitPolls, abort_s);
      __syncwarp();
    };
    // This row of an item's queries (nullptr: it does not exist) goes to shared memory during the
    // item before and from there to tensor memory, as the S MMAs' A operand; both by the owner of
    // that item's last tile.  The 16-byte pieces are swizzled by the row so that a warp's accesses
    // spread over the banks.
    uint8_t* qrow = Qs + r * (DH * 2);
    auto row_of = [&](const Walk& w) -> const __nv_bfloat16* {
      const int t = w.i * TB + tl;
      return tl < TB && t < w.s.nq ? a.Q + (w.s.q0 + t) * a.q_ts + (w.g * a.G + hh) * DH : nullptr;
    };
    auto fetch_q = [&](const __nv_bfloat16* row) {
#pragma unroll
      for (int c = 0; c < DH / 8; ++c)
        cp_async16(qrow + ((c ^ (r & 7)) << 4), (row ? row : a.Q) + (row ? c * 8 : 0), row != nullptr);
    };
    auto place_q = [&]() {
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
    uint32_t g0 = 0, nseg = 0;  // tiles and items before this one
    for (Walk w(sp, start); w.more(); w.next(p, sp), ++nseg) {
      const int t = w.i * TB + tl, n = w.n;
      const bool rvalid = tl < TB && t < w.s.nq;
      if (nseg == 0 && wg == 0) {
        fetch_q(row_of(w));
        place_q();
      }
      // local keys [0, seen) are visible to this row (rows that do not exist follow the last one)
      const int seen = w.s.len - w.s.nq + (rvalid ? t : min(w.i * TB + TB, w.s.nq) - 1) + 1;
      // the owner of the item's last tile sees to the next item's Q
      const bool next_q = ((g0 + n - 1) & 1) == (uint32_t)wg && w.another(sp);
      const int first = w.s.len - w.s.nq + w.i * TB;  // position of the block's first token
      const int j0 = (int)((g0 ^ wg) & 1);
      float m = -INFINITY, l_run = 0.f;  // this warpgroup's reference maximum (a whole number) and row sum
      for (int j = j0; j < n; j += 2) {
        const uint32_t g = g0 + j;
        const int st = g & 1, tile = w.t0 + j;
        const bool mem = tile < w.s.nm;
        // a memory tile's segment counts (one byte per segment), loaded before the wait
        uint4 segc = make_uint4(0u, 0u, 0u, 0u);
        if (mem) segc = __ldg(reinterpret_cast<const uint4*>(a.seg_cnt + w.b * p.Smax + tile * kTileSegs));
        hold(&s_full[st], (g >> 1) & 1);
        tc_fence_after();
        if (next_q && j == j0) {
          // this item's S has begun, so its Q has left the shared memory
          Walk wn = w;
          wn.next(p, sp);
          fetch_q(row_of(wn));
        }
        if (next_q && j == n - 1) place_q();  // the item's last S is done: Q's columns are free
        float s[kKeys];
        tmem_ld128(tS0 + lane_off + st * kKeys, s);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(&s_free[st]);
        if (mem) {
          // key c of the tile is row c % kSegRows of segment c / kSegRows
          static_assert(kTileSegs == 16 && kSegRows == 8, "four segment counts per word");
          const uint32_t full8 = 0x08080808u;
          if (!(segc.x == full8 && segc.y == full8 && segc.z == full8 && segc.w == full8)) {
            const uint32_t cw[4] = {segc.x, segc.y, segc.z, segc.w};
#pragma unroll
            for (int c = 0; c < kKeys; ++c) {
              const uint32_t cnt = (cw[c >> 5] >> (((c >> 3) & 3) * 8)) & 0xffu;
              s[c] = (uint32_t)(c & 7) < cnt ? s[c] : -INFINITY;
            }
            const uint32_t vs = g % kKV;
            hold(&v_full[vs], (g / kKV) & 1);  // see below
            if ((uint32_t)(r & 7) >= ((q == 0 ? cw[0] : q == 1 ? cw[1] : q == 2 ? cw[2] : cw[3]) >> ((lane >> 3) * 8) & 0xffu))
              zero_row<DH>(Vs + vs * L::kK, r);
            fence_async_smem();
            __syncwarp();
          }
        } else {
          const int base = (tile - w.s.nm) * kKeys;
          const int lim = seen - base;
          if (__any_sync(0xffffffffu, lim < kKeys)) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c) s[c] = c < lim ? s[c] : -INFINITY;
          }
          // Rows of V that not every row of the block sees (tile_row).  The copy that filled the
          // stage has landed (S read K of the same tile, not V): this wait makes it visible here.
          if (base + kKeys - 1 > first) {
            const uint32_t vs = g % kKV;
            hold(&v_full[vs], (g / kKV) & 1);
            uint8_t* vt = Vs + vs * L::kK;
            const int key = base + r;
            if (key >= w.s.len) zero_row<DH>(vt, r);
            else if (key > first && row_not_finite<DH>(vt, r)) {
              *odd_s = 1;
              drop_not_finite<DH>(vt, r);
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
        // the reference moves only when a score passes it by 2^8, to the next whole number: every
        // later change of scale is then a power of two, exact in any type
        const float mt = mx * sl2;
        if (mt > m + kRescaleLog2) {
          const float up = ceilf(mt);
          l_run *= m == -INFINITY ? 0.f : fast_exp2(m - up);
          m = up;
        }
        const float nm = m == -INFINITY ? 0.f : -m;  // no key seen yet: 2^(-inf) below is 0
        // P in registers (a pair of keys per word); the scaled arguments and the row sums in packed
        // pairs (one f32x2 instruction for two keys).  All on the transcendental unit (1,024 cycles
        // of its time a tile): a share of the exponentials as polynomials on the FMA pipes gained
        // nothing (the 4096-token part over 32,096 keys 2.10 ms with 2 of 16 pairs, 2.29 with 8; without,
        // 1.9 to 2.2 from run to run; 23 requests with heads of 64 130 us with 1 pair, 119 without).
        const uint64_t sl2x2 = f2_pack(sl2, sl2), nmx2 = f2_pack(nm, nm);
        uint64_t lsa2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        uint32_t pw[kKeys / 2];
#pragma unroll
        for (int i = 0; i < kKeys / 2; ++i) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(s[2 * i], s[2 * i + 1]), sl2x2, nmx2), x0, x1);
          const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
          lsa2[i & 1] = f2_add(lsa2[i & 1], f2_pack(e0, e1));
          pw[i] = pack_bf16x2(e0, e1);
        }
        float lsa[4];
        f2_unpack(lsa2[0], lsa[0], lsa[1]);
        f2_unpack(lsa2[1], lsa[2], lsa[3]);
        l_run += (lsa[0] + lsa[1]) + (lsa[2] + lsa[3]);
        // P goes into tensor memory once the PV of the tile before has read its own.  (A barrier of
        // its own for even and odd tiles: with one, a warp two tiles ahead would take the phase
        // before the last for the one it waits for.)
        if (g > 0) {
          hold(&p_free[(g - 1) & 1], ((g - 1) >> 1) & 1);
        }
        tc_fence_after();
        // the reference that O has, as the owner of the tile before left it (before its arrival on
        // p_full, which the PV behind p_free waited for).  Tiles publish in order, so this is the
        // place where the two warpgroups' references meet.
        const float ms = j > 0 ? m_s[r] : -INFINITY;
        if (__any_sync(0xffffffffu, m != ms)) {
          float fo = 1.f, fp = 1.f;  // factors of O and of P
          if (m > ms) {
            if (ms != -INFINITY) fo = fast_exp2(ms - m);  // else no key so far: O is 0 (or not begun)
          } else if (m < ms) {
            fp = m == -INFINITY ? 0.f : fast_exp2(m - ms);  // -inf: P is 0 already
            l_run *= fp;
            m = ms;
          }
          m_s[r] = m;
          if (__any_sync(0xffffffffu, fo != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < DH; c += 16) {
              float o[16];
              tmem_ld16(tO + lane_off + c, o);
              tmem_ld_wait();
              uint32_t wv[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) wv[i] = __float_as_uint(o[i] * fo);
              tmem_st16(tO + lane_off + c, wv);
            }
          }
          if (__any_sync(0xffffffffu, fp != 1.f)) {
            const __nv_bfloat162 f2 = __float2bfloat162_rn(fp);
#pragma unroll
            for (int i = 0; i < kKeys / 2; ++i) {
              __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&pw[i]);
              v = __hmul2(v, f2);
              pw[i] = *reinterpret_cast<uint32_t*>(&v);
            }
          }
        }
        if (j == 0) m_s[r] = m;
#pragma unroll
        for (int c = 0; c < kKeys / 2; c += 16) tmem_st16(tP + lane_off + c, *reinterpret_cast<const uint32_t(*)[16]>(&pw[c]));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full);
      }
      // The item's end belongs to the owner of its last tile; the other warpgroup leaves its sum and
      // goes on to the next item, whose first tile is its own.
      const uint32_t gl = g0 + n - 1;
      g0 += n;
      if ((int)(gl & 1) != wg) {
        if (nseg > 0) hold(o_read, (nseg - 1) & 1);  // the last item's sum has been read
        ml_s[r] = make_float2(m, l_run);
        mbar_arrive(&l_ready[q]);
        continue;
      }
      hold(&l_ready[q], nseg & 1);
      const float2 ml = ml_s[r];
      // this warpgroup stored the last P, so its reference is O's, and no smaller than the other's
      const float l = l_run + (ml.y == 0.f ? 0.f : ml.y * fast_exp2(ml.x - m));
      hold(&p_free[gl & 1], (gl >> 1) & 1);
      tc_fence_after();
      float o[DH];
#pragma unroll
      for (int c = 0; c < DH; c += 16) tmem_ld16(tO + lane_off + c, *reinterpret_cast<float(*)[16]>(&o[c]));
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(o_read);
      // O / l, lse = (m + log2 l) ln 2; the sum is 0 only for a row that saw no key: O = 0, lse = -inf
      const bool none = l == 0.f, whole = w.whole();
      const float inv = none ? 0.f : 1.f / l;
      const int64_t row = w.s.q0 + t;
      const int h = w.g * a.G + hh;
      if (rvalid) {
        if (whole) {
          __nv_bfloat16* orow = a.O + (row * a.Hq + h) * DH;
#pragma unroll
          for (int c = 0; c < DH; c += 8) {
            float f[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = none ? 0.f : o[c + x] * inv;
            *reinterpret_cast<uint4*>(orow + c) = pack(f);
          }
          if (a.lse) a.lse[(int64_t)h * p.N + row] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          float* slot = a.slots + slot_of(blockIdx.x, w.f, start->f0) * slot_floats(kRows, DH);
#pragma unroll
          for (int c = 0; c < DH; c += 4)
            *reinterpret_cast<float4*>(slot + ((c >> 2) * kRows + r) * 4) =
                make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
          *reinterpret_cast<float2*>(slot + kRows * DH + 2 * r) = make_float2(m, l);
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
  if (threadIdx.x == 0) {
    if (*abort_s) raise_flag(p.err_flag, MSA_FLAG_TIMEOUT);
    say_odd(a.marks, gridDim.x, blockIdx.x, *odd_s);
  }
}

// setmaxnreg.inc waits for registers that the launch must have brought: were the kernel ever compiled
// to fewer than the split needs, it would wait forever.  Looked up once per kernel.
template <int DH>
cudaError_t registers_cover_split() {
  static const bool enough = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, paged_prefill_kernel<DH>) == cudaSuccess &&
           at.numRegs * kThreads >= 256 * kSoftRegs + 128 * kOtherRegs;
  }();
  return enough ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int DH>
cudaError_t prefill_t(const PagedAttnArgs& a, cudaStream_t s) {
  using L = Layout<DH>;
  TileMaps maps;
  PreParams d;
  if (!make_tile_maps<DH>(a, &maps, &d.pm)) return cudaErrorInvalidValue;
  const int grid = sm_count(), G = a.Hq / a.p.Hkv;
  d.p = a.p;
  d.Q = reinterpret_cast<const __nv_bfloat16*>(a.Q);
  d.q_ts = a.q_ts;
  d.seg_row = a.seg_row;
  d.seg_cnt = a.seg_cnt;
  d.Hq = a.Hq;
  d.G = G;
  d.TB = kRows / G;
  d.O = reinterpret_cast<__nv_bfloat16*>(a.O);
  d.lse = a.lse;
  d.marks = reinterpret_cast<Mark*>(a.part);
  d.slots = reinterpret_cast<float*>(reinterpret_cast<char*>(a.part) + marks_bytes(grid));
  d.scale_log2 = a.scale * 1.4426950408889634f;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = registers_cover_split<DH>();
  if (e != cudaSuccess) return e;
  e = allow_smem(paged_prefill_kernel<DH>, L::kSmem, done);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_pdl(paged_prefill_kernel<DH>, dim3((unsigned)grid), dim3(kThreads), (size_t)L::kSmem, s, maps, d);
  if (e != cudaSuccess) return e;
  return launch_merge(MSA_BF16, true, MergeArgs{a, d.marks, d.slots, grid, kRows, d.TB, 1.f}, s);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedAttnArgs& a, cudaStream_t s) {
  return a.d == 64 ? prefill_t<64>(a, s) : prefill_t<128>(a, s);
}

}  // namespace msa
