// Attention over a paged cache for a few query rows per KV head (paged_attn.cu):
// the R = G * max_q <= 16 rows of one sequence and KV head against
// [selected memory rows ++ cached tokens], bf16.
//
// Every K and V row is read once and used for at most 16 dot products, so the
// kernel is shaped for HBM bandwidth; the contractions run on the tensor cores
// with the 128 keys of a tile as the MMA's M (one TMEM lane each) and the query
// rows as its N = 16:
//   S^T[key, row] = K_tile (TMA, 128-byte swizzle) x Q^T
//   O^T[d, row]  += V_tile^T (MN-major, straight from the tile) x P^T
// S^T is double-buffered in TMEM and P^T in shared memory; the MMA thread polls
// its barriers without blocking and issues each tile's S and P V as soon as
// their inputs are ready.  A softmax thread owns one TMEM lane: a key of S^T, a
// dimension of O^T.  The running maximum moves (and O^T is rescaled) only when
// it grows by more than 2^8; weights are rounded to bf16 for the P V product
// (2^-9 each, averaged over the keys), their sum is kept from the fp32 values.
// A tile's K and V arrive as one box per page (128 rows from pages of 128 and
// more), one lane each, straight from the block table's pages (paged_tma.cuh); rows
// past the sequence's end are never visible, and their V rows are zeroed in shared
// memory before the product.
// The split over CTAs is that of paged_sched.cuh: one CTA per SM, equal shares.
// Warp roles (192 threads): warp 0 TMA producer, warp 1 TMEM owner + MMA
// issuer, warps 2..5 softmax / output.  Every wait is bounded; after the first
// expired wait the CTA runs its loops out without data and raises
// MSA_FLAG_TIMEOUT.
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

constexpr int kMaxRows = 16;            // R = G * Tq (the MMA's N, padded to 16)
constexpr int kThreads = 192;
constexpr int kItemCost = 2, kSlack = 0;  // see Split
constexpr uint32_t kWaitPolls = 1u << 24;
constexpr uint32_t kSpinLimit = 1u << 28;  // non-blocking polls of the MMA issuer without progress
constexpr float kRescaleLog2 = 8.0f;

using Walk = WalkT<true>;  // one block of tokens per sequence

struct DecParams {
  PagedBatch p;
  const __nv_bfloat16* Q;
  int64_t q_ts;
  const int32_t* seg_row;
  const uint8_t* seg_cnt;
  int Hq, G, R;      // R = G * max_q
  PageMap pm;
  __nv_bfloat16* O;
  float* lse;
  Mark* marks;
  float* slots;
  float scale_log2;
};

template <int DH>
struct DLayout {
  static constexpr int kStages = DH == 64 ? 6 : 3;    // of K and V: 192 KB in flight either way
  static constexpr int kTile = Tile<DH>::kBytes;     // one K (or V) tile
  static constexpr int kStage = 2 * kTile;
  static constexpr int kQ = kMaxRows * DH * 2;        // Q rows, K-major, 128-byte swizzle (two buffers)
  static constexpr int kP = kMaxRows * kKeys * 2;     // P^T rows (query rows x keys); two buffers
  static constexpr int kRed = 2 * kMaxRows * 4 * 4;    // [maxima, sums][rows][4 warps]
  static constexpr int kBars = 2 * kStages + 13;       // and tensor memory's address, the stop flag, the odd flag
  static constexpr int kSmem = 1024 + kStages * kStage + 2 * kQ + 2 * kP + kRed + 8 * kBars + (int)sizeof(Start);
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static constexpr uint32_t kTmemCols = 64;           // S0, S1, O (16 columns each)
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Whether v holds in any of the 128 softmax threads (a barrier among them).
__device__ __forceinline__ bool any_softmax(bool v) {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n bar.red.popc.u32 %0, 1, 128, p;\n}"
               : "=r"(r)
               : "r"((uint32_t)v)
               : "memory");
  return r != 0;
}
// Maximum of v over the 32 lanes, in every lane (one instruction on sm_100a).
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Byte offset of element (row, col) in a K-major, 128-byte-swizzled tile whose
// rows hold 64 elements per box and `rows` rows per box.
__device__ __forceinline__ int sw128_off(int row, int col, int rows) {
  const int box = col >> 6, c = col & 63;
  return box * (rows * 128) + row * 128 + ((((c >> 3) ^ (row & 7))) << 4) + (c & 7) * 2;
}

// kR >= R is the number of query rows the softmax threads handle (4, 8 or 16);
// the MMA's N stays 16 and the columns past kR are never read.
template <int DH, int kR>
__global__ void __launch_bounds__(kThreads, 1)
paged_decode_kernel(const __grid_constant__ TileMaps maps, DecParams a) {
  using L = DLayout<DH>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* Qs = ring + kStages * L::kStage;  // two buffers, alternating by segment
  uint8_t* Ps = Qs + 2 * L::kQ;
  float* red_s = reinterpret_cast<float*>(Ps + 2 * L::kP);  // [2][16 rows][4 warps]
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red_s) + L::kRed);
  uint64_t* kv_full = bars;                  // [kStages]
  uint64_t* kv_empty = kv_full + kStages;    // [kStages]
  uint64_t* s_full = kv_empty + kStages;     // [2]
  uint64_t* s_free = s_full + 2;             // [2]
  uint64_t* q_ready = s_free + 2;
  uint64_t* p_full = q_ready + 1;            // [2] per P buffer
  uint64_t* o_done = p_full + 2;             // [2] per P buffer: its P V has completed
  uint64_t* drain = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* odd_s = abort_s + 1;  // values were left out of a product (drop_not_finite)
  Start* start = reinterpret_cast<Start*>(bars + L::kBars);

  const PagedBatch& p = a.p;
  const Split sp{p.max_q, kItemCost, kSlack};  // one block of tokens per sequence
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 128);
    }
    mbar_init(q_ready, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(drain, 1);
    *abort_s = 0;
    *odd_s = 0;
    fence_mbar_init();
  }
  // a programmatic dependent: nothing an earlier kernel writes is read before this wait
  pdl_wait();
  find_start<true>(p, sp, blockIdx.x, gridDim.x, blockIdx.x == 0, start, reinterpret_cast<ScanScratch*>(red_s));
  if (tid == 0) leave_mark(start, sp, blockIdx.x, a.marks + blockIdx.x);
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
  const uint32_t tS = tmem, tO = tmem + 32;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    // Lane 0 waits and arms the barriers.  A tile is up to 16 boxes of K and of V, one lane
    // each: the plan's segments of kSegRows bank rows, or the pages (parts of pages) that hold
    // cached tokens.  A lane's place in the block table is looked up one tile ahead.
    uint32_t it = 0;
    bool stop = false;
    auto locate = [&](const Walk& w, int t) {
      return locate_box(p, a.pm, a.seg_row, w.b, w.s.nm, w.s.len, t, lane);
    };
    for (Walk w(sp, start); w.more() && !stop; w.next(p, sp)) {
      Box x = locate(w, w.t0);
      for (int t = w.t0; t < w.t0 + w.n; ++t, ++it) {
        const uint32_t st = it % kStages;
        const bool mem = t < w.s.nm;
        const int rows = mem ? kSegRows : a.pm.box_rows;
        check_box(p, mem, &x);
        Box nx{false, 0, 0};
        if (t + 1 < w.t0 + w.n) nx = locate(w, t + 1);
        const int boxes = __popc(__ballot_sync(0xffffffffu, x.mine));
        int ok = 1;
        if (lane == 0) {
          ok = mbar_wait_or_stop(&kv_empty[st], ((it / kStages) & 1) ^ 1, kWaitPolls, abort_s);
          if (ok) mbar_arrive_expect_tx(&kv_full[st], (uint32_t)(boxes * rows * DH * 2 * 2));
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          stop = true;
          break;
        }
        if (x.mine) {
          uint8_t* Kd = ring + st * L::kStage;
          load_box<DH>(Kd, &maps.k, &maps.kbar, a.pm, mem, x, w.g, lane, &kv_full[st]);
          load_box<DH>(Kd + L::kTile, &maps.v, &maps.vbar, a.pm, mem, x, w.g, lane, &kv_full[st]);
        }
        x = nx;
      }
    }
    if (lane == 0) {
      // the copies in flight land before the CTA leaves its shared memory
      const uint32_t fills = it;
      for (uint32_t st = 0; st < (uint32_t)kStages && st < fills; ++st) {
        const uint32_t last = (fills - 1 - st) / kStages * kStages + st;
        if (!mbar_wait(&kv_full[st], (last / kStages) & 1, kWaitPolls)) *abort_s = 1;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(kKeys, kMaxRows);                              // K x Q^T
      constexpr uint32_t idO = idesc_bf16_f32(DH, kMaxRows, /*b_mn=*/false, /*a_mn=*/true);  // V^T x P^T
      const uint32_t p0 = smem_u32(Ps);
      uint32_t it = 0, nseg = 0;  // it: tiles (K/V stages, S and P buffers); nseg: segments
      for (Walk w(sp, start); w.more() && !*abort_s; w.next(p, sp), ++nseg) {
        const int T = w.n;
        const uint32_t q0 = smem_u32(Qs + (nseg & 1) * L::kQ);
        if (!mbar_wait_or_stop(q_ready, nseg & 1, kWaitPolls, abort_s)) break;
        // Issue S = K Q^T of a tile as soon as its K/V stage and an S buffer are
        // ready, and O += V^T P^T of a tile as soon as its P is: one thread polls
        // both (test_wait does not block), so a tile's P V is never held back by
        // the next tile's copy.
        int nS = 0, nP = 0;
        uint32_t spins = 0;
        while (nP < T && !*abort_s) {
          bool prog = false;
          if (nS < T) {
            const uint32_t g = it + nS, st = g % kStages, round = g / kStages, sb = g & 1;
            if (mbar_test(&kv_full[st], round & 1) && mbar_test(&s_free[sb], ((g >> 1) & 1) ^ 1)) {
              tc_fence_after();
              const uint32_t k0 = smem_u32(ring + st * L::kStage);
#pragma unroll
              for (int k = 0; k < DH / 16; ++k) {
                const int box = k >> 2, kk = k & 3;
                mma_bf16_ss(tS + sb * 16, desc_k_sw128_sbo(k0 + box * 1024 + kk * 32, Tile<DH>::kGroup),
                            desc_k_sw128(q0 + box * (kMaxRows * 128) + kk * 32), idS, k > 0 ? 1u : 0u);
              }
              mma_commit(&s_full[sb]);
              ++nS;
              prog = true;
            }
          }
          if (nP < nS) {
            const uint32_t g = it + nP, st = g % kStages, pb = g & 1;
            if (mbar_test(&p_full[pb], (g >> 1) & 1)) {
              tc_fence_after();
              const uint32_t v0 = smem_u32(ring + st * L::kStage + L::kTile);
              const uint32_t pp = p0 + pb * L::kP;
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k) {
                const int box = k >> 2, kk = k & 3;
                mma_bf16_ss(tO, desc_mn_sw128_sbo(v0 + k * 2 * Tile<DH>::kGroup, 1024, Tile<DH>::kGroup),
                            desc_k_sw128(pp + box * (kMaxRows * 128) + kk * 32), idO, (nP > 0 || k > 0) ? 1u : 0u);
              }
              mma_commit(&o_done[pb]);
              mma_commit(&kv_empty[st]);
              ++nP;
              prog = true;
            }
          }
          if (prog) spins = 0;
          else if (++spins > kSpinLimit) *abort_s = 1;
        }
        it += T;
      }
      mma_commit(drain);
      if (!mbar_wait(drain, 0, kWaitPolls)) *abort_s = 1;
    }
  } else {
    // ---------------------------------------------------------------- softmax / output
    const int q = warp & 3;
    const int r_lane = q * 32 + lane;               // this thread's TMEM lane: key of S^T
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    // this thread's dimension of O^T: a product of M = 64 leaves its rows in the first 16 lanes of
    // each warp's 32
    const int dim = DH == 128 ? r_lane : (lane < 16 ? q * 16 + lane : -1);
    const int et = tid - 64;                        // 0..127
    // Q rows of a segment into a swizzled K-major buffer: 16-byte piece i of 16 rows is row
    // r = i / (DH / 8) (token r / G, head g * G + r % G); rows of tokens the sequence does not have
    // are zeros.
    constexpr int kPieces = DH / 8, kEach = kMaxRows * kPieces / 128;
    auto load_q = [&](const Walk& w, uint4 (&v)[kEach]) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int i = et + 128 * k, r = i / kPieces, c8 = (i % kPieces) * 8;
        v[k] = make_uint4(0, 0, 0, 0);
        const int t = r / a.G, h = w.g * a.G + r % a.G;
        if (t < w.s.nq) v[k] = __ldg(reinterpret_cast<const uint4*>(a.Q + (w.s.q0 + t) * a.q_ts + h * DH + c8));
      }
    };
    auto store_q = [&](uint8_t* buf, const uint4 (&v)[kEach]) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int i = et + 128 * k, r = i / kPieces, c8 = (i % kPieces) * 8;
        *reinterpret_cast<uint4*>(buf + sw128_off(r, c8, kMaxRows)) = v[k];
      }
    };
    Walk w(sp, start);
    {
      uint4 v[kEach];
      load_q(w, v);
      store_q(Qs, v);
    }
    fence_async_smem();
    tc_fence_before();
    mbar_arrive(q_ready);

    // A wait that runs out stops the waiting, not the loops: the four warps meet at named
    // barriers, so each goes on (without data) to the end of the share.
    auto hold = [&](uint64_t* bar, uint32_t parity) {
      if (!*abort_s) mbar_wait_or_stop(bar, parity, kWaitPolls, abort_s);
      __syncwarp();
    };
    uint32_t it = 0, nseg = 0;
    while (w.more()) {
      // the next segment's Q rows, loaded now and stored after this segment's first tile
      Walk wn = w;
      wn.next(p, sp);
      const bool more = wn.more();
      uint4 qn[kEach];
      if (more) load_q(wn, qn);
      const int T = w.n, rows = w.s.nq * a.G;  // rows < kR that exist
      const int pos0 = w.s.len - w.s.nq;       // position of the first new token
      float m_run[kR], l_run[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        m_run[r] = -INFINITY;
        l_run[r] = 0.f;
      }
      for (int j = 0; j < T; ++j) {
        const int t = w.t0 + j;
        const uint32_t g = it + j, sb = g & 1;
        const bool mem = t < w.s.nm;
        // a memory tile: this thread's key is row (r_lane % kSegRows) of segment 16 t + r_lane / kSegRows
        int seg_n = 0;
        if (mem) seg_n = __ldg(a.seg_cnt + w.b * p.Smax + t * kTileSegs + (r_lane >> 3));
        hold(&s_full[sb], (g >> 1) & 1);
        tc_fence_after();
        float sc[kR];
        tmem_ld_cols<kR>(tS + sb * 16 + lane_off, sc);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(&s_free[sb]);
        // mask; scale into the log2 domain
        const int key = (t - w.s.nm) * kKeys + r_lane;  // cache position of a local key
        // rows from `low` on see the key: token r / G >= key - pos0 means r >= (key - pos0) G
        const int low = mem ? ((r_lane & (kSegRows - 1)) < seg_n ? 0 : kR)
                            : (key < pos0 ? 0 : min(key - pos0, kR) * a.G);
#pragma unroll
        for (int r = 0; r < kR; ++r) sc[r] = r >= low && r < rows ? sc[r] * a.scale_log2 : -INFINITY;
        // Rows of V that not every query row sees (paged_tma.cuh).  The copy that filled the stage
        // has landed (S read the same barrier's K); this wait makes it visible here.
        if (mem ? __any_sync(0xffffffffu, low > 0) : key - r_lane + kKeys - 1 > pos0) {
          hold(&kv_full[g % kStages], (g / kStages) & 1);
          uint8_t* vt = ring + (g % kStages) * L::kStage + L::kTile;
          if (mem ? low > 0 : key >= w.s.len) zero_row<DH>(vt, r_lane);
          else if (!mem && key > pos0 && row_not_finite<DH>(vt, r_lane)) {
            drop_not_finite<DH>(vt, r_lane);
            *odd_s = 1;
          }
          __syncwarp();
        }
        // The maximum moves only where a score passes it by 2^8 (always in the first tile with a
        // visible key): one vote over the 128 keys, and the column maxima (a warp reduction per
        // column, then the four warps' through shared memory) only if it says so.
        bool over = false;
#pragma unroll
        for (int r = 0; r < kR; ++r) over |= sc[r] > m_run[r] + kRescaleLog2;
        const bool grow = any_softmax(over);
        float corr[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) corr[r] = 1.f;
        if (grow) {
          float mine = -INFINITY;  // lane r < kR keeps this warp's maximum of column r
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const float v = warp_max(sc[r]);
            mine = lane == r ? v : mine;
          }
          if (lane < kR) red_s[lane * 4 + q] = mine;
          bar_softmax();
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const float4 wv = *reinterpret_cast<const float4*>(red_s + r * 4);
            const float mt = fmaxf(fmaxf(wv.x, wv.y), fmaxf(wv.z, wv.w));
            if (mt > m_run[r] + kRescaleLog2) {  // same decision in every thread
              corr[r] = m_run[r] == -INFINITY ? 0.f : fast_exp2(m_run[r] - mt);
              m_run[r] = mt;
            }
          }
        }
        float pr[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          pr[r] = sc[r] == -INFINITY ? 0.f : fast_exp2(sc[r] - m_run[r]);
          l_run[r] = l_run[r] * corr[r] + pr[r];
        }
        // P buffer g & 1 was last read by the P V of tile g - 2; O is rescaled
        // only after the P V of tile g - 1
        if (g >= 2) hold(&o_done[g & 1], ((g - 2) >> 1) & 1);
        if (j > 0 && grow) hold(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
        if (j > 0 && grow) {
          tc_fence_after();
          float o[kR];
          tmem_ld_cols<kR>(tO + lane_off, o);
          tmem_ld_wait();
          uint32_t wr[kR];
#pragma unroll
          for (int r = 0; r < kR; ++r) wr[r] = __float_as_uint(o[r] * corr[r]);
          tmem_st_cols<kR>(tO + lane_off, wr);
          tmem_st_wait();
        }
#pragma unroll
        for (int r = 0; r < kR; ++r)
          *reinterpret_cast<__nv_bfloat16*>(Ps + (g & 1) * L::kP + sw128_off(r, r_lane, kMaxRows)) =
              __float2bfloat16_rn(pr[r]);
        // The other Q buffer was last read by the previous segment's S MMAs,
        // all complete before that segment's last P V.
        if (j == 0 && more) store_q(Qs + ((nseg + 1) & 1) * L::kQ, qn);
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&p_full[g & 1]);
        if (j == 0 && more) mbar_arrive(q_ready);
      }
      // segment result: O^T[d = r_lane][row], the row maxima and the summed weights
      {
        const uint32_t g = it + T - 1;  // the segment's last tile
        hold(&o_done[g & 1], (g >> 1) & 1);
      }
      tc_fence_after();
      float o[kR];
      tmem_ld_cols<kR>(tO + lane_off, o);
      tmem_ld_wait();
      float* red_l = red_s + kMaxRows * 4;  // the segment's row sums, apart from the maxima
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float v = l_run[r];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) red_l[r * 4 + q] = v;
      }
      bar_softmax();
      const bool whole = w.whole();
      float* slot = a.slots + slot_of(blockIdx.x, w.f, start->f0) * slot_floats(a.R, DH);
      int t = 0, hh = 0;  // row r's token and head of the group
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r >= rows) break;
        const float4 lv = *reinterpret_cast<const float4*>(red_l + r * 4);
        const float l = (lv.x + lv.y) + (lv.z + lv.w);
        if (whole) {
          // a sum of 0: no key was visible
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int h = w.g * a.G + hh;
          if (dim >= 0) a.O[((w.s.q0 + t) * a.Hq + h) * DH + dim] = __float2bfloat16_rn(l == 0.f ? 0.f : o[r] * inv);
          if (a.lse && et == 0)
            a.lse[(int64_t)h * p.N + w.s.q0 + t] =
                l == 0.f ? -INFINITY : (m_run[r] + log2f(l)) * 0.69314718055994531f;
        } else {
          if (dim >= 0) slot[r * DH + dim] = o[r];
          if (et == 0) *reinterpret_cast<float2*>(slot + a.R * DH + 2 * r) = make_float2(m_run[r], l);
        }
        if (++hh == a.G) {
          hh = 0;
          ++t;
        }
      }
      bar_softmax();
      tc_fence_before();
      it += T;
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
  if (tid == 0) {
    if (*abort_s) raise_flag(p.err_flag, MSA_FLAG_TIMEOUT);
    say_odd(a.marks, gridDim.x, blockIdx.x, *odd_s);
  }
}

template <int DH>
cudaError_t decode_t(const PagedAttnArgs& a, cudaStream_t s) {
  using L = DLayout<DH>;
  TileMaps maps;
  DecParams d;
  if (!make_tile_maps<DH>(a, &maps, &d.pm)) return cudaErrorInvalidValue;
  const int grid = sm_count(), G = a.Hq / a.p.Hkv;
  d.p = a.p;
  d.Q = reinterpret_cast<const __nv_bfloat16*>(a.Q);
  d.q_ts = a.q_ts;
  d.seg_row = a.seg_row;
  d.seg_cnt = a.seg_cnt;
  d.Hq = a.Hq;
  d.G = G;
  d.R = G * a.p.max_q;
  d.O = reinterpret_cast<__nv_bfloat16*>(a.O);
  d.lse = a.lse;
  d.marks = reinterpret_cast<Mark*>(a.part);
  d.slots = reinterpret_cast<float*>(reinterpret_cast<char*>(a.part) + marks_bytes(grid));
  d.scale_log2 = a.scale * 1.4426950408889634f;
  auto kern = d.R <= 4   ? paged_decode_kernel<DH, 4>
              : d.R <= 8 ? paged_decode_kernel<DH, 8>
                         : paged_decode_kernel<DH, 16>;
  static std::atomic<uint64_t> done[3];
  cudaError_t e = allow_smem(kern, L::kSmem, done[d.R <= 4 ? 0 : (d.R <= 8 ? 1 : 2)]);
  if (e != cudaSuccess) return e;
  count_launch();
  e = launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), (size_t)L::kSmem, s, maps, d);
  if (e != cudaSuccess) return e;
  return launch_merge(MSA_BF16, false, MergeArgs{a, d.marks, d.slots, grid, d.R, a.p.max_q, 1.f}, s);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedAttnArgs& a, cudaStream_t s) {
  return a.d == 64 ? decode_t<64>(a, s) : decode_t<128>(a, s);
}

}  // namespace msa
