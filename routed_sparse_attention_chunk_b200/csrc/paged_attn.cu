// Attention of new tokens over [selected memory rows ++ cached tokens], the cached
// keys and values in pages: O = softmax(scale q K^T) V over the rows of the
// documents selected for the token's sequence and the cached positions up to the
// token's own.  This file holds the dispatcher, the kernel that merges items cut
// by the work split (paged_sched.cuh) and the fp32 kernel; bf16 runs on the
// tensor cores (paged_decode.cu, paged_prefill.cu).
//
// The fp32 kernels are a single pass over the keys with running row maxima and sums:
// blocks of 32 or 64 query rows over tiles of keys in shared memory
// (paged_f32_kernel), and up to d / 16 rows per KV head with the keys streamed through
// registers (paged_f32_rows_kernel).  All arithmetic is fp32 FMA; scores are compared and subtracted unscaled, so the
// exponent's argument (s - max) * scale carries only its own rounding.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged_sched.cuh"
#include "sm100.cuh"
#include "tma_host.h"

namespace msa {

cudaError_t launch_paged_decode(const PagedAttnArgs& a, cudaStream_t s);
cudaError_t launch_paged_prefill(const PagedAttnArgs& a, cudaStream_t s);

namespace paged {
namespace {

using namespace sm100;

constexpr int kF32Threads = 256;
constexpr int kF32ItemCost = 1, kF32Slack = 2;  // see Split
constexpr int kF32FewRows = 8;  // rows of a partial result of paged_f32_rows_kernel

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(have ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The block kernel.  RG groups of 16 query rows times 8 / RG parts of a tile's 128 keys, a warp
// each: a thread keeps 4 rows (ty + 4 j) x 4 or 8 keys (tx + 8 i) of the scores and 4 x DH / 8
// values of the output.  Every warp has running maxima and sums of its own over its keys, merged at
// the segment's end, so its weights never leave it.  K of the next tile is copied while P V runs, V
// while Q K^T does.  1,050 tokens x 32 heads of 128 over 2,200 keys take 849 us, 45 TFLOP/s: shared
// memory's way into the registers (128 bytes a clock for 128 FMA; 12 loads of 16 bytes per 128 FMA of
// a thread in Q K^T, 20 per 256 in P V) is 61 % busy, the FMA pipe 50 %, the rest latencies of two
// warps per scheduler.  Scores of 4 x 4 at a time took 887 us, one value an instruction instead of
// pairs (f32x2) and a question about the key at every weight 1,231, blocks of 64 rows x 32 keys with
// 4 x 2 scores a thread 1,127.
template <int DH, int RG>
struct F32Smem {
  static constexpr int RB = 16 * RG;              // query rows
  static constexpr int kParts = 8 / RG;           // warps that share a tile's keys
  static constexpr int kPerWarp = kKeys / kParts;
  static constexpr int kCtas = DH == 64 && RG == 2 ? 2 : 1;  // per SM, by registers and shared memory
  float Q[RB][DH + 4];
  float K[kKeys][DH + 4];  // at a segment's end the outputs of the parts
  float V[kKeys][DH + 4];
  float P[8][16][kPerWarp + 8];
  float2 ml[kParts][RB];   // row maxima and sums of the parts
  int64_t row[2][kKeys];   // element offset of each key of this tile and the next in its tensor, -1: no key,
                           // -2: a page outside the pool, read as zeros
  Start st;
  static_assert(kParts * RB * DH <= kKeys * (DH + 4), "the outputs of the parts");
};

template <int DH, int RG>
__global__ void __launch_bounds__(kF32Threads, F32Smem<DH, RG>::kCtas)
paged_f32_kernel(PagedAttnArgs a, int TB, Mark* marks, float* slots) {
  using S = F32Smem<DH, RG>;
  constexpr int RB = S::RB, kSteps = S::kPerWarp / 32, kVec = DH / 32;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const PagedBatch& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, ty = (tid >> 3) & 3, tx = tid & 7;
  const int r0 = warp % RG * 16 + ty, part = warp / RG, k0 = part * S::kPerWarp;  // first row, part, its first key
  const int G = a.Hq / p.Hkv;
  const Split sp{TB, kF32ItemCost, kF32Slack};
  pdl_wait();
  find_start<false>(p, sp, blockIdx.x, gridDim.x, blockIdx.x == 0, &sm.st, reinterpret_cast<ScanScratch*>(sm.row));
  if (tid == 0) leave_mark(&sm.st, sp, blockIdx.x, marks + blockIdx.x);
  pdl_trigger();
  if (!sm.st.any) return;
  const float sl2 = a.scale * 1.4426950408889634f;
  const float* Q = reinterpret_cast<const float*>(a.Q);
  const float minf = -INFINITY;

  for (WalkT<false> w(sp, &sm.st); w.more(); w.next(p, sp)) {
    const Seq& s = w.s;
    const int tb0 = w.i * TB, tend = w.t0 + w.n;
    const int rows = min(TB, s.nq - tb0) * G;  // that exist
    const int last = s.len - s.nq + min(tb0 + TB, s.nq) - 1;  // the block's last visible position
    auto locate = [&](int t) -> int64_t {  // this thread's entry of `row`
      if (t < s.nm) {
        const int sg = t * kTileSegs + tid / kSegRows, x = tid % kSegRows;
        if (sg < p.Smax && x < __ldg(a.seg_cnt + w.b * p.Smax + sg))
          return ((int64_t)(__ldg(a.seg_row + w.b * p.Smax + sg) + x) * p.Hkv + w.g) * DH;
        return -1;
      }
      const int at = (t - s.nm) * kKeys + tid;
      if (at > last) return -1;
      const int pi = at / p.page;
      const int64_t pg = __ldg(p.table + w.b * p.max_pages + pi);
      if (pg >= 0 && pg < p.num_pages) return pg * a.page_stride + (at - pi * p.page) * a.row_stride + w.g * a.head_stride;
      raise_flag(p.err_flag, MSA_FLAG_INDEX_OOB);
      return -2;
    };
    // Tile t of K or V; keys that do not exist are zeros.
    auto copy = [&](float (*dst)[DH + 4], const void* local, const void* bank, int t) {
      const float* src = reinterpret_cast<const float*>(t < s.nm ? bank : local);
      const int64_t* row = sm.row[(t - w.t0) & 1];
#pragma unroll
      for (int e = tid; e < kKeys * (DH / 4); e += kF32Threads) {
        const int r = e / (DH / 4), c = e % (DH / 4) * 4;
        const int64_t off = row[r];
        cp_async16(&dst[r][c], off >= 0 ? src + off + c : Q, off >= 0);
      }
    };
    __syncthreads();  // the previous segment's readers are done
    for (int e = tid; e < RB * (DH / 4); e += kF32Threads) {
      const int r = e / (DH / 4), c = e % (DH / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) v = __ldg(reinterpret_cast<const float4*>(Q + (s.q0 + tb0 + r / G) * a.q_ts + (w.g * G + r % G) * DH + c));
      *reinterpret_cast<float4*>(&sm.Q[r][c]) = v;
    }
    if (tid < kKeys) sm.row[0][tid] = locate(w.t0);
    __syncthreads();
    copy(sm.K, a.K, a.Kbar, w.t0);
    int pos[4];  // last visible cache position of this thread's rows
    float m_run[4], l_run[4];
    uint64_t o[4][2 * kVec];  // pairs
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + 4 * j;
      pos[j] = r < rows ? s.len - s.nq + tb0 + r / G : -1;
      m_run[j] = minf;
      l_run[j] = 0.f;  // over this thread's keys
#pragma unroll
      for (int c = 0; c < 2 * kVec; ++c) o[j][c] = 0;
    }

    for (int t = w.t0; t < tend; ++t) {
      const int buf = (t - w.t0) & 1;
      const bool mem = t < s.nm;
      const int key0 = (mem ? 0 : (t - s.nm) * kKeys) + k0;
      const bool live = mem || key0 <= last;  // the warp's part has a visible key
      cp_async_wait();
      __syncthreads();  // K is here; V and the other half of `row` are read
      copy(sm.V, a.V, a.Vbar, t);
      if (t + 1 < tend && tid < kKeys) sm.row[buf ^ 1][tid] = locate(t + 1);
      float (&P)[16][S::kPerWarp + 8] = sm.P[warp];
      bool all = true;  // every row of the warp sees every key of its part
      if (live) {
        float sc[kSteps][4][4];
        {
          uint64_t acc[kSteps][4][4];  // sums over the even and the odd dimensions
#pragma unroll
          for (int x = 0; x < kSteps * 16; ++x) acc[x / 16][x / 4 % 4][x % 4] = 0;
#pragma unroll 16
          for (int c = 0; c < DH; c += 4) {
            ulonglong2 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const ulonglong2*>(&sm.Q[r0 + 4 * j][c]);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
              ulonglong2 k[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) k[i] = *reinterpret_cast<const ulonglong2*>(&sm.K[k0 + st * 32 + tx + 8 * i][c]);
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[st][j][i] = f2_fma(q[j].y, k[i].y, f2_fma(q[j].x, k[i].x, acc[st][j][i]));
            }
          }
#pragma unroll
          for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float x, y;
                f2_unpack(acc[st][j][i], x, y);
                sc[st][j][i] = x + y;
              }
        }
        float top[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) top[j] = minf;
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = st * 32 + tx + 8 * i;
            const bool have = sm.row[buf][k0 + k] != -1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool sees = have && (mem || key0 + k <= pos[j]);
              all = all && sees;
              if (!sees) sc[st][j][i] = minf;
              top[j] = fmaxf(top[j], sc[st][j][i]);
            }
          }
        all = __all_sync(0xffffffffu, all);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int x = 4; x > 0; x >>= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], x));
          const float m_new = fmaxf(m_run[j], top[j]);
          // a row that has seen no key yet keeps weight 0 for everything
          const float corr = m_run[j] == minf ? 0.f : exp2f((m_run[j] - m_new) * sl2);
          m_run[j] = m_new;
          l_run[j] *= corr;
#pragma unroll
          for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a weight of 0 below is a key that the row does not see, so one it sees keeps at least 2^-149
              // (NaN is larger as an unsigned number and stays)
              const float e = sc[st][j][i] == minf ? 0.f
                            : __uint_as_float(max(__float_as_uint(exp2f((sc[st][j][i] - m_new) * sl2)), 1u));
              l_run[j] += e;
              P[ty + 4 * j][st * 32 + tx + 8 * i] = e;
            }
#pragma unroll
          for (int c = 0; c < 2 * kVec; ++c) o[j][c] = f2_mul(o[j][c], f2_pack(corr, corr));
        }
      }
      cp_async_wait();
      __syncthreads();  // V and the next tile's places are here, K is read
      if (t + 1 < tend) copy(sm.K, a.K, a.Kbar, t + 1);
      auto add_values = [&](auto all) {  // all: every weight is of a key that its row sees
#pragma unroll 4
        for (int kc = 0; kc < S::kPerWarp; kc += 4) {
          float4 pr[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) pr[j] = *reinterpret_cast<const float4*>(&P[ty + 4 * j][kc]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            ulonglong2 v[kVec];
#pragma unroll
            for (int c = 0; c < kVec; ++c) v[c] = *reinterpret_cast<const ulonglong2*>(&sm.V[k0 + kc + q][c * 32 + tx * 4]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float pw = q == 0 ? pr[j].x : q == 1 ? pr[j].y : q == 2 ? pr[j].z : pr[j].w;
              if (!all && pw == 0.f) continue;  // keeps a masked key out even where its value is not finite
              const uint64_t p2 = f2_pack(pw, pw);
#pragma unroll
              for (int c = 0; c < kVec; ++c) {
                o[j][2 * c] = f2_fma(p2, v[c].x, o[j][2 * c]);
                o[j][2 * c + 1] = f2_fma(p2, v[c].y, o[j][2 * c + 1]);
              }
            }
          }
        }
      };
      if (live) {
        if (all) add_values(std::true_type());
        else add_values(std::false_type());
      }
    }

    // the parts of a row, in their order; a sum of 0 is a part whose keys the row did not see
    float (*parts)[DH] = reinterpret_cast<float (*)[DH]>(&sm.K[0][0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int x = 4; x > 0; x >>= 1) l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], x);
      const int r = r0 + 4 * j;
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        *reinterpret_cast<ulonglong2*>(&parts[part * RB + r][c * 32 + tx * 4]) = make_ulonglong2(o[j][2 * c], o[j][2 * c + 1]);
      if (tx == 0) sm.ml[part][r] = make_float2(m_run[j], l_run[j]);
    }
    __syncthreads();
    const bool whole = w.whole();
    float* slot = slots + slot_of(blockIdx.x, w.f, sm.st.f0) * slot_floats(RB, DH);
    for (int e = tid; e < rows * (DH / 4); e += kF32Threads) {
      const int r = e / (DH / 4), c = e % (DH / 4) * 4;
      float top = minf, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < S::kParts; ++x) top = fmaxf(top, sm.ml[x][r].x);
#pragma unroll
      for (int x = 0; x < S::kParts; ++x) {
        const float2 ml = sm.ml[x][r];
        if (ml.y == 0.f) continue;
        const float f = exp2f((ml.x - top) * sl2);
        const float4 v = *reinterpret_cast<const float4*>(&parts[x * RB + r][c]);
        sum += ml.y * f;
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      const int tk = tb0 + r / G, h = w.g * G + r % G;
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.O) + ((s.q0 + tk) * a.Hq + h) * DH + c) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (a.lse && c == 0)
          a.lse[(int64_t)h * p.N + s.q0 + tk] = sum == 0.f ? minf : top * a.scale + logf(sum);
      } else {
        *reinterpret_cast<float4*>(slot + r * DH + c) = acc;
        if (c == 0) *reinterpret_cast<float2*>(slot + RB * DH + 2 * r) = make_float2(top, sum);
      }
    }
  }
}

// O = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s over an item's segments, in the
// order of the CTAs.  Block x merges the item of mark x + 1, if there is one; block y
// takes kMergeRows of its rows, a thread four values of a row.  A chain of dependent
// loads (mark, maxima, values) bounds it; all blocks are resident at once.
constexpr int kMergeThreads = 256, kMergeRows = 32;
constexpr int kAtOnce = 8;  // segments whose loads are in flight together

// Row of the V pages of cache position `at` of sequence b for KV head g; null: its page is outside the pool.
__device__ __forceinline__ const __nv_bfloat16* value_row(const PagedAttnArgs& a, int64_t b, int g, int at) {
  const int pi = at / a.p.page;
  const int64_t pg = __ldg(a.p.table + b * a.p.max_pages + pi);
  if (pg < 0 || pg >= a.p.num_pages) return nullptr;
  return reinterpret_cast<const __nv_bfloat16*>(a.V) + pg * a.page_stride + (at - pi * a.p.page) * a.row_stride + g * a.head_stride;
}
// The values that are not finite which an item's tiles left out (paged_tma.cuh): of the keys after its
// first token's, to the rows that see them.
// Four dimensions of the output of packed row `row`, for an item that is being merged:
__device__ __forceinline__ void add_odd_to_row(const PagedAttnArgs& a, const Mark& mk, int64_t row, int quad,
                                               float (&acc)[4]) {
  const Seq s = load_seq(a.p, mk.b);
  const int pos0 = s.len - s.nq, first = pos0 + (int)(mk.row - s.q0), pos = pos0 + (int)(row - s.q0);
#pragma unroll 1
  for (int key = max(first + 1, 0); key <= pos; ++key) {
    const __nv_bfloat16* v = value_row(a, mk.b, mk.g, key);
    if (!v) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = __bfloat162float(v[quad * 4 + i]);
      if (!isfinite(f)) acc[i] += f;
    }
  }
}
// ... and the outputs of all items that no mark names, which their CTA has written: a warp takes every
// `warps`-th item, a lane the sums of its dimensions over the keys so far, and a token's rows take
// those up to its own key.  Here, because the attention kernels run slower the more code lies around
// their loops (23 requests with heads of 64: 120.5 us, with this at each item's end 132, at the CTA's
// end 126), and not inlined, because the merge's registers spill then (one token 11.5 us instead of
// 10.4).
template <int DH>
__device__ __noinline__ void add_odd_values(const MergeArgs& ma, int64_t warp, int64_t warps) {
  constexpr int kEach = DH / 32;
  const PagedAttnArgs& a = ma.a;
  const PagedBatch& p = a.p;
  const int lane = threadIdx.x & 31, G = a.Hq / p.Hkv;
  int64_t turn = warp;  // items until this warp's next one
#pragma unroll 1
  for (int64_t b = 0; b < p.B; ++b) {
    const Seq s = load_seq(p, b);
    const int64_t items = (int64_t)blocks_of(s, ma.TB) * p.Hkv;
    for (; turn < items; turn += warps) {
      const int i = (int)(turn / p.Hkv), g = (int)(turn - (int64_t)i * p.Hkv), t0 = i * ma.TB;
      bool merged = false;
      for (int c = 1 + lane; c < ma.grid; c += 32) {
        const Mark mk = ma.marks[c];
        merged = merged || (mk.tokens > 0 && mk.b == b && mk.g == g && mk.row == s.q0 + t0);
      }
      if (__any_sync(0xffffffffu, merged)) continue;
      const int tokens = min(ma.TB, s.nq - t0), first = s.len - s.nq + t0, from = max(1, -first);
      float sum[kEach] = {};
#pragma unroll 1
      for (int t = from; t < tokens; ++t) {
        const __nv_bfloat16* v = value_row(a, b, g, first + t);
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
          const float f = v ? __bfloat162float(v[lane * kEach + x]) : 0.f;
          if (!isfinite(f)) sum[x] += f;
        }
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.O) + ((s.q0 + t0 + t) * a.Hq + g * G) * DH + lane * kEach;
#pragma unroll 1
        for (int h = 0; h < G; ++h, dst += DH)
#pragma unroll
          for (int x = 0; x < kEach; ++x)
            if (sum[x] != 0.f) dst[x] = __float2bfloat16_rn(__bfloat162float(dst[x]) + sum[x]);
      }
    }
    turn -= items;
  }
}

template <typename T, int DH, bool kQuads>
__global__ void __launch_bounds__(kMergeThreads, 4) merge_kernel(const __grid_constant__ MergeArgs ma) {
  constexpr int kPairs = kMergeRows * (DH / 4);  // (row, four values) pairs of the block
  pdl_wait();
  const PagedAttnArgs& a = ma.a;
  const Mark mk = ma.marks[blockIdx.x + 1];
  bool odd = false;  // values may have been left out
  if constexpr (sizeof(T) == 2) odd = any_odd(ma.marks, ma.grid);
  const int G = a.Hq / a.p.Hkv;
  const int last = mk.tokens * G;  // rows of the item
  const size_t sf = slot_floats(ma.rows, DH);
  const float* first = ma.slots + (2 * (int64_t)mk.c0 + mk.late) * sf;
  const float* rest = ma.slots + 2 * (int64_t)mk.c0 * sf;  // segment x > 0 is in slot 2 (c0 + x)
  for (int e = threadIdx.x; e < kPairs; e += kMergeThreads) {
    // consecutive threads: rows first in the quads layout, values of a row first in the other
    const int quad = kQuads ? e / kMergeRows : e % (DH / 4);
    const int r = blockIdx.y * kMergeRows + (kQuads ? e % kMergeRows : e / (DH / 4));
    if (r >= last) continue;
    const int ml_at = ma.rows * DH + 2 * r, v_at = kQuads ? (quad * ma.rows + r) * 4 : r * DH + quad * 4;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int x0 = 0; x0 < mk.n; x0 += kAtOnce) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce];
      float top = m;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (x0 + j >= mk.n) continue;
        const float* src = x0 + j == 0 ? first : rest + 2 * (size_t)(x0 + j) * sf;
        ml[j] = *reinterpret_cast<const float2*>(src + ml_at);
        v[j] = *reinterpret_cast<const float4*>(src + v_at);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (x0 + j < mk.n) top = fmaxf(top, ml[j].x);
      const float corr = l == 0.f ? 0.f : exp2f((m - top) * ma.unit_log2);
      l *= corr;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= corr;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (x0 + j >= mk.n) continue;
        const float w = ml[j].y == 0.f ? 0.f : exp2f((ml[j].x - top) * ma.unit_log2);  // sum 0: no key was visible
        l += w * ml[j].y;
        acc[0] += w * v[j].x;
        acc[1] += w * v[j].y;
        acc[2] += w * v[j].z;
        acc[3] += w * v[j].w;
      }
      m = top;
    }
    const bool seen = l != 0.f;
    const float inv = seen ? 1.f / l : 0.f;
    const int tl = r / G, h = mk.g * G + (r - tl * G);
    const int64_t row = mk.row + tl;
    T* dst = reinterpret_cast<T*>(a.O) + (row * a.Hq + h) * DH + quad * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= inv;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
      if (odd) add_odd_to_row(a, mk, row, quad, acc);
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    }
    if (a.lse && quad == 0)
      a.lse[(int64_t)h * a.p.N + row] = seen ? (m * ma.unit_log2 + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
  if (odd)
    add_odd_values<DH>(ma, ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5),
                       (int64_t)gridDim.x * gridDim.y * (kMergeThreads / 32));
}

// fp32 for RW rows per KV head: 256 threads stream the tiles' rows straight into registers.  Eight
// lanes share a key (DH / 8 dimensions each), so a warp takes four keys at once, kAhead times; every
// group of eight lanes keeps running maxima, sums and outputs of its own for the RW rows, merged
// within the CTA at the segment's end.  At 4 rows 0.75 of the copy rate (64 requests of 4,096 keys,
// heads of 128: 434 us), at 8 rows 831 us: twice the rows, twice the time, so the rows' arithmetic and
// its shuffles bound it, with the loads' latency uncovered beside them (a warp asks for its next keys
// when the last ones are used up).
template <int DH, int RW>
struct RowsSmem {
  static constexpr int kWarps = 8;  // share the keys of a tile
  float Q[RW][DH];
  float part[8][RW][DH];
  float2 ml[8][RW];
  int64_t row[2][kKeys];  // as in F32Smem
  Start st;
};

template <int DH, int RW>
__global__ void __launch_bounds__(kF32Threads, 1) paged_f32_rows_kernel(PagedAttnArgs a, Mark* marks, float* slots) {
  using S = RowsSmem<DH, RW>;
  constexpr int kVec = DH / 32, kAhead = RW == 4 ? 4 : 2, kPerWarp = kKeys / S::kWarps;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const PagedBatch& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = lane >> 3, sub = lane & 7;
  const int G = a.Hq / p.Hkv;
  const Split sp{p.max_q, kF32ItemCost, kF32Slack};
  pdl_wait();
  find_start<true>(p, sp, blockIdx.x, gridDim.x, blockIdx.x == 0, &sm.st, reinterpret_cast<ScanScratch*>(sm.row));
  if (tid == 0) leave_mark(&sm.st, sp, blockIdx.x, marks + blockIdx.x);
  pdl_trigger();
  if (!sm.st.any) return;
  const float sl2 = a.scale * 1.4426950408889634f;
  const float* Q = reinterpret_cast<const float*>(a.Q);
  const float minf = -INFINITY;

  for (WalkT<true> w(sp, &sm.st); w.more(); w.next(p, sp)) {
    const Seq& s = w.s;
    const int rows = s.nq * G, pos0 = s.len - s.nq;  // rows that exist, position of the first new token
    // element offset of one key of a tile in its tensor, -1: no key, -2: zeros
    auto locate = [&](int t) -> int64_t {
      if (t < s.nm) {
        const int sg = t * kTileSegs + tid / kSegRows, x = tid % kSegRows;
        if (sg < p.Smax && x < __ldg(a.seg_cnt + w.b * p.Smax + sg))
          return ((int64_t)(__ldg(a.seg_row + w.b * p.Smax + sg) + x) * p.Hkv + w.g) * DH;
        return -1;
      }
      const int at = (t - s.nm) * kKeys + tid;
      if (at >= s.len) return -1;
      const int pi = at / p.page;
      const int64_t pg = __ldg(p.table + w.b * p.max_pages + pi);
      if (pg >= 0 && pg < p.num_pages) return pg * a.page_stride + (at - pi * p.page) * a.row_stride + w.g * a.head_stride;
      raise_flag(p.err_flag, MSA_FLAG_INDEX_OOB);
      return -2;
    };
    __syncthreads();  // the previous segment's readers are done
    for (int e = tid; e < RW * (DH / 4); e += kF32Threads) {
      const int r = e / (DH / 4), c = (e - r * (DH / 4)) * 4, t = r / G;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < s.nq) v = __ldg(reinterpret_cast<const float4*>(Q + (s.q0 + t) * a.q_ts + (w.g * G + r % G) * DH + c));
      *reinterpret_cast<float4*>(&sm.Q[r][c]) = v;
    }
    if (tid < kKeys) sm.row[0][tid] = locate(w.t0);
    float m[RW], l[RW], o[RW][4 * kVec];
    int last[RW];  // last visible cache position of a row
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      m[r] = minf;
      l[r] = 0.f;
      last[r] = r < rows ? pos0 + r / G : -1;
#pragma unroll
      for (int c = 0; c < 4 * kVec; ++c) o[r][c] = 0.f;
    }
    for (int t = w.t0; t < w.t0 + w.n; ++t) {
      const int buf = (t - w.t0) & 1;
      const bool mem = t < s.nm;
      __syncthreads();  // this tile's rows are written, the last one's read
      if (t + 1 < w.t0 + w.n && tid < kKeys) sm.row[buf ^ 1][tid] = locate(t + 1);
      const float* Ks = reinterpret_cast<const float*>(mem ? a.Kbar : a.K) + sub * 4;
      const float* Vs = reinterpret_cast<const float*>(mem ? a.Vbar : a.V) + sub * 4;
      const int base = mem ? 0 : (t - s.nm) * kKeys;
#pragma unroll 1
      for (int k0 = warp * kPerWarp; k0 < (warp + 1) * kPerWarp; k0 += 4 * kAhead) {
        int64_t off[kAhead];
        float4 kv[kAhead][kVec], vv[kAhead][kVec];
        bool all = true;  // every row of the warp sees every key of the step
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          const int k = k0 + n * 4 + grp;
          off[n] = sm.row[buf][k];
          all = all && off[n] != -1 && (mem || base + k <= pos0);
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            kv[n][i] = vv[n][i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (off[n] >= 0) {
              kv[n][i] = __ldg(reinterpret_cast<const float4*>(Ks + off[n] + i * 32));
              vv[n][i] = __ldg(reinterpret_cast<const float4*>(Vs + off[n] + i * 32));
            }
          }
        }
        all = __all_sync(0xffffffffu, all);
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          float sc[kAhead];
#pragma unroll
          for (int n = 0; n < kAhead; ++n) sc[n] = 0.f;
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(&sm.Q[r][sub * 4 + i * 32]);
#pragma unroll
            for (int n = 0; n < kAhead; ++n)
              sc[n] = fmaf(q.x, kv[n][i].x, fmaf(q.y, kv[n][i].y, fmaf(q.z, kv[n][i].z, fmaf(q.w, kv[n][i].w, sc[n]))));
          }
          float top = m[r];
#pragma unroll
          for (int n = 0; n < kAhead; ++n) {
#pragma unroll
            for (int x = 4; x > 0; x >>= 1) sc[n] += __shfl_xor_sync(0xffffffffu, sc[n], x);
            if (!all && !(off[n] != -1 && (mem ? r < rows : base + k0 + n * 4 + grp <= last[r]))) sc[n] = minf;
            top = fmaxf(top, sc[n]);
          }
          const float corr = m[r] == minf ? 0.f : exp2f((m[r] - top) * sl2);
          const float ref = top == minf ? 0.f : top;  // nothing above -inf yet: keys of score -inf weigh 0
          m[r] = top;
          l[r] *= corr;
#pragma unroll
          for (int c = 0; c < 4 * kVec; ++c) o[r][c] = corr == 1.f ? o[r][c] : o[r][c] * corr;
#pragma unroll
          for (int n = 0; n < kAhead; ++n) {
            if (!all && sc[n] == minf) continue;  // not seen: whatever V holds stays out
            const float pw = exp2f((sc[n] - ref) * sl2);
            l[r] += pw;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
              o[r][4 * i] = fmaf(pw, vv[n][i].x, o[r][4 * i]);
              o[r][4 * i + 1] = fmaf(pw, vv[n][i].y, o[r][4 * i + 1]);
              o[r][4 * i + 2] = fmaf(pw, vv[n][i].z, o[r][4 * i + 2]);
              o[r][4 * i + 3] = fmaf(pw, vv[n][i].w, o[r][4 * i + 3]);
            }
          }
        }
      }
    }
    // the warp's four groups, then the warps; a sum of 0 is a group whose rows saw no key
#pragma unroll
    for (int r = 0; r < RW; ++r) {
#pragma unroll
      for (int x = 8; x < 32; x <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, m[r], x), lo = __shfl_xor_sync(0xffffffffu, l[r], x);
        const float top = fmaxf(m[r], mo);
        const float f = l[r] == 0.f ? 0.f : exp2f((m[r] - top) * sl2), fo = lo == 0.f ? 0.f : exp2f((mo - top) * sl2);
        m[r] = top;
        l[r] = l[r] * f + lo * fo;
#pragma unroll
        for (int c = 0; c < 4 * kVec; ++c) {
          const float y = __shfl_xor_sync(0xffffffffu, o[r][c], x);
          o[r][c] = o[r][c] * f + y * fo;  // (0 where no key was seen; an infinity is not lost to a factor of 0)
        }
      }
      if (grp == 0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          *reinterpret_cast<float4*>(&sm.part[warp][r][sub * 4 + i * 32]) =
              make_float4(o[r][4 * i], o[r][4 * i + 1], o[r][4 * i + 2], o[r][4 * i + 3]);
        if (sub == 0) sm.ml[warp][r] = make_float2(m[r], l[r]);
      }
    }
    __syncthreads();
    const bool whole = w.whole();
    float* slot = slots + slot_of(blockIdx.x, w.f, sm.st.f0) * slot_floats(kF32FewRows, DH);
    for (int e = tid; e < rows * (DH / 4); e += kF32Threads) {
      const int r = e / (DH / 4), c = (e - r * (DH / 4)) * 4;
      float top = minf, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < S::kWarps; ++x) top = fmaxf(top, sm.ml[x][r].x);
#pragma unroll
      for (int x = 0; x < S::kWarps; ++x) {
        const float2 ml = sm.ml[x][r];
        if (ml.y == 0.f) continue;
        const float f = exp2f((ml.x - top) * sl2);
        const float4 v = *reinterpret_cast<const float4*>(&sm.part[x][r][c]);
        sum += ml.y * f;
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      const int t = r / G, h = w.g * G + r % G;
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.O) + ((s.q0 + t) * a.Hq + h) * DH + c) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (a.lse && c == 0)
          a.lse[(int64_t)h * p.N + s.q0 + t] = sum == 0.f ? minf : top * a.scale + logf(sum);
      } else {
        *reinterpret_cast<float4*>(slot + r * DH + c) = acc;
        if (c == 0) *reinterpret_cast<float2*>(slot + kF32FewRows * DH + 2 * r) = make_float2(top, sum);
      }
    }
  }
}

// Rows of a block of the fp32 block kernel.  64 where 32 hold less than half as many tokens, and
// where the blocks of 64 are at least twice the SMs (1,050 tokens x 32 heads over 2,200 keys: heads
// of 128 849 us, with 32 rows 947; heads of 64 475 and 493); else 32, two CTAs per SM with heads of
// 64 (100 tokens over 1,100 keys 86 us, with 64 rows 96).
int f32_block_rows(int Hq, int Hkv, int64_t N) {
  const int G = Hq / Hkv;
  return 64 / G > 2 * (32 / G) || N * Hq >= 2 * 64 * (int64_t)sm_count() ? 64 : 32;
}

template <typename Kernel, typename... Args>
cudaError_t f32_launch(Kernel kernel, size_t smem, std::atomic<uint64_t>& done, int grid, int rows,
                       const PagedAttnArgs& a, cudaStream_t s, Args... args) {
  cudaError_t e = allow_smem(kernel, (int)smem, done);
  if (e != cudaSuccess) return e;
  Mark* marks = reinterpret_cast<Mark*>(a.part);
  float* slots = reinterpret_cast<float*>(reinterpret_cast<char*>(a.part) + marks_bytes(grid));
  count_launch();
  e = launch_pdl(kernel, dim3((unsigned)grid), dim3(kF32Threads), smem, s, a, args..., marks, slots);
  if (e != cudaSuccess) return e;
  return launch_merge(MSA_F32, false, MergeArgs{a, marks, slots, grid, rows, 0, a.scale * 1.4426950408889634f}, s);
}
template <int DH, int RG>
cudaError_t f32_block(const PagedAttnArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  return f32_launch(paged_f32_kernel<DH, RG>, sizeof(F32Smem<DH, RG>), done, F32Smem<DH, RG>::kCtas * sm_count(), 16 * RG,
                    a, s, 16 * RG / (a.Hq / a.p.Hkv));
}
template <int DH>
cudaError_t f32_blocks(const PagedAttnArgs& a, cudaStream_t s) {
  return f32_block_rows(a.Hq, a.p.Hkv, a.p.N) == 32 ? f32_block<DH, 2>(a, s) : f32_block<DH, 4>(a, s);
}
template <int DH, int RW>
cudaError_t f32_few(const PagedAttnArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  return f32_launch(paged_f32_rows_kernel<DH, RW>, sizeof(RowsSmem<DH, RW>), done, sm_count(), kF32FewRows, a, s);
}

// Whether the kernels for few rows take a call, by the rows G * max_q that a sequence may have per KV
// head.  Measured against the kernels for blocks of rows (us, few / blocks; 64 requests of 4,096 keys
// and of 900, 16 of 1,000, one of 1,000, 4 of 30,000):
//   bf16, heads of 128   4 rows 171/187  56/83  18/20  10/19  82/94     8 rows 177/188  62/85  20/20  11/19  84/93
//                       12 rows 189/190  82/87  25/21  14/19  89/95    16 rows 199/189  90/86  26/21  14/19  90/94
//   bf16, heads of 64    4 rows 136/141  42/64  17/18  11/14  56/71    16 rows 151/142  71/66  23/18  13/15  66/71
//   fp32, heads of 128   4 rows 435/1058 126/274 42/82 12/18 201/485    8 rows 831/1101 232/285 69/85 17/18 379/504
//                       12 rows 1607/1145 426/299 123/88 25/21 730/525
//   fp32, heads of 64    4 rows 352/597 102/159 26/49 10/14 165/276     8 rows 673/605 187/161 47/50 14/14 308/279
// So up to 16 rows in bf16 (few at 12 and 16 gain for one request and for long caches about what they
// lose for some tens of short ones), in fp32 up to 8 with heads of 128 and 4 with heads of 64.
bool few_rows(msa_dtype dt, int d, int Hq, int Hkv, int max_q) {
  return (int64_t)(Hq / Hkv) * max_q <= (dt == MSA_F32 ? d / 16 : 16);
}

}  // namespace

cudaError_t launch_merge(msa_dtype dt, bool quads, const MergeArgs& m, cudaStream_t s) {
  const int d = m.a.d;
  auto k = dt == MSA_F32 ? (d == 64 ? merge_kernel<float, 64, false> : merge_kernel<float, 128, false>)
           : !quads      ? (d == 64 ? merge_kernel<__nv_bfloat16, 64, false> : merge_kernel<__nv_bfloat16, 128, false>)
                         : (d == 64 ? merge_kernel<__nv_bfloat16, 64, true> : merge_kernel<__nv_bfloat16, 128, true>);
  const dim3 grid((unsigned)(m.grid - 1), (unsigned)((m.rows + kMergeRows - 1) / kMergeRows));
  count_launch();
  return launch_pdl(k, grid, dim3(kMergeThreads), 0, s, m);
}

}  // namespace paged

size_t paged_attn_partial_bytes(msa_dtype dt, int Hq, int Hkv, int d, int max_q) {
  const bool few = paged::few_rows(dt, d, Hq, Hkv, max_q);
  // fp32 blocks: as many rows with two CTAs of 32 per SM as with one of 64
  const int grid = dt == MSA_F32 && !few ? 2 * sm_count() : sm_count();
  const int rows = dt == MSA_F32 ? (few ? paged::kF32FewRows : 32) : (few ? Hq / Hkv * max_q : 128);
  return paged::marks_bytes(grid) + 2 * (size_t)grid * paged::slot_floats(rows, d) * sizeof(float);
}

cudaError_t launch_paged_attn(msa_dtype dt, const PagedAttnArgs& a, cudaStream_t s) {
  const bool few = paged::few_rows(dt, a.d, a.Hq, a.p.Hkv, a.p.max_q);
  if (dt != MSA_F32) return few ? launch_paged_decode(a, s) : launch_paged_prefill(a, s);
  if (a.d == 64) return few ? paged::f32_few<64, 4>(a, s) : paged::f32_blocks<64>(a, s);
  if (!few) return paged::f32_blocks<128>(a, s);
  return a.Hq / a.p.Hkv * a.p.max_q <= 4 ? paged::f32_few<128, 4>(a, s) : paged::f32_few<128, 8>(a, s);
}

}  // namespace msa
