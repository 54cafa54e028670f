// The sliding-window and paged-cache attention forward on the tensor cores
// (tcgen05), bf16 and fp16, D = 16, 32, 64 or 128.
//
// Mathematics: softmax(Q K^T / sqrt(D)) V over the visible keys in one pass,
// with each row's running maximum and sum in fp32; P is rounded to the input
// format for the second product (the tensor cores take 16-bit operands; fp16 as
// 2^7 P, see kUp), the sum is of the unrounded values.
//
// Layout.  The G query heads of a key/value head read the same keys, so a
// tile's 128 rows are 128 / G tokens by G heads.  A CTA owns two row tiles (A
// and B) of one key/value head and streams 64-key blocks through one ring that
// both tiles read: a key block is fetched once for 256 rows.  It visits only
// the blocks the mask reaches (those with sinks, then those of the window).
//   warps 0-3, 4-7  softmax of tile A and B, a thread per row: scores from
//                   TMEM, P back over them in the input format, O rescaled in
//                   TMEM only when the row maximum grew by more than 2^8
//   warp 8          TMA loads; a block of a paged cache is a box per page
//   warps 9, 10     MMA issue for tile A and B: per block, P V and then the
//                   scores two blocks further on.  One warp for both tiles is
//                   busy all the time and sets the pace (3370 cycles per 64
//                   keys at D = 128 where the softmax takes 1050)
// TMEM: two 64-column score buffers per tile, so that a tile's next scores are
// there when its softmax asks for them, and two D-column accumulators.
// With fewer rows than one tile per key/value head (short chunks over a long
// cache) both streams take the same tile and alternate blocks.  A paged call
// with few row tiles is cut along the keys too: into pieces of nearly equal
// runs of blocks, as many as SMs, which each CTA works out for itself from the
// lengths on the device; join_kernel adds them.  (Three chunks of up to 1024
// tokens over 8K keys, 8/2 heads of 128, 96 row-tile pairs of very different
// lengths: 141 us uncut, 49 and 17 for the join cut.)
// Bound: neither pipe alone, but the chain of a block from its scores over its
// softmax to its second product; the tensor cores work 37 % of the cycles at D =
// 128 and the exponentials' unit 38 %.  Measured: 8192 tokens, 12/4 heads of 64,
// window 1024: 68 us (357 TFLOP/s of visible products); 16384 tokens, 8 heads of
// 128, window 4096: 242 us (995); two chunks of up to 4096 tokens over up to 16384
// keys, 16/4 heads of 128: 709 us (1092).
// Slots past a sequence's keys may hold anything: their scores are masked
// before use and their value rows are overwritten with zeros in shared memory.
// Every wait is bounded; on a timeout the kernel records the status word,
// stops issuing, drains what it issued and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "attn_args.cuh"
#include "tc_ptx.cuh"
#include "window_tc.cuh"

namespace longnet {
namespace wt {
using namespace tc;

constexpr int kThreads = 352;
constexpr int kTma = 8, kMma = 9;  // warps; kMma + 1 issues for the second stream
constexpr int kBlk = 64;           // keys of a block
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;  // after two score buffers per stream
constexpr int kSms = 148;

template <int kD>
struct L : Panels<kD> {
  using P = Panels<kD>;
  static constexpr int kQBytes = kTile * kD * 2;     // one row tile
  static constexpr int kHalf = kBlk * kD * 2;        // one block of keys or values
  static constexpr int kStageBytes = 2 * kHalf;      // values of block n, keys of block n + ahead
  static constexpr int kStages = kD == 128 ? 5 : 6;
  static constexpr int kBars = 2 * kQBytes + kStages * kStageBytes;
  // one CTA per SM at every D: its TMEM columns are all of the SM's
  static constexpr int kSmem = kBars + 512 + 1024 > 120 * 1024 ? kBars + 512 + 1024 : 120 * 1024;
};

// The blocks of a CTA's list that one stream takes: a run [begin, end), or
// every second one.  A run has no gap, since the softmax asks for a block's
// scores before it hands over the P of the block before; so a stream with
// sinks also takes the few blocks between them and its window that only the
// other stream sees, all masked.
struct Range {
  int begin, end, step, count;
  __device__ __forceinline__ bool has(int n) const {
    return n >= begin && n < end && (step == 1 || ((n - begin) & 1) == 0);
  }
};

constexpr int kMaxItems = 320;  // ten per lane of the numbering warp
constexpr int kMinRun = 8;      // blocks of a piece: shorter ones cost more in joining than they spread

// base[i] = pieces of the items before i, of one head, by one warp.  The run
// length is the least, in steps of an eighth, for which all heads' pieces fit
// one CTA per SM (or, with more items than SMs, for which none is cut).
__device__ __forceinline__ void number_pieces(const AttnArgs& a, const Plan& plan, int* base, int lane) {
  int c[kMaxItems / 32], sum = 0, some = 0;
#pragma unroll
  for (int k = 0; k < kMaxItems / 32; ++k) {
    const int it = lane + 32 * k;
    c[k] = 0;
    if (it < plan.items) {
      const Seq q = seq_of(a, it / plan.pairs);
      const int t0 = (it % plan.pairs) * 2 * plan.tokens, t1 = t0 + 2 * plan.tokens < q.nq ? t0 + 2 * plan.tokens : q.nq;
      if (t0 < q.nq) c[k] = blocks_of<kBlk>(a, q.first + t0, q.first + t1 - 1).count;
      if (t0 < q.nq && c[k] == 0) c[k] = 1;  // rows that see nothing are written too
    }
    sum += c[k];
    some += c[k] > 0 ? 1 : 0;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  some = __reduce_add_sync(0xffffffffu, some);
  const int limit = (some * a.Hkv > kSms ? some * a.Hkv : kSms) / a.Hkv;  // pieces of one head
  int run = limit > 0 ? (sum + limit - 1) / limit : 1;
  if (run < kMinRun) run = kMinRun;
  while (true) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kMaxItems / 32; ++k) n += (c[k] + run - 1) / run;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n <= limit) break;  // at the latest when no item is cut
    run += run / 8;
  }
  int before = 0;
#pragma unroll
  for (int k = 0; k < kMaxItems / 32; ++k) {
    const int n = (c[k] + run - 1) / run;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int it = lane + 32 * k;
    if (it <= plan.items) base[it] = before + x - n;
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  if (plan.items == kMaxItems && lane == 0) base[kMaxItems] = before;
}

template <int kFmt, int kD, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Maps maps, const Plan plan) {
  using LL = L<kD>;
  constexpr int kPanels = LL::kPanels, S = LL::kStages;
  constexpr int kQPanel = kTile * LL::kRowBytes, kKVPanel = kBlk * LL::kRowBytes;
  constexpr uint32_t kDescHi = LL::kDescHi;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sStage = smem + 2 * LL::kQBytes;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // the join may be scheduled; and what the launch before this one wrote is
  // read only from here on
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tpt = plan.tokens;  // tokens of a row tile
  const bool alternate = kPaged && plan.alternate;
  int s, f, pair, slot = 0, piece = 0, pieces = 1;
  if (kPaged && plan.items) {
    // this CTA's piece: of `pieces` equal runs of an item's blocks, run `piece`
    int* base = reinterpret_cast<int*>(sStage);
    if (warp == 0) number_pieces(a, plan, base, lane);
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i <= plan.items; i += kThreads) plan.base[i] = base[i];
    slot = blockIdx.x;
    int lo = 0, hi = plan.items;
    const bool none = slot >= base[hi] * a.Hkv;
    while (!none && hi - lo > 1) {  // the last item with base Hkv <= slot
      const int mid = (lo + hi) >> 1;
      if (base[mid] * a.Hkv <= slot) lo = mid;
      else hi = mid;
    }
    pieces = base[lo + 1] - base[lo];
    const int in = slot - base[lo] * a.Hkv;
    __syncthreads();  // base is read: the ring may take its place
    if (none) return;
    s = lo / plan.pairs;
    pair = lo % plan.pairs;
    f = in / pieces;
    piece = in % pieces;
  } else {
    s = blockIdx.y / a.Hkv;
    f = blockIdx.y % a.Hkv;
    pair = (int)gridDim.x - 1 - blockIdx.x;  // the longest first
  }
  const Seq q = seq_of(a, s);
  const int t0 = pair * 2 * tpt;  // alternate: pair 0
  if (t0 >= q.nq) return;         // whole CTA, before any barrier or TMEM use
  const int t1 = t0 + (alternate ? tpt : 2 * tpt) < q.nq ? t0 + (alternate ? tpt : 2 * tpt) : q.nq;
  const BlockList bl = blocks_of<kBlk>(a, q.first + t0, q.first + t1 - 1);
  const int per = (bl.count + pieces - 1) / pieces;
  const int n0 = piece * per < bl.count ? piece * per : bl.count;
  const int cnt = n0 + per < bl.count ? per : bl.count - n0;  // blocks [n0, n0 + cnt) of the list
  auto block_key = [&](int n) { return bl.at(n0 + n) * kBlk; };
  // tokens [ta, tb) of stream st, empty when it has none
  auto tok_begin = [&](int st) { return alternate ? t0 : t0 + st * tpt; };
  auto tok_end = [&](int st) {
    const int e = tok_begin(st) + tpt;
    return e < t1 ? e : t1;
  };
  auto range_of = [&](int st) {
    Range r;
    const int tb = tok_begin(st), te = tok_end(st);
    const int lo = q.first + tb, low = a.window == 0 || lo < a.window ? 0 : (lo - a.window + 1) / kBlk;
    if (alternate) {
      r.begin = st;
      r.end = cnt;
      r.step = 2;
      r.count = (cnt + 1 - st) / 2;
      return r;
    }
    r.begin = n0 * kBlk < a.sinks ? 0 : bl.n_sink + low - bl.win0 - n0;
    if (r.begin < 0) r.begin = 0;
    const int end = q.first + te - 1 < 0 ? 0 : bl.n_sink + (q.first + te - 1) / kBlk - bl.win0 + 1 - n0;
    r.end = tb < te ? (end < cnt ? end : cnt) : 0;
    r.step = 1;
    r.count = r.end > r.begin ? r.end - r.begin : 0;
    return r;
  };
  // The scores of block n + ahead are issued after P V of block n: two blocks
  // of a stream further on.  Item n of the ring holds what that step takes:
  // the values of block n (none for n < 0) and the keys of block n + ahead
  // (none past the last).
  const int ahead = alternate ? 4 : 2;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LL::kBars);
  uint64_t* bar_q = bars;
  uint64_t* bar_full = bars + 1;       // [S]
  uint64_t* bar_empty = bars + 1 + S;  // [S]
  uint64_t* bar_s = bars + 1 + 2 * S;  // [stream][buffer] scores in TMEM
  uint64_t* bar_p = bar_s + 4;         // [stream][buffer] P in TMEM
  uint64_t* bar_pv = bar_s + 8;        // [stream] the last product but one done
  uint64_t* bar_o = bar_s + 10;        // [stream] the last one done
  uint64_t* bar_tail = bar_s + 12;     // the values of a block with slots past the sequence
  uint64_t* bar_drain = bar_s + 13;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_s + 14);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    for (int i = 0; i < S; ++i) {
      mbar_init(bar_full + i, 1);
      mbar_init(bar_empty + i, 2);  // both streams
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_pv + i, 1);
      mbar_init(bar_o + i, 1);
    }
    mbar_init(bar_tail, 1);
    mbar_init(bar_drain, 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kTma && lane < 3) prefetch_tmap(&maps.m[lane]);
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  Waiter wt{abort_flag, a.status, kWaitLimitNs};

  if (warp == kTma) {
    // ------------------------------------------------------------ loads
    bool ok = true;
    const int qtiles = alternate || t0 + tpt >= t1 ? 1 : 2;
    if (cnt > 0 && lane == 0) {
      mbar_arrive_expect_tx(bar_q, (uint32_t)(qtiles * kPanels * tpt * a.G * LL::kRowBytes));
      for (int st = 0; st < qtiles; ++st)
#pragma unroll
        for (int pn = 0; pn < kPanels; ++pn)
          tma_load_3d(sQ + st * LL::kQBytes + pn * kQPanel, &maps.m[0], bar_q, LL::kPanelElems * pn, f * a.G,
                      (int)(q.q0 + t0 + st * tpt));
    }
    int issued = 0;
    for (int n = -ahead; n < cnt && ok; ++n, ++issued) {
      const int st = issued % S;
      if (issued >= S) ok = wt.wait_warp(bar_empty + st, ((issued / S) - 1) & 1);
      if (!ok) break;
      uint8_t* dst = sStage + st * LL::kStageBytes;
      const bool v = n >= 0, k = n + ahead < cnt;
      if (!kPaged) {
        if (lane == 0) {
          mbar_arrive_expect_tx(bar_full + st, ((v ? 1 : 0) + (k ? 1 : 0)) * LL::kHalf);
#pragma unroll
          for (int pn = 0; pn < kPanels; ++pn) {
            if (v)
              tma_load_4d(dst + pn * kKVPanel, &maps.m[2], bar_full + st, LL::kPanelElems * pn, f, block_key(n), s);
            if (k)
              tma_load_4d(dst + LL::kHalf + pn * kKVPanel, &maps.m[1], bar_full + st, LL::kPanelElems * pn, f,
                          block_key(n + ahead), s);
          }
        }
      } else {
        // expect each half's bytes, then arrive once
        if (k) load_pages<kD>(a, q, s, f, block_key(n + ahead), kBlk, &maps.m[1], dst + LL::kHalf, bar_full + st, lane);
        if (v) {
          const int j0 = block_key(n);
          const bool tail = j0 + kBlk > q.kv;  // the sequence's last block, with no keys after it in this item
          load_pages<kD>(a, q, s, f, j0, kBlk, &maps.m[2], dst, tail ? bar_tail : bar_full + st, lane);
          if (tail) {
            if (lane == 0) mbar_arrive(bar_tail);
            ok = wt.wait_warp(bar_tail, 0);
            if (!ok) break;
            zero_rows<kD>(dst, kBlk, q.kv - j0, lane);
          }
        }
        if (lane == 0) mbar_arrive(bar_full + st);
      }
    }
    // drain: every issued load has landed before the CTA may exit
    if (lane == 0) {
      if (cnt > 0 && !mbar_wait(bar_q, 0, kWaitLimitNs)) record_status(a.status, kStatusTimeout);
      // (the last item's values, when they end in a tail; worked out here, as a flag
      // that the loop sets cost 1 % of the kernel)
      const bool tail = kPaged && cnt > 0 && issued >= cnt - 1 + ahead && block_key(cnt - 1) + kBlk > q.kv;
      if (tail && !mbar_wait(bar_tail, 0, kWaitLimitNs)) record_status(a.status, kStatusTimeout);
      drain_loads(bar_full, issued, S, a.status);
    }
  } else if (warp >= kMma) {
    // ------------------------------------------------------------ MMA issue
    if (cnt > 0) {
      constexpr uint32_t kIdS = idesc_f16kind(kTile, kBlk, false, kFmt);  // 128 x 64, B K-major
      constexpr uint32_t kIdO = idesc_f16kind(kTile, kD, true, kFmt);     // 128 x D, B MN-major
      constexpr uint32_t lbo_mn = ((uint32_t)kKVPanel >> 4) << 16;        // V's panel stride along D
      const int st = warp - kMma;
      const uint32_t leader = elect_leader();
      const Range r = range_of(st);
      const int left = r.count;
      const uint32_t q_lo = (smem_u32(sQ + (alternate ? 0 : st) * LL::kQBytes) >> 4) | (1u << 16);
      const uint32_t ring_lo = smem_u32(sStage) >> 4;
      const uint32_t s_base = tmem + 2 * kBlk * st, o_base = tmem + kColO + kD * st;
      int asked = 0, done = 0;   // blocks whose scores, whose P V are issued
      int stage = 0, phase = 0;  // of the ring
      bool ok = wt.wait_warp(bar_q, 0);
      for (int n = -ahead; n < cnt && ok; ++n) {
        const bool pv = n >= 0 && r.has(n), sc = n + ahead < cnt && r.has(n + ahead);
        // (an item that only the other stream uses is released once it is
        // there, so that this stream stays within a ring of the other)
        ok = wt.wait_warp(bar_full + stage, phase);
        if (!ok) break;
        const uint32_t v_lo = ring_lo + stage * (LL::kStageBytes >> 4);
        if (pv) {  // O += P V of block n
          ok = wt.wait_warp(bar_p + 2 * st + (done & 1), (done >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t p_col = s_base + kBlk * (done & 1);
#pragma unroll
          for (int kk = 0; kk < kBlk / 16; ++kk)
            mma_ts_if(leader, o_base, p_col + kk * 8, desc_from((v_lo | lbo_mn) + kk * (16 * LL::kRowBytes >> 4), kDescHi),
                      kIdO, (done > 0 || kk > 0) ? 1u : 0u);
          ++done;
          if (done >= left - 1) tc_commit_if(leader, done == left ? bar_o + st : bar_pv + st);
        }
        if (sc) {  // the scores of block n + ahead
          tc_fence_after();
          const uint32_t k_lo = (v_lo + (LL::kHalf >> 4)) | (1u << 16);
          const uint32_t s_col = s_base + kBlk * (asked & 1);
#pragma unroll
          for (int pn = 0; pn < kPanels; ++pn)
#pragma unroll
            for (int kk = 0; kk < LL::kPanelElems / 16; ++kk)
              mma_ss_if(leader, s_col, desc_from(q_lo + pn * (kQPanel >> 4) + kk * 2, kDescHi),
                        desc_from(k_lo + pn * (kKVPanel >> 4) + kk * 2, kDescHi), kIdS, (pn > 0 || kk > 0) ? 1u : 0u);
          tc_commit_if(leader, bar_s + 2 * st + (asked & 1));
          ++asked;
        }
        if (pv || sc)
          tc_commit_if(leader, bar_empty + stage);
        else
          mbar_arrive_if(leader, bar_empty + stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
      // drain: all issued MMAs complete before TMEM is released
      tc_commit_if(leader, bar_drain);
      if (!mbar_wait(bar_drain, 0, kWaitLimitNs)) record_status(a.status, kStatusTimeout);
    }
  } else {
    // ------------------------------------------------------------ softmax and epilogue
    const int st = warp >> 2;
    const int row = 32 * (warp & 3) + lane;  // TMEM lane = tile row
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t o_col = tmem + lane_base + kColO + kD * st;
    const int ta = tok_begin(st), tb = tok_end(st);
    const int i = ta + row / a.G;
    const bool row_ok = row < tpt * a.G && i < tb;
    const int pos = row_ok ? q.first + i : -1;
    const int x_lo = q.first + ta, x_hi = q.first + tb - 1;
    const uint64_t sc2 = f32x2(a.scale_log2, a.scale_log2);
    const Range r = range_of(st);
    const int left = r.count;
    float m_use = -INFINITY, l_run = 0.f;
    int done = 0;
    bool ok = true;
    // Scores of block n from TMEM, what the row does not see at -inf.
    auto take = [&](int n, int k, uint32_t(&x)[kBlk]) {
      const uint32_t s_col = tmem + lane_base + kBlk * (2 * st + (k & 1));
      ok = wt.wait_warp(bar_s + 2 * st + (k & 1), (k >> 1) & 1);
      if (!ok) return;
      tc_fence_after();
      LN_TMEM_LD32(s_col, (x + 0));
      LN_TMEM_LD32(s_col + 32, (x + 32));
      tmem_wait_ld();
      const int j0 = block_key(n);
      // a block that some row of the tile does not see whole
      if (j0 + kBlk - 1 > x_lo || (a.window && x_hi - j0 >= a.window && j0 + kBlk > a.sinks) || !row_ok) {
        const int hi = pos - j0, lo = a.window ? hi - a.window + 1 : -1, sk = a.sinks - j0;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t keep = below(hi + 1 - 32 * w) & (~below(lo - 32 * w) | below(sk - 32 * w));
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((keep >> c) & 1)) x[32 * w + c] = __float_as_uint(-INFINITY);
        }
      }
    };
    auto maximum = [&](const uint32_t(&x)[kBlk]) -> float {
      float pm[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pm[e] = max3(__uint_as_float(x[e]), __uint_as_float(x[e + 4]), __uint_as_float(x[e + 8]));
#pragma unroll
      for (int c = 12; c + 8 <= kBlk; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          pm[e] = max3(pm[e], __uint_as_float(x[c + e]), __uint_as_float(x[c + e + 4]));
#pragma unroll
      for (int e = 0; e < 4; ++e) pm[e] = fmaxf(pm[e], __uint_as_float(x[kBlk - 4 + e]));
      return max3(fmaxf(pm[0], pm[1]), pm[2], pm[3]) * a.scale_log2;
    };
    uint32_t x[kBlk], pk[32];
    for (int n = r.begin; n < r.end; n += r.step) {
      take(n, done, x);
      if (!ok) break;
      const float m_blk = maximum(x);
      float corr = 1.f;
      if (m_blk > m_use + 8.f) {  // also from -inf, the first visible key
        corr = ex2(m_use - m_blk);
        m_use = m_blk;
      }
      // P = 2^(s scale - m + kUp), packed over the buffer's first 32 columns
      const float base = m_use == -INFINITY ? 0.f : m_use - kUp<kFmt>;  // a row with nothing to see so far
      const uint64_t nm2 = f32x2(-base, -base);
      uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        float xa, xb;
        f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, nm2), xa, xb);
        const float pa = ex2(xa), pb = ex2(xb);
        ls[c & 3] = add_f32x2(ls[c & 3], f32x2(pa, pb));
        pk[c] = pack2<kFmt>(pa, pb);
      }
      if (done > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
        // O holds the products up to the block before, the latest that may
        // still run: it is done when the next block's scores are, which were
        // issued after it
        ok = done + 1 < left ? wt.wait_warp(bar_s + 2 * st + ((done + 1) & 1), ((done + 1) >> 1) & 1)
                             : wt.wait_warp(bar_pv + st, 0);
        if (!ok) break;
        tc_fence_after();
        l_run *= corr;
        constexpr int kChunk = kD < 32 ? kD : 32;
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += kChunk) {
          uint32_t rr[kChunk];
          tmem_load<kChunk>(o_col + c0, rr);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kChunk; ++c) rr[c] = __float_as_uint(__uint_as_float(rr[c]) * corr);
          tmem_store<kChunk>(o_col + c0, rr);
        }
      }
      LN_TMEM_ST32(tmem + lane_base + kBlk * (2 * st + (done & 1)), pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_p + 2 * st + (done & 1));
      float t0s, t1s;
      f32x2_split(add_f32x2(add_f32x2(ls[0], ls[1]), add_f32x2(ls[2], ls[3])), t0s, t1s);
      l_run += t0s + t1s;
      ++done;
    }
    if (ok && done > 0) ok = wt.wait_warp(bar_o + st, 0);
    // (a tile that met no block is still written below: not before its load landed)
    if (ok && cnt > 0) ok = wt.wait_warp(bar_q, 0);
    if (ok && ta < tb) {
      tc_fence_after();
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // (a sum of NaN stays one)
      const int h = f * a.G + row % a.G;
      const bool whole = !kPaged || (!alternate && pieces == 1);
      const int64_t prow = ((int64_t)slot * 2 + st) * plan.slot_rows + row;
      if (!whole && kD >= 64 && !alternate) {
        if constexpr (kD >= 64)  // (a slot has 128 rows of this stream)
          store_rows_f32<kD>(sQ + st * LL::kQBytes, o_col, done > 0, inv, 32 * (warp & 3), lane,
                             plan.part_out + prow * kD);
      } else if (!whole) {
        constexpr int kChunk = kD < 32 ? kD : 32;
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += kChunk) {
          uint32_t rr[kChunk];
          if (done > 0) {
            tmem_load<kChunk>(o_col + c0, rr);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < kChunk; ++c) rr[c] = 0;
          }
          if (row_ok) {
            float4* o = reinterpret_cast<float4*>(plan.part_out + prow * kD + c0);
#pragma unroll
            for (int c = 0; c < kChunk; c += 4)
              o[c / 4] = make_float4(__uint_as_float(rr[c]) * inv, __uint_as_float(rr[c + 1]) * inv,
                                     __uint_as_float(rr[c + 2]) * inv, __uint_as_float(rr[c + 3]) * inv);
          }
        }
      } else {
        // this tile's queries are read: its last product is done
        store_rows<kFmt, kD>(sQ + st * LL::kQBytes, o_col, done > 0, inv, 32 * (warp & 3), lane,
                             static_cast<uint16_t*>(a.out) + ((q.q0 + i) * a.H + h) * (int64_t)kD, row_ok);
      }
      if (row_ok) {
        const float lse2 = l_run == 0.f ? -INFINITY : m_use - kUp<kFmt> + log2f(l_run);
        if (!whole)
          plan.part_lse[prow] = lse2;
        else if (a.lse)
          a.lse[lse_index(a, q, s, i, h)] = lse2 * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the pieces of every row: out = sum_p 2^(lse_p - m) O_p / sum_p 2^(lse_p - m).
// A block per 32 rows of an item and head, a warp per row; a row's pieces (each
// with both streams' halves when they alternate) are added in order.
template <int kFmt, int kD>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnArgs a, const Plan plan) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x / a.Hkv, f = blockIdx.x % a.Hkv;
  const int pieces = plan.base[item + 1] - plan.base[item];
  if (pieces == 0 || (!plan.alternate && pieces == 1)) return;  // no rows, or written by their CTA
  const int s = item / plan.pairs, t0 = (item % plan.pairs) * 2 * plan.tokens;
  const Seq q = seq_of(a, s);
  const int halves = plan.alternate ? 2 : 1, parts = halves * pieces;
  const int64_t first = (int64_t)plan.base[item] * a.Hkv + f * pieces;
  const int tokens = (2 / halves) * plan.tokens < q.nq - t0 ? (2 / halves) * plan.tokens : q.nq - t0;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < tokens * a.G; r += gridDim.y * 8) {
    const int in = r / a.G, g = r % a.G, st = in / plan.tokens, i = t0 + in, h = f * a.G + g;
    const int at = (in - st * plan.tokens) * a.G + g;
    auto row_of = [&](int p) {  // of part p: piece p / halves
      return ((first + p / halves) * 2 + (halves == 2 ? (p & 1) : st)) * plan.slot_rows + at;
    };
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, plan.part_lse[row_of(p)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    constexpr int kE = kD / 32 > 0 ? kD / 32 : 1;  // values of a lane
    const bool on = lane * kE < kD;
    float acc[kE] = {}, sum = 0.f;
    for (int p0 = 0; p0 < parts; p0 += 32) {
      const float wl = p0 + lane < parts ? ex2(plan.part_lse[row_of(p0 + lane)] - base) : 0.f;
      const int n = parts - p0 < 32 ? parts - p0 : 32;
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        const float w = __shfl_sync(0xffffffffu, wl, p);
        sum += w;
        if (on) {
          const float* src = plan.part_out + row_of(p0 + p) * kD + lane * kE;
          float t[kE];
          if constexpr (kE == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            t[0] = v.x;
            t[1] = v.y;
            t[2] = v.z;
            t[3] = v.w;
          } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) t[e] = src[e];
          }
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[e] = fmaf(w, t[e], acc[e]);
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (on) {
      uint16_t* o = static_cast<uint16_t*>(a.out) + ((q.q0 + i) * a.H + h) * (int64_t)kD + lane * kE;
      if constexpr (kE == 1) {
        o[0] = (uint16_t)pack2<kFmt>(acc[0] * inv, 0.f);
      } else {
#pragma unroll
        for (int e = 0; e < kE; e += 2)
          *reinterpret_cast<uint32_t*>(o + e) = pack2<kFmt>(acc[e] * inv, acc[e + 1] * inv);
      }
    }
    if (lane == 0 && a.lse) a.lse[lse_index(a, q, s, i, h)] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
  }
}

template <int kFmt, int kD>
int launch_typed(const AttnArgs& a, const Plan& plan, cudaStream_t stream) {
  using LL = L<kD>;
  Maps maps;
  EncodeTiledFn enc = get_encoder();
  if (!enc) return LONGNET_ERR_CUDA;
  if (!encode_q(enc, &maps.m[0], a.q, a, plan.tokens) || !encode_kv(enc, &maps.m[1], a.k, a, kBlk) ||
      !encode_kv(enc, &maps.m[2], a.v, a, kBlk))
    return LONGNET_ERR_CUDA;
  if (!(a.cu_q ? opt_in_smem<fwd_kernel<kFmt, kD, true>>(LL::kSmem) : opt_in_smem<fwd_kernel<kFmt, kD, false>>(LL::kSmem)))
    return LONGNET_ERR_CUDA;
  auto fn = a.cu_q ? fwd_kernel<kFmt, kD, true> : fwd_kernel<kFmt, kD, false>;
  const dim3 grid = plan.items ? dim3((unsigned)plan.grid) : dim3((unsigned)plan.pairs, (unsigned)(a.S * a.Hkv));
  int rc = launch_after(fn, grid, kThreads, LL::kSmem, stream, a, maps, plan);
  if (rc || !plan.items) return rc;
  // four rows a warp, at most
  const int rows = (plan.alternate ? a.nq_max : 2 * plan.tokens) * a.G;
  return launch_after(join_kernel<kFmt, kD>, dim3((unsigned)(plan.items * a.Hkv), (unsigned)((rows + 31) / 32)), 256, 0,
                      stream, a, plan);
}

}  // namespace wt

bool window_tc_supports(const AttnArgs& a) {
  return (a.dtype == LONGNET_DTYPE_BF16 || a.dtype == LONGNET_DTYPE_F16) && a.G <= wt::kTile;
}

#define LN_TC_BY(FN, ...)                                                                              \
  (a.dtype == LONGNET_DTYPE_F16                                                                        \
       ? (a.D == 16 ? FN<tc::kFmtF16, 16>(__VA_ARGS__) : a.D == 32 ? FN<tc::kFmtF16, 32>(__VA_ARGS__)   \
          : a.D == 64 ? FN<tc::kFmtF16, 64>(__VA_ARGS__) : FN<tc::kFmtF16, 128>(__VA_ARGS__))           \
       : (a.D == 16 ? FN<tc::kFmtBF16, 16>(__VA_ARGS__) : a.D == 32 ? FN<tc::kFmtBF16, 32>(__VA_ARGS__) \
          : a.D == 64 ? FN<tc::kFmtBF16, 64>(__VA_ARGS__) : FN<tc::kFmtBF16, 128>(__VA_ARGS__)))

// A contiguous call is never cut along the keys (its row tiles fill the GPU,
// and training sequences are of one length); a paged one is when its row tiles
// would not keep every SM busy twice over.
WindowTcPlan window_tc_plan(const AttnArgs& a) {
  WindowTcPlan p;
  memset(&p, 0, sizeof(p));
  p.tokens = wt::kTile / a.G;
  p.alternate = a.cu_q && a.nq_max <= p.tokens && a.S <= wt::kMaxItems;
  p.pairs = p.alternate ? 1 : (int)(((int64_t)a.nq_max + 2 * p.tokens - 1) / (2 * p.tokens));
  const int64_t items = (int64_t)p.pairs * a.S;
  if (!a.cu_q || items > wt::kMaxItems || (!p.alternate && items * a.Hkv >= 2 * wt::kSms)) return p;
  p.items = (int)items;
  p.grid = (int)(items * a.Hkv > wt::kSms ? items * a.Hkv : wt::kSms);
  p.slot_rows = p.alternate ? a.nq_max * a.G : wt::kTile;
  return p;
}

namespace {
int64_t round64(int64_t floats) { return (floats + 63) / 64 * 64; }  // 256 bytes
}  // namespace

int64_t window_tc_part_floats(const AttnArgs& a, const WindowTcPlan& p) {
  if (!p.items) return 0;
  const int64_t rows = (int64_t)p.grid * 2 * p.slot_rows;
  return round64(p.items + 1) + round64(rows) + round64(rows * a.D);
}

int launch_window_fwd_tc(const AttnArgs& a, float* workspace, cudaStream_t stream) {
  WindowTcPlan p = window_tc_plan(a);
  if (p.items) {
    p.base = reinterpret_cast<int*>(workspace);
    p.part_lse = workspace + round64(p.items + 1);
    p.part_out = p.part_lse + round64((int64_t)p.grid * 2 * p.slot_rows);
  }
  return LN_TC_BY(wt::launch_typed, a, p, stream);
}

}  // namespace longnet
