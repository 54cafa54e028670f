// The backward of the sliding-window attention on the tensor cores (tcgen05),
// bf16 and fp16, D = 16, 32, 64 or 128.
//
// Mathematics.  With P = e^{s - lse} and delta = <dout, out>, dS = P (dout V^T -
// delta):
//   dV = P^T dout, dK = dS^T Q / sqrt(D), dQ = dS K / sqrt(D).
// P and dS are computed in fp32 and rounded to the input format for their
// products (the tensor cores take 16-bit operands); every sum is fp32 and each
// gradient is rounded once, when it is written.  Two measures against what the
// roundings cost:
//   - delta from the forward's out carries that tensor's rounding, which shows
//     in dS where few keys are seen (and dout V^T - delta nearly cancels).  Up
//     to kExactKeys visible keys, delta is summed as P dout V^T in fp32 instead,
//     by a first pass over the same blocks (relative error of dq and dk at a
//     window of 64: 2.6e-3 -> 2.4e-3, where the plain 32-bit form rounded once has
//     1.7e-3).  Beyond, the rounding is left where it shows most: with values whose
//     mean is five times their spread, 900 keys, bf16: 1.4e-2 in dq, 1.0e-2 in dk;
//   - in fp16, P is rounded as 2^8 P, since a weight of one in thousands of keys
//     is below that format's normal range; dV is scaled back at the end.  And dS
//     is rounded as 2^e dS, where gradients may be of any size: e is such that
//     2^15 >= 2^e 2 max |dout_x| max |v_j| >= |2^e dS| (the norms' maxima are found by the
//     pass that makes delta, or one of its own: launch_window_peaks); dQ and dK
//     are scaled back at the end.  (dk of 4096 tokens, window 2048, D = 64, dout
//     of 1e-4: relative error 1.5e-2 without, 2.7e-3 with, which is the exact
//     gradient's own rounding.)
//
// Design.  Two kernels, so that no gradient row is summed by two CTAs and no
// atomics are needed (the same bits every run), at the price of computing the
// two score products twice (7 products instead of 5):
//   key-centric    a CTA holds tiles of 128 keys (K, V) and streams 64-row
//                  blocks of packed query rows (Q, dout, lse, delta):
//                  S^T = K Q^T, dP^T = V dout^T, then dV += P^T dout and
//                  dK += dS^T Q with P^T and dS^T read from TMEM.  The block's
//                  rows are 64 / G tokens by the G query heads that share the
//                  keys, so shared heads sum in the accumulators.
//   query-centric  a CTA holds two tiles of 128 packed query rows (Q, dout) and
//                  streams 64-key blocks (K, V): S, dP, then dQ += dS K.  Where
//                  delta takes a pass of its own it runs first; else delta
//                  comes from its own kernel, and both run as one launch.
// Two score slots (S and dP, 64 columns each) in TMEM, each with two compute
// warpgroups, one for each half of a block's columns: no row statistic is
// shared between columns, so a block's scores are worked off by 256 threads.
// Query-centric, and key-centric up to D = 64, a slot belongs to one of two tiles
// that share every streamed block; key-centric at D = 128 the accumulators of
// one tile fill the rest of TMEM, and the slots take alternate blocks.
// What the tiles' tensor work must not wait for is the arithmetic on the block
// before.  So S of the next block is issued as soon as this one's scores are in
// registers; P and dS go over dP's columns, and dP of the next block follows the
// products that read them.  Query-centric up to D = 64 TMEM has room for dS
// beside the scores, and dP comes early as well.  (All after the products of
// the block before, with half the warps: 274 us for the step of 8192 tokens, 12/4
// heads of 64, against 240; 1222 against 1093 for 16384 tokens, 8 heads of 128.)
// The compute warps are held up by what they read from shared memory: a column's
// -lse and -delta, the same for all 32 lanes, cost a load's full bandwidth (512
// bytes of registers for 16).  Key-centric up to D = 64 they are therefore added
// by the tensor cores: the tiles get a further 16 operand columns, constants,
// and the blocks three parts of each number in the input format, which makes
// the scores s - lse / scale and dP - delta (three_parts: what the parts hold).
// Warps 0-15 compute (slot 0, slot 1, and the same for the other half), warp 16
// loads (TMA; its lanes fetch lse and delta), warps 17 and 18 issue, one for each
// tile (one tile: warp 17 alone, as both slots add to the same accumulators).  Every wait is bounded.
// Bound: query-centric the exponentials' unit while the compute warps work (1024
// cycles of the 1950 that a block takes both tiles at D = 64), key-centric the
// products, whose 64-row blocks make the tensor cores read a tile again for every
// 64 columns (tensor cores at work 30 and 42 % of the cycles at D = 64, 53 and 52 %
// at D = 128).  Turns of the two tiles at the arithmetic, which kept their
// exponentials apart, were slower (240 -> 307 us).  Measured, both kernels: 8192
// tokens, 12/4 heads of 64, window 1024: 148 us and 7 for delta; 16384 tokens, 8 heads of 128, window
// 4096, fp16: 775 us (1088 TFLOP/s of the seven products), in one launch.  608 threads
// leave each 96 registers; at D = 128 the one launch spills 72 bytes of stores and 152
// of loads a thread in bf16, 24 and 36 in fp16.
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
namespace wb {
using namespace wt;

constexpr int kThreads = 608;
constexpr int kTma = 16, kMma = 17;  // warps
constexpr int kBlk = 64;           // streamed rows
constexpr uint32_t kTmemCols = 512, kColAcc = 256, kColDs = 384;

template <int kD, bool kKeys>
struct B : Panels<kD> {
  using P = Panels<kD>;
  static constexpr int kTiles = kKeys && kD > 64 ? 1 : 2;
  static constexpr int kTileBytes = kTile * kD * 2;
  static constexpr int kBlkBytes = kBlk * kD * 2;
  // Key-centric up to D = 64, -lse and -delta come into the scores as one more
  // step of the products (kFold), from extra operand columns; at D = 128 the
  // compute warps add them from shared memory.
  static constexpr bool kFold = kKeys && kD <= 64;
  // Query-centric up to D = 64, TMEM has room for dS beside the scores (two
  // buffers a tile): both products of the next block run during this one's.
  static constexpr bool kBeside = !kKeys && kD <= 64;
  static constexpr int kFoldBytes = kFold ? 2 * kTile * 32 : 0;  // the extra columns of K's and of V's tiles: 128 rows of 16
  static constexpr int kStageBytes = 2 * kBlkBytes + (kFold ? 2 * kBlk * 32 : kKeys ? 1024 : 0);  // two blocks, then these
  static constexpr int kStages = kD == 128 ? (kKeys ? 4 : 3) : 6;
  static constexpr int kStage0 = kTiles * 2 * kTileBytes;
  static constexpr int kFold0 = kStage0 + kStages * kStageBytes;
  static constexpr int kBars = kFold0 + kFoldBytes;
  // one CTA per SM at every D: its TMEM columns are all of the SM's
  static constexpr int kSmem = kBars + 512 + 1024 > 120 * 1024 ? kBars + 512 + 1024 : 120 * 1024;
};

struct __align__(64) BMaps {
  CUtensorMap t[2], b[2];  // the tiles' two tensors, the blocks' two
};

constexpr int kExactKeys = 512;

struct BPlan {
  int tokens;    // of a tile (query-centric) or of a block (key-centric)
  int exact;     // query-centric: delta by a pass of its own (else it is there)
  int peaks;     // fp16: blocks that left their rows' largest norms in g.peaks
  KeyPlan key;
};

struct Run {
  int begin, end, step, count;
  __device__ __forceinline__ bool has(int n) const { return n >= begin && n < end; }  // of a run of step 1
};

// P and dS of 32 streamed rows for this thread's tile row, packed in pairs:
// P = 2^(s scale log2(e) - lse log2(e)), dS = P (dP - delta); 0 where keep has
// no bit.  In fp16, dS comes times the call's unit 2^e; key-centric, P is 2^8 P
// (its lse says so), so that 2^e dS is 2^8 P times 2^(e-8) (dP - delta).
template <int kFmt>
constexpr float kPScale = kFmt == kFmtF16 ? 256.f : 1.f;

// 2^e from the largest |dout_x|^2 and |v_j|^2: |dP| <= B = |dout_x| |v_j| < 2^k, and
// delta, a mean of dP, too, so e = 14 - k keeps 2^e (dP - delta) within 2^15.  (1
// when there is nothing to scale.)
__device__ __forceinline__ float grad_unit(float dout2, float v2) {
  const float b2 = dout2 * v2;  // of fp16 values: 0 or from 2^-96 to 2^79
  if (b2 == 0.f) return 1.f;
  const int k = (((int)(__float_as_uint(b2) >> 23) - 127) >> 1) + 1;
  return __uint_as_float((uint32_t)(127 + 14 - k) << 23);
}

// x as three parts of the input format whose sum, times the tiles' constant, is
// x: by is 1 / constant.  bf16, constant 1: to 2^-24 of x.  fp16: to 2^-33 of x, or
// 2^-25 of the constant where that is more.  For lse / scale the constant is 256,
// which keeps |x| up to 1.6e7 in range and |x| to 1e-5; for delta it is 2^-e, as
// far as fp16 has it, which leaves parts of at most 2^15 and an error of 2^-39 of
// the largest |dP| there may be.
constexpr float kLseUnit = 256.f;
template <int kFmt>
__device__ __forceinline__ uint4 three_parts(float x, float by) {
  x *= by;
  float hi, mid, none;
  unpack2<kFmt>(pack2<kFmt>(x, 0.f), hi, none);
  unpack2<kFmt>(pack2<kFmt>(x - hi, 0.f), mid, none);
  return make_uint4(pack2<kFmt>(hi, mid), pack2<kFmt>(x - hi - mid, 0.f), 0u, 0u);
}
// Byte of 16-byte chunk c of row r of the extra columns (32-byte rows and swizzle).
__device__ __forceinline__ int fold_at(int r, int c) { return r * 32 + ((c ^ ((r >> 2) & 1)) << 4); }

// The same with -lse and -delta already in sr (times the softmax scale) and dr.
// up2: 2^(e-8) in fp16, twice.
template <int kFmt, bool kMask>
__device__ __forceinline__ void p_ds_folded(const uint32_t (&sr)[32], const uint32_t (&dr)[32], uint64_t sc2,
                                            uint64_t up2, uint32_t keep, uint32_t (&pk)[16], uint32_t (&dk)[16]) {
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float x0, x1;
    const uint64_t s2 = f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
    // fp16: 2^8 P
    f32x2_split(kPScale<kFmt> == 1.f ? mul_f32x2(s2, sc2) : fma_f32x2(s2, sc2, f32x2(8.f, 8.f)), x0, x1);
    float p0 = ex2(x0), p1 = ex2(x1), d0, d1;
    const uint64_t pp = f32x2(p0, p1);
    uint64_t dp = f32x2(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1]));
    if (kFmt == kFmtF16) dp = mul_f32x2(dp, up2);
    f32x2_split(mul_f32x2(pp, dp), d0, d1);
    if (kMask) {
      const bool v0 = (keep >> c) & 1, v1 = (keep >> (c + 1)) & 1;
      p0 = v0 ? p0 : 0.f;
      p1 = v1 ? p1 : 0.f;
      d0 = v0 ? d0 : 0.f;
      d1 = v1 ? d1 : 0.f;
    }
    pk[c / 2] = pack2<kFmt>(p0, p1);
    dk[c / 2] = pack2<kFmt>(d0, d1);
  }
}

// The others, with -lse and -delta of the columns or of the row, delta in fp16
// times up2: key-centric 2^(e-8), query-centric 2^e, twice.
template <int kFmt, bool kKeys, bool kMask>
__device__ __forceinline__ void p_ds_half(const uint32_t (&sr)[32], const uint32_t (&dr)[32], const float* nl_col,
                                          const float* nd_col, uint64_t nl_row, uint64_t nd_row, uint64_t sc2,
                                          uint64_t up2, uint32_t keep, uint32_t (&pk)[16], uint32_t (&dk)[16]) {
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    uint64_t nl[2], nd[2];
    if (kKeys) {
      const float4 l4 = *reinterpret_cast<const float4*>(nl_col + c);
      const float4 d4 = *reinterpret_cast<const float4*>(nd_col + c);
      nl[0] = f32x2(l4.x, l4.y);
      nl[1] = f32x2(l4.z, l4.w);
      nd[0] = f32x2(d4.x, d4.y);
      nd[1] = f32x2(d4.z, d4.w);
    } else {
      nl[0] = nl[1] = nl_row;
      nd[0] = nd[1] = nd_row;
    }
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      float x0, x1;
      f32x2_split(fma_f32x2(f32x2(__uint_as_float(sr[c + e]), __uint_as_float(sr[c + e + 1])), sc2, nl[e / 2]), x0,
                  x1);
      float p0 = ex2(x0), p1 = ex2(x1), d0, d1;
      const uint64_t dp = f32x2(__uint_as_float(dr[c + e]), __uint_as_float(dr[c + e + 1]));
      f32x2_split(mul_f32x2(f32x2(p0, p1), kFmt == kFmtF16 ? fma_f32x2(dp, up2, nd[e / 2]) : add_f32x2(dp, nd[e / 2])),
                  d0, d1);
      if (kMask) {
        const bool v0 = (keep >> (c + e)) & 1, v1 = (keep >> (c + e + 1)) & 1;
        p0 = v0 ? p0 : 0.f;
        p1 = v1 ? p1 : 0.f;
        d0 = v0 ? d0 : 0.f;
        d1 = v1 ? d1 : 0.f;
      }
      if (kKeys) pk[(c + e) / 2] = pack2<kFmt>(p0, p1);
      dk[(c + e) / 2] = pack2<kFmt>(d0, d1);
    }
  }
}

// The work of CTA bx of nx of (batch, key/value head) by.
template <int kFmt, int kD, bool kKeys>
__device__ __forceinline__ void bwd_body(const AttnArgs& a, const WindowBwdArgs& g, const BMaps& maps,
                                         const BPlan& plan, int bx, int nx, int by) {
  using LL = B<kD, kKeys>;
  constexpr int kTiles = LL::kTiles, kPanels = LL::kPanels, S = LL::kStages;
  constexpr int kTilePanel = kTile * LL::kRowBytes, kBlkPanel = kBlk * LL::kRowBytes;
  constexpr uint32_t kDescHi = LL::kDescHi;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // the next launch may be scheduled; and what the one before wrote (key-centric:
  // delta) is read only from here on
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = by / a.Hkv, f = by % a.Hkv;
  const int N = a.nq_max, G = a.G, tok = plan.tokens;
  // ---- the CTA's tiles and the streamed rows
  int first;                // key-centric: first key; query-centric: first token
  int i0 = 0, cnt = 0;      // key-centric: first streamed token; blocks
  int i1 = 0;               // key-centric: end of the streamed tokens
  int slot_no = -1;         // key-centric: the item's slot
  BlockList bl = {0, 0, 0};
  if (kKeys) {
    const KeyItem it = key_item(a, plan.key, bx);
    first = it.tile * kTiles * kTile;
    i0 = it.i0;
    i1 = it.i1;
    slot_no = it.slot;
    cnt = i1 > i0 ? (i1 - i0 + tok - 1) / tok : 0;
  } else {
    first = (nx - 1 - bx) * 2 * tok;  // the longest first
    if (first >= N) return;
    const int end = first + 2 * tok < N ? first + 2 * tok : N;
    bl = blocks_of<kBlk>(a, first, end - 1);
    cnt = bl.count;
  }
  // the blocks of slot st: a run of those streamed, or every second one
  auto run_of = [&](int st) {
    Run r = {0, 0, 1, 0};
    if (kTiles == 1) {
      r = {st, cnt, 2, (cnt + 1 - st) / 2};
      return r;
    }
    if (kKeys) {
      const int jt = first + st * kTile;
      if (jt < N) {
        r.begin = jt > i0 ? (jt - i0) / tok : 0;  // the first with a token at or after the tile's first key
        // and up to the last whose first token's window reaches the tile's last key
        const int64_t reach = (int64_t)jt + kTile - 1 + a.window - i0;
        const int64_t end = jt < a.sinks ? cnt : reach <= 0 ? 0 : (reach + tok - 1) / tok;
        r.end = end < cnt ? (int)end : cnt;
      }
    } else {
      const int t0 = first + st * tok, t1 = t0 + tok < N ? t0 + tok : N;
      if (t0 < t1) {
        // (with sinks, also the few blocks between them and the tile's window
        // that only the other tile sees, all masked)
        const int low = t0 < a.window ? 0 : (t0 - a.window + 1) / kBlk;
        r.begin = a.sinks > 0 ? 0 : bl.n_sink + low - bl.win0;
        r.end = bl.n_sink + (t1 - 1) / kBlk - bl.win0 + 1;
      }
    }
    r.count = r.end > r.begin ? r.end - r.begin : 0;
    return r;
  };

  uint8_t* sStage = smem + LL::kStage0;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LL::kBars);
  uint64_t* bar_tile = bars;
  uint64_t* bar_full = bars + 1;       // [S]
  uint64_t* bar_empty = bars + 1 + S;  // [S]
  uint64_t* bar_s = bars + 1 + 2 * S;  // [2] scores of a slot in TMEM
  uint64_t* bar_p = bar_s + 2;         // [2] P and dS of a slot in TMEM
  uint64_t* bar_acc = bar_s + 4;       // [2] accumulators done
  uint64_t* bar_drain = bar_s + 6;
  uint64_t* bar_ld = bar_s + 7;        // [2] scores of a slot read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_s + 9);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // fp16: the largest norms, by warps; all of it between the set-up's steps, whose
  // waits it shares (numbers from 0 up compare as their bits do)
  uint32_t* s_top = reinterpret_cast<uint32_t*>(smem + LL::kBars + 256);  // [2][warps]
  uint32_t top[2] = {0, 0};
  if constexpr (kFmt == kFmtF16)
    for (int i = threadIdx.x; i < plan.peaks; i += kThreads) {
      const uint2 x = reinterpret_cast<const uint2*>(g.peaks)[i];
      top[0] = max(top[0], x.x);
      top[1] = max(top[1], x.y);
    }
  if (threadIdx.x == 0) {
    mbar_init(bar_tile, 1);
    for (int i = 0; i < S; ++i) {
      mbar_init(bar_full + i, 32);  // the loading warp's lanes, and the TMA bytes
      mbar_init(bar_empty + i, kTiles);  // the issuing warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, 256);
      mbar_init(bar_acc + i, 1);
      mbar_init(bar_ld + i, 256);
    }
    mbar_init(bar_drain, kTiles);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (LL::kFold) {
    // K's tiles' extra columns, three constants and zeros (V's: the loading warp),
    // and the blocks' second chunk of theirs, zeros
    const float c = kFmt == kFmtF16 ? kLseUnit : 1.f;
    const uint32_t one = pack2<kFmt>(c, c);
    for (int e = threadIdx.x; e < kTile * 2; e += kThreads)
      *reinterpret_cast<uint4*>(smem + LL::kFold0 + fold_at(e >> 1, e & 1)) =
          (e & 1) ? make_uint4(0, 0, 0, 0) : make_uint4(one, one & 0xffffu, 0, 0);
    for (int e = threadIdx.x; e < S * 2 * kBlk; e += kThreads)
      *reinterpret_cast<uint4*>(sStage + (e / (2 * kBlk)) * LL::kStageBytes + 2 * LL::kBlkBytes +
                                (e / kBlk % 2) * kBlk * 32 + fold_at(e % kBlk, 1)) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (kKeys && tok * G < kBlk) {
    // rows of a block that no token has: zeros, as the products read them
    const int rows = kBlk - tok * G, chunks = LL::kRowBytes / 16;
    for (int e = threadIdx.x; e < S * 2 * kPanels * rows * chunks; e += kThreads) {
      const int c = e % chunks, r = (e / chunks) % rows, pn = e / chunks / rows;  // pn over stages, blocks, panels
      const int stg = pn / (2 * kPanels);
      *reinterpret_cast<uint4*>(sStage + stg * LL::kStageBytes + (pn % (2 * kPanels)) * kBlkPanel +
                                (tok * G + r) * LL::kRowBytes + c * 16) = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kTma && lane < 4) prefetch_tmap(lane < 2 ? &maps.t[lane] : &maps.b[lane - 2]);
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if constexpr (kFmt == kFmtF16) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, top[w]);
      if (lane == 0) s_top[w * (kThreads / 32) + warp] = m;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  Waiter wt{abort_flag, a.status, kWaitLimitNs};
  float unit = 1.f;  // fp16: the call's 2^e
  if constexpr (kFmt == kFmtF16) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
      top[w] = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? s_top[w * (kThreads / 32) + lane] : 0u);
    unit = grad_unit(__uint_as_float(top[0]), __uint_as_float(top[1]));
  }
  const int passes = !kKeys && plan.exact ? 2 : 1;  // over the blocks; the first of two sums delta
  auto tile_ptr = [&](int st, int which) { return smem + (st * 2 + which) * LL::kTileBytes; };

  if (warp == kTma) {
    // ------------------------------------------------------------ loads
    bool ok = true;
    if (cnt > 0 && lane == 0) {
      const int tiles = kTiles == 2 && first + (kKeys ? kTile : tok) < N ? 2 : 1;
      mbar_arrive_expect_tx(bar_tile,
                            (uint32_t)(tiles * 2 * (kKeys ? LL::kTileBytes : kPanels * tok * G * LL::kRowBytes)));
      for (int st = 0; st < tiles; ++st)
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int pn = 0; pn < kPanels; ++pn)
            tma_load_4d(tile_ptr(st, w) + pn * kTilePanel, &maps.t[w], bar_tile, LL::kPanelElems * pn,
                        kKeys ? f : f * G, first + st * (kKeys ? kTile : tok), s);
    }
    // the constant of delta's parts: 2^-e as far as fp16 holds it, 2^-24 to 2^15
    const float part_unit = kFmt == kFmtF16 ? fminf(fmaxf(1.f / unit, 5.9604645e-8f), 32768.f) : 1.f;
    if (LL::kFold) {  // V's tiles' extra columns, there before the first block is (it arrives after the fence)
      const uint32_t one = pack2<kFmt>(part_unit, part_unit);
      for (int e = lane; e < kTile * 2; e += 32)
        *reinterpret_cast<uint4*>(smem + LL::kFold0 + kTile * 32 + fold_at(e >> 1, e & 1)) =
            (e & 1) ? make_uint4(0, 0, 0, 0) : make_uint4(one, one & 0xffffu, 0, 0);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    // key-centric: -lse (log2 domain) and -delta of a block's rows, fetched a
    // block ahead (their latency would otherwise stand between the loads)
    float l2[2] = {0.f, 0.f}, dl[2] = {0.f, 0.f};
    const int c_tok[2] = {lane / G, (lane + 32) / G}, c_head[2] = {lane % G, (lane + 32) % G};
    // (loaded from a valid address in any case: a load under a condition is
    // waited for where the condition ends)
    auto fetch = [&](int n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = i0 + n * tok + c_tok[e];
        const int64_t idx = ((int64_t)s * a.H + f * G + c_head[e]) * N + (i < N ? i : N - 1);
        l2[e] = a.lse[idx];
        dl[e] = g.delta[idx];
      }
    };
    if (kKeys) fetch(0);
    int issued = 0;
    for (int n = 0; n < passes * cnt && ok; ++n) {
      const int st = n % S;
      if (n >= S) ok = wt.wait_warp(bar_empty + st, ((n / S) - 1) & 1);
      if (!ok) break;
      uint8_t* stage = sStage + st * LL::kStageBytes;
      const int at = kKeys ? i0 + n * tok : bl.at(n < cnt ? n : n - cnt) * kBlk;
      if (lane == 0) {
        mbar_expect_tx(bar_full + st,
                       (uint32_t)(2 * (kKeys ? kPanels * tok * G * LL::kRowBytes : LL::kBlkBytes)));
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int pn = 0; pn < kPanels; ++pn)
            tma_load_4d(stage + w * LL::kBlkBytes + pn * kBlkPanel, &maps.b[w], bar_full + st, LL::kPanelElems * pn,
                        kKeys ? f * G : f, at, s);
      }
      if (LL::kFold) {
        uint8_t* fold = stage + 2 * LL::kBlkBytes;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          *reinterpret_cast<uint4*>(fold + fold_at(lane + 32 * e, 0)) =
              three_parts<kFmt>(-l2[e] / a.scale, kFmt == kFmtF16 ? 1.f / kLseUnit : 1.f);
          *reinterpret_cast<uint4*>(fold + kBlk * 32 + fold_at(lane + 32 * e, 0)) = three_parts<kFmt>(-dl[e], 1.f / part_unit);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      } else if (kKeys) {
        float* sl = reinterpret_cast<float*>(stage + 2 * LL::kBlkBytes);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sl[lane + 32 * e] = fmaf(-l2[e], kLog2e, kFmt == kFmtF16 ? 8.f : 0.f);
          sl[kBlk + lane + 32 * e] = -dl[e] * (unit / kPScale<kFmt>);
        }
      }
      __syncwarp();  // the bytes are expected before the phase can complete
      mbar_arrive(bar_full + st);
      if (kKeys) fetch(n + 1);
      issued = n + 1;
    }
    // drain: every issued load has landed before the CTA may exit
    if (lane == 0) {
      if (cnt > 0 && !mbar_wait(bar_tile, 0, kWaitLimitNs)) record_status(a.status, kStatusTimeout);
      drain_loads(bar_full, issued, S, a.status);
    }
  } else if (warp >= kMma) {
    // ------------------------------------------------------------ MMA issue
    if (cnt > 0 && warp < kMma + kTiles) {
      constexpr uint32_t kIdScore = idesc_f16kind(kTile, kBlk, false, kFmt);  // 128 x 64, B K-major
      constexpr uint32_t kIdGrad = idesc_f16kind(kTile, kD, true, kFmt);      // 128 x D, B MN-major
      constexpr uint32_t lbo_mn = ((uint32_t)kBlkPanel >> 4) << 16;           // panel stride along D
      constexpr uint32_t kStep16 = 16 * LL::kRowBytes >> 4;                   // 16 rows of an MN-major operand
      const int st = warp - kMma;  // the tile
      const uint32_t leader = elect_leader();
      const Run r = run_of(st);
      const uint32_t t_lo[2] = {(smem_u32(tile_ptr(st, 0)) >> 4) | (1u << 16), (smem_u32(tile_ptr(st, 1)) >> 4) | (1u << 16)};
      const uint32_t ring_lo = smem_u32(sStage) >> 4;
      const uint32_t acc = tmem + kColAcc + (kTiles == 2 ? (kKeys ? 2 : 1) * kD * st : 0);
      // product w (0: S, 1: dP) of the block in `stage` into slot `slot`
      auto score = [&](int w, int stage, int slot) {
        const uint32_t b_lo = (ring_lo + stage * (LL::kStageBytes >> 4)) | (1u << 16);
#pragma unroll
        for (int pn = 0; pn < kPanels; ++pn)
#pragma unroll
          for (int kk = 0; kk < LL::kPanelElems / 16; ++kk)
            mma_ss_if(leader, tmem + 128 * slot + 64 * w, desc_from(t_lo[w] + pn * (kTilePanel >> 4) + kk * 2, kDescHi),
                      desc_from(b_lo + w * (LL::kBlkBytes >> 4) + pn * (kBlkPanel >> 4) + kk * 2, kDescHi), kIdScore,
                      (pn > 0 || kk > 0) ? 1u : 0u);
        if (LL::kFold) {
          constexpr uint32_t kHi = (uint32_t)(8 * 32 >> 4) | (1u << 14) | (6u << 29);  // 32-byte rows and swizzle
          const uint32_t fa = (smem_u32(smem + LL::kFold0 + w * kTile * 32) >> 4) | (1u << 16);
          const uint32_t fb = b_lo + (2 * LL::kBlkBytes >> 4);
          mma_ss_if(leader, tmem + 128 * slot + 64 * w, desc_from(fa, kHi), desc_from(fb + w * (kBlk * 32 >> 4), kHi),
                    kIdScore, 1u);
        }
      };
      // the gradient products of item e, in `stage`; P and dS in slot `slot`
      auto grads = [&](int stage, int slot, int e, bool fresh) {
        tc_fence_after();
        const uint32_t b0 = (ring_lo + stage * (LL::kStageBytes >> 4)) | lbo_mn, b1 = b0 + (LL::kBlkBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kBlk / 16; ++kk) {
          const uint32_t add = fresh && kk == 0 ? 0u : 1u;
          // 16 rows' P (8 columns) and, 16 columns on, dS; in each half of dP's columns those of its rows
          const uint32_t p = tmem + 128 * slot + 64 + 32 * (kk >> 1) + 8 * (kk & 1);
          if (kKeys) {
            // dV += P^T dout, dK += dS^T Q
            mma_ts_if(leader, acc, p, desc_from(b1 + kk * kStep16, kDescHi), kIdGrad, add);
            mma_ts_if(leader, acc + kD, p + 16, desc_from(b0 + kk * kStep16, kDescHi), kIdGrad, add);
          } else {
            // dQ += dS K
            const uint32_t d = LL::kBeside ? tmem + kColDs + 64 * slot + 32 * (e & 1) + 8 * kk : p + 16;
            mma_ts_if(leader, acc, d, desc_from(b0 + kk * kStep16, kDescHi), kIdGrad, add);
          }
        }
      };
      bool ok = wt.wait_warp(bar_tile, 0);
      if (kTiles == 2) {
        // Item e (the e-th block of the tile's run, first pass and second): its
        // S is issued as soon as the scores before it are read, its dP then too
        // where dS lies beside them, else after the products that read P and dS
        // in its place.
        const int sums = (passes - 1) * r.count, all = passes * r.count;
        int stage = 0, phase = 0, asked = 0, used = 0, held = -1;  // held: stage of the item asked for and not used
        auto use = [&]() {
          ok = wt.wait_warp(bar_p + st, used & 1);
          if (!ok) return;
          if (used >= sums) {
            grads(held, st, used, used == sums);
            tc_commit_if(leader, bar_empty + held);
            if (used == all - 1) tc_commit_if(leader, bar_acc + st);
          }
          ++used;
          held = -1;
        };
        for (int m = 0; m < passes * cnt && ok; ++m) {
          const bool sum = m < (passes - 1) * cnt;  // the pass for delta
          const int n = m < cnt ? m : m - cnt;
          // (a block that only the other tile uses is released once it is
          // there, so that this warp stays within a ring of the other)
          ok = wt.wait_warp(bar_full + stage, phase);
          if (!ok) break;
          if (r.has(n)) {
            if (asked > 0) ok = wt.wait_warp(bar_ld + st, (asked - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            score(0, stage, st);
            if (LL::kBeside) {
              score(1, stage, st);
              tc_commit_if(leader, bar_s + st);
            }
            if (held >= 0) use();
            if (!ok) break;
            if (!LL::kBeside) {
              score(1, stage, st);
              tc_commit_if(leader, bar_s + st);
            }
            if (sum) tc_commit_if(leader, bar_empty + stage);
            ++asked;
            held = stage;
          } else {
            if (held >= 0) use();
            if (!ok) break;
            mbar_arrive_if(leader, bar_empty + stage);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok && held >= 0) use();
      } else {
        // a block's scores are issued before the P and dS of the one before
        // are waited for
        int stage = 0, before = 0, phase = 0;
        for (int n = 0; n <= cnt && ok; ++n) {
          if (n < cnt) {
            ok = wt.wait_warp(bar_full + stage, phase);
            if (!ok) break;
            tc_fence_after();
            score(0, stage, n & 1);
            score(1, stage, n & 1);
            tc_commit_if(leader, bar_s + (n & 1));
          }
          if (n > 0) {
            ok = wt.wait_warp(bar_p + ((n - 1) & 1), ((n - 1) >> 1) & 1);
            if (!ok) break;
            grads(before, (n - 1) & 1, n - 1, n == 1);
            tc_commit_if(leader, bar_empty + before);
          }
          before = stage;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok) {
          tc_commit_if(leader, bar_acc + 0);
          tc_commit_if(leader, bar_acc + 1);
        }
      }
      // drain: all issued MMAs complete before TMEM is released
      tc_commit_if(leader, bar_drain);
      if (!mbar_wait(bar_drain, 0, kWaitLimitNs)) record_status(a.status, kStatusTimeout);
    }
  } else {
    // ------------------------------------------------------------ P, dS and the epilogue
    const int st = (warp >> 2) & 1, hf = warp >> 3;  // slot, half of the block's columns
    const int row = 32 * (warp & 3) + lane;          // TMEM lane = tile row
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t slot = tmem + lane_base + 128 * st + 32 * hf;
    // key-centric: this thread's key; query-centric: its token and head
    const int j = first + (kTiles == 2 ? st * kTile : 0) + row;
    const int t0 = first + st * tok, i = t0 + row / G, h = f * G + row % G;
    const bool row_ok = kKeys ? j < N : row < tok * G && i < N;
    float lse2 = 0.f, delta = 0.f;
    const int64_t stat = ((int64_t)s * a.H + h) * N + i;  // of lse and delta
    if (!kKeys && row_ok) lse2 = a.lse[stat] * kLog2e;
    if (!kKeys && passes == 1 && row_ok) delta = g.delta[stat];
    const uint64_t sc2 = f32x2(a.scale_log2, a.scale_log2);
    const uint64_t nl_row = f32x2(-lse2, -lse2);
    const Run r = run_of(st);
    int done = 0;
    bool ok = true;
    // query-centric: the columns of this half of block n that the row sees, as bits
    auto seen = [&](int n) {
      const int j0 = bl.at(n) * kBlk + 32 * hf;
      const int hi = row_ok ? i - j0 + 1 : 0, lo = i - j0 - a.window + 1, sk = a.sinks - j0;
      return below(hi) & (~below(lo) | below(sk));
    };
    if (!kKeys && passes == 2) {
      // delta = sum of P dP over the row
      uint64_t acc = 0;
      for (int n = r.begin; n < r.end && ok; ++n) {
        ok = wt.wait_warp(bar_s + st, done & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t keep = seen(n);
        uint32_t sr[32], dr[32];
        LN_TMEM_LD32(slot, sr);
        LN_TMEM_LD32(slot + 64, dr);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(bar_ld + st);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float x0, x1;
          f32x2_split(fma_f32x2(f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc2, nl_row), x0, x1);
          const bool v0 = (keep >> c) & 1, v1 = (keep >> (c + 1)) & 1;
          // (an unseen pair's dP may be anything, where a row is no token's)
          acc = fma_f32x2(f32x2(v0 ? ex2(x0) : 0.f, v1 ? ex2(x1) : 0.f),
                          f32x2(v0 ? __uint_as_float(dr[c]) : 0.f, v1 ? __uint_as_float(dr[c + 1]) : 0.f), acc);
        }
        mbar_arrive(bar_p + st);
        ++done;
      }
      float d0, d1;
      f32x2_split(acc, d0, d1);
      // the other half's sum comes through TMEM, in accumulators not yet in use
      const uint32_t swap = tmem + lane_base + kColAcc + kD * st;
      asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(swap + hf), "f"(d0 + d1) : "memory");
      tmem_wait_st();
      tc_fence_before();
      asm volatile("bar.sync %0, 256;" ::"r"(1 + st) : "memory");  // the slot's two warpgroups, also after a timeout
      tc_fence_after();
      float other;
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(other) : "r"(swap + (hf ^ 1)));
      tmem_wait_ld();
      asm volatile("" : "+f"(other));  // used after the wait only
      tc_fence_before();
      delta = hf ? other + (d0 + d1) : (d0 + d1) + other;
    }
    if (!kKeys && passes == 2 && row_ok && hf == 0) g.delta[stat] = delta;  // the key-centric kernel's
    const uint64_t nd_row = f32x2(-delta * unit, -delta * unit);
    const float up = kKeys ? unit / kPScale<kFmt> : unit;
    const uint64_t up2 = f32x2(up, up);
    for (int n = r.begin; n < r.end && ok; n += r.step) {
      const float* sl = reinterpret_cast<const float*>(sStage + (n % S) * LL::kStageBytes + 2 * LL::kBlkBytes);
      uint32_t keep;  // the half's columns that pair with this row, as bits
      if (kKeys) {
        const int b0 = i0 + n * tok;
        const int n_tok = i1 - b0 < tok ? i1 - b0 : tok;
        const int from = j - b0, to = j + a.window - b0;  // tokens
        const int lo = (from < 0 ? 0 : from > kBlk ? kBlk : from) * G;
        const int hi = (j < a.sinks || to > n_tok ? n_tok : to < 0 ? 0 : to) * G;
        keep = below(hi - 32 * hf) & ~below(lo - 32 * hf);
      } else {
        keep = seen(n);
      }
      if (kKeys && !LL::kFold) ok = wt.wait_warp(bar_full + n % S, (n / S) & 1);  // for what sl holds
      if (ok) ok = wt.wait_warp(bar_s + st, done & 1);
      if (!ok) break;
      tc_fence_after();
      const bool whole = __all_sync(0xffffffffu, keep == 0xffffffffu);
      uint32_t sr[32], dr[32], pk[16], dk[16];
      LN_TMEM_LD32(slot, sr);
      LN_TMEM_LD32(slot + 64, dr);
      tmem_wait_ld();
      if (kTiles == 2) {
        tc_fence_before();
        mbar_arrive(bar_ld + st);
      }
      if (LL::kFold) {
        if (whole)
          p_ds_folded<kFmt, false>(sr, dr, sc2, up2, 0, pk, dk);
        else
          p_ds_folded<kFmt, true>(sr, dr, sc2, up2, keep, pk, dk);
      } else if (whole)
        p_ds_half<kFmt, kKeys, false>(sr, dr, sl + 32 * hf, sl + kBlk + 32 * hf, nl_row, nd_row, sc2, up2, 0, pk, dk);
      else
        p_ds_half<kFmt, kKeys, true>(sr, dr, sl + 32 * hf, sl + kBlk + 32 * hf, nl_row, nd_row, sc2, up2, keep, pk, dk);
      if (kKeys) LN_TMEM_ST16(slot + 64, pk);
      LN_TMEM_ST16(LL::kBeside ? tmem + lane_base + kColDs + 64 * st + 32 * (done & 1) + 16 * hf : slot + 80, dk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_p + st);
      ++done;
    }
    const bool any = kTiles == 2 ? done > 0 : cnt > 0;
    if (ok && any) ok = wt.wait_warp(bar_acc + st, 0);
    // (a tile that met no block is still written below: not before its load landed)
    if (ok && cnt > 0) ok = wt.wait_warp(bar_tile, 0);
    if (ok) {
      tc_fence_after();
      const bool partial = kKeys && slot_no >= 0;
      // key-centric with two tiles: a warpgroup writes both gradients of its
      // tile; with one tile, the first dV and the second dK
#pragma unroll 1
      for (int w = 0; w < (kKeys ? 2 : 1); ++w) {
        if (kTiles == 1 ? w != st || hf : w != hf) continue;
        // w = 0: dV or dQ, w = 1: dK
        const float sc = kKeys && w == 0 ? 1.f / kPScale<kFmt> : a.scale / unit;
        const uint32_t acc = tmem + lane_base + kColAcc + (kTiles == 2 ? (kKeys ? 2 : 1) * kD * st : 0) + w * kD;
        uint16_t* dst = kKeys ? static_cast<uint16_t*>(w == 0 ? g.dv : g.dk) + (((int64_t)s * N + j) * a.Hkv + f) * kD
                              : static_cast<uint16_t*>(g.dq) + (((int64_t)s * N + i) * a.H + h) * kD;
        if (!partial) {
          // through an operand tile that nothing reads any more
          store_rows<kFmt, kD>(tile_ptr(kTiles == 2 ? st : 0, w), acc, any, sc, 32 * (warp & 3), lane, dst, row_ok);
          continue;
        }
        // [S Hkv][slot][dK, dV][tile rows][D]
        float* part = g.partial + (((int64_t)by * plan.key.slots() + slot_no) * 2 + (w == 0 ? 1 : 0)) *
                                      (int64_t)(kTiles * kTile * kD) + (int64_t)(j - first) * kD;
        if constexpr (kD >= 64) {
          store_rows_f32<kD>(tile_ptr(kTiles == 2 ? st : 0, w), acc, any, sc, 32 * (warp & 3), lane, part);
          continue;
        }
        constexpr int kChunk = kD < 32 ? kD : 32;
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += kChunk) {
          uint32_t rr[kChunk];
          if (any) {
            tmem_load<kChunk>(acc + c0, rr);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < kChunk; ++c) rr[c] = 0;
          }
          float4* o = reinterpret_cast<float4*>(part + c0);
#pragma unroll
          for (int c = 0; c < kChunk; c += 4)
            o[c / 4] = make_float4(__uint_as_float(rr[c]) * sc, __uint_as_float(rr[c + 1]) * sc,
                                   __uint_as_float(rr[c + 2]) * sc, __uint_as_float(rr[c + 3]) * sc);
        }
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

template <int kFmt, int kD, bool kKeys>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ WindowBwdArgs g,
               const __grid_constant__ BMaps maps, const __grid_constant__ BPlan plan) {
  bwd_body<kFmt, kD, kKeys>(a, g, maps, plan, blockIdx.x, gridDim.x, blockIdx.y);
}

// Both at once, when delta is there: first the CTAs that take longer, key-centric
// (256 keys by three heads' rows, say) up to D = 64 and query-centric (256 rows
// against 128 keys) at D = 128; the others fill up their last wave.  nq: query-centric
// ones of a (batch, head).  One launch after the other: 240 us for the step of 8192
// tokens, 12/4 heads of 64, against 237; 1093 against 1015 for 16384 tokens, 8 heads of
// 128; 78 against 60 for 1024 tokens, 8 heads of 64, window 600.
template <int kFmt, int kD>
__global__ void __launch_bounds__(kThreads, 1)
    both_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ WindowBwdArgs g,
                const __grid_constant__ BMaps mq, const __grid_constant__ BMaps mk, const __grid_constant__ BPlan pq,
                const __grid_constant__ BPlan pk, int nq) {
  const int nk = pk.key.items(), first = (kD > 64 ? nq : nk) * a.S * a.Hkv;
  const bool head = (int)blockIdx.x < first;
  const int x = head ? blockIdx.x : blockIdx.x - first;
  if (head == (kD > 64))
    bwd_body<kFmt, kD, false>(a, g, mq, pq, x % nq, nq, x / nq);
  else
    bwd_body<kFmt, kD, true>(a, g, mk, pk, x % nk, nk, x / nk);
}

// Query rows [B, N, H, D] as (d, h, token, batch): a box is one panel of G
// heads by `tokens` tokens.
bool encode_rows(EncodeTiledFn enc, CUtensorMap* map, const void* base, const AttnArgs& a, int tokens) {
  const cuuint64_t row = (cuuint64_t)a.D * 2;
  cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.H, (cuuint64_t)a.nq_max, (cuuint64_t)a.S};
  cuuint64_t strides[3] = {row, row * a.H, row * a.H * a.nq_max};
  const int pe = a.D >= 64 ? 64 : a.D;
  cuuint32_t box[4] = {(cuuint32_t)pe, (cuuint32_t)a.G, (cuuint32_t)tokens, 1};
  cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, a.dtype == LONGNET_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             pe == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
             : pe == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                        : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kFmt, int kD>
int launch_typed(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return LONGNET_ERR_CUDA;
  constexpr bool kF16 = kFmt == kFmtF16;
  BPlan pk, pq;
  pk.tokens = kBlk / a.G;
  pq.tokens = kTile / a.G;
  pk.exact = pk.peaks = pq.peaks = 0;
  pq.exact = (int64_t)a.window + a.sinks <= kExactKeys || a.nq_max <= kExactKeys;
  using LK = B<kD, true>;
  using LQ = B<kD, false>;
  pk.key = pq.key =
      key_plan(a.S, a.nq_max, a.H, a.Hkv, a.window, a.sinks, LK::kTiles * kTile, kTcMinBlocks, kTcCtas);
  BMaps mk, mq;
  if (!encode_kv(enc, &mk.t[0], a.k, a, kTile) || !encode_kv(enc, &mk.t[1], a.v, a, kTile) ||
      !encode_rows(enc, &mk.b[0], a.q, a, pk.tokens) || !encode_rows(enc, &mk.b[1], g.dout, a, pk.tokens) ||
      !encode_rows(enc, &mq.t[0], a.q, a, pq.tokens) || !encode_rows(enc, &mq.t[1], g.dout, a, pq.tokens) ||
      !encode_kv(enc, &mq.b[0], a.k, a, kBlk) || !encode_kv(enc, &mq.b[1], a.v, a, kBlk))
    return LONGNET_ERR_CUDA;
  if (!opt_in_smem<bwd_kernel<kFmt, kD, true>>(LK::kSmem) || !opt_in_smem<bwd_kernel<kFmt, kD, false>>(LQ::kSmem))
    return LONGNET_ERR_CUDA;
  const int64_t pairs = ((int64_t)a.nq_max + 2 * pq.tokens - 1) / (2 * pq.tokens);
  if (!pq.exact) {
    if ((pairs + pk.key.items()) * a.S * a.Hkv > INT32_MAX) return LONGNET_ERR_UNSUPPORTED;
    int rc = kF16 ? launch_window_peaks(a, g, true, &pk.peaks, stream) : launch_window_delta(a, g, stream);
    if (rc) return rc;
    pq.peaks = pk.peaks;
    constexpr int smem = LK::kSmem > LQ::kSmem ? LK::kSmem : LQ::kSmem;
    if (!opt_in_smem<both_kernel<kFmt, kD>>(smem)) return LONGNET_ERR_CUDA;
    rc = launch_after(both_kernel<kFmt, kD>, dim3((unsigned)((pairs + pk.key.items()) * a.S * a.Hkv)), kThreads,
                      smem, stream, a, g, mq, mk, pq, pk, (int)pairs);
    return rc ? rc : launch_key_reduce(a, g, pk.key, stream);
  }
  int rc = kF16 ? launch_window_peaks(a, g, false, &pk.peaks, stream) : LONGNET_OK;
  if (rc) return rc;
  pq.peaks = pk.peaks;
  // dq first: it leaves delta for dk and dv
  rc = launch_after(bwd_kernel<kFmt, kD, false>, dim3((unsigned)pairs, (unsigned)(a.S * a.Hkv)), kThreads, LQ::kSmem,
                        stream, a, g, mq, pq);
  if (rc) return rc;
  rc = launch_after(bwd_kernel<kFmt, kD, true>, dim3((unsigned)pk.key.items(), (unsigned)(a.S * a.Hkv)), kThreads, LK::kSmem,
                    stream, a, g, mk, pk);
  if (rc) return rc;
  return launch_key_reduce(a, g, pk.key, stream);
}

}  // namespace wb

// Shared groups of up to 64 heads: a token's rows fit one streamed block.
bool window_bwd_tc_supports(const AttnArgs& a) {
  return (a.dtype == LONGNET_DTYPE_BF16 || a.dtype == LONGNET_DTYPE_F16) && a.G <= wb::kBlk;
}
int window_bwd_tc_tile(int64_t D) { return (D > 64 ? 1 : 2) * wt::kTile; }

int launch_window_bwd_tc(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream) {
  const bool f16 = a.dtype == LONGNET_DTYPE_F16;
  switch (a.D) {
    case 16:
      return f16 ? wb::launch_typed<tc::kFmtF16, 16>(a, g, stream) : wb::launch_typed<tc::kFmtBF16, 16>(a, g, stream);
    case 32:
      return f16 ? wb::launch_typed<tc::kFmtF16, 32>(a, g, stream) : wb::launch_typed<tc::kFmtBF16, 32>(a, g, stream);
    case 64:
      return f16 ? wb::launch_typed<tc::kFmtF16, 64>(a, g, stream) : wb::launch_typed<tc::kFmtBF16, 64>(a, g, stream);
    default:
      return f16 ? wb::launch_typed<tc::kFmtF16, 128>(a, g, stream) : wb::launch_typed<tc::kFmtBF16, 128>(a, g, stream);
  }
}

}  // namespace longnet
