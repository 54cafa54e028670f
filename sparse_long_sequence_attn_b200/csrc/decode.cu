// Attention of few new tokens over a paged cache (bf16 and fp16): at most 16
// packed query rows, i * G + g, per key/value head.
//
// Such a call reads every cached key and value once for a handful of
// multiply-adds each, so it is bound by DRAM; what matters is that all SMs
// stream all the time, whatever the sequences' lengths.
//
// Work.  The visible 64-key blocks of all (sequence, key/value head) pairs are
// numbered in order, and each CTA takes an equal run of them (at least
// kMinRun), cutting pairs where its run begins and ends.  Lengths live on the
// device: each CTA computes the numbering (a prefix sum over the sequences)
// itself.  A pair that one CTA holds whole is written at once; a cut pair's
// pieces go to the workspace, at slot CTA + pair, and join_kernel adds them in
// order.
//
// A CTA.  Warp 4 loads blocks through a ring (TMA, a box per page).  Warps 0-3
// each take 16 keys of every block: S = Q K^T and O += P V by mma.sync (16
// rows is its tile, and the tensor rate is not the bound), with a running
// maximum and sum of the warp's own, so the warps meet only where a pair ends.
// Two CTAs share an SM, so one streams while the other joins its warps.
//
// Weight sums.  The scores are written to the workspace as they are made (4
// bytes per row and key, against 2 D bytes of the key itself), and the join
// turns them into weights when lse is known, so keys are not read again.  They
// lie in the order of the visible blocks, so a window's keys alone have a
// place, and a call whose scores would take more than kMaxScores runs as
// several, each of as many sequences as fit.
//
// Measured (with the join and the append; the kernel itself in brackets): 4
// sequences of up to 131072 keys, 16/2 heads of 128, fp16: 87 us (75, 6.1 TB/s); 64
// sequences of up to 8192 keys, 32/8 heads of 128, weights too: 238 us (204, 6.1
// TB/s).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "attn_args.cuh"
#include "decode.cuh"
#include "tc_ptx.cuh"
#include "window_tc.cuh"

namespace longnet {
namespace dc {
using namespace wt;

constexpr int kBlk = 64;
constexpr int kWarps = 4;                      // computing; one more loads
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMinRun = 4;                     // blocks: shorter runs cost more in joining than they spread
constexpr int kMaxRows = 16;

struct Args {
  AttnArgs a;
  int rows;          // nq_max G
  int* plan;         // [S + 1] blocks before each sequence (of one head), then the run length
  float* part_out;   // [slots, rows, D] normalised pieces
  float* part_lse;   // [slots, rows] log2 domain
  float* scores;     // [S Hkv, rows, kept] log2 domain, key by key of the visible blocks, or null
  int64_t kept;      // keys that the visible blocks have, at most
  float* weights;
};

template <int kD>
struct L : Panels<kD> {
  static constexpr int kHalf = kBlk * kD * 2;     // keys or values of a block
  static constexpr int kStageBytes = 2 * kHalf;
  __device__ static uint32_t at(int row, int chunk) {  // byte of a 16-byte chunk of a row
    using P = Panels<kD>;
    constexpr int kCpr = P::kRowBytes / 16;
    const int c = chunk % kCpr;
    const int sw = P::kRowBytes == 128 ? (row & 7) : P::kRowBytes == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1);
    return (uint32_t)((chunk / kCpr) * kBlk * P::kRowBytes + row * P::kRowBytes + ((c ^ sw) << 4));
  }
};

template <int kFmt>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kFmt == kFmtBF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ int seq_blocks(const AttnArgs& a, int s) {
  const Seq q = seq_of(a, s);
  return q.nq > 0 ? blocks_of<kBlk>(a, q.first, q.kv - 1).count : 0;
}

// The run length for `total` blocks over `ctas` CTAs.
__device__ __forceinline__ int run_length(int64_t total, int ctas) {
  const int64_t r = (total + ctas - 1) / ctas;
  return r < kMinRun ? kMinRun : (int)r;
}

// A piece of a pair: blocks [n0, n0 + cnt) of its list.
struct Piece {
  int s, f, n0, cnt, all;
};
__device__ __forceinline__ Piece piece_at(const int* prefix, int S, int Hkv, int64_t w, int64_t end) {
  // the sequence whose blocks hold w: the last with prefix[s] Hkv <= w
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)prefix[mid] * Hkv <= w) lo = mid;
    else hi = mid;
  }
  Piece p;
  p.s = lo;
  p.all = prefix[lo + 1] - prefix[lo];
  const int64_t in = w - (int64_t)prefix[lo] * Hkv;
  p.f = (int)(in / p.all);
  p.n0 = (int)(in % p.all);
  p.cnt = end - w < p.all - p.n0 ? (int)(end - w) : p.all - p.n0;
  return p;
}

template <int kFmt, int kD>
__global__ void __launch_bounds__(kThreads)
    decode_kernel(const __grid_constant__ Args A, const __grid_constant__ Maps maps, int stages) {
  using LL = L<kD>;
  const AttnArgs& a = A.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sStage = smem;
  float* s_o = reinterpret_cast<float*>(smem + stages * LL::kStageBytes);  // [warp][row][D]
  float* s_m = s_o + kWarps * A.rows * kD;                                 // [warp][16]
  float* s_l = s_m + kWarps * kMaxRows;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(s_l + kWarps * kMaxRows);
  uint64_t* bar_empty = bar_full + 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_full + 16);
  int* prefix = reinterpret_cast<int*>(bar_full + 17);  // [S + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(bar_full + i, 1);
      mbar_init(bar_empty + i, kWarps);
    }
    *abort_flag = 0;
    prefix[0] = 0;
    fence_barrier_init();
  }
  if (warp == kWarps && lane < 2) prefetch_tmap(&maps.m[1 + lane]);
  // the join may be scheduled; and what the launch before this one wrote is
  // read only from here on
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- the numbering: warp 0 sums the sequences' blocks, 32 at a time
  if (warp == 0) {
    int base = 0;
    for (int s0 = 0; s0 < a.S; s0 += 32) {
      int x = s0 + lane < a.S ? seq_blocks(a, s0 + lane) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (s0 + lane < a.S) prefix[s0 + lane + 1] = base + x;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const int64_t total = (int64_t)prefix[a.S] * a.Hkv;
  const int run = run_length(total, gridDim.x);
  if (blockIdx.x == 0) {
    for (int s = threadIdx.x; s <= a.S; s += kThreads) A.plan[s] = prefix[s];
    if (threadIdx.x == 0) A.plan[a.S + 1] = run;
  }
  const int64_t w0 = (int64_t)blockIdx.x * run;
  const int64_t w1 = w0 + run < total ? w0 + run : total;
  if (w0 >= w1) return;
  Waiter wt{abort_flag, a.status, kWaitLimitNs};

  if (warp == kWarps) {
    // ------------------------------------------------------------ loads
    bool ok = true;
    int it = 0;
    for (int64_t w = w0; w < w1 && ok;) {
      const Piece p = piece_at(prefix, a.S, a.Hkv, w, w1);
      const Seq q = seq_of(a, p.s);
      const BlockList bl = blocks_of<kBlk>(a, q.first, q.kv - 1);
      for (int n = 0; n < p.cnt && ok; ++n, ++it) {
        const int st = it % stages;
        if (it >= stages) ok = wt.wait_warp(bar_empty + st, ((it / stages) - 1) & 1);
        if (!ok) break;
        const int j0 = bl.at(p.n0 + n) * kBlk;
        uint8_t* dst = sStage + st * LL::kStageBytes;
        // both halves' boxes on one barrier
        const int box = a.page < kBlk ? a.page : kBlk, boxes = kBlk / box;
        const int j = j0 + lane * box;
        const bool live = lane < boxes && j < q.kv;
        int pg = 0;
        if (live) {
          pg = a.table[(int64_t)p.s * a.max_pages + (j >> a.page_shift)];
          if (pg < 0 || pg >= a.n_pages) {
            record_status(a.status, kStatusBounds);
            pg = a.n_pages;  // past the tensor: zeros
          }
        }
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, live));
        if (lane == 0) mbar_arrive_expect_tx(bar_full + st, 2 * count * (uint32_t)(box * kD * 2));
        __syncwarp();
        if (live) {
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int pn = 0; pn < LL::kPanels; ++pn)
              tma_load_4d(dst + half * LL::kHalf + pn * kBlk * LL::kRowBytes + lane * box * LL::kRowBytes,
                          &maps.m[1 + half], bar_full + st, LL::kPanelElems * pn, p.f, j & (a.page - 1), pg);
        }
      }
      w += p.cnt;
    }
    // drain: every issued load has landed before the CTA may exit
    if (lane == 0) drain_loads(bar_full, it, stages, a.status);
    return;
  }
  // -------------------------------------------------------------- compute
  const int gr = lane >> 2, t4 = lane & 3;
  int it = 0;
  bool ok = true;  // a warp whose wait ran out goes on to the meetings below, without waiting or computing
  for (int64_t w = w0; w < w1;) {
    const Piece p = piece_at(prefix, a.S, a.Hkv, w, w1);
    const Seq q = seq_of(a, p.s);
    const BlockList bl = blocks_of<kBlk>(a, q.first, q.kv - 1);
    const int rows = q.nq * a.G;  // of this pair
    const int pair = p.s * a.Hkv + p.f;
    // Q fragments and positions of rows gr and gr + 8
    uint32_t qf[kD / 16][4];
    int x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = gr + 8 * e;
      const bool in = r < rows;
      const int i = in ? r / a.G : 0, h = p.f * a.G + (in ? r % a.G : 0);
      x[e] = in ? q.first + i : -1;
      const uint32_t* src =
          reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + ((q.q0 + i) * a.H + h) * (int64_t)kD);
#pragma unroll
      for (int kk = 0; kk < kD / 16; ++kk) {
        qf[kk][e] = in ? src[kk * 8 + t4] : 0u;
        qf[kk][2 + e] = in ? src[kk * 8 + 4 + t4] : 0u;
      }
    }
    float o[kD / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int n = 0; n < p.cnt && ok; ++n, ++it) {
      const int st = it % stages;
      ok = wt.wait_warp(bar_full + st, (it / stages) & 1);
      if (!ok) break;
      const int j0 = bl.at(p.n0 + n) * kBlk + 16 * warp;  // this warp's keys
      if (j0 < q.kv) {
        const uint32_t k_at = smem_u32(sStage + st * LL::kStageBytes), v_at = k_at + LL::kHalf;
        float sc[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          uint32_t b[4];
          ldsm4(k_at + LL::at(16 * warp + (lane >> 4) * 8 + (lane & 7), 2 * kk + ((lane >> 3) & 1)), b);
          mma16816<kFmt>(sc[0], qf[kk], b[0], b[1]);
          mma16816<kFmt>(sc[1], qf[kk], b[2], b[3]);
        }
        float mx[2] = {-INFINITY, -INFINITY};
        // rows of x = -1 see nothing; below the first query every key is seen
        // unless a window hides it
        const bool whole = a.window == 0 && j0 + 15 <= q.first;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int e = c >> 1, j = j0 + 8 * nt + 2 * t4 + (c & 1);
            sc[nt][c] = (whole ? x[e] >= 0 : sees(a, x[e], j)) ? sc[nt][c] * a.scale_log2 : -INFINITY;
            mx[e] = fmaxf(mx[e], sc[nt][c]);
          }
        if (A.scores) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (gr + 8 * e < rows) {
              float* dst =
                  A.scores + ((int64_t)pair * A.rows + gr + 8 * e) * A.kept + (p.n0 + n) * kBlk + 16 * warp + 2 * t4;
#pragma unroll
              for (int nt = 0; nt < 2; ++nt)
                *reinterpret_cast<float2*>(dst + 8 * nt) = make_float2(sc[nt][2 * e], sc[nt][2 * e + 1]);
            }
        }
        float base[2];
        bool grow = false;
        float corr[2] = {1.f, 1.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          if (mx[e] > m[e] + 8.f) {  // the maximum moves only when it grew by more than 2^8
            corr[e] = ex2(m[e] - mx[e]);
            m[e] = mx[e];
            grow = true;
          }
          base[e] = m[e] == -INFINITY ? 0.f : m[e] - kUp<kFmt>;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) l[e] *= corr[e];
#pragma unroll
          for (int d = 0; d < kD / 8; ++d)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[d][c] *= corr[c >> 1];
        }
        uint32_t pf[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p0 = ex2(sc[nt][2 * e] - base[e]), p1 = ex2(sc[nt][2 * e + 1] - base[e]);
            l[e] += p0 + p1;
            pf[2 * nt + e] = pack2<kFmt>(p0, p1);  // the second product takes 16-bit operands
          }
        // slots past the sequence's keys may hold anything: their value rows
        // count as zeros
        const int live = q.kv - j0 - 2 * t4;
        const uint32_t z0 = live >= 2 ? 0xffffffffu : live == 1 ? 0x0000ffffu : 0u;
        const uint32_t z1 = live >= 10 ? 0xffffffffu : live == 9 ? 0x0000ffffu : 0u;
#pragma unroll
        for (int d = 0; d < kD / 16; ++d) {
          uint32_t b[4];
          ldsm4_t(v_at + LL::at(16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7), 2 * d + (lane >> 4)), b);
          mma16816<kFmt>(o[2 * d], pf, b[0] & z0, b[1] & z1);
          mma16816<kFmt>(o[2 * d + 1], pf, b[2] & z0, b[3] & z1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_empty + st);
    }
    // ---- the pair's piece ends: join the warps
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      const int r = gr + 8 * e;
      if (r < rows) {
        if (t4 == 0) {
          s_m[warp * kMaxRows + r] = m[e];
          s_l[warp * kMaxRows + r] = l[e];
        }
        float* dst = s_o + ((int64_t)warp * A.rows + r) * kD + 2 * t4;
#pragma unroll
        for (int d = 0; d < kD / 8; ++d)
          *reinterpret_cast<float2*>(dst + 8 * d) = make_float2(o[d][2 * e], o[d][2 * e + 1]);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    const bool direct = p.cnt == p.all;
    const int64_t slot = (int64_t)blockIdx.x + pair;
    for (int e = threadIdx.x; e < rows * (kD / 4); e += 32 * kWarps) {
      const int r = e / (kD / 4), d = (e % (kD / 4)) * 4;
      float mm = s_m[r];
#pragma unroll
      for (int v = 1; v < kWarps; ++v) mm = fmaxf(mm, s_m[v * kMaxRows + r]);
      const float bs = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float sc = ex2(s_m[v * kMaxRows + r] - bs);
        const float4 t = *reinterpret_cast<const float4*>(s_o + ((int64_t)v * A.rows + r) * kD + d);
        ll = fmaf(sc, s_l[v * kMaxRows + r], ll);
        acc.x = fmaf(sc, t.x, acc.x);
        acc.y = fmaf(sc, t.y, acc.y);
        acc.z = fmaf(sc, t.z, acc.z);
        acc.w = fmaf(sc, t.w, acc.w);
      }
      const float inv = ll == 0.f ? 0.f : 1.f / ll;  // (a sum of NaN stays one)
      const float lse2 = ll == 0.f ? -INFINITY : mm - kUp<kFmt> + log2f(ll);
      if (direct) {
        const int i = r / a.G, h = p.f * a.G + r % a.G;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + ((q.q0 + i) * a.H + h) * (int64_t)kD + d) =
            make_uint2(pack2<kFmt>(acc.x * inv, acc.y * inv), pack2<kFmt>(acc.z * inv, acc.w * inv));
        if (d == 0 && a.lse) a.lse[(q.q0 + i) * a.H + h] = lse2 * kLn2;
      } else {
        *reinterpret_cast<float4*>(A.part_out + (slot * A.rows + r) * kD + d) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (d == 0) A.part_lse[slot * A.rows + r] = lse2;
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    w += p.cnt;
  }
}

// lse (log2 domain) of a row of a pair: its pieces' joined, or the one written
// directly.
struct Pieces {
  int64_t first;  // slot of the first
  int count;
};
__device__ __forceinline__ Pieces pieces_of(const Args& A, int s, int f, int blocks) {
  Pieces p = {0, 0};
  if (blocks == 0) return p;
  const int run = A.plan[A.a.S + 1];
  const uint32_t w = (uint32_t)(A.plan[s] * A.a.Hkv + f * blocks);  // fewer than 2^30 blocks in all
  const uint32_t c0 = w / (uint32_t)run, c1 = (w + blocks - 1) / (uint32_t)run;
  p.first = (int64_t)c0 + s * A.a.Hkv + f;
  p.count = (int)(c1 - c0) + 1;
  return p;
}

constexpr int kJoinThreads = 256;
constexpr int kKeysPerBlock = 1024;

// Blocks [0, row_blocks): kSplit warps per (pair, row) join the row's pieces,
// each an equal run of them, then the runs in order.  The others: the weights
// of kKeysPerBlock keys of a pair.
template <int kFmt, int kD, int kSplit>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args A, int row_blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttnArgs& a = A.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x < row_blocks) {
    constexpr int kWarpsPerBlock = kJoinThreads / 32;
    constexpr int kE = kD / 32 > 0 ? kD / 32 : 1;  // values of a lane
    __shared__ float s_acc[kSplit > 1 ? kWarpsPerBlock : 1][kSplit > 1 ? kD : 1], s_sum[kWarpsPerBlock];
    const int64_t id = (int64_t)blockIdx.x * (kWarpsPerBlock / kSplit) + warp / kSplit;
    const int64_t pair = id / A.rows;
    const int r = (int)(id % A.rows), s = (int)(pair / a.Hkv), f = (int)(pair % a.Hkv);
    Seq q = {0, 0, 0, 0};
    Pieces p = {0, 1};
    if (pair < (int64_t)a.S * a.Hkv) {
      q = seq_of(a, s);
      if (r < q.nq * a.G) p = pieces_of(A, s, f, A.plan[s + 1] - A.plan[s]);
    }
    const bool mine = p.count != 1;  // one piece was written by its CTA; none: zeros
    const bool on = lane * kE < kD;
    float m = -INFINITY, acc[kE] = {}, sum = 0.f;
    if (mine) {
      for (int c = lane; c < p.count; c += 32) m = fmaxf(m, A.part_lse[(p.first + c) * A.rows + r]);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.f : m;
      const int per = (p.count + kSplit - 1) / kSplit;
      const int b0 = (warp % kSplit) * per, b1 = b0 + per < p.count ? b0 + per : p.count;
      // 32 pieces at a time: a lane weighs one, then all lanes add them in
      // order (independent loads, so their latencies overlap)
      for (int c0 = b0; c0 < b1; c0 += 32) {
        const float wl = c0 + lane < b1 ? ex2(A.part_lse[(p.first + c0 + lane) * A.rows + r] - base) : 0.f;
        const int n = b1 - c0 < 32 ? b1 - c0 : 32;
#pragma unroll 8
        for (int c = 0; c < n; ++c) {
          const float wgt = __shfl_sync(0xffffffffu, wl, c);
          sum += wgt;
          if (on) {
            const float* src = A.part_out + ((p.first + c0 + c) * A.rows + r) * kD + lane * kE;
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
            for (int e = 0; e < kE; ++e) acc[e] = fmaf(wgt, t[e], acc[e]);
          }
        }
      }
    }
    if (kSplit > 1) {
      if (on) {
#pragma unroll
        for (int e = 0; e < kE; ++e) s_acc[warp][lane * kE + e] = acc[e];
      }
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();
      if (warp % kSplit != 0) return;
#pragma unroll
      for (int v = 1; v < kSplit; ++v) {
        sum += s_sum[warp + v];
        if (on) {
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[e] += s_acc[warp + v][lane * kE + e];
        }
      }
    }
    if (!mine) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i = r / a.G, h = f * a.G + r % a.G;
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
    if (lane == 0 && a.lse) a.lse[(q.q0 + i) * a.H + h] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
    return;
  }
  // ---- weights
  __shared__ float s_lse[kMaxRows];
  const int64_t keys = (int64_t)a.max_pages << a.page_shift;
  const int chunks = (int)((keys + kKeysPerBlock - 1) / kKeysPerBlock);
  const int64_t id = (int64_t)blockIdx.x - row_blocks;
  const int64_t pair = id / chunks;
  const int s = (int)(pair / a.Hkv), f = (int)(pair % a.Hkv);
  const int j0 = (int)(id % chunks) * kKeysPerBlock;
  const Seq q = seq_of(a, s);
  if (j0 >= q.kv || q.nq == 0) return;
  const int rows = q.nq * a.G;
  const BlockList bl = blocks_of<kBlk>(a, q.first, q.kv - 1);
  const Pieces p = pieces_of(A, s, f, bl.count);
  for (int r = warp; r < rows; r += kJoinThreads / 32) {
    float l2 = -INFINITY;
    if (p.count == 1) {
      l2 = a.lse[(q.q0 + r / a.G) * a.H + f * a.G + r % a.G] * kLog2e;
    } else {
      float m = -INFINITY, sum = 0.f;
      for (int c = lane; c < p.count; c += 32) m = fmaxf(m, A.part_lse[(p.first + c) * A.rows + r]);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.f : m;
      for (int c = lane; c < p.count; c += 32) sum += ex2(A.part_lse[(p.first + c) * A.rows + r] - base);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (sum != 0.f) l2 = m + log2f(sum);
    }
    if (lane == 0) s_lse[r] = l2;
  }
  __syncthreads();
  const int j = j0 + 4 * (int)threadIdx.x;  // keys is a multiple of 8, j of 4
  if (j >= q.kv) return;
  const int block = j / kBlk;
  if (block >= bl.n_sink && block < bl.win0) return;  // no row sees it
  // the place of the key's block among the visible ones
  const int64_t at = (int64_t)(block < bl.n_sink ? block : bl.n_sink + block - bl.win0) * kBlk + j % kBlk;
  float acc[4] = {};
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const int x = q.first + r / a.G;
    if (x < 0) continue;
    const float4 sc = *reinterpret_cast<const float4*>(A.scores + (pair * A.rows + r) * A.kept + at);
    const float v[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (sees(a, x, j + e)) acc[e] += ex2(v[e] - s_lse[r]);
  }
  float* wp = A.weights + pair * keys + j;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j + e < q.kv) wp[e] += acc[e];
}

// ---- host
constexpr int kMaxSeq = 2048;  // the numbering is kept in shared memory
constexpr int64_t kMaxScores = (int64_t)1 << 26;  // floats: 256 MiB

int rows_of(const AttnArgs& a) { return a.nq_max * a.G; }
int ctas_of(const AttnArgs& a) {
  // as many as the cache's capacity can occupy, at most two per SM
  const int64_t blocks = (((int64_t)a.max_pages << a.page_shift) + kBlk - 1) / kBlk * a.S * a.Hkv;
  const int64_t want = (blocks + kMinRun - 1) / kMinRun;
  return (int)(want < 296 ? want : 296);
}
int64_t round64(int64_t floats) { return (floats + 63) / 64 * 64; }  // 256 bytes
// The keys of the blocks that a sequence's rows see, at most: all, or the
// window of nq_max tokens and the sinks, in whole blocks.
int64_t kept_keys(const AttnArgs& a) {
  const int64_t all = (((int64_t)a.max_pages << a.page_shift) + kBlk - 1) / kBlk;
  if (!a.window) return all * kBlk;
  const int64_t seen = ((int64_t)a.window + a.nq_max - 2) / kBlk + 2 + ((int64_t)a.sinks + kBlk - 1) / kBlk;
  return (seen < all ? seen : all) * kBlk;
}
// Sequences of one launch: all, or with weights as many as kMaxScores holds.
int group_of(const AttnArgs& a, bool weights) {
  if (!weights) return a.S;
  const int64_t fit = kMaxScores / (a.Hkv * rows_of(a) * kept_keys(a));
  return fit < 1 ? 1 : fit < a.S ? (int)fit : a.S;
}
struct Sizes {
  int64_t plan, out, lse, scores;  // floats, each rounded to 256 bytes
  int64_t all() const { return plan + out + lse + scores; }
};
// Of one launch over a's sequences.
Sizes sizes_of(const AttnArgs& a, bool weights) {
  const int64_t slots = (int64_t)ctas_of(a) + (int64_t)a.S * a.Hkv;
  Sizes z;
  z.plan = round64(a.S + 2);
  z.out = round64(slots * rows_of(a) * a.D);
  z.lse = round64(slots * rows_of(a));
  z.scores = weights ? round64((int64_t)a.S * a.Hkv * rows_of(a) * kept_keys(a)) : 0;
  return z;
}

template <int kFmt, int kD>
int launch_typed(const AttnArgs& a, float* workspace, float* weights, cudaStream_t stream) {
  using LL = L<kD>;
  Args A;
  A.a = a;
  A.rows = rows_of(a);
  const Sizes z = sizes_of(a, weights != nullptr);
  A.plan = reinterpret_cast<int*>(workspace);
  A.part_out = workspace + z.plan;
  A.part_lse = A.part_out + z.out;
  A.scores = weights ? A.part_lse + z.lse : nullptr;
  A.kept = kept_keys(a);
  A.weights = weights;
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  EncodeTiledFn enc = get_encoder();
  if (!enc) return LONGNET_ERR_CUDA;
  if (!encode_kv(enc, &maps.m[1], a.k, a, kBlk) || !encode_kv(enc, &maps.m[2], a.v, a, kBlk)) return LONGNET_ERR_CUDA;
  // two CTAs per SM: stages of what is left of half an SM's shared memory
  const int fixed = kWarps * A.rows * kD * 4 + 2 * kWarps * kMaxRows * 4 + 20 * 8 + (a.S + 2) * 4 + 1024;
  int stages = (112 * 1024 - fixed) / LL::kStageBytes;
  if (stages > 8) stages = 8;
  const int smem = fixed + stages * LL::kStageBytes;
  if (!opt_in_smem<decode_kernel<kFmt, kD>>(112 * 1024)) return LONGNET_ERR_CUDA;
  int rc = launch_after(decode_kernel<kFmt, kD>, dim3((unsigned)ctas_of(a)), kThreads, smem, stream, A, maps, stages);
  if (rc) return rc;
  const int64_t pairs = (int64_t)a.S * a.Hkv;
  // pairs cut into many pieces (few pairs over the CTAs) are joined by eight
  // warps a row: 8 pairs of 37 pieces took 14 us with one
  const bool many = ctas_of(a) >= 8 * pairs;
  const int per = kJoinThreads / 32 / (many ? 8 : 1);  // rows of a block
  const int row_blocks = (int)((pairs * A.rows + per - 1) / per);
  const int64_t keys = (int64_t)a.max_pages << a.page_shift;
  const int64_t blocks = row_blocks + (weights ? pairs * ((keys + kKeysPerBlock - 1) / kKeysPerBlock) : 0);
  return launch_after(many ? join_kernel<kFmt, kD, 8> : join_kernel<kFmt, kD, 1>, dim3((unsigned)blocks), kJoinThreads,
                      0, stream, A, row_blocks);
}

int launch_group(const AttnArgs& a, float* workspace, float* weights, bool f16, cudaStream_t stream) {
  switch (a.D) {
    case 16:
      return f16 ? launch_typed<tc::kFmtF16, 16>(a, workspace, weights, stream)
                 : launch_typed<tc::kFmtBF16, 16>(a, workspace, weights, stream);
    case 32:
      return f16 ? launch_typed<tc::kFmtF16, 32>(a, workspace, weights, stream)
                 : launch_typed<tc::kFmtBF16, 32>(a, workspace, weights, stream);
    case 64:
      return f16 ? launch_typed<tc::kFmtF16, 64>(a, workspace, weights, stream)
                 : launch_typed<tc::kFmtBF16, 64>(a, workspace, weights, stream);
    default:
      return f16 ? launch_typed<tc::kFmtF16, 128>(a, workspace, weights, stream)
                 : launch_typed<tc::kFmtBF16, 128>(a, workspace, weights, stream);
  }
}

}  // namespace dc

// At most 16 rows per key/value head and kMaxSeq sequences.
bool decode_supports(const AttnArgs& a) {
  if (a.dtype != LONGNET_DTYPE_BF16 && a.dtype != LONGNET_DTYPE_F16) return false;
  const int64_t keys = (int64_t)a.max_pages << a.page_shift;
  return (int64_t)a.nq_max * a.G <= dc::kMaxRows && a.S <= dc::kMaxSeq &&
         // block numbers are 32-bit, and so is the grid of the join
         (int64_t)a.S * a.Hkv * ((keys + dc::kBlk - 1) / dc::kBlk) < ((int64_t)1 << 30);
}

int64_t decode_workspace_floats(const AttnArgs& a, bool weights) {
  AttnArgs g = a;
  g.S = dc::group_of(a, weights);
  return dc::sizes_of(g, weights).all();
}

int launch_decode(const AttnArgs& all, float* workspace, float* weights, cudaStream_t stream) {
  const bool f16 = all.dtype == LONGNET_DTYPE_F16;
  const int group = dc::group_of(all, weights != nullptr);
  for (int s = 0; s < all.S; s += group) {
    AttnArgs a = all;  // sequences [s, s + S): token rows stay where they are
    a.S = all.S - s < group ? all.S - s : group;
    a.cu_q += s;
    a.kv_len += s;
    a.table += (int64_t)s * a.max_pages;
    float* w = weights ? weights + ((int64_t)s * a.Hkv * a.max_pages << a.page_shift) : nullptr;
    const int rc = dc::launch_group(a, workspace, w, f16, stream);
    if (rc) return rc;
  }
  return LONGNET_OK;
}

}  // namespace longnet
