// The attention weight that each cached key received from a chunk of new
// tokens, on the tensor cores (tcgen05), bf16 and fp16:
//   weights[s, f, j] += sum over the rows that see key j of e^{s_xj - lse_x}.
//
// The forward has written lse, so the scores are made once more, transposed:
// S^T = K Q^T, a TMEM lane per key, and each thread sums its key's row.  No
// second product, no exchange between threads, one addition per key and call,
// so the result does not depend on any order.  Bound: the exponentials (16 per
// clock and SM: 17 us of them for three chunks of up to 1024 tokens over up to 8192
// keys, 8/2 heads of 128, which take 37 us).
//
// A CTA holds a tile of 128 keys of one key/value head and streams blocks of
// 128 packed query rows (128 / G tokens by G heads) with their lse.  Two
// warpgroups take alternate blocks, each with two 128-column score buffers in
// TMEM, so that a block's scores are there when the one before is summed.
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
namespace ww {
using namespace wt;

constexpr int kThreads = 320;
constexpr int kTma = 8, kMma = 9;  // warps
constexpr uint32_t kTmemCols = 512;
constexpr int kSlots = 4;  // score buffers

template <int kD>
struct L : Panels<kD> {
  static constexpr int kTileBytes = kTile * kD * 2;
  static constexpr int kStageBytes = kTileBytes + 1024;  // a block of query rows, then their -lse
  static constexpr int kStages = kD == 128 ? 5 : 6;
  static constexpr int kBars = kTileBytes + kStages * kStageBytes;
  // one CTA per SM: its TMEM columns are all of the SM's
  static constexpr int kSmem = kBars + 1024 + 1024 > 120 * 1024 ? kBars + 1024 + 1024 : 120 * 1024;
};

// acc += the sum over 128 columns of 2^(s scale log2(e) - lse log2(e)), of those
// in [lo, hi) with kMask.
template <bool kMask>
__device__ __forceinline__ void sum_block(uint32_t s_col, const float* sl, uint64_t sc2, int lo, int hi,
                                          uint64_t (&acc)[2]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t sr[32];
    LN_TMEM_LD32(s_col + 32 * w, sr);
    tmem_wait_ld();
    const uint32_t keep = below(hi - 32 * w) & ~below(lo - 32 * w);
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      const float4 l4 = *reinterpret_cast<const float4*>(sl + 32 * w + c);
      float x[4];
      f32x2_split(fma_f32x2(f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc2, f32x2(l4.x, l4.y)), x[0],
                  x[1]);
      f32x2_split(fma_f32x2(f32x2(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), sc2, f32x2(l4.z, l4.w)),
                  x[2], x[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = ex2(x[e]);
        if (kMask) x[e] = (keep >> (c + e)) & 1 ? x[e] : 0.f;
      }
      acc[0] = add_f32x2(acc[0], f32x2(x[0], x[1]));
      acc[1] = add_f32x2(acc[1], f32x2(x[2], x[3]));
    }
  }
}

template <int kFmt, int kD>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Maps maps, float* weights, int tok) {
  using LL = L<kD>;
  constexpr int kPanels = LL::kPanels, kPanelBytes = kTile * LL::kRowBytes, S = LL::kStages;
  constexpr uint32_t kDescHi = LL::kDescHi;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int s = blockIdx.y / a.Hkv, f = blockIdx.y % a.Hkv;
  const Seq q = seq_of(a, s);
  const int j0 = blockIdx.x * kTile, G = a.G;
  if (j0 >= q.kv || q.nq == 0) return;  // whole CTA, before any barrier or TMEM use
  // tokens [i0, i1): from the first at or after the tile's first key on, and,
  // unless the tile holds a sink, up to the last whose window reaches it
  const int i0 = j0 > q.first ? j0 - q.first : 0;
  int i1 = q.nq;
  if (a.window && j0 >= a.sinks) {
    const int64_t last = (int64_t)j0 + kTile - 1 + a.window - q.first;
    if (last < i1) i1 = last < 0 ? 0 : (int)last;
  }
  if (i0 >= i1) return;
  const int cnt = (i1 - i0 + tok - 1) / tok;

  uint8_t* sStage = smem + LL::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + LL::kBars);
  uint64_t* bar_k = bars;
  uint64_t* bar_full = bars + 1;       // [S]
  uint64_t* bar_empty = bars + 1 + S;  // [S] the block's scores done, and read
  uint64_t* bar_s = bars + 1 + 2 * S;  // [kSlots] scores in TMEM
  uint64_t* bar_r = bar_s + kSlots;    // [kSlots] scores read
  uint64_t* bar_drain = bar_s + 2 * kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_s + 2 * kSlots + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_sum = reinterpret_cast<float*>(smem + LL::kBars + 256);  // [128]

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar_k, 1);
    for (int i = 0; i < S; ++i) {
      mbar_init(bar_full + i, 32);        // the loading warp's lanes, and the TMA bytes
      mbar_init(bar_empty + i, 1 + 128);  // the scores' commit, and the threads that read the -lse
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar_s + i, 1);
      mbar_init(bar_r + i, 128);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kTma && lane < 2) prefetch_tmap(&maps.m[lane]);
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
  float sum = 0.f;

  if (warp == kTma) {
    // ------------------------------------------------------------ loads
    bool ok = true;
    load_pages<kD>(a, q, s, f, j0, kTile, &maps.m[1], smem, bar_k, lane);
    if (lane == 0) mbar_arrive(bar_k);
    // -lse (log2 domain) of a block's rows, fetched a block ahead (their
    // latency would otherwise stand between the loads)
    // (loaded from a valid address in any case: a load under a condition is
    // waited for where the condition ends)
    float l2[4];
    int c_tok[4], c_head[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c_tok[e] = (lane + 32 * e) / G;
      c_head[e] = f * G + (lane + 32 * e) % G;
    }
    auto fetch = [&](int n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + n * tok + c_tok[e];
        l2[e] = a.lse[(q.q0 + (i < i1 ? i : i0)) * a.H + c_head[e]];
      }
    };
    fetch(0);
    int issued = 0;
    for (int n = 0; n < cnt && ok; ++n) {
      const int st = n % S;
      if (n >= S) ok = wt.wait_warp(bar_empty + st, ((n / S) - 1) & 1);
      if (!ok) break;
      uint8_t* stage = sStage + st * LL::kStageBytes;
      if (lane == 0) {
        mbar_expect_tx(bar_full + st, (uint32_t)(kPanels * tok * G * LL::kRowBytes));
#pragma unroll
        for (int pn = 0; pn < kPanels; ++pn)
          tma_load_3d(stage + pn * kPanelBytes, &maps.m[0], bar_full + st, LL::kPanelElems * pn, f * G,
                      (int)(q.q0 + i0 + n * tok));
      }
      float* sl = reinterpret_cast<float*>(stage + LL::kTileBytes);
#pragma unroll
      for (int e = 0; e < 4; ++e) sl[lane + 32 * e] = -l2[e] * kLog2e;  // (not looked at past the block's rows)
      __syncwarp();  // the bytes are expected before the phase can complete
      mbar_arrive(bar_full + st);
      fetch(n + 1);
      issued = n + 1;
    }
    // drain: every issued load has landed before the CTA may exit
    if (lane == 0) {
      if (!mbar_wait(bar_k, 0, kWaitLimitNs)) record_status(a.status, kStatusTimeout);
      drain_loads(bar_full, issued, S, a.status);
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t kIdS = idesc_f16kind(kTile, kTile, false, kFmt);
    const uint32_t leader = elect_leader();
    const uint32_t k_lo = (smem_u32(smem) >> 4) | (1u << 16), ring_lo = smem_u32(sStage) >> 4;
    bool ok = wt.wait_warp(bar_k, 0);
    for (int n = 0; n < cnt && ok; ++n) {
      ok = wt.wait_warp(bar_full + n % S, (n / S) & 1);
      if (ok && n >= kSlots) ok = wt.wait_warp(bar_r + n % kSlots, (n / kSlots - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t q_lo = (ring_lo + (n % S) * (LL::kStageBytes >> 4)) | (1u << 16);
#pragma unroll
      for (int pn = 0; pn < kPanels; ++pn)
#pragma unroll
        for (int kk = 0; kk < LL::kPanelElems / 16; ++kk)
          mma_ss_if(leader, tmem + kTile * (n % kSlots), desc_from(k_lo + pn * (kPanelBytes >> 4) + kk * 2, kDescHi),
                    desc_from(q_lo + pn * (kPanelBytes >> 4) + kk * 2, kDescHi), kIdS, (pn > 0 || kk > 0) ? 1u : 0u);
      tc_commit_if(leader, bar_s + n % kSlots);
      tc_commit_if(leader, bar_empty + n % S);
    }
    // drain: all issued MMAs complete before TMEM is released
    tc_commit_if(leader, bar_drain);
    if (!mbar_wait(bar_drain, 0, kWaitLimitNs)) record_status(a.status, kStatusTimeout);
  } else {
    // ------------------------------------------------------------ exponentials and sums
    const int wg = warp >> 2;
    const int j = j0 + 32 * (warp & 3) + lane;  // TMEM lane = key
    const uint32_t s_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint64_t sc2 = f32x2(a.scale_log2, a.scale_log2);
    uint64_t acc[2] = {0, 0};
    bool ok = true;
    for (int n = wg; n < cnt && ok; n += 2) {
      const int st = n % S;
      const float* sl = reinterpret_cast<const float*>(sStage + st * LL::kStageBytes + LL::kTileBytes);
      // the columns [lo, hi) that see this key
      const int at = i0 + n * tok, n_tok = i1 - at < tok ? i1 - at : tok;
      const int from = j - q.first - at;
      const int64_t to = (int64_t)from + a.window;
      const int lo = (from < 0 ? 0 : from > kTile ? kTile : from) * G;
      const int hi = (a.window == 0 || j < a.sinks || to > n_tok ? n_tok : to < 0 ? 0 : (int)to) * G;
      const bool whole = __all_sync(0xffffffffu, lo == 0 && hi == kTile);
      ok = wt.wait_warp(bar_full + st, (n / S) & 1);
      if (ok) ok = wt.wait_warp(bar_s + n % kSlots, (n / kSlots) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t s_col = s_lane + kTile * (n % kSlots);
      if (whole)
        sum_block<false>(s_col, sl, sc2, lo, hi, acc);
      else
        sum_block<true>(s_col, sl, sc2, lo, hi, acc);
      tc_fence_before();
      mbar_arrive(bar_r + n % kSlots);
      mbar_arrive(bar_empty + st);
    }
    float t0, t1;
    f32x2_split(add_f32x2(acc[0], acc[1]), t0, t1);
    sum = t0 + t1;
    if (wg == 1) s_sum[threadIdx.x - 128] = sum;
  }
  tc_fence_before();
  __syncthreads();
  if (warp < 4) {
    const int j = j0 + (int)threadIdx.x;
    if (j < q.kv)
      weights[(int64_t)blockIdx.y * ((int64_t)a.max_pages << a.page_shift) + j] += sum + s_sum[threadIdx.x];
  }
  if (warp == kMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

template <int kFmt, int kD>
int launch_typed(const AttnArgs& a, float* weights, cudaStream_t stream) {
  using LL = L<kD>;
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  EncodeTiledFn enc = get_encoder();
  if (!enc) return LONGNET_ERR_CUDA;
  const int tok = kTile / a.G;
  if (!encode_q(enc, &maps.m[0], a.q, a, tok) || !encode_kv(enc, &maps.m[1], a.k, a, kTile)) return LONGNET_ERR_CUDA;
  if (!opt_in_smem<weights_kernel<kFmt, kD>>(LL::kSmem)) return LONGNET_ERR_CUDA;
  const int64_t tiles = (((int64_t)a.max_pages << a.page_shift) + kTile - 1) / kTile;
  weights_kernel<kFmt, kD><<<dim3((unsigned)tiles, (unsigned)(a.S * a.Hkv)), kThreads, LL::kSmem, stream>>>(a, maps, weights, tok);
  return cudaGetLastError() == cudaSuccess ? LONGNET_OK : LONGNET_ERR_CUDA;
}

}  // namespace ww

int launch_weights_tc(const AttnArgs& a, float* weights, cudaStream_t stream) {
  const bool f16 = a.dtype == LONGNET_DTYPE_F16;
  switch (a.D) {
    case 16:
      return f16 ? ww::launch_typed<tc::kFmtF16, 16>(a, weights, stream) : ww::launch_typed<tc::kFmtBF16, 16>(a, weights, stream);
    case 32:
      return f16 ? ww::launch_typed<tc::kFmtF16, 32>(a, weights, stream) : ww::launch_typed<tc::kFmtBF16, 32>(a, weights, stream);
    case 64:
      return f16 ? ww::launch_typed<tc::kFmtF16, 64>(a, weights, stream) : ww::launch_typed<tc::kFmtBF16, 64>(a, weights, stream);
    default:
      return f16 ? ww::launch_typed<tc::kFmtF16, 128>(a, weights, stream) : ww::launch_typed<tc::kFmtBF16, 128>(a, weights, stream);
  }
}

}  // namespace longnet
