// Eviction from a paged cache by accumulated attention weight.
//
// A sequence of n > budget keys keeps, for each key/value head, its first
// `sinks` keys, its last `recent` keys, and of the others the budget - sinks -
// recent with the largest weights (equal weights: the lowest index first; NaN
// below every number).  A sequence of n <= budget keys keeps them all.  Kept
// keys stay in order: the j-th kept key becomes key j of the new cache.
//
// Two kernels.  Select, one CTA per (sequence, head): the need-th largest weight
// by a radix select on the weights' order-preserving 32-bit images (digits of
// 11, 11 and 10 bits, a histogram in shared memory each), then one pass in index
// order that writes the kept indices and their weights.  The images stay in
// shared memory where they fit (48K keys), so the weights are read once.  (A
// cluster of CTAs per pair, its histograms added over distributed shared
// memory, was slower: 49 us against 32 for 128 pairs of 32K keys, 12 against 7
// for 400 keys.)
// Move: a thread copies four 16-byte chunks of kept key and value rows, with
// all its index and page look-ups and then all its loads in flight together;
// neighbours along the row and then the heads of a slot, so both sides move
// whole sectors.
// Bound: DRAM, the kept rows read and written once.  16 sequences of up to 32K
// keys, 8 heads, D = 128, cut to 8192: 28 us select (bound by its instructions) and
// 164 us move (5.8 TB/s).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_args.cuh"
#include "launch_util.cuh"

namespace longnet {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kPer = 8;  // keys of a thread in a tile of the ordered pass
constexpr int kBins = 2048;
constexpr int kHeld = 48 * 1024;  // images kept in shared memory

// Unsigned image of a weight: larger weight, larger image; +0 and -0 equal;
// NaN 0, below -infinity.
__device__ __forceinline__ uint32_t image(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the block; total gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const uint32_t before = warp ? warp_sums[warp - 1] : 0u;
  *total = warp_sums[31];
  __syncthreads();
  return before + inc - x;
}

// kHold: the images are kept in shared memory; else they are made again from
// the weights for every digit.
template <bool kHold>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t held[];
  __shared__ uint32_t hist[kBins], warp_sums[32], s_digit, s_need;
  const int pair = blockIdx.x, s = pair / a.Hkv, f = pair % a.Hkv;
  const int64_t cap = (int64_t)a.max_pages << a.page_shift, out_cap = (int64_t)a.max_out_pages << a.page_shift;
  int n = a.kv_len[s];
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0) record_status(a.status, kStatusBounds);
    n = 0;
  }
  const float* w = a.weights + (int64_t)pair * cap;
  float* nw = a.new_weights + (int64_t)pair * out_cap;
  int* kept = a.kept + (int64_t)pair * a.budget;
  const int left = n < a.budget ? n : a.budget;
  if (threadIdx.x == 0 && f == 0) a.new_len[s] = left;
  for (int64_t j = left + threadIdx.x; j < out_cap; j += kSelThreads) nw[j] = 0.f;
  for (int j = left + threadIdx.x; j < a.budget; j += kSelThreads) kept[j] = -1;
  if (n <= a.budget) {
    for (int j = threadIdx.x; j < n; j += kSelThreads) {
      kept[j] = j;
      nw[j] = w[j];
    }
    return;
  }
  const int lo = a.sinks, hi = n - a.recent;  // the keys that compete
  const uint32_t need = (uint32_t)(a.budget - a.sinks - a.recent);
  uint32_t prefix = 0, rest = need;  // digits found so far; how many equal to them are needed
  // 16 bytes a load where the weights allow it (a row is a multiple of 32 bytes)
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  if (kHold && need > 0) {
    const int n4 = wide ? n / 4 : 0;
#pragma unroll 8
    for (int j = threadIdx.x; j < n4; j += kSelThreads) {
      const float4 x = reinterpret_cast<const float4*>(w)[j];
      reinterpret_cast<uint4*>(held)[j] = make_uint4(image(x.x), image(x.y), image(x.z), image(x.w));
    }
    for (int j = 4 * n4 + threadIdx.x; j < n; j += kSelThreads) held[j] = image(w[j]);
  }
  if (need > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = lo + threadIdx.x; j < hi; j += kSelThreads) {
        const uint32_t u = kHold ? held[j] : image(w[j]);
        if (pass == 0 || (u >> (shift + bits)) == prefix) atomicAdd(&hist[(u >> shift) & ((1u << bits) - 1)], 1u);
      }
      __syncthreads();
      // the digit whose count, added to those above it, first reaches rest:
      // two bins a thread, the largest first
      const uint32_t c0 = hist[kBins - 1 - 2 * threadIdx.x], c1 = hist[kBins - 2 - 2 * threadIdx.x];
      uint32_t total;
      const uint32_t above = block_scan(c0 + c1, warp_sums, &total);
      if (above < rest && above + c0 + c1 >= rest) {
        const bool second = above + c0 < rest;
        s_digit = kBins - 1 - 2 * threadIdx.x - (second ? 1 : 0);
        s_need = rest - above - (second ? c0 : 0u);
      }
      __syncthreads();
      prefix = (prefix << bits) | s_digit;
      rest = s_need;
    }
  }
  // in index order, kPer consecutive keys a thread and tile: forced keys, those
  // above the threshold, and the first `rest` equal to it
  uint32_t sure_before = 0, equal_before = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads * kPer) {
    const int j0 = t0 + threadIdx.x * kPer;
    float x[kPer];  // all loaded at once: one latency a tile
    if (wide && j0 + kPer <= n) {
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(w + j0 + i);
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = j0 + i < n ? w[j0 + i] : 0.f;
    }
    uint32_t kind[kPer], count = 0;  // 1 << 16 surely kept, 1 equal to the threshold, 0 not kept
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = j0 + i;
      const uint32_t u = image(x[i]);
      kind[i] = j >= n ? 0u : j < lo || j >= hi ? 1u << 16 : need == 0 ? 0u : u > prefix ? 1u << 16 : u == prefix ? 1u : 0u;
      count += kind[i];
    }
    uint32_t total;
    const uint32_t before = block_scan(count, warp_sums, &total);
    uint32_t sure = sure_before + (before >> 16), equal = equal_before + (before & 0xffffu);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kind[i] == (1u << 16) || (kind[i] == 1u && equal < rest)) {
        const uint32_t at = sure + (equal < rest ? equal : rest);
        kept[at] = j0 + i;
        nw[at] = x[i];
      }
      sure += kind[i] >> 16;
      equal += kind[i] & 0xffffu;
    }
    sure_before += total >> 16;
    equal_before += total & 0xffffu;
  }
}

constexpr int kMoveThreads = 256;
constexpr int kChunksPer = 4;  // of a thread

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a, int head_chunks) {
  const int s = blockIdx.y;
  const uint32_t row_chunks = a.Hkv * head_chunks;
  const uint32_t e0 = blockIdx.x * (kMoveThreads * kChunksPer) + threadIdx.x;  // fewer than 2^31 a sequence
  int64_t src[kChunksPer], dst[kChunksPer];
  int from[kChunksPer];
#pragma unroll
  for (int k = 0; k < kChunksPer; ++k) {
    const uint32_t e = e0 + k * kMoveThreads, j = e / row_chunks, c = e - j * row_chunks, f = c / head_chunks;
    from[k] = (int)j < a.budget ? a.kept[((int64_t)s * a.Hkv + f) * a.budget + j] : -1;
    src[k] = c;
    dst[k] = j;
  }
#pragma unroll
  for (int k = 0; k < kChunksPer; ++k) {
    if (from[k] < 0) continue;
    const int j = (int)dst[k];
    const int64_t c = src[k];
    const int pg = a.table[(int64_t)s * a.max_pages + (from[k] >> a.page_shift)];
    const int to = a.new_table[(int64_t)s * a.max_out_pages + (j >> a.page_shift)];
    if (pg < 0 || pg >= a.n_pages || to < 0 || to >= a.n_out_pages) {
      record_status(a.status, kStatusBounds);
      from[k] = -1;
      continue;
    }
    src[k] = (((int64_t)pg << a.page_shift) + (from[k] & (a.page - 1))) * row_chunks + c;
    dst[k] = (((int64_t)to << a.page_shift) + (j & (a.page - 1))) * row_chunks + c;
  }
  uint4 kk[kChunksPer], vv[kChunksPer];
#pragma unroll
  for (int k = 0; k < kChunksPer; ++k)
    if (from[k] >= 0) {
      kk[k] = static_cast<const uint4*>(a.k)[src[k]];
      vv[k] = static_cast<const uint4*>(a.v)[src[k]];
    }
#pragma unroll
  for (int k = 0; k < kChunksPer; ++k)
    if (from[k] >= 0) {
      static_cast<uint4*>(a.k_out)[dst[k]] = kk[k];
      static_cast<uint4*>(a.v_out)[dst[k]] = vv[k];
    }
}

}  // namespace

int launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int es = a.dtype == LONGNET_DTYPE_F32 ? 4 : 2;
  const int head_chunks = a.D * es / 16;
  const int64_t chunks = (int64_t)a.budget * a.Hkv * head_chunks;  // of a sequence
  if (chunks + kMoveThreads * kChunksPer > 0x7fffffffLL) return LONGNET_ERR_UNSUPPORTED;
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  const unsigned pairs = (unsigned)(a.S * a.Hkv);
  if (cap <= kHeld) {
    if (!opt_in_smem<select_kernel<true>>(kHeld * 4)) return LONGNET_ERR_CUDA;
    select_kernel<true><<<pairs, kSelThreads, (size_t)cap * 4, stream>>>(a);
  } else {
    select_kernel<false><<<pairs, kSelThreads, 0, stream>>>(a);
  }
  if (cudaGetLastError() != cudaSuccess) return LONGNET_ERR_CUDA;
  move_kernel<<<dim3((unsigned)((chunks + kMoveThreads * kChunksPer - 1) / (kMoveThreads * kChunksPer)), (unsigned)a.S),
                kMoveThreads, 0, stream>>>(a, head_chunks);
  return cudaGetLastError() == cudaSuccess ? LONGNET_OK : LONGNET_ERR_CUDA;
}

}  // namespace longnet
