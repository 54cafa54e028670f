// Eviction from a paged cache by accumulated attention weight.
//
// A sequence of n > budget keys keeps, for each key/value head, its first
// `sinks` keys, its last `recent` keys, and of the others the budget - sinks -
// recent with the largest weights (equal weights: the lowest index first; NaN
// below every number).  A sequence of n <= budget keys keeps them all.  Kept
// keys stay in order: the j-th kept key becomes key j of the new cache.
//
// Two kernels.  Select, one CTA per (sequence, head): the need-th largest
// weight by a radix select on the weights' order-preserving 32-bit images (four
// 8-bit digits, each a histogram in shared memory), then one pass in index
// order that writes the kept indices and their weights.  Move: one thread per
// 16-byte chunk of a kept key and value row, neighbours along the row and then
// the heads of a slot, so both sides move whole sectors.
// Bound: DRAM, the kept rows read and written once; the weights are read from
// DRAM once and from L2 after that.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_args.cuh"

namespace longnet {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kPer = 4;  // keys of a thread in the ordered pass

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

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[256], warp_sums[32];
  __shared__ uint32_t s_prefix, s_need;
  const int s = blockIdx.x / a.Hkv, f = blockIdx.x % a.Hkv;
  const int64_t cap = (int64_t)a.max_pages << a.page_shift, out_cap = (int64_t)a.max_out_pages << a.page_shift;
  int n = a.kv_len[s];
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0) record_status(a.status, kStatusBounds);
    n = 0;
  }
  const float* w = a.weights + (int64_t)blockIdx.x * cap;
  float* nw = a.new_weights + (int64_t)blockIdx.x * out_cap;
  int* kept = a.kept + (int64_t)blockIdx.x * a.budget;
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
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (threadIdx.x < 256) hist[threadIdx.x] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int j = lo + threadIdx.x; j < hi; j += kSelThreads) {
        const uint32_t u = image(w[j]);
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255], 1u);
      }
      __syncthreads();
      // the digit whose count, added to those above it, first reaches rest
      const uint32_t c = threadIdx.x < 256 ? hist[255 - threadIdx.x] : 0u;
      uint32_t total;
      const uint32_t above = block_scan(c, warp_sums, &total);
      if (threadIdx.x < 256 && above < rest && above + c >= rest) {
        s_prefix = prefix | ((uint32_t)(255 - threadIdx.x) << shift);
        s_need = rest - above;
      }
      __syncthreads();
      prefix = s_prefix;
      rest = s_need;
      __syncthreads();
    }
  }
  // in index order: forced keys, those above the threshold, and the first
  // `rest` equal to it
  uint32_t sure_before = 0, equal_before = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads * kPer) {
    const int j0 = t0 + threadIdx.x * kPer;
    float x[kPer];
    uint32_t kind[kPer], count = 0;  // 0 no, 1 << 16 surely kept, 1 equal to the threshold
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = j0 + i;
      kind[i] = 0;
      x[i] = 0.f;
      if (j < n) {
        x[i] = w[j];
        if (j < lo || j >= hi) {
          kind[i] = 1u << 16;
        } else if (need > 0) {
          const uint32_t u = image(x[i]);
          kind[i] = u > prefix ? 1u << 16 : u == prefix ? 1u : 0u;
        }
      }
      count += kind[i];
    }
    uint32_t total;
    uint32_t before = block_scan(count, warp_sums, &total);
    uint32_t sure = sure_before + (before >> 16), equal = equal_before + (before & 0xffffu);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool keep = kind[i] == (1u << 16) || (kind[i] == 1u && equal < rest);
      if (keep) {
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

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a, int head_chunks) {
  const int row_chunks = a.Hkv * head_chunks;
  const int64_t e = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x;
  const int64_t sj = e / row_chunks;
  if (sj >= (int64_t)a.S * a.budget) return;
  const int c = (int)(e % row_chunks), f = c / head_chunks;
  const int s = (int)(sj / a.budget), j = (int)(sj % a.budget);
  const int from = a.kept[((int64_t)s * a.Hkv + f) * a.budget + j];
  if (from < 0) return;
  const int pg = a.table[(int64_t)s * a.max_pages + (from >> a.page_shift)];
  const int to = a.new_table[(int64_t)s * a.max_out_pages + (j >> a.page_shift)];
  if (pg < 0 || pg >= a.n_pages || to < 0 || to >= a.n_out_pages) {
    record_status(a.status, kStatusBounds);
    return;
  }
  const int64_t src = (((int64_t)pg << a.page_shift) + (from & (a.page - 1))) * row_chunks + c;
  const int64_t dst = (((int64_t)to << a.page_shift) + (j & (a.page - 1))) * row_chunks + c;
  static_cast<uint4*>(a.k_out)[dst] = static_cast<const uint4*>(a.k)[src];
  static_cast<uint4*>(a.v_out)[dst] = static_cast<const uint4*>(a.v)[src];
}

}  // namespace

int launch_evict(const EvictArgs& a, cudaStream_t stream) {
  select_kernel<<<(unsigned)(a.S * a.Hkv), kSelThreads, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return LONGNET_ERR_CUDA;
  const int es = a.dtype == LONGNET_DTYPE_F32 ? 4 : 2;
  const int head_chunks = a.D * es / 16;
  const int64_t work = (int64_t)a.S * a.budget * a.Hkv * head_chunks;
  const int64_t blocks = (work + kMoveThreads - 1) / kMoveThreads;
  if (blocks > 0x7fffffffLL) return LONGNET_ERR_UNSUPPORTED;
  move_kernel<<<(unsigned)blocks, kMoveThreads, 0, stream>>>(a, head_chunks);
  return cudaGetLastError() == cudaSuccess ? LONGNET_OK : LONGNET_ERR_CUDA;
}

}  // namespace longnet
