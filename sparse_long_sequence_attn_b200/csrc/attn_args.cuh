// Arguments and index arithmetic shared by the sliding-window and paged-cache
// attention kernels.
//
// Both attend causally with one mask: the query at position x sees key j when
// j <= x and (window == 0 or x - j < window or j < sinks).  The contiguous
// form (training) has S batches of N tokens; the paged form (serving) has S
// sequences whose new tokens are packed one after the other (cu_q) and whose
// keys and values lie in pages (table).  Query head h reads key/value head
// h / G, G = H / Hkv, so the G * nq query rows of one key/value head are taken
// as packed rows, row = i * G + g, and share every key they read.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_util.cuh"
#include "params.h"

namespace longnet {

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;       // [S, H, N] (contiguous) or [T, H] (paged); may be null
  int64_t T;        // token rows of q
  int S;            // batches or sequences
  int nq_max;       // N, or the most new tokens a sequence has
  int H, Hkv, G, D;
  int dtype;
  int window, sinks;  // window 0: every earlier key
  // paged form; null / zero for the contiguous one
  const int* cu_q;    // [S + 1] first token row of each sequence
  const int* kv_len;  // [S] cached keys, the new tokens' among them
  const int* table;   // [S, max_pages] page of keys [p page, (p + 1) page)
  int n_pages, page, max_pages;
  int page_shift;     // log2 page
  float scale, scale_log2;
  int* status;
};

// One sequence: its token rows [q0, q0 + nq), the position of the first, its
// keys [0, kv).  A sequence whose entries are out of range records the
// bounds status and is taken as empty.
struct Seq {
  int64_t q0;
  int nq, first, kv;
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int s) {
  Seq r;
  if (!a.cu_q) {
    r.q0 = (int64_t)s * a.nq_max;
    r.nq = a.nq_max;
    r.first = 0;
    r.kv = a.nq_max;
    return r;
  }
  const int c0 = a.cu_q[s], c1 = a.cu_q[s + 1], kv = a.kv_len[s];
  r.q0 = c0;
  r.nq = c1 - c0;
  r.kv = kv;
  r.first = kv - r.nq;
  if (c0 < 0 || c1 < c0 || c1 > a.T || c1 - c0 > a.nq_max || kv < 0 || kv > (int64_t)a.max_pages << a.page_shift) {
    record_status(a.status, kStatusBounds);
    r.q0 = 0;
    r.nq = r.first = r.kv = 0;
  }
  return r;
}

// Index of (sequence s at token i, head h) in lse.
__device__ __forceinline__ int64_t lse_index(const AttnArgs& a, const Seq& q, int s, int i, int h) {
  return a.cu_q ? (q.q0 + i) * a.H + h : ((int64_t)s * a.H + h) * a.nq_max + i;
}

// Element offset of key j's row (head f), or -1 when its page is out of range
// (recorded in the status word; the row then counts as zeros).
__device__ __forceinline__ int64_t kv_row(const AttnArgs& a, const Seq& q, int s, int f, int j) {
  if (!a.cu_q) return ((q.q0 + j) * a.Hkv + f) * a.D;
  const int pg = a.table[(int64_t)s * a.max_pages + (j >> a.page_shift)];
  if (pg < 0 || pg >= a.n_pages) {
    record_status(a.status, kStatusBounds);
    return -1;
  }
  return ((((int64_t)pg << a.page_shift) + (j & (a.page - 1))) * a.Hkv + f) * a.D;
}

__device__ __forceinline__ bool sees(const AttnArgs& a, int x, int j) {
  return j <= x && (a.window == 0 || x - j < a.window || j < a.sinks);
}

// The key blocks (of kBlk keys) that queries at positions [lo, hi] see: the
// blocks holding sinks, then those from the window's first key on.  Block n
// (n < count) is block at(n); ascending, none twice.
struct BlockList {
  int n_sink, win0, count;
  __device__ __forceinline__ int at(int n) const { return n < n_sink ? n : win0 + (n - n_sink); }
};
template <int kBlk>
__device__ __forceinline__ BlockList blocks_of(const AttnArgs& a, int lo, int hi) {
  BlockList b;
  if (hi < 0) {
    b.n_sink = b.win0 = b.count = 0;
    return b;
  }
  if (lo < 0) lo = 0;
  const int last = hi / kBlk;
  const int low = a.window == 0 || lo < a.window ? 0 : lo - a.window + 1;
  b.win0 = low / kBlk;
  // sink blocks below the window's first block
  b.n_sink = a.sinks > 0 ? (a.sinks - 1) / kBlk + 1 : 0;
  if (b.n_sink > b.win0) b.n_sink = b.win0;
  b.count = b.n_sink + last - b.win0 + 1;
  return b;
}

// Launchers (host).  Each returns a longnet_status.
int launch_window_fwd_simt(const AttnArgs& a, cudaStream_t stream);
int launch_weights_simt(const AttnArgs& a, float* weights, cudaStream_t stream);

// The backward's extra arguments: gradients in the inputs' dtype, and the
// workspace: delta [S, H, N] fp32, then the far partials of the sink tiles.
struct WindowBwdArgs {
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  float* delta;
  float* partial;
};
// Key tiles (of window_tile(impl) keys) holding sinks take the queries past
// their window in `chunks` further work items, each summed on its own.
struct FarPlan {
  int tile;         // keys of a tile
  int sink_tiles;   // tiles with far work
  int chunk;        // queries of a far item
  int chunks;       // far items of the first tile (the most any has)
};
FarPlan far_plan(int64_t S, int64_t N, int64_t H, int64_t Hkv, int64_t window, int64_t sinks, int tile);
int64_t far_partial_floats(const FarPlan& f, int64_t S, int64_t Hkv, int64_t D);
int launch_window_bwd_simt(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream);
// The last steps both families share: delta = <dout, out>, and the far
// partials of the sink tiles summed in order into dk and dv.
int launch_window_delta(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream);
int launch_far_reduce(const AttnArgs& a, const WindowBwdArgs& g, const FarPlan& f, cudaStream_t stream);

int launch_paged_append(const AttnArgs& a, const void* k_tok, const void* v_tok, float* weights, cudaStream_t stream);

struct EvictArgs {
  const void* k;
  const void* v;
  const float* weights;  // [S, Hkv, max_pages * page]
  const int* kv_len;
  const int* table;      // [S, max_pages]
  void* k_out;
  void* v_out;
  float* new_weights;    // [S, Hkv, max_out_pages * page]
  int* new_len;
  int* kept;             // [S, Hkv, budget]
  const int* new_table;  // [S, max_out_pages]
  int S, Hkv, D, n_pages, page, page_shift, max_pages, n_out_pages, max_out_pages;
  int budget, sinks, recent, dtype;
  int* status;
};
int launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace longnet
