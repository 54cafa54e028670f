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
// workspace: delta [S, H, N] fp32, fp16's peaks, then the partials of the key
// tiles.
struct WindowBwdArgs {
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  float* delta;
  float* peaks;  // [kPeakBlocks][2]
  float* partial;
};
constexpr int kPeakBlocks = 148 * 6;  // of launch_window_peaks, at most
// How dk and dv are cut into work items, one CTA each: a tile of keys by a
// range of the queries that see it.  A tile's near queries (those its window
// reaches) are cut into `near` ranges where the tiles alone would leave SMs
// idle; a tile holding sinks has far queries past its window, in ranges of
// `chunk`.  A tile with more than one item gets a partial (a slot) from each,
// which launch_key_reduce adds in order.
struct KeyPlan {
  int tile, tiles;   // keys of a tile, tiles
  int near;          // near items of a tile
  int sink_tiles;    // tiles with far items
  int chunk, chunks; // queries of a far item; far items of a tile
  __host__ __device__ int items() const { return sink_tiles * chunks + tiles * near; }
  // slots of the tiles before t, of one (batch, head)
  __host__ __device__ int slot_of(int t) const {
    return t <= sink_tiles ? t * (near + chunks) : sink_tiles * (near + chunks) + (near > 1 ? (t - sink_tiles) * near : 0);
  }
  __host__ __device__ int slots() const { return slot_of(tiles); }
  __host__ __device__ int reduced() const { return near > 1 ? tiles : sink_tiles; }  // tiles with partials
};
// One item: queries [i0, i1) (none when i0 >= i1) for the tile, into a slot, or
// straight into dk and dv (slot -1).
struct KeyItem {
  int tile, i0, i1, slot;
};
__device__ __forceinline__ KeyItem key_item(const AttnArgs& a, const KeyPlan& k, int x) {
  KeyItem it;
  const int N = a.nq_max, fars = k.sink_tiles * k.chunks;
  const bool far = x < fars;  // far items first: they are as long as any
  const int part = far ? x % k.chunks : (x - fars) % k.near;
  it.tile = far ? x / k.chunks : (x - fars) / k.near;
  const int first = it.tile * k.tile;
  // the near queries end where the window of the tile's last key does, or, for
  // a tile with sinks whose far queries have no items, with the sequence
  const int64_t reach = (int64_t)first + k.tile - 1 + a.window;
  const int end = reach >= N || (first < a.sinks && it.tile >= k.sink_tiles) ? N : (int)reach;
  const int len = far ? k.chunk : (end - first + k.near - 1) / k.near;
  const int64_t i0 = (int64_t)(far ? end : first) + (int64_t)part * len, stop = far ? N : end;
  it.i0 = i0 < stop ? (int)i0 : (int)stop;
  it.i1 = i0 + len < stop ? (int)(i0 + len) : (int)stop;
  it.slot = k.near > 1 || it.tile < k.sink_tiles ? k.slot_of(it.tile) + (far ? k.near + part : part) : -1;
  return it;
}
KeyPlan key_plan(int64_t S, int64_t N, int64_t H, int64_t Hkv, int64_t window, int64_t sinks, int tile, int min_blocks,
                 int ctas);
int64_t key_partial_floats(const KeyPlan& k, int64_t S, int64_t Hkv, int64_t D);
// the SIMT family's
KeyPlan simt_key_plan(int64_t S, int64_t N, int64_t H, int64_t Hkv, int64_t window, int64_t sinks);
int launch_window_bwd_simt(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream);
// delta = <dout, out> of every row, and the last step both families share.
int launch_window_delta(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream);
// fp16: the largest |dout_x|^2 and |v_j|^2 of each of its *blocks blocks' rows, to
// g.peaks, and with them, when asked for, delta.
int launch_window_peaks(const AttnArgs& a, const WindowBwdArgs& g, bool with_delta, int* blocks, cudaStream_t stream);
int launch_key_reduce(const AttnArgs& a, const WindowBwdArgs& g, const KeyPlan& k, cudaStream_t stream);

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
