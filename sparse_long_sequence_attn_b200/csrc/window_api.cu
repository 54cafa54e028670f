// C entry points of the sliding-window and paged-cache attention: argument
// checks, family choice and launches.  Everything the host can see is checked
// before anything is enqueued; what only the device holds (lengths, page
// numbers) is checked by the kernels and recorded in the status word.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "attn_args.cuh"
#include "decode.cuh"
#include "longnet.h"
#include "params.h"
#include "window_tc.cuh"

using namespace longnet;

namespace longnet {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int dtype) {
  return dtype == LONGNET_DTYPE_F32 || dtype == LONGNET_DTYPE_BF16 || dtype == LONGNET_DTYPE_F16;
}
bool dim_ok(int64_t D) { return D == 16 || D == 32 || D == 64 || D == 128; }

int shift_of(int64_t page) {
  int s = 0;
  while (((int64_t)1 << s) < page) ++s;
  return s;
}

void set_heads(AttnArgs* a, int64_t H, int64_t Hkv, int64_t D, int dtype) {
  a->H = (int)H;
  a->Hkv = (int)Hkv;
  a->G = (int)(H / Hkv);
  a->D = (int)D;
  a->dtype = dtype;
  a->scale = 1.f / sqrtf((float)D);
  a->scale_log2 = 1.4426950408889634f * a->scale;
}

// Sizes of the contiguous form.
int check_window(int64_t B, int64_t N, int64_t H, int64_t Hkv, int64_t D, int64_t window, int64_t sinks, int dtype) {
  if (B <= 0 || N <= 0 || H <= 0 || Hkv <= 0 || D <= 0 || window < 1 || sinks < 0 || !dtype_ok(dtype))
    return LONGNET_ERR_INVALID_ARG;
  if (H % Hkv != 0) return LONGNET_ERR_INVALID_ARG;
  if (!dim_ok(D)) return LONGNET_ERR_UNSUPPORTED;
  // packed rows and token rows are 32-bit in the kernels; (batch, head) pairs
  // are a grid's second dimension
  if (B > 65535 || H > 65535 || B * Hkv > 65535 || N > ((int64_t)1 << 30) || N * H > ((int64_t)1 << 30) ||
      B * N > ((int64_t)1 << 30))
    return LONGNET_ERR_UNSUPPORTED;
  return LONGNET_OK;
}

void fill_window(AttnArgs* a, const void* q, const void* k, const void* v, void* out, float* lse, int64_t B,
                 int64_t N, int64_t H, int64_t Hkv, int64_t D, int64_t window, int64_t sinks, int dtype) {
  memset(a, 0, sizeof(*a));
  a->q = q;
  a->k = k;
  a->v = v;
  a->out = out;
  a->lse = lse;
  a->T = B * N;
  a->S = (int)B;
  a->nq_max = (int)N;
  set_heads(a, H, Hkv, D, dtype);
  a->window = (int)(window < N ? window : N);  // N: every earlier key
  a->sinks = (int)(sinks < N ? sinks : N);
}

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

// The workspace of the backward: delta, fp16's peaks, then the partials of the
// family that needs most, so that it does not depend on the family.
int64_t peak_bytes(int dtype) { return dtype == LONGNET_DTYPE_F16 ? round256(8 * kPeakBlocks) : 0; }
int64_t bwd_workspace(int64_t B, int64_t N, int64_t H, int64_t Hkv, int64_t D, int64_t window, int64_t sinks,
                      int dtype) {
  window = window < N ? window : N;
  sinks = sinks < N ? sinks : N;
  const KeyPlan ks = simt_key_plan(B, N, H, Hkv, window, sinks);
  const KeyPlan kt = key_plan(B, N, H, Hkv, window, sinks, window_bwd_tc_tile(D), kTcMinBlocks, kTcCtas);
  const int64_t simt = key_partial_floats(ks, B, Hkv, D), tc = key_partial_floats(kt, B, Hkv, D);
  return round256(4 * B * N * H) + peak_bytes(dtype) + round256(4 * (simt > tc ? simt : tc));
}

int check_cache(int64_t S, int64_t Hkv, int64_t D, int64_t n_pages, int64_t page, int64_t max_pages, int dtype) {
  if (S <= 0 || Hkv <= 0 || D <= 0 || n_pages <= 0 || page <= 0 || max_pages <= 0 || !dtype_ok(dtype))
    return LONGNET_ERR_INVALID_ARG;
  if (!dim_ok(D) || page < 8 || page > 256 || (page & (page - 1)) != 0) return LONGNET_ERR_UNSUPPORTED;
  // each factor before its product, which could pass 64 bits
  constexpr int64_t kMost = (int64_t)1 << 30;
  if (S > 65535 || Hkv > 65535 || S * Hkv > 65535 || n_pages > kMost || max_pages > kMost || max_pages * page > kMost)
    return LONGNET_ERR_UNSUPPORTED;
  return LONGNET_OK;
}

void fill_cache(AttnArgs* a, const void* k_pages, const void* v_pages, const int32_t* cu_q, const int32_t* kv_len,
                const int32_t* table, int64_t T, int64_t S, int64_t n_pages, int64_t page, int64_t max_pages) {
  a->k = k_pages;
  a->v = v_pages;
  a->cu_q = cu_q;
  a->kv_len = kv_len;
  a->table = table;
  a->T = T;
  a->S = (int)S;
  a->n_pages = (int)n_pages;
  a->page = (int)page;
  a->page_shift = shift_of(page);
  a->max_pages = (int)max_pages;
}

}  // namespace
}  // namespace longnet

extern "C" int longnet_window_attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int64_t B,
                                       int64_t N, int64_t H, int64_t Hkv, int64_t D, int64_t window, int64_t sinks,
                                       int dtype, int impl, longnet_stream_t stream) {
  if (!q || !k || !v || !out) return LONGNET_ERR_INVALID_ARG;
  if (impl != LONGNET_IMPL_AUTO && impl != LONGNET_IMPL_SIMT && impl != LONGNET_IMPL_TCGEN05)
    return LONGNET_ERR_INVALID_ARG;
  int rc = check_window(B, N, H, Hkv, D, window, sinks, dtype);
  if (rc) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)))
    return LONGNET_ERR_MISALIGNED;
  AttnArgs a;
  fill_window(&a, q, k, v, out, lse, B, N, H, Hkv, D, window, sinks, dtype);
  const bool tc = window_tc_supports(a);
  if (impl == LONGNET_IMPL_TCGEN05 && !tc) return LONGNET_ERR_UNSUPPORTED;
  int dev = 0;
  rc = device_state(&dev, &a.status);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return tc && impl != LONGNET_IMPL_SIMT ? launch_window_fwd_tc(a, nullptr, st) : launch_window_fwd_simt(a, st);
}

extern "C" int64_t longnet_window_bwd_workspace_bytes(int64_t B, int64_t N, int64_t H, int64_t Hkv, int64_t D,
                                                      int64_t window, int64_t sinks, int dtype) {
  const int rc = check_window(B, N, H, Hkv, D, window, sinks, dtype);
  if (rc) return rc;
  return bwd_workspace(B, N, H, Hkv, D, window, sinks, dtype);
}

extern "C" int longnet_window_attn_bwd(const void* q, const void* k, const void* v, const void* out,
                                       const float* lse, const void* dout, void* dq, void* dk, void* dv, int64_t B,
                                       int64_t N, int64_t H, int64_t Hkv, int64_t D, int64_t window, int64_t sinks,
                                       int dtype, int impl, void* workspace, int64_t workspace_bytes,
                                       longnet_stream_t stream) {
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv) return LONGNET_ERR_INVALID_ARG;
  if (impl != LONGNET_IMPL_AUTO && impl != LONGNET_IMPL_SIMT && impl != LONGNET_IMPL_TCGEN05)
    return LONGNET_ERR_INVALID_ARG;
  int rc = check_window(B, N, H, Hkv, D, window, sinks, dtype);
  if (rc) return rc;
  if (!workspace ||
      workspace_bytes < longnet_window_bwd_workspace_bytes(B, N, H, Hkv, D, window, sinks, dtype))
    return LONGNET_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, out, dout, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!aligned(p, 16)) return LONGNET_ERR_MISALIGNED;
  if (!aligned(lse, 4) || !aligned(workspace, 256)) return LONGNET_ERR_MISALIGNED;
  AttnArgs a;
  fill_window(&a, q, k, v, const_cast<void*>(out), const_cast<float*>(lse), B, N, H, Hkv, D, window, sinks, dtype);
  const bool tc = window_bwd_tc_supports(a);
  if (impl == LONGNET_IMPL_TCGEN05 && !tc) return LONGNET_ERR_UNSUPPORTED;
  int dev = 0;
  rc = device_state(&dev, &a.status);
  if (rc) return rc;
  WindowBwdArgs g;
  g.dout = dout;
  g.dq = dq;
  g.dk = dk;
  g.dv = dv;
  g.delta = static_cast<float*>(workspace);
  g.peaks = reinterpret_cast<float*>(static_cast<char*>(workspace) + round256(4 * B * N * H));
  g.partial = reinterpret_cast<float*>(reinterpret_cast<char*>(g.peaks) + peak_bytes(dtype));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return tc && impl != LONGNET_IMPL_SIMT ? launch_window_bwd_tc(a, g, st) : launch_window_bwd_simt(a, g, st);
}

extern "C" int longnet_paged_append(const void* k_tok, const void* v_tok, void* k_pages, void* v_pages,
                                    float* weights, const int32_t* cu_q, const int32_t* kv_len,
                                    const int32_t* table, int64_t T, int64_t S, int64_t Hkv, int64_t D,
                                    int64_t n_pages, int64_t page, int64_t max_pages, int dtype,
                                    longnet_stream_t stream) {
  if (T < 0) return LONGNET_ERR_INVALID_ARG;
  int rc = check_cache(S, Hkv, D, n_pages, page, max_pages, dtype);
  if (rc) return rc;
  if (!k_pages || !v_pages || !cu_q || !kv_len || !table || (T > 0 && (!k_tok || !v_tok)))
    return LONGNET_ERR_INVALID_ARG;
  if (T > ((int64_t)1 << 30)) return LONGNET_ERR_UNSUPPORTED;
  if (!aligned(k_tok, 16) || !aligned(v_tok, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(cu_q, 4) || !aligned(kv_len, 4) || !aligned(table, 4) || !aligned(weights, 4))
    return LONGNET_ERR_MISALIGNED;
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  set_heads(&a, Hkv, Hkv, D, dtype);
  fill_cache(&a, k_pages, v_pages, cu_q, kv_len, table, T, S, n_pages, page, max_pages);
  int dev = 0;
  rc = device_state(&dev, &a.status);
  if (rc) return rc;
  if (T == 0) return LONGNET_OK;
  return launch_paged_append(a, k_tok, v_tok, weights, reinterpret_cast<cudaStream_t>(stream));
}

namespace longnet {
namespace {
int check_paged(int64_t S, int64_t max_q, int64_t H, int64_t Hkv, int64_t D, int64_t page, int64_t max_pages,
                int64_t window, int64_t sinks, int dtype) {
  const int rc = check_cache(S, Hkv, D, 1, page, max_pages, dtype);
  if (rc) return rc;
  if (max_q <= 0 || H <= 0 || H % Hkv != 0 || window < 0 || sinks < 0) return LONGNET_ERR_INVALID_ARG;
  if (H > 65535 || max_q > ((int64_t)1 << 30) || max_q * H > ((int64_t)1 << 30)) return LONGNET_ERR_UNSUPPORTED;
  return LONGNET_OK;
}

// The sizes of a checked paged call (no pointers): what its plan goes by.
void fill_paged(AttnArgs* a, int64_t S, int64_t max_q, int64_t H, int64_t Hkv, int64_t D, int64_t page,
                int64_t max_pages, int64_t window, int64_t sinks, int dtype) {
  static const int32_t paged = 0;  // cu_q set: the paged form
  memset(a, 0, sizeof(*a));
  set_heads(a, H, Hkv, D, dtype);
  fill_cache(a, nullptr, nullptr, &paged, nullptr, nullptr, 0, S, 0, page, max_pages);
  a->nq_max = (int)max_q;
  const int64_t cap = max_pages * page;
  a->window = window == 0 || window >= cap ? 0 : (int)window;
  a->sinks = (int)(sinks < cap ? sinks : cap);
}

// The workspace of a paged call: the parts of the family that needs most, so
// that it does not depend on the family.
int64_t paged_workspace(const AttnArgs& a, bool weights) {
  if (!window_tc_supports(a)) return 0;
  const int64_t tc = window_tc_part_floats(a, window_tc_plan(a));
  const int64_t dec = decode_supports(a) ? decode_workspace_floats(a, weights) : 0;
  return round256(4 * (tc > dec ? tc : dec));
}
}  // namespace
}  // namespace longnet

extern "C" int64_t longnet_paged_workspace_bytes(int64_t S, int64_t max_q, int64_t H, int64_t Hkv, int64_t D,
                                                 int64_t page, int64_t max_pages, int64_t window, int64_t sinks,
                                                 int dtype, int weights) {
  const int rc = check_paged(S, max_q, H, Hkv, D, page, max_pages, window, sinks, dtype);
  if (rc) return rc;
  if (weights != 0 && weights != 1) return LONGNET_ERR_INVALID_ARG;
  AttnArgs a;
  fill_paged(&a, S, max_q, H, Hkv, D, page, max_pages, window, sinks, dtype);
  return paged_workspace(a, weights != 0);
}

extern "C" int longnet_paged_attn_fwd(const void* q, const void* k_pages, const void* v_pages, void* out, float* lse,
                                      float* weights, const int32_t* cu_q, const int32_t* kv_len,
                                      const int32_t* table, int64_t T, int64_t S, int64_t max_q, int64_t H,
                                      int64_t Hkv, int64_t D, int64_t n_pages, int64_t page, int64_t max_pages,
                                      int64_t window, int64_t sinks, int dtype, int impl, void* workspace,
                                      int64_t workspace_bytes, longnet_stream_t stream) {
  if (T < 0 || n_pages <= 0) return LONGNET_ERR_INVALID_ARG;
  if (impl != LONGNET_IMPL_AUTO && impl != LONGNET_IMPL_SIMT && impl != LONGNET_IMPL_TCGEN05 &&
      impl != LONGNET_IMPL_DECODE)
    return LONGNET_ERR_INVALID_ARG;
  int rc = check_paged(S, max_q, H, Hkv, D, page, max_pages, window, sinks, dtype);
  if (rc) return rc;
  rc = check_cache(S, Hkv, D, n_pages, page, max_pages, dtype);
  if (rc) return rc;
  if (!k_pages || !v_pages || !cu_q || !kv_len || !table || (T > 0 && (!q || !out || (weights && !lse))))
    return LONGNET_ERR_INVALID_ARG;
  if (T > ((int64_t)1 << 30)) return LONGNET_ERR_UNSUPPORTED;
  const int64_t need =
      longnet_paged_workspace_bytes(S, max_q, H, Hkv, D, page, max_pages, window, sinks, dtype, weights ? 1 : 0);
  if (workspace_bytes < need || (need > 0 && !workspace)) return LONGNET_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(weights, 4) || !aligned(cu_q, 4) || !aligned(kv_len, 4) || !aligned(table, 4) ||
      !aligned(workspace, 256))
    return LONGNET_ERR_MISALIGNED;
  AttnArgs a;
  fill_paged(&a, S, max_q, H, Hkv, D, page, max_pages, window, sinks, dtype);
  fill_cache(&a, k_pages, v_pages, cu_q, kv_len, table, T, S, n_pages, page, max_pages);
  a.q = q;
  a.out = out;
  a.lse = lse;
  const bool tc = window_tc_supports(a), dec = decode_supports(a);
  if ((impl == LONGNET_IMPL_DECODE && !dec) || (impl == LONGNET_IMPL_TCGEN05 && !tc)) return LONGNET_ERR_UNSUPPORTED;
  int dev = 0;
  rc = device_state(&dev, &a.status);
  if (rc) return rc;
  if (T == 0) return LONGNET_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dec && (impl == LONGNET_IMPL_AUTO || impl == LONGNET_IMPL_DECODE))
    return launch_decode(a, static_cast<float*>(workspace), weights, st);
  if (tc && impl != LONGNET_IMPL_SIMT) {
    rc = launch_window_fwd_tc(a, static_cast<float*>(workspace), st);
    return rc || !weights ? rc : launch_weights_tc(a, weights, st);
  }
  rc = launch_window_fwd_simt(a, st);
  return rc || !weights ? rc : launch_weights_simt(a, weights, st);
}

extern "C" int longnet_cache_evict(const void* k_pages, const void* v_pages, const float* weights,
                                   const int32_t* kv_len, const int32_t* table, void* k_out, void* v_out,
                                   float* new_weights, int32_t* new_len, int32_t* kept, const int32_t* new_table,
                                   int64_t S, int64_t Hkv, int64_t D, int64_t n_pages, int64_t page,
                                   int64_t max_pages, int64_t n_out_pages, int64_t max_out_pages, int64_t budget,
                                   int64_t sinks, int64_t recent, int dtype, longnet_stream_t stream) {
  int rc = check_cache(S, Hkv, D, n_pages, page, max_pages, dtype);
  if (rc) return rc;
  rc = check_cache(S, Hkv, D, n_out_pages, page, max_out_pages, dtype);
  if (rc) return rc;
  if (!k_pages || !v_pages || !weights || !kv_len || !table || !k_out || !v_out || !new_weights || !new_len ||
      !kept || !new_table)
    return LONGNET_ERR_INVALID_ARG;
  if (budget <= 0 || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks ||
      budget > max_out_pages * page)
    return LONGNET_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
      !aligned(weights, 4) || !aligned(kv_len, 4) || !aligned(table, 4) || !aligned(new_weights, 4) ||
      !aligned(new_len, 4) || !aligned(kept, 4) || !aligned(new_table, 4))
    return LONGNET_ERR_MISALIGNED;
  EvictArgs e;
  memset(&e, 0, sizeof(e));
  e.k = k_pages;
  e.v = v_pages;
  e.weights = weights;
  e.kv_len = kv_len;
  e.table = table;
  e.k_out = k_out;
  e.v_out = v_out;
  e.new_weights = new_weights;
  e.new_len = new_len;
  e.kept = kept;
  e.new_table = new_table;
  e.S = (int)S;
  e.Hkv = (int)Hkv;
  e.D = (int)D;
  e.n_pages = (int)n_pages;
  e.page = (int)page;
  e.page_shift = shift_of(page);
  e.max_pages = (int)max_pages;
  e.n_out_pages = (int)n_out_pages;
  e.max_out_pages = (int)max_out_pages;
  e.budget = (int)budget;
  e.sinks = (int)sinks;
  e.recent = (int)recent;
  e.dtype = dtype;
  int dev = 0;
  rc = device_state(&dev, &e.status);
  if (rc) return rc;
  return launch_evict(e, reinterpret_cast<cudaStream_t>(stream));
}
