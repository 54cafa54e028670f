// The sliding-window and paged-cache attention on the CUDA cores: forward,
// weight sums and backward in fp32 arithmetic for every dtype, D = 16, 32, 64
// or 128.  AUTO takes it for fp32; the 16-bit formats run on the tensor-core
// families and are checked against it.
//
// Mathematics.  Forward: softmax(Q K^T / sqrt(D)) V over the visible keys, one
// pass with the running maximum and sum of each row.  Weight sums: per key,
// the sum over its queries of P = e^{s - lse}.  Backward, with
// delta = <dout, out>: P = e^{s - lse}, dS = P (dout V^T - delta),
// dQ = dS K / sqrt(D), dK = dS^T Q / sqrt(D), dV = P^T dout.
//
// Layout.  A CTA of 16 x 16 threads owns 16 RT rows (packed query rows, or keys;
// RT = 4, or 1 for small problems) and streams 64-row blocks of the other
// side through shared memory as fp32; a thread holds an RT x 4 piece of the
// scores and an RT x D/16 piece of the accumulators, so that at RT = 4 every
// value read from shared memory feeds four multiply-adds.  Rows are padded by four
// floats, which keeps the 16-byte reads of 8 lanes in different banks.  Products
// stay fp32 for fp32 inputs (no TF32).  The bound is shared memory, which hands out
// 128 bytes a clock: at two bytes or more for each multiply-add, half of the fp32
// pipe's rate at most; and for small problems a CTA's latency.  Measured, fp32,
// forward, dq, and dk with dv: 997 tokens, 6/2 heads of 32, window 200: 22, 23 and 34
// us; 1500 tokens, 8 heads of 128, window 500: 171, 224 and 304 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_args.cuh"
#include "launch_util.cuh"

namespace longnet {
namespace ws {

constexpr int kT = 64;        // rows of a tile, keys of a block
constexpr int kThreads = 256;
constexpr int kPS = kT + 4;   // row stride of a score tile
constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct L {
  static constexpr int kStride = D + 4;
  static constexpr int kTile = kT * kStride;  // floats
  static constexpr int kC = D / 16;           // accumulator columns of a thread
  static constexpr int kV = kC < 4 ? kC : 4;  // consecutive ones
  __device__ static int col(int tx, int c) { return (c / kV) * (16 * kV) + tx * kV + c % kV; }
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// ROWS rows of D elements on their way to shared memory: fetched into registers
// (16 bytes at a time; off(r) is a row's element offset, negative for a row of
// zeros), then stored as fp32.  A block is fetched while the one before is
// computed.
template <typename T, int D, int ROWS = kT>
struct Fetch {
  static constexpr int kVec = 16 / sizeof(T);  // elements of a 16-byte load
  static constexpr int kChunks = D / kVec;
  static constexpr int kAll = ROWS * kChunks, kN = (kAll + kThreads - 1) / kThreads;
  uint4 x[kN];
  template <typename Off>
  __device__ __forceinline__ void get(const T* src, Off off) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = threadIdx.x + i * kThreads;
      const int64_t o = kAll % kThreads == 0 || e < kAll ? off(e / kChunks) : -1;
      x[i] = o < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(src + o + (e % kChunks) * kVec);
    }
  }
  __device__ __forceinline__ void put(float* dst) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = threadIdx.x + i * kThreads;
      if (kAll % kThreads != 0 && e >= kAll) continue;
      T t[kVec];
      *reinterpret_cast<uint4*>(t) = x[i];
      float* o = dst + (e / kChunks) * L<D>::kStride + (e % kChunks) * kVec;
#pragma unroll
      for (int j = 0; j < kVec; j += 4)
        *reinterpret_cast<float4*>(o + j) = make_float4(to_f<T>(t[j]), to_f<T>(t[j + 1]), to_f<T>(t[j + 2]), to_f<T>(t[j + 3]));
    }
  }
};
template <typename T, int D, int ROWS = kT, typename Off>
__device__ __forceinline__ void load_rows(float* dst, const T* src, Off off) {
  Fetch<T, D, ROWS> f;
  f.get(src, off);
  f.put(dst);
}

// Two fp32 multiply-adds in one instruction: the pipe's rate is the same, but the
// loads beside them find the issue slots (1500 tokens, 8 heads of 128, window 500:
// forward 201 -> 171 us, dq 236 -> 224, dk and dv 325 -> 304).
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t r) {
  float2 x;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(r));
  return x;
}
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

// acc[r][c] = <A row RT ty + r, B row tx + 16 c>, even and odd elements apart
template <int D, int RT>
__device__ __forceinline__ void dots(const float* A, const float* B, int ty, int tx, float (&acc)[RT][4]) {
  constexpr int ST = L<D>::kStride;
  uint64_t s[RT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[r][c] = 0;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    ulonglong2 x[RT], y[4];
#pragma unroll
    for (int r = 0; r < RT; ++r) x[r] = *reinterpret_cast<const ulonglong2*>(A + (RT * ty + r) * ST + d);
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * r) * ST + d);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        fma2(s[r][c], x[r].x, y[c].x);
        fma2(s[r][c], x[r].y, y[c].y);
      }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 t = unpack2(s[r][c]);
      acc[r][c] = t.x + t.y;
    }
}

// The accumulators of RT rows by a thread's columns, in pairs of columns.
template <int D, int RT>
struct Acc {
  static constexpr int C = L<D>::kC, kP = (C + 1) / 2;  // at D = 16 the second of the pair is unused
  uint64_t v[RT][kP];
  __device__ __forceinline__ Acc() {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < kP; ++c) v[r][c] = 0;
  }
  __device__ __forceinline__ void scale(int r, float f) {
#pragma unroll
    for (int c = 0; c < kP; ++c) {
      const float2 t = unpack2(v[r][c]);
      v[r][c] = pack2(t.x * f, t.y * f);
    }
  }
  // to rows of D values
  __device__ __forceinline__ void put(float* dst, int ty, int tx) const {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) dst[(RT * ty + r) * D + L<D>::col(tx, c)] = at(r, c);
  }
  __device__ __forceinline__ float at(int r, int c) const {
    const float2 t = unpack2(v[r][c / 2]);
    return c % 2 ? t.y : t.x;
  }
};

// acc[r][c] += sum_j P[RT ty + r][j] X[j][col c]
template <int D, int RT>
__device__ __forceinline__ void accumulate(const float* P, const float* X, int ty, int tx, Acc<D, RT>& acc) {
  constexpr int ST = L<D>::kStride, C = L<D>::kC, V = L<D>::kV;
#pragma unroll 2
  for (int j = 0; j < kT; j += 4) {
    float p[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float4 t = *reinterpret_cast<const float4*>(P + (RT * ty + r) * kPS + j);
      p[r][0] = t.x;
      p[r][1] = t.y;
      p[r][2] = t.z;
      p[r][3] = t.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c0 = 0; c0 < C; c0 += V) {
        const float* src = X + (j + i) * ST + L<D>::col(tx, c0);
        uint64_t x[(V + 1) / 2];
        if constexpr (V == 4) {
          const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(src);
          x[0] = t.x;
          x[1] = t.y;
        } else if constexpr (V == 2) {
          x[0] = *reinterpret_cast<const uint64_t*>(src);
        } else {
          x[0] = pack2(src[0], 0.f);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int u = 0; u < (V + 1) / 2; ++u) fma2(acc.v[r][c0 / 2 + u], pack2(p[r][i], p[r][i]), x[u]);
      }
  }
}

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float max16(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// A query tile's key blocks are shared by the CTAs of a cluster (1 to 8),
// each with a run of them: part `rank` of `parts`.
struct Part {
  int rank, parts, tile;
  __device__ Part() {
    parts = (int)cooperative_groups::this_cluster().num_blocks();
    rank = (int)cooperative_groups::this_cluster().block_rank();
    tile = (gridDim.x - 1 - blockIdx.x) / parts;  // the longest rows first
  }
  __device__ int first(int blocks) const { return (int)((int64_t)blocks * rank / parts); }
  __device__ int last(int blocks) const { return (int)((int64_t)blocks * (rank + 1) / parts); }
};

// A tile of packed query rows of (sequence s, key/value head f).
struct Rows {
  Seq q;
  int s, f, G, r0, n;  // first packed row, rows in the tile
  __device__ int token(int r) const { return (r0 + r) / G; }
  __device__ int head(int r) const { return f * G + (r0 + r) % G; }
  __device__ int pos(int r) const { return q.first + token(r); }
  __device__ int64_t elem(int r, int H, int D) const { return ((q.q0 + token(r)) * H + head(r)) * (int64_t)D; }
};

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const AttnArgs a) {
  constexpr int kR = 16 * RT;  // rows of the tile
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sK = sm + kR * L<D>::kStride;
  float* sV = sK + L<D>::kTile;
  float* sP = sV + L<D>::kTile;
  Rows R;
  R.s = blockIdx.y / a.Hkv;
  R.f = blockIdx.y % a.Hkv;
  R.q = seq_of(a, R.s);
  R.G = a.G;
  const Part part;
  R.r0 = part.tile * kR;
  R.n = R.q.nq * a.G - R.r0;
  if (R.n <= 0) return;
  if (R.n > kR) R.n = kR;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  load_rows<T, D, kR>(sQ, static_cast<const T*>(a.q), [&](int r) { return r < R.n ? R.elem(r, a.H, D) : -1; });
  Acc<D, RT> acc;
  float m[RT], l[RT];
  int x[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    x[r] = RT * ty + r < R.n ? R.pos(RT * ty + r) : -1;
  }
  const BlockList bl = blocks_of<kT>(a, R.pos(0), R.pos(R.n - 1));
  Fetch<T, D> fk, fv;
  auto fetch = [&](int n) {
    const int j0 = bl.at(n) * kT;
    auto row = [&](int r) -> int64_t { return j0 + r < R.q.kv ? kv_row(a, R.q, R.s, R.f, j0 + r) : -1; };
    fk.get(static_cast<const T*>(a.k), row);
    fv.get(static_cast<const T*>(a.v), row);
  };
  const int n0 = part.first(bl.count), n1 = part.last(bl.count);
  if (n0 < n1) fetch(n0);
  for (int n = n0; n < n1; ++n) {
    const int j0 = bl.at(n) * kT;
    __syncthreads();
    fk.put(sK);
    fv.put(sV);
    __syncthreads();
    if (n + 1 < n1) fetch(n + 1);
    float s[RT][4];
    dots<D, RT>(sQ, sK, ty, tx, s);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[r][c] = sees(a, x[r], j0 + tx + 16 * c) ? s[r][c] * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[r][c]);
      }
      mx = fmaxf(max16(mx), m[r]);
      const float base = mx == -INFINITY ? 0.f : mx;  // a row with nothing to see so far
      const float corr = exp2f(m[r] - base);
      m[r] = mx;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = exp2f(s[r][c] - base);
        sum += p;
        sP[(RT * ty + r) * kPS + tx + 16 * c] = p;
      }
      l[r] = l[r] * corr + sum16(sum);
      acc.scale(r, corr);
    }
    __syncthreads();
    accumulate<D, RT>(sP, sV, ty, tx, acc);
  }
  if (part.parts > 1) {  // each CTA adds the parts of some of the rows, in order
    auto cluster = cooperative_groups::this_cluster();
    float* sA = sK;  // [kR][D]
    float* sM = sK + kR * D;
    float* sL = sM + kR;
    __syncthreads();
    acc.put(sA, ty, tx);
    if (tx == 0)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        sM[RT * ty + r] = m[r];
        sL[RT * ty + r] = l[r];
      }
    cluster.sync();
    for (int e = part.rank * kThreads + threadIdx.x; e < R.n * D; e += part.parts * kThreads) {
      const int i = e / D;
      float top = -INFINITY, sum = 0.f, o = 0.f;
      for (int c = 0; c < part.parts; ++c) top = fmaxf(top, cluster.map_shared_rank(sM, c)[i]);
      const float base = top == -INFINITY ? 0.f : top;
      for (int c = 0; c < part.parts; ++c) {
        const float w = exp2f(cluster.map_shared_rank(sM, c)[i] - base);
        sum = fmaf(w, cluster.map_shared_rank(sL, c)[i], sum);
        o = fmaf(w, cluster.map_shared_rank(sA, c)[e], o);
      }
      static_cast<T*>(a.out)[R.elem(i, a.H, D) + e % D] = from_f<T>(o * (sum == 0.f ? 0.f : 1.f / sum));
      if (e % D == 0 && a.lse)
        a.lse[lse_index(a, R.q, R.s, R.token(i), R.head(i))] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
    }
    cluster.sync();  // no CTA ends while another reads its part
    return;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int i = RT * ty + r;
    if (i >= R.n) continue;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];  // (a sum of NaN stays one)
    T* o = static_cast<T*>(a.out) + R.elem(i, a.H, D);
#pragma unroll
    for (int c = 0; c < L<D>::kC; ++c) o[L<D>::col(tx, c)] = from_f<T>(acc.at(r, c) * inv);
    if (tx == 0 && a.lse)
      a.lse[lse_index(a, R.q, R.s, R.token(i), R.head(i))] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
  }
}

// weights[s, f, j] += sum over the rows that see key j of e^{s - lse}.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) weights_kernel(const AttnArgs a, float* weights) {
  extern __shared__ __align__(16) float sm[];
  float* sK = sm;
  float* sQ = sm + L<D>::kTile;
  __shared__ float s_lse[kT];
  __shared__ int s_pos[kT];
  const int s = blockIdx.y / a.Hkv, f = blockIdx.y % a.Hkv;
  const Seq q = seq_of(a, s);
  const int j0 = blockIdx.x * kT;
  if (j0 >= q.kv || q.nq == 0) return;
  // rows from the first query at or after the tile on
  int i0 = j0 - q.first;
  if (i0 < 0) i0 = 0;
  // and up to the last one whose window reaches it, unless the tile holds a sink
  int i1 = q.nq;
  if (a.window && j0 >= a.sinks) {
    const int64_t last = (int64_t)j0 + kT - 1 + a.window - q.first;
    if (last < i1) i1 = last < 0 ? 0 : (int)last;
  }
  if (i0 >= i1) return;  // keys that no query sees are not read
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  load_rows<T, D>(sK, static_cast<const T*>(a.k),
                  [&](int r) -> int64_t { return j0 + r < q.kv ? kv_row(a, q, s, f, j0 + r) : -1; });
  float acc[4] = {};
  for (int r0 = i0 * a.G; r0 < i1 * a.G; r0 += kT) {
    Rows R{q, s, f, a.G, r0, i1 * a.G - r0 < kT ? i1 * a.G - r0 : kT};
    __syncthreads();
    load_rows<T, D>(sQ, static_cast<const T*>(a.q), [&](int r) { return r < R.n ? R.elem(r, a.H, D) : -1; });
    for (int r = threadIdx.x; r < kT; r += kThreads) {
      s_pos[r] = r < R.n ? R.pos(r) : -1;
      s_lse[r] = r < R.n ? a.lse[lse_index(a, q, s, R.token(r), R.head(r))] * kLog2e : 0.f;
    }
    __syncthreads();
    float st[4][4];
    dots<D, 4>(sK, sQ, ty, tx, st);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = tx + 16 * c;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (sees(a, s_pos[col], j0 + 4 * ty + r)) acc[r] += exp2f(fmaf(st[r][c], a.scale_log2, -s_lse[col]));
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float t = sum16(acc[r]);
    const int j = j0 + 4 * ty + r;
    if (tx == 0 && j < q.kv)
      weights[((int64_t)s * a.Hkv + f) * ((int64_t)a.max_pages << a.page_shift) + j] += t;
  }
}

// The sum of a 16-byte chunk's products x y.
template <typename T>
__device__ __forceinline__ float dot16(const uint4& x, const uint4& y, float acc) {
  T a[16 / sizeof(T)], b[16 / sizeof(T)];
  *reinterpret_cast<uint4*>(a) = x;
  *reinterpret_cast<uint4*>(b) = y;
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) acc = fmaf(to_f<T>(a[i]), to_f<T>(b[i]), acc);
  return acc;
}

// delta of every row, [S, H, N] fp32: a warp's 8 lanes per row.  kPeaks: also the
// largest |dout_x|^2 and |v_j|^2 of the block's rows, to peaks[2 block] and the next
// (rows with an infinity or NaN not counted); with delta null, these alone.  (A pair
// of maxima by atomics wants zeros there first, one launch more: the gradients of
// 2 x 128 tokens, 4/2 heads of 64, captured: 22.4 us against 20.5.)
template <typename T, int D, bool kPeaks>
__global__ void __launch_bounds__(256) delta_kernel(const AttnArgs a, const T* out, const T* dout, float* delta,
                                                    float* peaks) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kLanes = D / kVec < 8 ? D / kVec : 8;
  const int64_t rows = a.T * a.H;
  const int64_t per = 256 / kLanes;
  const int sub = threadIdx.x % kLanes;
  float top[2] = {0.f, 0.f};
  if (kPeaks) {  // launched while the kernel before ends, as the next one is
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  auto sum = [&](float x) {
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  for (int64_t r0 = blockIdx.x * per; r0 < rows; r0 += gridDim.x * per) {
    const int64_t r = r0 + threadIdx.x / kLanes;
    float acc = 0.f, square = 0.f;
    if (r < rows) {
#pragma unroll
      for (int c = sub * kVec; c < D; c += kLanes * kVec) {
        const uint4 y = *reinterpret_cast<const uint4*>(dout + r * D + c);
        if (!kPeaks || delta) acc = dot16<T>(*reinterpret_cast<const uint4*>(out + r * D + c), y, acc);
        if (kPeaks) square = dot16<T>(y, y, square);
      }
    }
    acc = sum(acc);
    if (kPeaks) {
      square = sum(square);
      if (square < INFINITY) top[0] = fmaxf(top[0], square);
    }
    if (r < rows && sub == 0 && (!kPeaks || delta)) {
      const int64_t h = r % a.H, t = r / a.H;
      const int64_t s = t / a.nq_max, i = t % a.nq_max;
      delta[(s * a.H + h) * a.nq_max + i] = acc;
    }
  }
  if constexpr (kPeaks) {
    const T* v = static_cast<const T*>(a.v);
    const int64_t keys = a.T * a.Hkv;
    for (int64_t r0 = blockIdx.x * per; r0 < keys; r0 += gridDim.x * per) {
      const int64_t r = r0 + threadIdx.x / kLanes;
      float square = 0.f;
      if (r < keys) {
#pragma unroll
        for (int c = sub * kVec; c < D; c += kLanes * kVec) {
          const uint4 y = *reinterpret_cast<const uint4*>(v + r * D + c);
          square = dot16<T>(y, y, square);
        }
      }
      square = sum(square);
      if (square < INFINITY) top[1] = fmaxf(top[1], square);
    }
    __shared__ uint32_t s_top[2][8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // (numbers from 0 up compare as their bits do)
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(top[w]));
      if (threadIdx.x % 32 == 0) s_top[w][threadIdx.x / 32] = m;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, s_top[threadIdx.x][i]);
      peaks[2 * blockIdx.x + threadIdx.x] = __uint_as_float(m);
    }
  }
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads) dq_kernel(const AttnArgs a, const WindowBwdArgs g) {
  constexpr int kR = 16 * RT;  // rows of the tile
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sO = sm + kR * L<D>::kStride;
  float* sK = sO + kR * L<D>::kStride;
  float* sV = sK + L<D>::kTile;
  float* sS = sV + L<D>::kTile;
  Rows R;
  R.s = blockIdx.y / a.Hkv;
  R.f = blockIdx.y % a.Hkv;
  R.q = seq_of(a, R.s);
  R.G = a.G;
  const Part part;
  R.r0 = part.tile * kR;
  R.n = R.q.nq * a.G - R.r0;
  if (R.n <= 0) return;
  if (R.n > kR) R.n = kR;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  auto qrow = [&](int r) { return r < R.n ? R.elem(r, a.H, D) : -1; };
  load_rows<T, D, kR>(sQ, static_cast<const T*>(a.q), qrow);
  load_rows<T, D, kR>(sO, static_cast<const T*>(g.dout), qrow);
  Acc<D, RT> acc;
  float lse2[RT], delta[RT];
  int x[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int i = RT * ty + r;
    const bool in = i < R.n;
    const int64_t at = in ? lse_index(a, R.q, R.s, R.token(i), R.head(i)) : 0;
    lse2[r] = in ? a.lse[at] * kLog2e : 0.f;
    delta[r] = in ? g.delta[at] : 0.f;
    x[r] = in ? R.pos(i) : -1;
  }
  const BlockList bl = blocks_of<kT>(a, R.pos(0), R.pos(R.n - 1));
  Fetch<T, D> fk, fv;
  auto fetch = [&](int n) {
    const int j0 = bl.at(n) * kT;
    auto row = [&](int r) -> int64_t { return j0 + r < R.q.kv ? kv_row(a, R.q, R.s, R.f, j0 + r) : -1; };
    fk.get(static_cast<const T*>(a.k), row);
    fv.get(static_cast<const T*>(a.v), row);
  };
  const int n0 = part.first(bl.count), n1 = part.last(bl.count);
  if (n0 < n1) fetch(n0);
  for (int n = n0; n < n1; ++n) {
    const int j0 = bl.at(n) * kT;
    __syncthreads();
    fk.put(sK);
    fv.put(sV);
    __syncthreads();
    if (n + 1 < n1) fetch(n + 1);
    float s[RT][4], dp[RT][4];
    dots<D, RT>(sQ, sK, ty, tx, s);
    dots<D, RT>(sO, sV, ty, tx, dp);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p =
            sees(a, x[r], j0 + tx + 16 * c) ? exp2f(fmaf(s[r][c], a.scale_log2, -lse2[r])) : 0.f;
        sS[(RT * ty + r) * kPS + tx + 16 * c] = p * (dp[r][c] - delta[r]);
      }
    __syncthreads();
    accumulate<D, RT>(sS, sK, ty, tx, acc);
  }
  if (part.parts > 1) {
    auto cluster = cooperative_groups::this_cluster();
    float* sA = sV;  // [kR][D]
    __syncthreads();
    acc.put(sA, ty, tx);
    cluster.sync();
    for (int e = part.rank * kThreads + threadIdx.x; e < R.n * D; e += part.parts * kThreads) {
      float sum = 0.f;
      for (int c = 0; c < part.parts; ++c) sum += cluster.map_shared_rank(sA, c)[e];
      static_cast<T*>(g.dq)[R.elem(e / D, a.H, D) + e % D] = from_f<T>(sum * a.scale);
    }
    cluster.sync();
    return;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int i = RT * ty + r;
    if (i >= R.n) continue;
    T* o = static_cast<T*>(g.dq) + R.elem(i, a.H, D);
#pragma unroll
    for (int c = 0; c < L<D>::kC; ++c) o[L<D>::col(tx, c)] = from_f<T>(acc.at(r, c) * a.scale);
  }
}

// dk, dv of a tile of 16 RT keys over one item's queries.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads, D <= 32 ? 2 : 1)  // two to an SM: 42 -> 34 us for 997 tokens, 6/2 heads of 32
    dkv_kernel(const AttnArgs a, const WindowBwdArgs g, const KeyPlan kp) {
  constexpr int kR = 16 * RT;
  extern __shared__ __align__(16) float sm[];
  float* sK = sm;
  float* sV = sm + kR * L<D>::kStride;
  float* sQ = sV + kR * L<D>::kStride;
  float* sO = sQ + L<D>::kTile;
  float* sP = sO + L<D>::kTile;
  float* sS = sP + kR * kPS;
  __shared__ float s_lse[kT], s_delta[kT];
  const int s = blockIdx.y / a.Hkv, f = blockIdx.y % a.Hkv;
  const Seq q = seq_of(a, s);
  const KeyItem it = key_item(a, kp, blockIdx.x);
  const int j0 = it.tile * kR, i0 = it.i0, i1 = it.i1;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  auto krow = [&](int r) -> int64_t { return j0 + r < q.kv ? kv_row(a, q, s, f, j0 + r) : -1; };
  load_rows<T, D, kR>(sK, static_cast<const T*>(a.k), krow);
  load_rows<T, D, kR>(sV, static_cast<const T*>(a.v), krow);
  Acc<D, RT> dk, dv;
  Fetch<T, D> fq, fo;
  float l2 = 0.f, dl = 0.f;  // of row threadIdx.x
  auto rows_at = [&](int r0) { return Rows{q, s, f, a.G, r0, i1 * a.G - r0 < kT ? i1 * a.G - r0 : kT}; };
  auto fetch = [&](int r0) {
    const Rows R = rows_at(r0);
    auto qrow = [&](int r) { return r < R.n ? R.elem(r, a.H, D) : -1; };
    fq.get(static_cast<const T*>(a.q), qrow);
    fo.get(static_cast<const T*>(g.dout), qrow);
    const int r = threadIdx.x;
    if (r < R.n) {
      const int64_t at = lse_index(a, q, s, R.token(r), R.head(r));
      l2 = a.lse[at] * kLog2e;
      dl = g.delta[at];
    }
  };
  if (i0 < i1) fetch(i0 * a.G);
  for (int r0 = i0 * a.G; r0 < i1 * a.G; r0 += kT) {
    const Rows R = rows_at(r0);
    __syncthreads();
    fq.put(sQ);
    fo.put(sO);
    if (threadIdx.x < kT) {
      s_lse[threadIdx.x] = l2;
      s_delta[threadIdx.x] = dl;
    }
    __syncthreads();
    if (r0 + kT < i1 * a.G) fetch(r0 + kT);
    float st[RT][4], dp[RT][4];
    dots<D, RT>(sK, sQ, ty, tx, st);
    dots<D, RT>(sV, sO, ty, tx, dp);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = tx + 16 * c;
      const int x = col < R.n ? R.pos(col) : -1;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float p =
            sees(a, x, j0 + RT * ty + r) ? exp2f(fmaf(st[r][c], a.scale_log2, -s_lse[col])) : 0.f;
        sP[(RT * ty + r) * kPS + col] = p;
        sS[(RT * ty + r) * kPS + col] = p * (dp[r][c] - s_delta[col]);
      }
    }
    __syncthreads();
    accumulate<D, RT>(sP, sO, ty, tx, dv);
    accumulate<D, RT>(sS, sQ, ty, tx, dk);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int j = j0 + RT * ty + r;
    if (it.slot >= 0) {
      // [S Hkv][slot][dk, dv][kR][D]
      float* p = g.partial + ((((int64_t)blockIdx.y * kp.slots() + it.slot) * 2) * kR + RT * ty + r) * D;
#pragma unroll
      for (int c = 0; c < L<D>::kC; ++c) {
        p[L<D>::col(tx, c)] = dk.at(r, c) * a.scale;
        p[kR * D + L<D>::col(tx, c)] = dv.at(r, c);
      }
    } else if (j < q.kv) {
      const int64_t at = ((q.q0 + j) * a.Hkv + f) * D;
#pragma unroll
      for (int c = 0; c < L<D>::kC; ++c) {
        static_cast<T*>(g.dk)[at + L<D>::col(tx, c)] = from_f<T>(dk.at(r, c) * a.scale);
        static_cast<T*>(g.dv)[at + L<D>::col(tx, c)] = from_f<T>(dv.at(r, c));
      }
    }
  }
}

// dk and dv of the tiles with partials, added in slot order (the order is
// fixed, so the result does not change from run to run).
template <typename T>
__global__ void __launch_bounds__(256) key_reduce_kernel(const AttnArgs a, const WindowBwdArgs g, const KeyPlan kp) {
  const int sf = blockIdx.z, tile = blockIdx.y;
  const int s = sf / a.Hkv, f = sf % a.Hkv;
  const int per = kp.tile * a.D;  // values of one gradient's tile
  const int e = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= 2 * per) return;
  const int s0 = kp.slot_of(tile), s1 = kp.slot_of(tile + 1);
  const float* p = g.partial + ((int64_t)sf * kp.slots() + s0) * 2 * per + e;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < s1 - s0; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(p + (int64_t)c * 2 * per);
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  const int which = e / per, r = (e % per) / a.D, d = e % a.D;
  const int j = tile * kp.tile + r;
  if (j >= a.nq_max) return;
  T* o = static_cast<T*>(which ? g.dv : g.dk) + (((int64_t)s * a.nq_max + j) * a.Hkv + f) * a.D + d;
  o[0] = from_f<T>(acc.x);
  o[1] = from_f<T>(acc.y);
  o[2] = from_f<T>(acc.z);
  o[3] = from_f<T>(acc.w);
}

bool set_smem(const void* fn, int bytes) {
  if (bytes <= 48 * 1024) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

int ok_launch() { return cudaGetLastError() == cudaSuccess ? LONGNET_OK : LONGNET_ERR_CUDA; }

// Query tiles have 64 rows, or 16 where the GPU holds all of those at once, two
// to an SM.  A small tile reads shared memory more often for each product, and is
// done sooner: forward and dq of 2 x 276 tokens, one head of 128, take 64 and 74 us
// with 64 rows, 37 and 49 with 16; of 600 tokens, 4/2 heads of 64, 42 and 50 with
// 64, 26 and 33 with 16.  (Tiles of 32 rows lie between: 32 and 38 us; and above
// the limit they lose, 36 us, where 94 tiles of 64 rows take 32, for dq at D = 32.)
bool small_tiles(const AttnArgs& a) {
  return ((int64_t)a.nq_max * a.G + 15) / 16 * a.S * a.Hkv <= 2 * kSms;
}

// CTAs that share a query tile's key blocks (a cluster): as many as there are
// blocks and the grid fits two to an SM (forward and dq of 2 x 276 tokens, one head
// of 128: 37 and 49 us with one, 19 and 23 with 5; of 997 tokens, 6/2 heads of 32,
// window 200: 27 and 31 us with one, 26 and 29 with 2, 22 and 23 with 3).
int key_parts(const AttnArgs& a, int64_t tiles, int rows) {
  int64_t keys = a.cu_q ? (int64_t)a.max_pages << a.page_shift : a.nq_max;
  if (a.window) {
    const int64_t seen = (int64_t)a.window + rows / a.G + 2 + (a.sinks + kT - 1) / kT * kT;
    if (seen < keys) keys = seen;
  }
  const int64_t fit = 2 * kSms / (tiles * a.S * a.Hkv), blocks = (keys + kT - 1) / kT;
  const int64_t parts = fit < blocks ? fit : blocks;
  return parts < 1 ? 1 : parts > 8 ? 8 : (int)parts;
}
// fn on (tiles, S Hkv) clusters of `parts` CTAs.
template <typename... P, typename... V>
int launch_tiles(void (*fn)(P...), const AttnArgs& a, int rows, int smem, cudaStream_t st, V&&... args) {
  if (!set_smem((const void*)fn, smem)) return LONGNET_ERR_CUDA;
  const int64_t tiles = ((int64_t)a.nq_max * a.G + rows - 1) / rows;
  const int parts = key_parts(a, tiles, rows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * parts), (unsigned)(a.S * a.Hkv));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess) return LONGNET_OK;
  cudaGetLastError();
  return LONGNET_ERR_CUDA;
}

template <typename T, int D, int RT>
int fwd_tiles(const AttnArgs& a, cudaStream_t st) {
  constexpr int kR = 16 * RT;
  return launch_tiles(fwd_kernel<T, D, RT>, a, kR, (kR * L<D>::kStride + 2 * L<D>::kTile + kR * kPS) * 4, st, a);
}
template <typename T, int D>
int fwd(const AttnArgs& a, cudaStream_t st) {
  return small_tiles(a) ? fwd_tiles<T, D, 1>(a, st) : fwd_tiles<T, D, 4>(a, st);
}
template <typename T, int D, int RT>
int dq_tiles(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t st) {
  constexpr int kR = 16 * RT;
  return launch_tiles(dq_kernel<T, D, RT>, a, kR, (2 * kR * L<D>::kStride + 2 * L<D>::kTile + kR * kPS) * 4, st, a, g);
}
template <typename T, int D>
int weights_sum(const AttnArgs& a, float* w, cudaStream_t st) {
  const int smem = 2 * L<D>::kTile * 4;
  auto fn = weights_kernel<T, D>;
  if (!set_smem((const void*)fn, smem)) return LONGNET_ERR_CUDA;
  const int64_t tiles = (((int64_t)a.max_pages << a.page_shift) + kT - 1) / kT;
  fn<<<dim3((unsigned)tiles, (unsigned)(a.S * a.Hkv)), kThreads, smem, st>>>(a, w);
  return ok_launch();
}
template <typename T, int D, int RT>
int dkv_tiles(const AttnArgs& a, const WindowBwdArgs& g, const KeyPlan& kp, cudaStream_t st) {
  constexpr int kR = 16 * RT;
  const int smem = (2 * kR * L<D>::kStride + 2 * L<D>::kTile + 2 * kR * kPS) * 4;
  auto fn = dkv_kernel<T, D, RT>;
  if (!set_smem((const void*)fn, smem)) return LONGNET_ERR_CUDA;
  fn<<<dim3((unsigned)kp.items(), (unsigned)(a.S * a.Hkv)), kThreads, smem, st>>>(a, g, kp);
  return ok_launch();
}
template <typename T, int D>
int bwd(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t st) {
  int rc = launch_window_delta(a, g, st);
  if (rc) return rc;
  const KeyPlan kp = simt_key_plan(a.S, a.nq_max, a.H, a.Hkv, a.window, a.sinks);
  rc = kp.tile == 16 ? dkv_tiles<T, D, 1>(a, g, kp, st) : dkv_tiles<T, D, 4>(a, g, kp, st);
  if (rc) return rc;
  rc = small_tiles(a) ? dq_tiles<T, D, 1>(a, g, st) : dq_tiles<T, D, 4>(a, g, st);
  if (rc) return rc;
  return launch_key_reduce(a, g, kp, st);
}
template <typename T, int D>
int delta_blocks(const AttnArgs& a, int most) {
  const int64_t rows = a.T * a.H, per = 256 / (D / (16 / (int)sizeof(T)) < 8 ? D / (16 / (int)sizeof(T)) : 8);
  const int64_t blocks = (rows + per - 1) / per;
  return (int)(blocks < most ? blocks : most);
}
template <typename T, int D>
int delta(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t st) {
  delta_kernel<T, D, false><<<delta_blocks<T, D>(a, 148 * 16), 256, 0, st>>>(
      a, static_cast<const T*>(a.out), static_cast<const T*>(g.dout), g.delta, nullptr);
  return ok_launch();
}
template <int D>
int peaks(const AttnArgs& a, const WindowBwdArgs& g, bool with_delta, int* blocks, cudaStream_t st) {
  *blocks = delta_blocks<__half, D>(a, kPeakBlocks);
  return launch_after(delta_kernel<__half, D, true>, dim3((unsigned)*blocks), 256, 0, st, a,
                      static_cast<const __half*>(a.out), static_cast<const __half*>(g.dout),
                      with_delta ? g.delta : nullptr, g.peaks);
}

#define LN_BY_D(FN, T, ...)                                      \
  (a.D == 16 ? FN<T, 16>(__VA_ARGS__)                            \
             : a.D == 32 ? FN<T, 32>(__VA_ARGS__)                \
                         : a.D == 64 ? FN<T, 64>(__VA_ARGS__) : FN<T, 128>(__VA_ARGS__))
#define LN_BY_TYPE(FN, ...)                                                        \
  (a.dtype == LONGNET_DTYPE_F32 ? LN_BY_D(FN, float, __VA_ARGS__)                  \
   : a.dtype == LONGNET_DTYPE_BF16 ? LN_BY_D(FN, __nv_bfloat16, __VA_ARGS__)       \
                                   : LN_BY_D(FN, __half, __VA_ARGS__))

}  // namespace ws

int launch_window_fwd_simt(const AttnArgs& a, cudaStream_t stream) { return LN_BY_TYPE(ws::fwd, a, stream); }
int launch_weights_simt(const AttnArgs& a, float* weights, cudaStream_t stream) {
  return LN_BY_TYPE(ws::weights_sum, a, weights, stream);
}
int launch_window_bwd_simt(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream) {
  return LN_BY_TYPE(ws::bwd, a, g, stream);
}
int launch_window_delta(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream) {
  return LN_BY_TYPE(ws::delta, a, g, stream);
}
int launch_window_peaks(const AttnArgs& a, const WindowBwdArgs& g, bool with_delta, int* blocks, cudaStream_t stream) {
  switch (a.D) {
    case 16:
      return ws::peaks<16>(a, g, with_delta, blocks, stream);
    case 32:
      return ws::peaks<32>(a, g, with_delta, blocks, stream);
    case 64:
      return ws::peaks<64>(a, g, with_delta, blocks, stream);
    default:
      return ws::peaks<128>(a, g, with_delta, blocks, stream);
  }
}

int launch_key_reduce(const AttnArgs& a, const WindowBwdArgs& g, const KeyPlan& k, cudaStream_t stream) {
  if (k.reduced() == 0) return LONGNET_OK;
  const dim3 grid((unsigned)((2 * k.tile * a.D / 4 + 255) / 256), (unsigned)k.reduced(), (unsigned)(a.S * a.Hkv));
  if (a.dtype == LONGNET_DTYPE_F32)
    ws::key_reduce_kernel<float><<<grid, 256, 0, stream>>>(a, g, k);
  else if (a.dtype == LONGNET_DTYPE_BF16)
    ws::key_reduce_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, g, k);
  else
    ws::key_reduce_kernel<__half><<<grid, 256, 0, stream>>>(a, g, k);
  return ws::ok_launch();
}

// Near ranges: so many that there are about `ctas` items, of at least min_blocks
// blocks of 64 query rows each, at most 16 a tile.  (Not to even out the last
// wave of many tiles: every tile then has partials, and adding them took 83 us
// for 16K tokens of 8 heads at D = 128, more than the wave.)  A far item has
// about as many queries as a near one, up to half as many more where the items
// then fit the waves that the tiles need anyway, and at least 64; a tile has at
// most 64.  With more than 16 sink tiles, or 1024 sinks in smaller tiles, there
// are enough of them to fill the GPU without: each then takes all its queries itself.
KeyPlan key_plan(int64_t S, int64_t N, int64_t H, int64_t Hkv, int64_t window, int64_t sinks, int tile,
                 int min_blocks, int ctas) {
  KeyPlan k = {tile, (int)((N + tile - 1) / tile), 1, 0, 0, 0};
  if (window > N) window = N;
  if (sinks > N) sinks = N;
  const int64_t pairs = S * Hkv, reach = tile + window < N ? tile + window : N;
  const int64_t blocks = reach * (H / Hkv) / 64;
  int64_t near = ctas / (k.tiles * pairs);
  if (near > blocks / min_blocks) near = blocks / min_blocks;
  if (near > 16) near = 16;
  if (near > 1) k.near = (int)near;
  // tiles with sinks and queries past their window
  int64_t t = (sinks + tile - 1) / tile;
  const int64_t past = N - (tile - 1 + window);  // queries past the first tile's window
  if (t <= 0 || past <= 0) return k;
  const int64_t has = (past + tile - 1) / tile;  // tiles that have any
  if (t > has) t = has;
  if (t > (tile < 64 ? 1024 / tile : 16)) return k;
  int64_t chunk = (window + tile) / k.near;
  if (chunk < 4 * tile / k.near) chunk = 4 * tile / k.near;
  if (chunk < 64) chunk = 64;
  int64_t n = (past + chunk - 1) / chunk;
  if (n > 64) n = 64;
  const int64_t fewest = (2 * past + 3 * chunk - 1) / (3 * chunk), items = pairs * k.tiles * k.near;
  const int64_t room = ((items + ctas - 1) / ctas * ctas - items) / (pairs * t);
  if (room >= fewest && room < n) n = room;
  k.sink_tiles = (int)t;
  k.chunk = (int)((past + n - 1) / n);
  k.chunks = (int)((past + k.chunk - 1) / k.chunk);
  return k;
}

// Ranges down to one block of queries; tiles of 64 keys, or 16 where the items of 64
// would leave half of the SMs idle.  (dk and dv of 2 x 276 tokens, one head of 128:
// 73 us with tiles of 64 keys, 41 with 16, both of two blocks at least, 27 with 16
// and one; of 600 tokens, 4/2 heads of 64: 33 us with two blocks at least, 25 with
// one.)
KeyPlan simt_key_plan(int64_t S, int64_t N, int64_t H, int64_t Hkv, int64_t window, int64_t sinks) {
  const KeyPlan k = key_plan(S, N, H, Hkv, window, sinks, 64, 1, 2 * ws::kSms);
  if (k.items() * S * Hkv >= ws::kSms / 2) return k;
  return key_plan(S, N, H, Hkv, window, sinks, 16, 1, 2 * ws::kSms);
}

int64_t key_partial_floats(const KeyPlan& k, int64_t S, int64_t Hkv, int64_t D) {
  return S * Hkv * k.slots() * 2 * (int64_t)k.tile * D;
}

}  // namespace longnet
