// Shared pieces of the tcgen05 kernels of the sliding-window and paged-cache
// attention: operand tile geometry, tensor maps, page-wise block loads and
// bounded waits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_args.cuh"
#include "launch_util.cuh"
#include "tc_ptx.cuh"

namespace longnet {

// How a forward call is cut.  tokens: of a 128-row tile; pairs: row-tile pairs
// of the longest sequence (1 when alternate); alternate: one row tile per
// key/value head, whose blocks the two streams take in turn.  items = 0: a CTA
// per (sequence, head, pair).  Else the items, (sequence, pair) for one head,
// are cut into pieces of at most a run of blocks each, one CTA per piece, and
// the pieces' results, in slots of slot_rows rows, are joined by a second
// kernel.
struct WindowTcPlan {
  int tokens, pairs, alternate;
  int items, grid, slot_rows;
  int* base;        // [items + 1] pieces before each item (of one head)
  float* part_out;  // [grid, slots of a piece, slot_rows, D]
  float* part_lse;  // [grid, slots of a piece, slot_rows], log2 domain
};

bool window_tc_supports(const AttnArgs& a);
WindowTcPlan window_tc_plan(const AttnArgs& a);
int64_t window_tc_part_floats(const AttnArgs& a, const WindowTcPlan& p);
int launch_window_fwd_tc(const AttnArgs& a, float* parts, cudaStream_t stream);
int launch_weights_tc(const AttnArgs& a, float* weights, cudaStream_t stream);
bool window_bwd_tc_supports(const AttnArgs& a);
int window_bwd_tc_tile(int64_t D);  // keys of a work item of the key-centric kernel
constexpr int kTcMinBlocks = 8, kTcCtas = 148;  // of key_plan, for the tcgen05 family
int launch_window_bwd_tc(const AttnArgs& a, const WindowBwdArgs& g, cudaStream_t stream);

namespace wt {
using namespace tc;

using Plan = WindowTcPlan;
constexpr int kTile = 128;  // rows of a tile, keys of a block
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
// P and its row sum in the forward are times 2^kUp.  fp16: a weight of 2^-21 of the
// row's largest is then still a normal number (beside a sink the others' weights
// are that small), and the largest, up to 2^8 while the running maximum lags, fits.
template <int kFmt>
constexpr float kUp = kFmt == kFmtF16 ? 7.f : 0.f;

// Rows of D 16-bit elements as swizzle panels: D = 64 or 128 is one or two
// panels of 128-byte rows, D = 32 or 16 one panel of 64- or 32-byte rows.
template <int kD>
struct Panels {
  static constexpr int kPanels = kD >= 64 ? kD / 64 : 1;
  static constexpr int kPanelElems = kD >= 64 ? 64 : kD;
  static constexpr int kRowBytes = kPanelElems * 2;
  // descriptor high word: stride between 8-row groups, sm_100 version, layout
  // type (128-byte swizzle 2, 64-byte 4, 32-byte 6)
  static constexpr uint32_t kDescHi = (uint32_t)(8 * kRowBytes >> 4) | (1u << 14) |
                                      ((kRowBytes == 128 ? 2u : kRowBytes == 64 ? 4u : 6u) << 29);
};

struct __align__(64) Maps {
  CUtensorMap m[3];  // q, k, v
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// MMA issue by a converged warp.  All lanes run the issuing loop and one (the
// leader, chosen once) executes the instructions: addresses and descriptors
// then stay in uniform registers, which the MMA instructions take, where a
// loop inside a one-lane branch moves each of them there first (60 to 90
// cycles an instruction, more than the tensor cores need for it).
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss_if(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_if(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// A warp's 32 rows of an accumulator (TMEM columns acc.., scaled) to global
// memory in the 16-bit format, through its own rows of `tile`, an operand tile
// (128 rows, swizzled panels) that nothing reads any more: written a row per
// lane, read back a whole row per group of lanes.  (Stores of 16 bytes a lane to
// 32 different rows took 3000 cycles of a CTA at D = 64, 6000 at D = 128.)
// dst: the lane's row; rows without live are not written.  any = false: zeros.
template <int kFmt, int kD>
__device__ __forceinline__ void store_rows(uint8_t* tile, uint32_t acc, bool any, float scale, int row0, int lane,
                                           uint16_t* dst, bool live) {
  using LL = Panels<kD>;
  constexpr int kCpr = LL::kRowBytes / 16, kRow16 = kD / 8;  // 16-byte chunks of a panel row, of a row
  constexpr int kChunk = kD < 32 ? kD : 32;
  auto at = [&](int r, int c) -> uint4* {
    const int cc = c % kCpr;
    const int sw = LL::kRowBytes == 128 ? (r & 7) : LL::kRowBytes == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
    return reinterpret_cast<uint4*>(tile + (c / kCpr) * kTile * LL::kRowBytes + r * LL::kRowBytes + ((cc ^ sw) << 4));
  };
#pragma unroll
  for (int c0 = 0; c0 < kD; c0 += kChunk) {
    uint32_t rr[kChunk];
    if (any) {
      if constexpr (kChunk == 32) {
        LN_TMEM_LD32(acc + c0, rr);
      } else {
        LN_TMEM_LD16(acc + c0, rr);
      }
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int c = 0; c < kChunk; ++c) rr[c] = 0;
    }
#pragma unroll
    for (int c = 0; c < kChunk; c += 8) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack2<kFmt>(__uint_as_float(rr[c + 2 * e]) * scale, __uint_as_float(rr[c + 2 * e + 1]) * scale);
      *at(row0 + lane, (c0 + c) / 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __syncwarp();
  const uint32_t mask = __ballot_sync(0xffffffffu, live);
  const uint64_t mine = reinterpret_cast<uint64_t>(dst);
#pragma unroll 4
  for (int r0 = 0; r0 < 32; r0 += 32 / kRow16) {
    const int r = r0 + lane / kRow16, c = lane % kRow16;
    const uint64_t to = __shfl_sync(0xffffffffu, mine, r);
    if ((mask >> r) & 1) reinterpret_cast<uint4*>(to)[c] = *at(row0 + r, c);
  }
}

// The same rows as fp32 to consecutive global rows of kD floats (dst: the
// lane's), 32 columns at a time through 128-byte rows of `tile` (16 KB).
template <int kD>
__device__ __forceinline__ void store_rows_f32(uint8_t* tile, uint32_t acc, bool any, float scale, int row0, int lane,
                                               float* dst) {
  float* first = dst - (int64_t)lane * kD;  // the warp's row 0
#pragma unroll 1
  for (int c0 = 0; c0 < kD; c0 += 32) {
    uint32_t rr[32];
    if (any) {
      LN_TMEM_LD32(acc + c0, rr);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) rr[c] = 0;
    }
    auto at = [&](int r, int c) { return reinterpret_cast<float4*>(tile + (row0 + r) * 128 + ((c ^ (r & 7)) << 4)); };
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *at(lane, c) = make_float4(__uint_as_float(rr[4 * c]) * scale, __uint_as_float(rr[4 * c + 1]) * scale,
                                 __uint_as_float(rr[4 * c + 2]) * scale, __uint_as_float(rr[4 * c + 3]) * scale);
    __syncwarp();
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 4) {
      const int r = r0 + lane / 8, c = lane % 8;
      *reinterpret_cast<float4*>(first + (int64_t)r * kD + c0 + 4 * c) = *at(r, c);
    }
    __syncwarp();
  }
}

// Adds bytes to the barrier's current phase without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

struct Waiter {
  volatile int* abort_flag;
  int* status;
  uint64_t limit;
  __device__ bool wait(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 1;; ++it) {
      if (mbar_try_wait(a, parity)) return true;
      if ((it & 15u) == 0) {
        if (*abort_flag) return false;
        if (global_ns() - t0 > limit) {
          *abort_flag = 1;
          record_status(status, kStatusTimeout);
          return false;
        }
      }
    }
  }
  __device__ bool wait_warp(uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); }
};

// Waits for the loads of a ring's last items: of `issued` items, item n lies in
// stage n % stages and completes the phase of parity n / stages there (those
// before the last `stages` landed before their stage was filled again).  wait(stage,
// parity) is bounded and says whether the load landed.  A CTA must not exit with
// loads in flight, which would land in the next one's shared memory, so this is
// called whatever became of the waits before it.
template <typename Wait>
__host__ __device__ __forceinline__ void drain_ring(int issued, int stages, Wait wait) {
  for (int n = issued > stages ? issued - stages : 0; n < issued; ++n)
    if (!wait(n % stages, (uint32_t)(n / stages) & 1u)) return;
}
__device__ __forceinline__ void drain_loads(uint64_t* bars, int issued, int stages, int* status) {
  drain_ring(issued, stages, [&](int stage, uint32_t parity) {
    const bool landed = mbar_wait(bars + stage, parity, kWaitLimitNs);
    if (!landed) record_status(status, kStatusTimeout);
    return landed;
  });
}

// The largest of three, in one instruction.
__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

template <int kN>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[kN]) {
  if constexpr (kN == 32) {
    LN_TMEM_LD32(taddr, r);
  } else {
    LN_TMEM_LD16(taddr, r);
  }
}
template <int kN>
__device__ __forceinline__ void tmem_store(uint32_t taddr, uint32_t (&r)[kN]) {
  if constexpr (kN == 32) {
    LN_TMEM_ST32(taddr, r);
  } else {
    LN_TMEM_ST16(taddr, r);
  }
}

// Rows [j0, j0 + rows) of a paged cache into a block in shared memory, by one
// warp: a lane looks up a page and issues its boxes, whose bytes are added to
// the barrier's current phase (the caller arrives).  Pages past the sequence's
// last key are not read.
template <int kD>
__device__ __forceinline__ void load_pages(const AttnArgs& a, const Seq& q, int s, int f, int j0, int rows,
                                           const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int lane) {
  using LL = Panels<kD>;
  const int box = a.page < rows ? a.page : rows;  // rows of a box
  const int boxes = rows / box;                   // at most 16
  const int j = j0 + lane * box;
  const bool live = lane < boxes && j < q.kv;
  int pg = 0;
  if (live) {
    pg = a.table[(int64_t)s * a.max_pages + (j >> a.page_shift)];
    if (pg < 0 || pg >= a.n_pages) {
      record_status(a.status, kStatusBounds);
      pg = a.n_pages;  // past the tensor: zeros
    }
  }
  const uint32_t count = __popc(__ballot_sync(0xffffffffu, live));
  if (lane == 0) mbar_expect_tx(bar, count * (uint32_t)(box * kD * 2));
  __syncwarp();
  if (live) {
#pragma unroll
    for (int pn = 0; pn < LL::kPanels; ++pn)
      tma_load_4d(dst + pn * rows * LL::kRowBytes + lane * box * LL::kRowBytes, map, bar, LL::kPanelElems * pn, f,
                  j & (a.page - 1), pg);
  }
}

// Rows [keep, rows) of a loaded block overwritten with zeros, for the products
// to read: slots past a sequence's keys may hold anything, and a weight of 0
// would turn a NaN there into a NaN row.
template <int kD>
__device__ __forceinline__ void zero_rows(uint8_t* dst, int rows, int keep, int lane) {
  using LL = Panels<kD>;
  const int chunks = (rows - keep) * (LL::kRowBytes / 16);  // of one panel
  for (int pn = 0; pn < LL::kPanels; ++pn)
    for (int c = lane; c < chunks; c += 32)
      *reinterpret_cast<uint4*>(dst + pn * rows * LL::kRowBytes + keep * LL::kRowBytes + c * 16) =
          make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// [T, H, D] as (d, h, t): a box is one panel of G heads by `tokens` tokens.
inline bool encode_q(EncodeTiledFn enc, CUtensorMap* map, const void* base, const AttnArgs& a, int tokens) {
  const cuuint64_t row = (cuuint64_t)a.D * 2;
  cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.H, (cuuint64_t)a.T};
  cuuint64_t strides[2] = {row, row * a.H};
  const int pe = a.D >= 64 ? 64 : a.D;
  cuuint32_t box[3] = {(cuuint32_t)pe, (cuuint32_t)a.G, (cuuint32_t)tokens};
  cuuint32_t one[3] = {1, 1, 1};
  return enc(map, a.dtype == LONGNET_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             pe == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
             : pe == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                        : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Keys or values as (d, head, slot, page) or, contiguous, (d, head, position,
// batch); a box is one panel of `rows` slots, or of a page with fewer.
inline bool encode_kv(EncodeTiledFn enc, CUtensorMap* map, const void* base, const AttnArgs& a, int rows) {
  const bool paged = a.cu_q != nullptr;
  const int64_t slots = paged ? a.page : a.nq_max, outer = paged ? a.n_pages : a.S;
  if (paged && rows > a.page) rows = a.page;
  const cuuint64_t row = (cuuint64_t)a.D * 2;
  cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.Hkv, (cuuint64_t)slots, (cuuint64_t)outer};
  cuuint64_t strides[3] = {row, row * a.Hkv, row * a.Hkv * slots};
  const int pe = a.D >= 64 ? 64 : a.D;
  cuuint32_t box[4] = {(cuuint32_t)pe, 1, (cuuint32_t)rows, 1};
  cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, a.dtype == LONGNET_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             pe == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
             : pe == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                        : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace wt
}  // namespace longnet
