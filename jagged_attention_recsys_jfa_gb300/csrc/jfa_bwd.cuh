// What the backward passes share (jfa_bwd.cu, and jfa_win_bwd.cu for the windowed call): their
// parameters, tile shapes and memory plans, and the transfers between TMEM, registers and memory.
#pragma once
#include <cuda_bf16.h>

#include "jfa_internal.h"
#include "sm100_ptx.cuh"
#include "jfa_sched.cuh"

namespace jfa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// dK/dV pass (512 threads): role warps, compute warpgroups, epilogue warpgroup
constexpr uint32_t kRegsLoadDkdv = 96, kRegsComputeDkdv = 168, kRegsEpiDkdv = 72;
static_assert(reg_split_fits_dkdv(kRegsLoadDkdv, kRegsComputeDkdv, kRegsEpiDkdv),
              "register split exceeds the launch allocation");
struct BwdParams {
  const int64_t* q_off;
  const int64_t* kv_off;
  int B, H;
  int64_t total_q, total_kv;
  float scale, scale_log2;
  int causal;
  const float* bias2;  // [H][num_buckets] bias * log2(e), or nullptr
  float* bias_grad;    // [H][num_buckets] gradient of the bias table (cleared by the planner), or nullptr
  int num_buckets, center;
  const __nv_bfloat16* jbias;  // general jagged bias [H][jb_plane], or nullptr
  const int64_t* jb_off;       // its block offsets [B+1]
  int64_t jb_plane;
  __nv_bfloat16* jb_grad;      // its gradient (dK/dV and fused passes), or nullptr
  const CUtensorMap* maps;
  const WorkItem* items;
  const int* n_items;
  int* claim;  // the list's claim counter (zeroed by the planner)
  int* status;
  const uint64_t* wait_ns;  // the planner's item hand-off wait limit for this launch (ns)
  const float* lse2;    // [H][qpad_cap]  -lse * log2(e), padded per sequence to 128 rows
  const float* delta;   // [H][qpad_cap]  -D, same layout
  const int64_t* qpad;  // [B+1] sequence offsets in the padded vectors
  int64_t qpad_cap;
  __nv_bfloat16* g0;   // dK (dK/dV and fused passes) or dQ (dQ pass)
  __nv_bfloat16* g1;   // dV (dK/dV and fused passes)
  __nv_bfloat16* g2;   // dQ (fused and non-sequence-parallel passes)
  float* dqacc;        // non-sequence-parallel pass: fp32 dQ sums [total_q][H][D]
  TraceBuf trace;
  // windowed call
  WindowSpec win;
  int group;                 // query heads per key/value head
  const CUtensorMap* smaps;  // the sinks' K / V maps
  int sink_rows;             // rows of their boxes
  float* spart;              // partial dK, dV of the sinks (dK/dV pass): [slot][2][sinks][D]
};

__device__ __forceinline__ void raise_status(int* status, int code) { atomicCAS(status, 0, code); }

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitTimeoutNs) return;
  }
}

template <int D>
struct BwdCfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kRingDkdv = D == 128 ? 4 : 8;  // single-tile ring entries
  static constexpr int kRingDq = D == 128 ? 5 : 8;
  static constexpr int kVecSlots = 4;                  // dK/dV: per-query-tile lse2 / D vectors
  // dK/dV pass: S^T, dP^T, dK, dV.   dQ pass: S, dP (two buffers), dQ.
  static constexpr uint32_t kColS = 0, kColP = 128, kColA0 = 256, kColA1 = 256 + D;
  static constexpr uint32_t kColP1 = 256, kColDQ = 384;
  // dK/dV pass: P^T and dS^T (bf16, keys x 128 queries, each compute warpgroup's 64 queries
  // in 32 columns) over S^T / dP^T at d = 128, two 64-column halves apart; at d = 64 in the
  // spare columns [384, 448) and [448, 512), so the next S^T / dP^T MMA does not write the
  // columns the previous dV / dK MMA is still reading
  static constexpr uint32_t kColPT = D == 64 ? 384 : kColS, kColDST = D == 64 ? 448 : kColP;
  static constexpr uint32_t kXHalf = D == 64 ? 32 : 64;
  // dQ pass at d = 64: the query tile's Q and dO rows copied into the free columns
  // [448, 480) and [480, 512) by the compute warpgroups feed the S and dP MMAs from TMEM, and
  // the shared-memory buffers are free for the next query tile once both copies are done
  static constexpr bool kDqQTmem = D == 64;
  static constexpr uint32_t kColDqQ = 448, kColDqDO = 480;
  static constexpr int kSmemDkdv = 2 * kTileBytes + kRingDkdv * kTileBytes + kVecSlots * 1024 + 1024;
  static constexpr int kSmemDq = 2 * kTileBytes + kRingDq * kTileBytes + 1024;
  // Fused short-query pass: Q and dO resident, K/V ring, dS^T staging (keys x 128 queries,
  // bf16), lse2 / D vectors.  TMEM: S^T [0,128), dP^T then dK [128,256), dV, dQ.
  static constexpr int kRingFused = D == 128 ? 3 : 8;
  static constexpr uint32_t kColFdV = 256, kColFdQ = 256 + D;
  static constexpr int kSmemFused = 2 * kTileBytes + kRingFused * kTileBytes + 32768 + 1024 + 1024;
  // Non-sequence-parallel pass: K, V resident, dO / Q ring, dS^T staging, lse2 / D vectors.
  // dQ_ij over dP^T at d = 128, in the columns d = 64 leaves free otherwise.
  static constexpr int kRingNsp = D == 128 ? 3 : 8;
  static constexpr uint32_t kColNspDq = D == 128 ? kColP : 384;
  static constexpr int kSmemNsp = 2 * kTileBytes + kRingNsp * kTileBytes + 32768 + kVecSlots * 1024 + 1024;
  static_assert(kSmemDkdv <= 232448 && kSmemDq <= 232448 && kSmemFused + 1024 <= 232448 && kSmemNsp + 1024 <= 232448,
                "shared memory per CTA");
};

// Load one row-tile (128 rows x D columns, D/64 boxes of 16 KB) through a tensor map.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int col0, int row0) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_2d(dst + c * 16384, m, bar, col0 + c * 64, row0);
}

// 64 columns from TMEM -> floats, both loads in flight before one wait.
__device__ __forceinline__ void ld_cols64(uint32_t taddr, float* x) {
  uint32_t r0[32], r1[32];
  tmem_ld32(taddr, r0);
  tmem_ld32(taddr + 32, r1);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    x[c] = __uint_as_float(r0[c]);
    x[32 + c] = __uint_as_float(r1[c]);
  }
}

// Store 64 fp32 values as 32 packed bf16x2 TMEM columns.
__device__ __forceinline__ void st_bf16_64(uint32_t taddr, const float* v) {
  uint32_t pk[32];
#pragma unroll
  for (int t = 0; t < 32; ++t) pk[t] = pack_bf16x2(v[2 * t], v[2 * t + 1]);
  tmem_st32(taddr, pk);
}

// Write NC (32 or 64) accumulator columns of this thread's TMEM lane, times `mul`, as bf16
// to global (or zeros when `zero`), one thread per row.
template <int NC>
__device__ __forceinline__ void store_acc_row_own(uint32_t taddr, float mul, __nv_bfloat16* dst, bool valid,
                                                  bool zero) {
#pragma unroll
  for (int cc = 0; cc < NC / 32; ++cc) {
    uint32_t r[32];
    if (!zero) {
      tmem_ld32(taddr + cc * 32, r);
      tmem_ld_wait();
    }
    uint32_t pk[16];
#pragma unroll
    for (int t = 0; t < 16; ++t)
      pk[t] = zero ? 0u : pack_bf16x2(__uint_as_float(r[2 * t]) * mul, __uint_as_float(r[2 * t + 1]) * mul);
    if (valid) {
      st_global_v8(dst + cc * 32, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
      st_global_v8(dst + cc * 32 + 16, pk[8], pk[9], pk[10], pk[11], pk[12], pk[13], pk[14], pk[15]);
    }
  }
}
// All D accumulator columns of this thread's TMEM lane, times `mul`, as bf16 to its own row,
// 32 columns at a time; arrives on `empty` as soon as the last columns are in registers.
template <int D>
__device__ __forceinline__ void drain_row_own(uint32_t taddr, float mul, __nv_bfloat16* dst, bool valid,
                                              uint64_t* empty) {
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + c0, r);
    tmem_ld_wait();
    if (c0 + 32 == D) {
      tc_fence_before();
      mbar_arrive(empty);
    }
    uint32_t pk[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) pk[t] = pack_bf16x2(__uint_as_float(r[2 * t]) * mul, __uint_as_float(r[2 * t + 1]) * mul);
    if (valid) {
      st_global_v8(dst + c0, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
      st_global_v8(dst + c0 + 16, pk[8], pk[9], pk[10], pk[11], pk[12], pk[13], pk[14], pk[15]);
    }
  }
}

// Write NC (32 or 64) accumulator columns of this thread's TMEM lane, times `mul`, as bf16
// to global (or zeros when `zero`).  All 32 lanes of the warp call it together: the rows'
// stores are shared across lanes so that each store instruction writes whole row segments.
template <int NC>
__device__ __forceinline__ void store_acc_row(uint32_t taddr, float mul, __nv_bfloat16* dst, bool valid, bool zero) {
  uint4 c[NC / 8];  // the row's NC bf16 values as 16-byte chunks
#pragma unroll
  for (int cc = 0; cc < NC / 32; ++cc) {
    uint32_t r[32];
    if (!zero) {
      tmem_ld32(taddr + cc * 32, r);
      tmem_ld_wait();
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w4[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int e = 8 * q + 2 * t;
        w4[t] = zero ? 0u : pack_bf16x2(__uint_as_float(r[e]) * mul, __uint_as_float(r[e + 1]) * mul);
      }
      c[4 * cc + q] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
    }
  }
  st_rows_coalesced<NC * 2>(c, valid ? static_cast<void*>(dst) : nullptr);
}

// Writes the D accumulator columns of this thread's TMEM lane, times `mul`, as bf16 to the
// row at `dst`, 32 columns at a time (coalesced across the warp), and arrives on `empty`
// once the last columns are in registers: the accumulator may be overwritten from then on.
// All 32 lanes of the warp call it together.
template <int D>
__device__ __forceinline__ void drain_acc_rows(uint32_t taddr, float mul, __nv_bfloat16* dst, bool valid,
                                               uint64_t* empty) {
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + c0, r);
    tmem_ld_wait();
    if (c0 + 32 == D) {
      tc_fence_before();
      mbar_arrive(empty);
    }
    uint4 c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      c[q] = make_uint4(pack_bf16x2(__uint_as_float(r[8 * q]) * mul, __uint_as_float(r[8 * q + 1]) * mul),
                        pack_bf16x2(__uint_as_float(r[8 * q + 2]) * mul, __uint_as_float(r[8 * q + 3]) * mul),
                        pack_bf16x2(__uint_as_float(r[8 * q + 4]) * mul, __uint_as_float(r[8 * q + 5]) * mul),
                        pack_bf16x2(__uint_as_float(r[8 * q + 6]) * mul, __uint_as_float(r[8 * q + 7]) * mul));
    st_rows_coalesced<64>(c, valid ? static_cast<void*>(dst + c0) : nullptr);
  }
}

enum BwdPass { kPassDkdv = 0, kPassDq = 1, kPassFused = 2, kPassNsp = 3 };

inline BwdParams make_params(const Problem& pr, const float* lse, void* ws, const WsLayout& L, int pass) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  BwdParams bp;
  bp.q_off = pr.q_off;
  bp.kv_off = pr.kv_off;
  bp.B = pr.B;
  bp.H = pr.H;
  bp.total_q = pr.total_q;
  bp.total_kv = pr.total_kv;
  bp.scale = pr.scale;
  bp.scale_log2 = pr.scale * kLog2e;
  bp.causal = pr.causal;
  bp.bias2 = pr.bias_table ? reinterpret_cast<const float*>(w + L.bias2) : nullptr;
  // the dK/dV, fused and non-sequence-parallel passes together see every visible pair once:
  // they add the bias gradient
  bp.bias_grad = (pr.bias_table && pass != kPassDq) ? pr.bias_grad : nullptr;
  bp.num_buckets = pr.num_buckets;
  bp.center = pr.center;
  bp.jbias = static_cast<const __nv_bfloat16*>(pr.jbias);
  bp.jb_off = pr.jb_off;
  bp.jb_plane = pr.jb_plane;
  bp.jb_grad = pass != kPassDq ? static_cast<__nv_bfloat16*>(pr.jb_grad) : nullptr;
  bp.maps = reinterpret_cast<const CUtensorMap*>(w + L.maps);
  bp.items = reinterpret_cast<const WorkItem*>(
      w + (pass == kPassDq ? L.dq : pass == kPassFused ? L.fused : pass == kPassNsp ? L.nsp : L.dkv));
  const WsHeader* hdr = reinterpret_cast<const WsHeader*>(w);
  bp.n_items = pass == kPassDq ? &hdr->n_dq : pass == kPassFused ? &hdr->n_fused
                                           : pass == kPassNsp ? &hdr->n_nsp : &hdr->n_dkv;
  WsHeader* mh = reinterpret_cast<WsHeader*>(w);
  bp.claim = pass == kPassDq ? &mh->claim_dq : pass == kPassFused ? &mh->claim_fused
                                             : pass == kPassNsp ? &mh->claim_nsp : &mh->claim_dkv;
  bp.status = &reinterpret_cast<WsHeader*>(w)->status;
  // list kinds of the planner: forward 0, dQ 1, dK/dV 2, fused 3, non-sequence-parallel 4
  bp.wait_ns = &hdr->wait_ns[pass == kPassDq ? 1 : pass == kPassFused ? 3 : pass == kPassNsp ? 4 : 2];
  bp.dqacc = reinterpret_cast<float*>(w + L.dqacc);
  (void)lse;
  bp.lse2 = reinterpret_cast<const float*>(w + L.lse2);
  bp.delta = reinterpret_cast<const float*>(w + L.delta);
  bp.qpad = reinterpret_cast<const int64_t*>(w + L.qpad);
  bp.qpad_cap = L.qpad_cap;
  bp.g0 = nullptr;
  bp.g1 = nullptr;
  bp.g2 = nullptr;
  bp.win = pr.win;
  bp.group = pr.win.window > 0 ? pr.H / pr.win.H_kv : 1;
  bp.smaps = reinterpret_cast<const CUtensorMap*>(w + L.smaps);
  bp.sink_rows = sink_rows(pr.win.sinks);
  bp.spart = reinterpret_cast<float*>(w + L.spart);
  bp.trace = pr.trace[pass == kPassDq ? JFA_KERNEL_BWD_DQ : pass == kPassFused ? JFA_KERNEL_BWD_FUSED
                     : pass == kPassNsp ? JFA_KERNEL_BWD_NSP : JFA_KERNEL_BWD_DKDV];
  return bp;
}

template <typename K>
cudaError_t launch_dkdv_k(K kern, int smem, int grid, const BwdParams& bp, cudaStream_t stream) {
  cudaError_t e = check_launch_registers(kern, kLaunchRegsDkdv);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kThreadsDkdv), smem, stream, bp);
}

}  // namespace
}  // namespace jfa
