// What the windowed kernels with two CTAs per SM share (jfa_win.cu: forward; jfa_win_dq.cu and
// jfa_win_dkdv.cu: the backward passes at d = 64): the query tiles that a CTA's scheduler hands to
// its warps, and their waits.
#pragma once
#include <cuda_bf16.h>

#include "jfa_internal.h"
#include "sm100_ptx.cuh"
#include "jfa_sched.cuh"

namespace jfa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWinThreads = 256;
constexpr int kSoftmaxWarps = 4;
constexpr int kWinConsumers = 3 + kSoftmaxWarps;  // of a metadata entry
constexpr uint32_t kWinTmemCols = 256;

// What the roles need to know of an item, a query tile, worked out once by the scheduler: its
// steps are nz of sinks, then the window part's 64-key tiles from a on, n in all.
struct WinTile {
  int b, h, t;          // sequence (-1: no more items), query head, query tile
  int nz, a, n;
  int rows;             // rows of the tile that are queries
  int pos;              // position of its first row, counted from the grid's start
  int Lq, Lk, org, ns, pad, skip;  // as in WinSeq
  int64_t qo, ko;       // first query row of the sequence, first row of its window part's grid
  int64_t qp;           // its first row in the padded per-query vectors (backward)
};
struct TileRing {
  WinTile e[kMetaSlots];
  uint64_t full[kMetaSlots], empty[kMetaSlots];
  const uint64_t* wait_ns;  // the planner's hand-off limit for this launch
};
// The scheduler (one thread): claims item k once item k - 2 is released by every role, so the
// CTA never holds more than one item that it has not started; an end marker closes the ring.
template <int kAlign, typename Params>
__device__ __forceinline__ bool publish_tiles(TileRing& r, const Params& p, const int64_t* qpad, volatile int* abort) {
  const int n_items = *p.n_items;
  for (uint32_t k = 0;; ++k) {
    if (k >= 2) {
      const uint32_t kp = k - 2;
      if (!mbar_wait(&r.empty[kp % kMetaSlots], (kp / kMetaSlots) & 1, abort, r.wait_ns, kWaitTimeoutNs)) return false;
    }
    const int idx = atomicAdd(p.claim, 1);
    WinTile w = {};
    w.b = -1;
    if (idx < n_items) {
      const WorkItem wi = p.items[idx / p.H];  // one entry for all heads
      w.b = wi.b;
      w.h = idx % p.H;
      w.t = wi.u0;
      w.qo = p.q_off[wi.b];
      if (qpad) w.qp = qpad[wi.b];
      w.ko = p.kv_off[wi.b];
      w.Lq = int(p.q_off[wi.b + 1] - w.qo);
      const WinSeq ws = win_seq(w.Lq, int(p.kv_off[wi.b + 1] - w.ko), p.win.window, p.win.sinks, kAlign);
      w.ko += ws.org;
      w.Lk = ws.Lk;
      w.org = ws.org;
      w.ns = ws.ns;
      w.pad = ws.pad;
      w.skip = ws.skip;
      int e;
      win_kv_tiles(w.t, w.Lq, ws, p.win.window, &w.a, &e, kWinKeys);
      w.nz = win_sees_sinks(w.t, w.Lq, ws) ? (ws.ns + kWinKeys - 1) / kWinKeys : 0;
      w.n = w.nz + e - w.a;
      w.rows = min(kBM, w.Lq - w.t * kBM);
      w.pos = w.t * kBM + w.Lk - w.Lq;
    }
    r.e[k % kMetaSlots] = w;
    mbar_arrive(&r.full[k % kMetaSlots]);  // release: the entry is visible to every thread that waits on it
    if (w.b < 0) {
      grid_launch_dependents();  // nothing left to claim: the next kernel may take freed SMs
      return true;
    }
  }
}
// Entry k, read in place until it is released; all lanes of a warp together (see meta_wait_warp).
__device__ __forceinline__ bool tile_wait(TileRing& r, uint32_t k, volatile int* abort) {
  return mbar_wait(&r.full[k % kMetaSlots], (k / kMetaSlots) & 1, abort, r.wait_ns, kWaitTimeoutNs);
}
__device__ __forceinline__ bool tile_wait_warp(TileRing& r, uint32_t k, volatile int* abort) {
  return __all_sync(0xffffffffu, tile_wait(r, k, abort));
}
__device__ __forceinline__ void tile_release_warp(TileRing& r, uint32_t k) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[k % kMetaSlots]);
}

// A ring position: entry and the parity of its current round.
template <int N>
struct Ring {
  uint32_t e = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++e == N) {
      e = 0;
      ph ^= 1;
    }
  }
};

__device__ __forceinline__ void raise_status(int* status, int code) { atomicCAS(status, 0, code); }

// A wait of a whole warp, whose lanes then agree on its outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, kWaitTimeoutNs));
}

// Wait that ignores the abort flag: used only to drain copies already in flight.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitTimeoutNs) return;
  }
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

}  // namespace
}  // namespace jfa
