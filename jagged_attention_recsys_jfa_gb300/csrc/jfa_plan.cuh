// What the planners share (jfa_plan.cu, and jfa_win_plan.cu for the windowed call): their
// parameters, block-wide scans and the padded query offsets.
#pragma once
#include "jfa_internal.h"
#include "sm100_ptx.cuh"

namespace jfa {
namespace {

struct PlanParams {
  const int64_t* q_off;
  const int64_t* kv_off;
  int B, H;
  int64_t total_q, total_kv;
  int causal, backward;
  int grid;  // persistent CTAs of the kernels that consume the lists
  int nsp_max_tiles;  // query tiles up to which a sequence takes the non-sequence-parallel pass
  int d;              // head dimension
  uint8_t* ws;
  WsLayout L;
  const float* bias;  // [H][nb] or nullptr
  float* bias_grad;   // [H][nb] gradient table to clear before the backward passes add into it, or nullptr
  int nb;
  const int64_t* jb_off;  // general jagged bias block offsets [B+1], or nullptr
  int64_t jb_plane;
  WindowSpec win;         // windowed call
};

enum ListKind { kListFwd = 0, kListDq = 1, kListDkv = 2, kListFused = 3, kListNsp = 4 };

// Block-wide inclusive scan of one 64-bit value per thread (blockDim.x == 1024).
__device__ long long block_scan_incl(long long v, long long* total) {
  __shared__ long long warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const long long w = warp_sums[lane];
    long long wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += y;
    }
    warp_sums[lane] = wi - w;
    if (lane == 31) *total = wi;
  }
  __syncthreads();
  const long long r = warp_sums[warp] + incl;
  __syncthreads();
  return r;
}

// Exclusive scan of hist[] in descending cost order: base[c] = sum_{c' > c} hist[c'].
// 1024 threads, kCostBuckets = 2048 buckets (two per thread).  Returns the total.
__device__ int scan_desc(const int* hist, int* base) {
  __shared__ long long total;
  const int tid = threadIdx.x;
  // thread tid owns descending positions r = 2*tid, 2*tid+1  (bucket c = kCostBuckets-1-r)
  const int c0 = kCostBuckets - 1 - 2 * tid, c1 = c0 - 1;
  const int v0 = hist[c0], v1 = hist[c1];
  const long long incl = block_scan_incl(v0 + v1, &total);
  const int excl = int(incl) - (v0 + v1);
  base[c0] = excl;
  base[c1] = excl + v0;
  __syncthreads();
  return int(total);
}

// Backward: offsets of each sequence in the 128-row-padded per-query vectors.
__device__ void write_qpad(const PlanParams& p) {
  __shared__ long long chunk_total;
  int64_t* qpad = reinterpret_cast<int64_t*>(p.ws + p.L.qpad);
  long long carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    long long v = 0;
    if (b < p.B) v = ((p.q_off[b + 1] - p.q_off[b]) + kBM - 1) / kBM * kBM;
    const long long incl = block_scan_incl(v, &chunk_total);
    if (b < p.B) qpad[b] = carry + incl - v;
    carry += chunk_total;
  }
  if (threadIdx.x == 0) {
    qpad[p.B] = carry;
    reinterpret_cast<WsHeader*>(p.ws)->total_qpad = carry;
  }
}

// The planner's arguments from a problem's.  `grid`: the CTAs that share a list's items.
inline PlanParams plan_params(const Problem& pr, void* ws, const WsLayout& L, bool backward, int grid) {
  PlanParams p;
  p.q_off = pr.q_off;
  p.kv_off = pr.kv_off;
  p.B = pr.B;
  p.H = pr.H;
  p.total_q = pr.total_q;
  p.total_kv = pr.total_kv;
  p.causal = pr.causal;
  p.backward = backward ? 1 : 0;
  p.grid = grid;
  p.nsp_max_tiles = pr.nsp_max_tiles;
  p.d = pr.d;
  p.ws = static_cast<uint8_t*>(ws);
  p.L = L;
  p.bias = pr.bias_table;
  p.bias_grad = backward ? pr.bias_grad : nullptr;
  p.jb_off = pr.jb_off;
  p.jb_plane = pr.jb_plane;
  p.nb = pr.num_buckets;
  p.win = pr.win;
  return p;
}

}  // namespace
}  // namespace jfa
