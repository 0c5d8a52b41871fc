// Planner kernel: validates the jagged offsets, builds one TMA tensor map per
// (sequence, tensor) whose row extent is that sequence's length -- so tile loads
// past a sequence end arrive as zeros, which the subtraction scheme of "Jagged
// Flash Attention (JFA)", "Four generations" item 1, relies on -- and writes the
// persistent kernels' work lists sorted longest first (counting sort on cost), which
// the kernels' CTAs claim one at a time from a counter, the scheduling that keeps SMs busy
// when short sequences finish early (same page, "Why standard FlashAttention falls short"
// and item 3).
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
  WindowSpec win;         // sliding window with sinks (window = 0: none)
};

enum ListKind { kListFwd = 0, kListDq = 1, kListDkv = 2, kListFused = 3, kListNsp = 4 };

// A sequence's window part and sinks; the forward's key tiles have kWinKeys rows.
__device__ __forceinline__ WinSeq plan_seq(const PlanParams& p, int Lq, int Lk) {
  return win_seq(Lq, Lk, p.win.window, p.win.sinks, p.backward ? kBN : kWinKeys);
}

// Backward: a sequence whose queries fit one tile (Lq <= 128) is done by the fused pass
// (one CTA per sequence and head, every key tile once); one of 2 .. kNspMaxTiles query
// tiles by the non-sequence-parallel pass (one CTA per sequence and head, every tile pair
// once); the others by the split dK/dV and dQ passes.  Units: key tiles, except for the
// forward (query-tile pairs) and the dQ pass (query tiles); a sequence without keys still
// gets one unit in the fused and non-sequence-parallel lists (its dq rows are zeroed there).
// With a sliding window the forward's units are query tiles, and every sequence goes through the forward, dQ and dK/dV lists; the dK/dV
// units are the key tiles of the window part, then the chunks of the sinks.
__device__ __forceinline__ int list_units(const PlanParams& p, int kind, int Lq, int Lk) {
  const int nsp_max = p.nsp_max_tiles;
  const int nq = (Lq + kBM - 1) / kBM;
  const int nk = (Lk + kBN - 1) / kBN;
  if (p.win.window > 0) {
    if (kind == kListFwd || kind == kListDq) return nq;
    const WinSeq s = plan_seq(p, Lq, Lk);
    return (s.Lk + kBN - 1) / kBN + win_sink_chunks(Lq, s, p.H / p.win.H_kv);
  }
  if (kind == kListFwd) return (nq + 1) / 2;
  if (kind == kListFused) return Lq <= kBM ? (nk > 0 ? nk : (Lq > 0 ? 1 : 0)) : 0;
  if (kind == kListNsp) return nsp_path(Lq, nsp_max) ? (nk > 0 ? nk : 1) : 0;
  if (Lq <= kBM || nsp_path(Lq, nsp_max)) return 0;
  return kind == kListDq ? nq : nk;
}

__device__ __forceinline__ int win_tile_cost(int t, int Lq, const WinSeq& s, int W, int keys) {
  int a, e;
  win_kv_tiles(t, Lq, s, W, &a, &e, keys);
  return e - a + (win_sees_sinks(t, Lq, s) ? 1 : 0);
}

__device__ __forceinline__ int unit_cost(const PlanParams& p, int kind, int u, int Lq, int Lk) {
  const bool causal = p.causal != 0;
  if (p.win.window > 0) {
    const WinSeq s = plan_seq(p, Lq, Lk);
    if (kind == kListFwd) return win_tile_cost(u, Lq, s, p.win.window, kWinKeys);
    if (kind == kListDq) return win_tile_cost(u, Lq, s, p.win.window, kBN);
    const WinKeyUnit k = win_key_unit(u, Lq, s, p.win.window, p.H / p.win.H_kv);
    return k.r1 - k.r0;
  }
  if (kind == kListFused) return 1;  // a key tile (its dK / dV rows are stored even when unseen)
  if (kind == kListNsp) {            // the query tiles that see key tile u (at least 1)
    int first, count;
    q_tiles_for_kv_tile(u, Lq, Lk, causal, &first, &count);
    return count > 0 ? count : 1;
  }
  if (kind == kListFwd)
    return kv_tiles_for_q_tile(2 * u, Lq, Lk, causal) + kv_tiles_for_q_tile(2 * u + 1, Lq, Lk, causal);
  if (kind == kListDq) return kv_tiles_for_q_tile(u, Lq, Lk, causal);
  int first, count;
  q_tiles_for_kv_tile(u, Lq, Lk, causal, &first, &count);
  return count;
}

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

// Walk the units of one sequence, cutting them into consecutive ranges whose summed
// cost stays <= cap (a unit costlier than cap forms its own range); calls f(u0, u1, cost).
template <typename F>
__device__ void for_each_range(const PlanParams& p, int kind, int Lq, int Lk, long long cap, F&& f) {
  const int n = list_units(p, kind, Lq, Lk);
  int start = 0;
  long long acc = 0;
  for (int u = 0; u < n; ++u) {
    const int c = unit_cost(p, kind, u, Lq, Lk);
    if (u > start && acc + c > cap) {
      f(start, u, acc);
      start = u;
      acc = 0;
    }
    acc += c;
  }
  if (n > 0) f(start, n, acc);
}

// The windowed lists.  A window bounds what a unit can cost, so every unit is an item of its own
// and the units, not the sequences, are dealt out to the threads: a thread finds its unit's
// sequence in the running sums of the threads' runs of sequences (1024 of them) and walks its run
// to it.  Long sequences then cost no more time than short ones (long-tail batch of 64 sequences:
// 31 -> 10 us against emit_list).  Costliest first by the same counting sort.  One entry stands
// for a unit of all `heads` heads: item i of the launch is entry i / heads, head i % heads, so that
// heads which share keys read them at the same time (and the list is written in a tenth of the time
// that one entry per head took).
__device__ void emit_window_list(const PlanParams& p, int kind, WorkItem* items, int64_t cap, int* count_out, int* hist,
                                 int* base) {
  __shared__ long long run_end[1024];
  __shared__ int run_q[1024], run_k[1024];  // lengths, when a run is one sequence
  __shared__ long long units_total, cost_total;
  __shared__ int cost_max;
  const int tid = threadIdx.x;
  const int heads = kind == kListDkv ? p.win.H_kv : p.H;
  const int run = (p.B + 1023) / 1024;
  auto len_q = [&](int b) { return int(p.q_off[b + 1] - p.q_off[b]); };
  auto len_k = [&](int b) { return int(p.kv_off[b + 1] - p.kv_off[b]); };
  for (int c = tid; c < kCostBuckets; c += blockDim.x) hist[c] = 0;
  if (tid == 0) cost_max = 0;
  long long mine = 0;
  for (int b = tid * run; b < min(p.B, (tid + 1) * run); ++b) {
    run_q[tid] = len_q(b);
    run_k[tid] = len_k(b);
    mine += list_units(p, kind, run_q[tid], run_k[tid]);
  }
  run_end[tid] = block_scan_incl(mine, &units_total);
  __syncthreads();
  const long long n = units_total;
  if (n > cap) {  // cannot happen for valid offsets (capacities are upper bounds)
    if (tid == 0) {
      atomicCAS(&reinterpret_cast<WsHeader*>(p.ws)->status, 0, int(JFA_ERR_WORKSPACE));
      *count_out = 0;
    }
    return;
  }
  // calls f(active, b, unit, cost) for this thread's units, all lanes of a warp together
  auto for_units = [&](auto&& f) {
    for (long long i = tid; i - tid < n; i += blockDim.x) {
      int b = 0, u = 0, cost = 0;
      if (i < n) {
        int lo = 0, hi = 1023;  // the first run that ends behind unit i
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (run_end[mid] > i) hi = mid;
          else lo = mid + 1;
        }
        long long at = lo ? run_end[lo - 1] : 0;
        int lq = run_q[lo], lk = run_k[lo];
        b = lo * run;
        if (run > 1) {
          for (;; ++b) {
            lq = len_q(b);
            lk = len_k(b);
            const int m = list_units(p, kind, lq, lk);
            if (at + m > i) break;
            at += m;
          }
        }
        u = int(i - at);
        cost = unit_cost(p, kind, u, lq, lk);
      }
      f(i < n, b, u, cost);
    }
  };
  // Position of this lane's entry in its bucket.  Most units cost the same, so lanes of
  // one bucket share one addition.
  auto claim = [&](int* counts, bool active, int bkt) -> int {
    const unsigned same = __match_any_sync(0xffffffffu, active ? bkt : -1);
    const int lane = tid & 31, first = __ffs(same) - 1;
    int pos = 0;
    if (active && lane == first) pos = atomicAdd(&counts[bkt], __popc(same));
    return __shfl_sync(0xffffffffu, pos, first) + __popc(same & ((1u << lane) - 1u));
  };
  auto bucket = [](int cost) { return cost < kCostBuckets - 1 ? cost : kCostBuckets - 1; };
  long long sum = 0;
  int mx = 0;
  for_units([&](bool active, int, int, int cost) {
    claim(hist, active, bucket(cost));
    sum += cost;
    mx = max(mx, cost);
  });
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((tid & 31) == 0) atomicMax(&cost_max, mx);
  block_scan_incl(sum, &cost_total);
  const int total = scan_desc(hist, base);
  for_units([&](bool active, int b, int u, int cost) {
    const int pos = claim(base, active, bucket(cost));
    if (active) *reinterpret_cast<int4*>(items + pos) = make_int4(b, 0, u, u + 1);
  });
  if (tid == 0) {
    *count_out = total * heads;
    reinterpret_cast<WsHeader*>(p.ws)->wait_ns[kind] =
        wait_limit_ns(cost_total * heads, p.grid, cost_max);
  }
}

__device__ void emit_list(const PlanParams& p, int kind, WorkItem* items, int64_t cap, int* count_out,
                          int* hist, int* base) {
  if (p.win.window > 0) return emit_window_list(p, kind, items, cap, count_out, hist, base);
  __shared__ long long total_cost;
  const int tid = threadIdx.x;
  const int heads = p.H;
  // total work, to cap range cost at about 1/kItemsPerCta of a CTA's share
  long long local = 0;
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int Lq = int(p.q_off[b + 1] - p.q_off[b]);
    const int Lk = int(p.kv_off[b + 1] - p.kv_off[b]);
    const int n = list_units(p, kind, Lq, Lk);
    for (int u = 0; u < n; ++u) local += unit_cost(p, kind, u, Lq, Lk);
  }
  block_scan_incl(local, &total_cost);
  const long long share = (total_cost * heads + (long long)kItemsPerCta * p.grid - 1) /
                          ((long long)kItemsPerCta * p.grid);
  // the fused and non-sequence-parallel passes own each sequence's dQ: their items are
  // never cut into ranges.  At d = 128 the dK/dV and dQ passes take one tile per item, and
  // a (sequence, head)'s items sit next to each other in the list (ordered by the group's
  // total cost, longest first): neighbouring CTAs claim them together and stream the
  // operand they share (Q / dO for dK/dV, K / V for dQ) at the same time, so more of it
  // comes from L2 (GEM-like shape: dK/dV 720 -> 699 us; long-tail causal 1172 -> 1122 us).
  // At d = 64 a tile is too short for the per-item cost (biased causal shape: dK/dV
  // 344 -> 398 us), so those lists keep capped ranges, and so does the forward (grouped
  // query-tile pairs: GEM-like forward 411 -> 447 us).
  const bool grouped = (kind == kListDkv || kind == kListDq) && p.d == 128;
  const long long range_cap =
      (kind == kListFused || kind == kListNsp) ? (1ll << 62) : (grouped ? 1 : (share > 1 ? share : 1));
  auto bucket = [](long long cost) { return cost < kCostBuckets - 1 ? int(cost) : kCostBuckets - 1; };

  for (int c = tid; c < kCostBuckets; c += blockDim.x) hist[c] = 0;
  __syncthreads();
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int Lq = int(p.q_off[b + 1] - p.q_off[b]);
    const int Lk = int(p.kv_off[b + 1] - p.kv_off[b]);
    if (grouped) {
      long long gcost = 0;
      int nr = 0;
      for_each_range(p, kind, Lq, Lk, range_cap, [&](int, int, long long cost) {
        gcost += cost;
        ++nr;
      });
      if (nr) atomicAdd(&hist[bucket(gcost)], heads * nr);
    } else {
      for_each_range(p, kind, Lq, Lk, range_cap,
                     [&](int, int, long long cost) { atomicAdd(&hist[bucket(cost)], heads); });
    }
  }
  __syncthreads();
  const int total = scan_desc(hist, base);
  if (total > cap) {  // cannot happen for valid offsets (capacities are upper bounds)
    if (tid == 0) {
      atomicCAS(&reinterpret_cast<WsHeader*>(p.ws)->status, 0, int(JFA_ERR_WORKSPACE));
      *count_out = 0;
    }
    return;
  }
  __shared__ unsigned long long max_item;
  if (tid == 0) max_item = 0;
  __syncthreads();
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int Lq = int(p.q_off[b + 1] - p.q_off[b]);
    const int Lk = int(p.kv_off[b + 1] - p.kv_off[b]);
    unsigned long long mx = 0;
    if (grouped) {
      long long gcost = 0;
      int nr = 0;
      for_each_range(p, kind, Lq, Lk, range_cap, [&](int, int, long long cost) {
        gcost += cost;
        ++nr;
      });
      if (nr) {
        // head h's tiles at pos + h * nr + r, in tile order
        const int pos = atomicAdd(&base[bucket(gcost)], heads * nr);
        int r = 0;
        for_each_range(p, kind, Lq, Lk, range_cap, [&](int u0, int u1, long long cost) {
          for (int h = 0; h < heads; ++h) items[pos + h * nr + r] = WorkItem{b, h, u0, u1};
          ++r;
          if ((unsigned long long)cost > mx) mx = (unsigned long long)cost;
        });
      }
    } else {
      for_each_range(p, kind, Lq, Lk, range_cap, [&](int u0, int u1, long long cost) {
        const int pos = atomicAdd(&base[bucket(cost)], heads);
        for (int h = 0; h < heads; ++h) items[pos + h] = WorkItem{b, h, u0, u1};
        if ((unsigned long long)cost > mx) mx = (unsigned long long)cost;
      });
    }
    if (mx) atomicMax(&max_item, mx);
  }
  __syncthreads();
  if (tid == 0) {
    *count_out = total;
    // the bounded waits of the kernel that walks this list scale with the planned work
    reinterpret_cast<WsHeader*>(p.ws)->wait_ns[kind] =
        wait_limit_ns(total_cost * heads, p.grid, (long long)max_item);
  }
  __syncthreads();
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

// The first CTAs validate the offsets and write one work list each (block-wide scans: the
// forward list, or the dK/dV (with the padded query offsets), dQ and fused lists); the
// other CTAs write the bias table, the tail copies and the tensor maps in parallel.
__global__ void __launch_bounds__(1024, 1) plan_kernel(const __grid_constant__ PlanMaps maps, PlanParams p) {
  __shared__ int hist[kCostBuckets];
  __shared__ int base[kCostBuckets];
  const int tid = threadIdx.x;
  WsHeader* hdr = reinterpret_cast<WsHeader*>(p.ws);
  grid_dependency_wait();    // the offsets and the workspace may come from earlier work
  grid_launch_dependents();  // the next kernel may start its prologue; it waits for this one

  const int list_ctas = !p.backward ? 1 : p.win.window > 0 ? 2 : 4;
  if (int(blockIdx.x) >= list_ctas) {
    const size_t gt = size_t(blockIdx.x - list_ctas) * blockDim.x + tid;
    const size_t gstride = size_t(gridDim.x - list_ctas) * blockDim.x;
    // ---- bias table pre-scaled to log2 units (the kernels work with exp2)
    if (p.bias) {
      float* b2 = reinterpret_cast<float*>(p.ws + p.L.bias2);
      for (size_t i = gt; i < size_t(p.H) * p.nb; i += gstride) b2[i] = p.bias[i] * 1.4426950408889634f;
    }
    if (p.bias_grad)
      for (size_t i = gt; i < size_t(p.H) * p.nb; i += gstride) p.bias_grad[i] = 0.f;
    // ---- tail copies: the last min(128, total) rows of each tensor, which the boxes that
    //      would otherwise read past the tensor's last row load from instead
    for (int slot = 0; slot < kNumMapSlots; ++slot) {
      if (!maps.used[slot]) continue;
      const int64_t total = (slot == kMapQ || slot == kMapDO) ? p.total_q : p.total_kv;
      if (total <= 0) continue;
      const int64_t n = total < kBM ? total : kBM;
      const size_t rb = maps.row_bytes[slot];
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(maps.base[slot]) +
                                                        size_t(total - n) * rb);
      uint4* dst = reinterpret_cast<uint4*>(p.ws + p.L.tail + size_t(slot) * kTailRows * p.L.row_bytes);
      const size_t nvec = size_t(n) * rb / 16;
      for (size_t i = gt; i < nvec; i += gstride) dst[i] = src[i];
    }
    // ---- per-sequence tensor maps: copy the template, point it at the sequence's first
    //      row and clip its row extent to the sequence length.  A sequence whose last tile
    //      would reach past the tensor's last row also gets a tail map over the tail copy,
    //      pointed at that tile's first row and clipped to the tile's rows.  (With invalid
    //      offsets CTA 0 leaves every list empty, so no map is used; a tail map is only
    //      written for a sequence inside its tensor, which keeps its index in range.)
    //      One warp per map: the replaces of a warp's lanes are done one after another, so lanes
    //      that each wrote a map would be what the planner waits for.
    const int sets = p.win.window > 0 && p.win.sinks > 0 ? 2 : 1;  // maps, and the sinks' maps
    const int lane = tid & 31;
    for (size_t job = gt / 32; job < size_t(p.B) * kNumMapSlots * 2 * sets; job += gstride / 32) {
      const bool tail = job & 1, sink = sets == 2 && ((job >> 1) & 1);
      const size_t idx = job / (2 * sets);
      const int b = int(idx / kNumMapSlots), slot = int(idx % kNumMapSlots);
      if (!maps.used[slot]) continue;
      const bool is_q_side = (slot == kMapQ || slot == kMapDO);
      int64_t row0 = is_q_side ? p.q_off[b] : p.kv_off[b];
      int64_t len = (is_q_side ? p.q_off[b + 1] : p.kv_off[b + 1]) - row0;
      int skip = 0;  // empty rows in front of the first key's tile
      if (is_q_side && sink) continue;
      if (p.win.window > 0 && !is_q_side) {  // the sinks, or the window part
        const int64_t lq = p.q_off[b + 1] - p.q_off[b];
        if (lq < 0 || len < 0 || lq > (int64_t(1) << 30) || len > (int64_t(1) << 30)) continue;
        const WinSeq ws = plan_seq(p, int(lq), int(len));
        skip = sink ? 0 : ws.skip;
        if (!sink) row0 += ws.org + ws.skip;
        len = sink ? ws.ns : ws.Lk - ws.skip;
      }
      const size_t rb = maps.row_bytes[slot];
      const int rows = maps.tile_rows[slot];
      const int64_t total = is_q_side ? p.total_q : p.total_kv;
      CUtensorMap* dst = reinterpret_cast<CUtensorMap*>(p.ws + (sink ? p.L.smaps : p.L.maps));
      const void* base;
      if (!tail) {
        dst += idx;
        base = static_cast<const uint8_t*>(maps.base[slot]) + row0 * int64_t(rb);
      } else {
        if (len <= 0 || row0 < 0 || row0 + len > total) continue;
        // the sequence's last tile: its box's first row, and its first row that holds something
        const int64_t g0 = row0 - skip + (skip + len - 1) / rows * rows, r0 = g0 > row0 ? g0 : row0;
        if (g0 + rows <= total) continue;
        const int64_t n = total < kBM ? total : kBM;  // rows in the tail copy; it starts at row total - n
        dst += size_t(p.B) * kNumMapSlots + size_t(slot) * kTailMaps + size_t(r0 + rows - total);
        base = p.ws + p.L.tail + size_t(slot) * kTailRows * p.L.row_bytes + size_t(r0 - (total - n)) * rb;
        len = row0 + len - r0;
      }
      const uint4* src = reinterpret_cast<const uint4*>(sink ? &maps.sink_tmpl[slot - kMapK] : &maps.tmpl[slot]);
      if (lane < 8) reinterpret_cast<uint4*>(dst)[lane] = src[lane];
      __syncwarp();
      if (lane == 0) {
        tmap_replace_address(dst, base);
        tmap_replace_dim1(dst, uint32_t(len > 0 ? len : 1));
      }
    }
    tmap_release();
    return;
  }

  // ---- list CTAs: validate offsets (each list CTA on its own, so all agree)
  int bad = 0;
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int64_t lq = p.q_off[b + 1] - p.q_off[b];
    const int64_t lk = p.kv_off[b + 1] - p.kv_off[b];
    if (lq < 0 || lk < 0 || lq > (int64_t(1) << 30) || lk > (int64_t(1) << 30)) bad = 1;
    // a general bias's blocks must hold exactly Lq x round_up(Lk, 8) elements each
    if (p.jb_off && !bad && p.jb_off[b + 1] - p.jb_off[b] != lq * ((lk + 7) / 8 * 8)) bad = 1;
  }
  if (tid == 0) {
    if (p.q_off[0] != 0 || p.kv_off[0] != 0 || p.q_off[p.B] != p.total_q || p.kv_off[p.B] != p.total_kv)
      bad = 1;
    if (p.jb_off && (p.jb_off[0] != 0 || p.jb_off[p.B] != p.jb_plane)) bad = 1;
  }
  if (blockIdx.x == 0 && tid == 0) hdr->claim_fwd = hdr->claim_dq = hdr->claim_dkv = hdr->claim_fused = hdr->claim_nsp = 0;
  bad = __syncthreads_or(bad);
  if (bad) {
    if (tid == 0) {
      atomicCAS(&hdr->status, 0, int(JFA_ERR_BAD_OFFSETS));
      hdr->n_fwd = hdr->n_dq = hdr->n_dkv = hdr->n_fused = hdr->n_nsp = 0;
      hdr->total_qpad = 0;  // the preprocess walks no rows
      if (blockIdx.x == 0) hdr->planned = 0;
    }
    return;
  }

  // ---- work lists
  if (blockIdx.x == 0 && tid == 0) hdr->planned = 1;
  if (!p.backward) {
    emit_list(p, kListFwd, reinterpret_cast<WorkItem*>(p.ws + p.L.fwd), p.L.cap_fwd, &hdr->n_fwd, hist, base);
  } else if (blockIdx.x == 0) {
    write_qpad(p);
    emit_list(p, kListDkv, reinterpret_cast<WorkItem*>(p.ws + p.L.dkv), p.L.cap_dkv, &hdr->n_dkv, hist,
              base);
    if (tid == 0 && p.win.window > 0) hdr->n_fused = hdr->n_nsp = 0;  // no such lists
  } else if (blockIdx.x == 1) {
    emit_list(p, kListDq, reinterpret_cast<WorkItem*>(p.ws + p.L.dq), p.L.cap_dq, &hdr->n_dq, hist, base);
  } else if (blockIdx.x == 2) {
    emit_list(p, kListFused, reinterpret_cast<WorkItem*>(p.ws + p.L.fused), p.L.cap_fused, &hdr->n_fused, hist,
              base);
  } else {
    emit_list(p, kListNsp, reinterpret_cast<WorkItem*>(p.ws + p.L.nsp), p.L.cap_nsp, &hdr->n_nsp, hist, base);
  }
}

// Failure-detection self test: one thread waits on an mbarrier that nothing arrives on,
// through the same bounded wait the pipelines use; when the limit runs out it records
// JFA_ERR_TIMEOUT in the workspace status word and the kernel returns normally.
__global__ void wait_timeout_selftest_kernel(int* status, uint64_t timeout_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar, 1);
    fence_mbar_init();
    if (!mbar_wait(&bar, 0, &abort_flag, timeout_ns)) atomicCAS(status, 0, int(JFA_ERR_TIMEOUT));
  }
}

}  // namespace

cudaError_t launch_wait_timeout_selftest(void* ws, uint64_t timeout_ns, cudaStream_t stream) {
  wait_timeout_selftest_kernel<<<1, 32, 0, stream>>>(&reinterpret_cast<WsHeader*>(ws)->status, timeout_ns);
  return cudaGetLastError();
}

cudaError_t launch_plan(const Problem& pr, const PlanMaps& maps, void* ws, const WsLayout& L, bool backward,
                        int num_sms, cudaStream_t stream) {
  PlanParams p;
  p.q_off = pr.q_off;
  p.kv_off = pr.kv_off;
  p.B = pr.B;
  p.H = pr.H;
  p.total_q = pr.total_q;
  p.total_kv = pr.total_kv;
  p.causal = pr.causal;
  p.backward = backward ? 1 : 0;
  p.grid = pr.win.window > 0 && !backward ? kWinCtasPerSm * num_sms : num_sms;
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
  // one CTA per list; helpers for the maps (one warp each), tail copies and bias table
  const int sets = pr.win.window > 0 && pr.win.sinks > 0 ? 2 : 1;
  const long long map_ctas = (static_cast<long long>(pr.B) * kNumMapSlots * 2 * sets + 31) / 32;
  const int helpers = int(map_ctas < 8 ? 8 : map_ctas > 120 ? 120 : map_ctas);
  return launch_pdl(plan_kernel, dim3((!backward ? 1 : pr.win.window > 0 ? 2 : 4) + helpers), dim3(1024), 0, stream, maps, p);
}

}  // namespace jfa
