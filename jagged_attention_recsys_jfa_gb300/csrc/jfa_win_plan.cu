// The windowed call's planner: validates the jagged offsets, builds the tensor maps of every
// sequence's queries, window part and sinks, and writes the work lists.  As in the plain call's
// (jfa_plan.cu) a map's row extent is its sequence's, so that rows past it load as zeros, and the
// lists are sorted costliest first.  A kernel of its own: every launch-bound microsecond of a
// planner is on the caller's path, and the plain one lost 1.4 of 27.5 us to the window's branches.
#include "jfa_plan.cuh"

namespace jfa {
namespace {

// A sequence's window part and sinks; the forward's key tiles have kWinKeys rows.
__device__ __forceinline__ WinSeq plan_seq(const PlanParams& p, int Lq, int Lk) {
  return win_seq(Lq, Lk, p.win.window, p.win.sinks, p.backward ? kBN : kWinKeys);
}

// Units of a sequence: query tiles in the forward and dQ lists; in the dK/dV list the key tiles
// of the window part, then the chunks of the sinks.
__device__ __forceinline__ int win_units(const PlanParams& p, int kind, int Lq, int Lk) {
  if (kind != kListDkv) return (Lq + kBM - 1) / kBM;
  const WinSeq s = plan_seq(p, Lq, Lk);
  return (s.Lk + kBN - 1) / kBN + win_sink_chunks(Lq, s, p.H / p.win.H_kv);
}
// A unit's cost: the tiles that it meets.
__device__ __forceinline__ int win_unit_cost(const PlanParams& p, int kind, int u, int Lq, int Lk) {
  const WinSeq s = plan_seq(p, Lq, Lk);
  if (kind == kListDkv) {
    const WinKeyUnit k = win_key_unit(u, Lq, s, p.win.window, p.H / p.win.H_kv);
    return k.r1 - k.r0;
  }
  int a, e;
  win_kv_tiles(u, Lq, s, p.win.window, &a, &e, kind == kListFwd ? kWinKeys : kBN);
  return e - a + (win_sees_sinks(u, Lq, s) ? 1 : 0);
}

// The windowed lists.  A window bounds what a unit can cost, so every unit is an item of its own
// and the units, not the sequences, are dealt out to the threads: 1024 sequences at a time, a thread
// finds its unit's sequence in the running sums of their units.  Long sequences then cost no more
// time than short ones (long-tail batch of 64 sequences: 31 -> 10 us against a thread per sequence).
// Costliest first by a counting sort.  One entry stands
// for a unit of all `heads` heads: item i of the launch is entry i / heads, head i % heads, so that
// heads which share keys read them at the same time (and the list is written in a tenth of the time
// that one entry per head took).
__device__ void emit_window_list(const PlanParams& p, int kind, WorkItem* items, int64_t cap, int* count_out, int* hist,
                                 int* base) {
  __shared__ long long seq_end[1024];       // units up to the end of each of these sequences
  __shared__ int seq_q[1024], seq_k[1024];  // their lengths
  __shared__ long long units, cost_total;
  __shared__ int cost_max;
  const int tid = threadIdx.x;
  const int heads = kind == kListDkv ? p.win.H_kv : p.H;
  for (int c = tid; c < kCostBuckets; c += blockDim.x) hist[c] = 0;
  if (tid == 0) cost_max = 0;
  int loaded = -1;  // first of the sequences in shared memory
  // calls f(active, b, unit, cost) for this thread's units, all lanes of a warp together
  auto for_units = [&](auto&& f) {
    for (int b0 = 0; b0 < p.B; b0 += 1024) {
      if (loaded != b0) {
        const int b = b0 + tid;
        long long mine = 0;
        __syncthreads();  // the sequences before have been read
        if (b < p.B) {
          seq_q[tid] = int(p.q_off[b + 1] - p.q_off[b]);
          seq_k[tid] = int(p.kv_off[b + 1] - p.kv_off[b]);
          mine = win_units(p, kind, seq_q[tid], seq_k[tid]);
        }
        seq_end[tid] = block_scan_incl(mine, &units);
        __syncthreads();
        loaded = b0;
      }
      const long long n = units;
      for (long long i = tid; i - tid < n; i += blockDim.x) {
        int lo = 0, u = 0, cost = 0;
        if (i < n) {
          int hi = 1023;  // the first sequence that ends behind unit i
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (seq_end[mid] > i) hi = mid;
            else lo = mid + 1;
          }
          u = int(i - (lo ? seq_end[lo - 1] : 0));
          cost = win_unit_cost(p, kind, u, seq_q[lo], seq_k[lo]);
        }
        f(i < n, b0 + lo, u, cost);
      }
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
  if (total > cap) {  // cannot happen for valid offsets (capacities are upper bounds)
    if (tid == 0) {
      atomicCAS(&reinterpret_cast<WsHeader*>(p.ws)->status, 0, int(JFA_ERR_WORKSPACE));
      *count_out = 0;
    }
    return;
  }
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

// The first CTAs validate the offsets and write one work list each: the forward list, or the
// dK/dV list (with the padded query offsets) and the dQ list.  The other CTAs write the tail
// copies and the tensor maps in parallel.
__global__ void __launch_bounds__(1024, 1) win_plan_kernel(const __grid_constant__ WinPlanMaps maps, PlanParams p) {
  __shared__ int hist[kCostBuckets];
  __shared__ int base[kCostBuckets];
  const int tid = threadIdx.x;
  WsHeader* hdr = reinterpret_cast<WsHeader*>(p.ws);
  grid_dependency_wait();    // the offsets and the workspace may come from earlier work
  grid_launch_dependents();  // the next kernel may start its prologue; it waits for this one

  const int list_ctas = p.backward ? 2 : 1;
  if (int(blockIdx.x) >= list_ctas) {
    const size_t gt = size_t(blockIdx.x - list_ctas) * blockDim.x + tid;
    const size_t gstride = size_t(gridDim.x - list_ctas) * blockDim.x;
    // ---- the tensors' last rows, which maps that start close to their end load from (zone_bytes)
    const size_t stride = zone_stride(p.L.row_bytes);
    for (int slot = 0; slot < kNumMapSlots; ++slot) {
      if (!maps.used[slot]) continue;
      const int64_t total = (slot == kMapQ || slot == kMapDO) ? p.total_q : p.total_kv;
      if (total <= 0) continue;
      const size_t rb = maps.row_bytes[slot];
      const int64_t n = zone_rows(total, rb);
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(maps.base[slot]) +
                                                        size_t(total - n) * rb);
      uint4* dst = reinterpret_cast<uint4*>(p.ws + p.L.tail + size_t(slot) * stride);
      const size_t nvec = size_t(n) * rb / 16;
      for (size_t i = gt; i < nvec; i += gstride) dst[i] = src[i];
    }
    // ---- per-sequence tensor maps: copy the template, point it at the sequence's first row (of its
    //      window part, of its sinks) and clip its row extent.  (With invalid offsets CTA 0 leaves
    //      every list empty, so no map is used.)
    //      One warp per map: the replaces of a warp's lanes are done one after another, so lanes
    //      that each wrote a map would be what the planner waits for.
    const int sets = p.win.sinks > 0 ? 2 : 1;  // maps, and the sinks' maps
    const int lane = tid & 31;
    for (size_t job = gt / 32; job < size_t(p.B) * kNumMapSlots * sets; job += gstride / 32) {
      const bool sink = sets == 2 && (job & 1);
      const size_t idx = job / sets;
      const int b = int(idx / kNumMapSlots), slot = int(idx % kNumMapSlots);
      if (!maps.used[slot]) continue;
      const bool is_q_side = (slot == kMapQ || slot == kMapDO);
      int64_t row0 = is_q_side ? p.q_off[b] : p.kv_off[b];
      int64_t len = (is_q_side ? p.q_off[b + 1] : p.kv_off[b + 1]) - row0;
      if (is_q_side && sink) continue;
      if (!is_q_side) {  // the sinks, or the window part
        const int64_t lq = p.q_off[b + 1] - p.q_off[b];
        if (lq < 0 || len < 0 || lq > (int64_t(1) << 30) || len > (int64_t(1) << 30)) continue;
        const WinSeq ws = plan_seq(p, int(lq), int(len));
        if (!sink) row0 += ws.org + ws.skip;
        len = sink ? ws.ns : ws.Lk - ws.skip;
      }
      const size_t rb = maps.row_bytes[slot];
      const int64_t total = is_q_side ? p.total_q : p.total_kv;
      const void* base = static_cast<const uint8_t*>(maps.base[slot]) + row0 * int64_t(rb);
      if (in_zone(row0, total, rb))
        base = p.ws + p.L.tail + size_t(slot) * stride + (row0 - (total - zone_rows(total, rb))) * int64_t(rb);
      CUtensorMap* dst = reinterpret_cast<CUtensorMap*>(p.ws + (sink ? p.L.smaps : p.L.maps)) + idx;
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
  }
  if (tid == 0) {
    if (p.q_off[0] != 0 || p.kv_off[0] != 0 || p.q_off[p.B] != p.total_q || p.kv_off[p.B] != p.total_kv)
      bad = 1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    hdr->claim_fwd = hdr->claim_dq = hdr->claim_dkv = hdr->claim_fused = hdr->claim_nsp = 0;
    if (p.L.total > kArrivedAt) hdr->counters_used = 1;
  }
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
    emit_window_list(p, kListFwd, reinterpret_cast<WorkItem*>(p.ws + p.L.fwd), p.L.cap_fwd, &hdr->n_fwd, hist, base);
  } else if (blockIdx.x == 0) {
    write_qpad(p);
    emit_window_list(p, kListDkv, reinterpret_cast<WorkItem*>(p.ws + p.L.dkv), p.L.cap_dkv, &hdr->n_dkv, hist, base);
    if (tid == 0) hdr->n_fused = hdr->n_nsp = 0;  // no such lists
  } else {
    emit_window_list(p, kListDq, reinterpret_cast<WorkItem*>(p.ws + p.L.dq), p.L.cap_dq, &hdr->n_dq, hist, base);
  }
}

}  // namespace

cudaError_t launch_win_plan(const Problem& pr, const WinPlanMaps& maps, void* ws, const WsLayout& L, bool backward,
                            int num_sms, cudaStream_t stream) {
  const PlanParams p = plan_params(pr, ws, L, backward, backward ? num_sms : kWinCtasPerSm * num_sms);
  // one CTA per list; helpers for the maps (one warp each) and tail copies
  const int sets = pr.win.sinks > 0 ? 2 : 1;
  const long long map_ctas = (static_cast<long long>(pr.B) * kNumMapSlots * sets + 31) / 32;
  const int helpers = int(map_ctas < 8 ? 8 : map_ctas > 120 ? 120 : map_ctas);
  return launch_pdl(win_plan_kernel, dim3((backward ? 2 : 1) + helpers), dim3(1024), 0, stream, maps, p);
}

}  // namespace jfa
