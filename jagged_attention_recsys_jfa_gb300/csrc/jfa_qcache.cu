// The attention of one new token per sequence over the paged cache held in 8 bits.
//
// G = H / H_kv query heads per key/value head; with codes kc, vc and scales ks, vs,
//   s_j = scale ks_j (q . kc_j),  lse = ln sum_j exp s_j,  out = sum_j exp(s_j - lse) vs_j vc_j.
// Visible codes are read once per block of 8, 16 or 32 query heads.
//
// Measured (e4m3, d = 128 unless stated; GB/s of codes, scales and rows): 936 MB of 128 sequences, 4 heads to a
// key, 144 us, 6500 GB/s: memory; 451 MB of two sequences, 77 us, 5830: some 10 us are the way to the first tile and
// the join of 152 partials at the end; 210 MB with 32 heads to a key, 71 us: its warps' latency, 2100 clk for a
// tile of 128 keys with two warps to a scheduler; 95 MB in windows, 33 us: the first tile is there after 5 (a CTA's
// sum of the lengths, the page, the copy), a CTA's tiles take 20 in the median (4800 GB/s; the first CTA is done with
// them at 21, the last at 28), and its joins another 4.
//
// Codes are exact in f16, and so the products run in f16 with fp32 sums, m16n8k16, keys (or output columns)
// as the 16 rows and 8 query heads as the columns, so that a code is converted once for all heads of a block:
//   S^T = K Q^T   (q scaled by a power of two, its largest element in [2^14, 2^15): exact but below 2^-39 of it)
//   O^T += V^T P^T
// P = exp2(s - base), base being a maximum that is raised only where a score exceeds it by more than 8 (then O^T
// and the sums are rescaled): P <= 2^8.  P is rounded to f16 as an operand, at most 2^-11 relative a term.  A
// 16-key group has one value scale vs, which multiplies its P before that: P' = 2^7 P vs / r, r being the
// largest |vs| met so far (2^-126 at least).  P' keeps f16's 11 bits down to 2^-14, so terms lose relative precision only where
// P vs is below 2^-21 of the largest scale, and are then off by 2^-32 of that.
//
// Work is dealt as in the bf16 kernel (jfa_cache.cuh), in tiles of 128 keys, a unit counting kExtra tiles more for
// its query and its join.  Up to 16 heads, four warps take 32 keys of each tile, two CTAs to an SM; above, eight
// warps take 16 keys (at d = 64 of two tiles at a time), one CTA to an SM, with q in shared memory.  A unit whose tiles
// lie in several CTAs is joined from their partial rows, in a fixed order: by the CTA that finishes last, and where
// there are many, by the last of each 16 first.
#include "jfa_qcache.cuh"

namespace jfa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kQTile = 128;
constexpr int kQJoinPitch = 36;  // 32 output columns; 4 modulo 32, so that rows 2c are 8 banks apart
constexpr int kJoinGroup = 16;

struct QAttnParams : CacheWalkParams {
  const __nv_bfloat16* q;       // [B][H][d]
  const float *k_scale, *v_scale;
  __nv_bfloat16* out;           // [B][H][d]
  float* lse;                   // [H][B]
  int H, G;
  int lb, blocks_per_page;      // log2 of the tokens of a scale's block
  float scale_log2;
  int rows;                     // query heads of a block that are real at most
  int* counters_used;           // nonzero: `arrived` and `grouped` may not be at 0
  unsigned* arrived;            // [units] partials (or groups of them) written (left at 0)
  unsigned* grouped;            // [2 * grid] partials of a group written, at its first's place (left at 0)
  float* partial;               // [2 * grid][rows][d + 4]: out, maximum, sum, two of nothing
};

// NT: blocks of 8 query heads.
template <int D, int NT>
struct QCfg {
  static constexpr int kWarps = NT == 4 ? 8 : 4;
  // A warp takes kU 16-key groups at a time: of one tile, or, where eight warps share a tile, of two, one behind the
  // other, which have to lie in the ring with others on their way (d = 64, 105 MB, 32 heads to a key: 57 us instead of 61
  // with a group at a time; d = 128, where the ring holds five tiles: 86 instead of 84 on 210 MB of int8, 72 either way of e4m3).
  static constexpr bool kApart = NT == 4 && D == 64;
  static constexpr int kU = NT == 4 && !kApart ? 1 : 2;
  static constexpr bool kSplitRegs = NT == 4;          // registers moved from the producer's warps to the others
  static constexpr int kThreads = 32 * (kWarps + (kSplitRegs ? 4 : 2));
  static constexpr int kHeads = 8 * NT;
  static constexpr int kTileBytes = kQTile * D;
  static constexpr int kStageBytes = 2 * kTileBytes;   // K, V
  static constexpr int kCtasPerSm = NT == 4 ? 1 : 2;
  static constexpr int kStages = (D == 128 ? 1 : 2) * (NT == 4 ? 5 : 3);
  static constexpr int kExtra = NT == 4 ? 6 : NT == 2 ? 4 : 3;  // tiles that a unit counts besides its own
  static constexpr int kQBytes = NT == 4 ? D * kHeads * 2 : 0;
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024 + kWarps * kHeads * kQJoinPitch * 4 + kQBytes;
  static_assert(33 * kHeads * 8 <= kWarps * kHeads * kQJoinPitch * 4, "a join's weights in the place of its rows");
  static_assert(kCtasPerSm * (kSmemBytes + 4096) <= 233472, "shared memory per SM (dynamic, static and reserved)");
};
// Registers a thread where they are split: 384 x 168 at launch, of which the producer's four warps keep 56 and the
// other eight get 224 (40 and 232: the producer spills, 72.2 us for 71.6 on 210 MB).
constexpr uint32_t kQLaunchRegs = 168, kQProducerRegs = 56, kQOtherRegs = 224;
static_assert(128 * kQProducerRegs + 256 * kQOtherRegs <= 384 * kQLaunchRegs, "register split");

// A join runs once in a while, at the end where all else waits for it, and would find its instructions far away (in
// L2, or behind the codes that stream through it), which takes longer than its work: 11300 clk for 20 partials.  So
// each CTA with more than a few tiles rehearses one while it waits for its first tile, on whatever its own partial
// holds (451 MB of two sequences: 77 us with, 80 without).
//
// Rows of n <= 32 partials, joined in order, by the whole CTA but its producer, and handed to `take` as (row, column,
// four columns, maximum and sum).  `weights` (shared) has room for 33 x rows pairs.  Ends behind a barrier.
// kAhead partials' columns are loaded at a time, kItems each.
template <int D, int kThreads, int kAhead, int kItems, typename Slot, typename Take>
__device__ __forceinline__ void join_slots(float2* weights, int rows, int n, int tid, const Slot& slot, const Take& take) {
  constexpr int kPitch = D + 4;
  const int lane = tid & 31;
#pragma unroll 1
  for (int i = tid; i < n * rows; i += kThreads) {
    const int s = i / rows, r = i - s * rows;
    weights[i] = __ldcg(reinterpret_cast<const float2*>(slot(s) + r * kPitch + D));
  }
  named_bar_sync(1, kThreads);
#pragma unroll 1
  for (int r = tid >> 5; r < rows; r += kThreads / 32) {  // a warp for a row, a lane for a partial
    const float2 ml = lane < n ? weights[lane * rows + r] : make_float2(-INFINITY, 0.f);
    float m = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float w = ml.y * ex2_approx(ml.x - (m == -INFINITY ? 0.f : m));
    float l = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane < n) weights[lane * rows + r].x = l != 0.f ? w / l : 0.f;
    if (lane == 0) weights[32 * rows + r] = make_float2(m, l);
  }
  named_bar_sync(1, kThreads);
  const int items = rows * (D / 4);
#pragma unroll 1
  for (int i0 = tid; i0 < items; i0 += kItems * kThreads) {
    float4 x[kItems] = {};
#pragma unroll 1
    for (int s0 = 0; s0 < n; s0 += kAhead) {
      float4 v[kAhead][kItems];
#pragma unroll
      for (int s = 0; s < kAhead; ++s)
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          // several items: the last one again in the place of those beyond the end, which costs no registers (with branches
          // the kernel of 32 heads spills: 210 MB 102 us instead of 77); one: only the partials there are (451 MB 77 us, else 80)
          const int i = min(i0 + k * kThreads, items - 1), r = i / (D / 4), c = 4 * (i - r * (D / 4));
          if (kItems > 1 || s0 + s < n) v[s][k] = __ldcg(reinterpret_cast<const float4*>(slot(min(s0 + s, n - 1)) + r * kPitch + c));
        }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        if (s0 + s >= n) break;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
          const float w = weights[(s0 + s) * rows + min(i0 + k * kThreads, items - 1) / (D / 4)].x;
          x[k].x += w * v[s][k].x;
          x[k].y += w * v[s][k].y;
          x[k].z += w * v[s][k].z;
          x[k].w += w * v[s][k].w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int i = i0 + k * kThreads, r = i / (D / 4), c = 4 * (i - r * (D / 4));
      if (i < items) take(r, c, x[k], weights[32 * rows + r]);
    }
  }
  named_bar_sync(1, kThreads);
}

template <int D, bool kInt8, int NT>
__global__ void __launch_bounds__(QCfg<D, NT>::kThreads, QCfg<D, NT>::kCtasPerSm)
    qcache_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                            const QAttnParams p) {
  using C = QCfg<D, NT>;
  constexpr int U = C::kU, kExtra = C::kExtra;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* join = reinterpret_cast<float*>(ring + C::kStages * C::kStageBytes);  // [warp][kHeads][kQJoinPitch], or weights
  uint2* q_shared = reinterpret_cast<uint2*>(join + C::kWarps * C::kHeads * kQJoinPitch);  // NT = 4: [D / 16][2][lane][2]
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ float2 scales[C::kStages][kQTile / 16];  // of each 16-key group: K's, V's
  __shared__ long long run_end[C::kThreads];          // tiles of all units before the end of each thread's run of sequences
  __shared__ float unit_shared[C::kHeads];            // NT = 4: a product of codes and scaled q in log2 units
  __shared__ int abort_sh, refused, is_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    abort_sh = 0;
    tmap_prefetch(&k_map);
    tmap_prefetch(&v_map);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], C::kWarps);
    }
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  volatile int* abort_flag = &abort_sh;

  // (one thread reads the word: another CTA whose wait has run out may be writing it)
  if (tid == 0) refused = *static_cast<volatile const int*>(p.counters_used);
  sum_tiles<kQTile, C::kThreads, kExtra>(p, tid, run_end);
  if (refused) {  // uniform over the CTA, nothing in flight
    if (tid == 0) raise_status(p.status, JFA_ERR_WORKSPACE);
    return;
  }
  const int64_t total = run_end[C::kThreads - 1];

  // ---- sequences that show no key: out 0, lse -inf
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (checked_len(p, b) > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + int64_t(b) * p.H * D);
    for (int i = tid; i < p.H * D / 8; i += C::kThreads) o[i] = make_uint4(0, 0, 0, 0);
    for (int h = tid; h < p.H; h += C::kThreads) p.lse[int64_t(h) * p.B + b] = -INFINITY;
  }

  const int ctas = total < gridDim.x ? int(total) : int(gridDim.x);
  if (int(blockIdx.x) >= ctas) return;  // uniform over the CTA, nothing in flight
  const int64_t t0 = first_tile(total, blockIdx.x, ctas), t1 = first_tile(total, blockIdx.x + 1, ctas);
  Walk w = walk_from<kQTile, C::kThreads, kExtra>(p, t0, run_end, lane);
  // On to the next segment: tile t of unit w, or false.  (No keys belong to what a unit counts besides its tiles.)
  auto next_segment = [&](int64_t& t) {
    for (;; next_unit<kQTile, kExtra>(p, w)) {
      t = max(t, w.unit0 + kExtra);
      if (t >= t1) return false;
      if (t < w.unit0 + w.s.n) return true;
    }
  };
  // First key of the unit's tile number i, and the keys [lo, hi) that count there.
  auto keys_of = [&](int i, int& j0, int& lo, int& hi) {
    const bool sink = i < w.s.n_sink;
    j0 = (sink ? i : w.s.lo / kQTile + i - w.s.n_sink) * kQTile;
    lo = sink ? 0 : w.s.lo;
    hi = sink ? w.s.s_end : w.s.len;
  };

  if (warp >= C::kWarps) {
    // ------------------------------------------------------------ producers: a warp for K, one for V
    // (A warp issues its lanes' copies one behind the other: one warp for both took 49 us instead of 41 on 115 MB of
    // d = 64 in pages of 16.)
    // A batch is up to four tiles of one unit: lane x has 16-key group x % 8 of its tile x / 8, whose page and
    // scales are looked up ahead of its copies, the page while the batch in front is under way.  A copy is a box
    // of 16 or 32 rows of one page, by the lane of its first group; a tile's scales go to shared memory behind
    // its copies, and then it counts as arrived.
    if (C::kSplitRegs) setmaxnreg_dec<kQProducerRegs>();
    if (warp > C::kWarps + 1) return;
    const bool is_v = warp == C::kWarps + 1;
    const CUtensorMap* map = is_v ? &v_map : &k_map;
    const float* all_scales = is_v ? p.v_scale : p.k_scale;
    const int box = p.page_size < 32 ? 16 : 32, per_box = box / 16;
    struct Batch {
      int tiles, hk, page, row;  // row: the group's first in its page
      bool seen;                 // a key of the group is visible
      float scale;
    };
    auto look_up = [&](int64_t& t, Batch& n) {  // the batch that starts at tile t; t and w go on
      n.tiles = 0;
      n.seen = false;
      const int64_t unit0 = w.unit0;
      if (!next_segment(t)) return;
      if (w.unit0 != unit0 && !is_v) {  // a new unit: its query rows into L2
        const char* q = reinterpret_cast<const char*>(p.q + (int64_t(w.b) * p.H + w.hk * p.G + w.rb * C::kHeads) * D);
        const int bytes = min(C::kHeads, p.G - w.rb * C::kHeads) * D * 2;
        for (int at = lane * 128; at < bytes; at += 32 * 128) prefetch_l2(q + at);
      }
      n.tiles = int(min(min(t1, w.unit0 + w.s.n) - t, int64_t(4)));
      n.hk = w.hk;
      int j, lo, hi;
      keys_of(int(t - w.unit0) - kExtra + min(lane / 8, n.tiles - 1), j, lo, hi);
      j += lane % 8 * 16;
      n.row = j % p.page_size;
      n.seen = lane / 8 < n.tiles && j < hi && j + 16 > lo;
      if (n.seen) n.page = __ldg(p.page_table + int64_t(w.b) * p.max_pages + j / p.page_size);
      t += n.tiles;
    };
    auto is_page = [&](const Batch& n) { return n.seen && n.page >= 0 && n.page < p.num_pages; };
    auto load_scales = [&](Batch& n) {
      if (is_page(n)) {
        const int64_t at = (int64_t(n.page) * p.Hkv + n.hk) * p.blocks_per_page + (n.row >> p.lb);
        n.scale = all_scales[at];
      }
    };
    int64_t t = t0;
    uint32_t n = 0;
    bool ok = true;
    Batch cur = {}, next = {};
    look_up(t, cur);
    load_scales(cur);
    while (cur.tiles > 0 && ok) {
      const bool good = is_page(cur);
      if (cur.seen && !good) raise_status(p.status, JFA_ERR_BAD_PAGES);
      // a box is copied where a key of it is visible: its first group's lane does
      const unsigned have = __ballot_sync(0xffffffffu, good);
      const int leader = lane & ~(per_box - 1);
      const unsigned any = (have >> leader) & ((1u << per_box) - 1u);
      const int page = __shfl_sync(0xffffffffu, cur.page, any ? leader + __ffs(any) - 1 : lane);  // (one page a box)
      const bool copies = lane == leader && any;
      const unsigned loads = __ballot_sync(0xffffffffu, copies);
      const int line = int(((int64_t(page) * p.Hkv + cur.hk) * p.page_size + (cur.row & ~(box - 1))) * D / 128);
      for (int x = 0; x < cur.tiles; ++x, ++n) {
        const uint32_t e = n % C::kStages, ph = (n / C::kStages) & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[e], ph ^ 1, abort_flag, kWaitTimeoutNs));
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&full[e], uint32_t(__popc(loads & (0xffu << (x * 8)))) * box * D);
        __syncwarp();
        if (copies && lane / 8 == x)
          tma_load_2d(ring + e * C::kStageBytes + (is_v ? C::kTileBytes : 0) + (lane % 8) * 16 * D, map, &full[e], 0, line);
        if (lane / 8 == x) reinterpret_cast<float*>(&scales[e][lane % 8])[is_v] = cur.scale;
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[e]);
        if (x == 0) look_up(t, next);
      }
      if (ok) load_scales(next);
      cur = next;
    }
    if (!ok && lane == 0) {
      raise_status(p.status, JFA_ERR_TIMEOUT);
      *p.counters_used = 1;  // units that this CTA leaves undone keep their counts
    }
    // every copy this warp started has landed before the CTA can exit
    const uint32_t first = n > uint32_t(C::kStages) ? n - C::kStages : 0;
    for (uint32_t m = first; m < n; ++m) {
      const uint64_t start = globaltimer_ns();
      while (!mbar_try_wait(&full[m % C::kStages], (m / C::kStages) & 1))
        if (globaltimer_ns() - start > kWaitTimeoutNs) break;
    }
    return;
  }

  // ------------------------------------------------------------ the other warps
  if (C::kSplitRegs) setmaxnreg_inc<kQOtherRegs>();
  constexpr int kThreads = C::kWarps * 32;
  const int g = lane >> 2, c = lane & 3;  // S^T: keys g, g + 8 and heads 2c, 2c + 1; O^T: columns 2g, 2g + 1 of 16, same heads
  // rows of a 16-key group as ldmatrix reads them: this lane's row and 16-byte chunk, whose place in its 128-byte
  // line is exchanged by the line's number (128-byte swizzle); d = 64 has two rows to a line
  uint32_t lane_row[U], lane_sw[U];
  auto group_of = [&](int u) { return C::kApart ? warp : warp * U + u; };  // the place of a group in its tile
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = group_of(u) * 16 + (lane & 15);
    const int line = r * D / 128;
    lane_row[u] = line * 128;
    lane_sw[u] = ((lane >> 4) + (D == 64 ? (r & 1) * 4 : 0)) ^ (line & 7);
  }
  uint32_t e = 0, ph = 0;  // the ring's stage and its phase
  bool ok = true;
  bool rehearsal = NT == 1 && t1 - t0 > 8;
  // the join at a segment's end: partials of CTAs xa, xa + 1, ... ; the first CTA's is its later one
  int rows = 1, h0 = 0, xa = blockIdx.x, count = 1;
  bool later = false;
  float2* weights = reinterpret_cast<float2*>(join);
  constexpr int kPitch = D + 4;  // a partial row: out, then maximum and sum
  // (210 MB with 32 heads to a key: 72 us, 74 with four partials of one item at a time, 73 with a rehearsal)
  constexpr int kJoinAhead = NT == 1 ? 10 : 2, kJoinItems = NT == 1 ? 1 : 4;
  // where CTA x puts a unit's rows: the place of its first segment, or of a later one
  auto slot_of = [&](int64_t x, bool later_one) { return p.partial + (2 * x + later_one) * p.rows * kPitch; };
  for (int64_t t = t0; ok && (rehearsal || next_segment(t)); rehearsal = false) {
    if (!rehearsal) {
      const int64_t first = w.unit0 + kExtra, seg0 = t, end = min(t1, w.unit0 + w.s.n);
      h0 = w.hk * p.G + w.rb * C::kHeads;   // first query head of the block
      rows = min(C::kHeads, p.G - w.rb * C::kHeads);
      // ---- q as the second operand: head g of each 8, elements 16 j + 4 c + {0, 1} and {2, 3}
      uint2 qb[NT == 4 ? 1 : D / 16][NT == 4 ? 1 : NT];
      float unit_log2[NT][2];  // of heads 2c, 2c + 1: a product of codes and scaled q in log2 units
#pragma unroll
      for (int k = 0; k < (NT == 4 ? 1 : NT); ++k) {
        const int t8 = NT == 4 ? warp & 3 : k, hl = t8 * 8 + g;  // (NT = 4: two warps share a block's columns)
        const uint2* src = reinterpret_cast<const uint2*>(p.q + (int64_t(w.b) * p.H + h0 + hl) * D + 4 * c);
        uint2 x[D / 16];
        uint32_t m2 = 0;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          x[j] = hl < rows ? src[4 * j] : make_uint2(0, 0);
          m2 = __vmaxu2(m2, __vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu));
        }
        uint32_t m = max(m2 & 0xffffu, m2 >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t e = min(max(m >> 7, 15u), 254u);
        const float f = __uint_as_float((268u - e) << 23);  // 2^(141 - e); its inverse
        const float back = __uint_as_float((e - 14u) << 23) * p.scale_log2;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint2 b = make_uint2(pack_f16x2(bf16lo(x[j].x) * f, bf16hi(x[j].x) * f),
                                     pack_f16x2(bf16lo(x[j].y) * f, bf16hi(x[j].y) * f));
          if (NT != 4) {
            qb[j][k] = b;
          } else if ((j & 1) == warp >> 2) {
            q_shared[((j * 2 + t8 / 2) * 32 + lane) * 2 + t8 % 2] = b;
          }
        }
        if (NT != 4) {
          unit_log2[k][0] = __shfl_sync(0xffffffffu, back, 8 * c);
          unit_log2[k][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
        } else if (c == 0 && warp < 4) {
          unit_shared[hl] = back;
        }
      }
      if (NT == 4) {
        named_bar_sync(1, kThreads);
#pragma unroll
        for (int t8 = 0; t8 < NT; ++t8) {
          unit_log2[t8][0] = unit_shared[t8 * 8 + 2 * c];
          unit_log2[t8][1] = unit_shared[t8 * 8 + 2 * c + 1];
        }
      }
      auto q_of = [&](int j, uint2 (&b)[NT]) {
#pragma unroll
        for (int t8 = 0; t8 < NT; ++t8) {
          if (NT != 4) {
            b[t8] = qb[j][t8];
          } else if (t8 % 2 == 0) {
            const uint4 v = reinterpret_cast<const uint4*>(q_shared)[(j * 2 + t8 / 2) * 32 + lane];
            b[t8] = make_uint2(v.x, v.y);
            b[t8 + (NT == 4)] = make_uint2(v.z, v.w);
          }
        }
      };
      float o[D / 16][NT][4];  // columns 16 j + 2g (heads 2c, 2c + 1), 16 j + 2g + 1
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int t8 = 0; t8 < NT; ++t8) o[j][t8][0] = o[j][t8][1] = o[j][t8][2] = o[j][t8][3] = 0.f;
      float lower[NT][2], sum[NT][2];  // the base, less than zero by as much as it is above, in log2 units; sums of this lane's keys until the end
      unsigned started = 0;           // bit 2 t8 + k: base is a score's
#pragma unroll
      for (int t8 = 0; t8 < NT; ++t8) lower[t8][0] = lower[t8][1] = sum[t8][0] = sum[t8][1] = 0.f;
      float ref = 1.1754944e-38f, inv_ref = 8.5070592e37f;  // the largest |value scale| so far (2^-126 at least), its inverse

      // U groups of 16 keys, in the stages at[], of which keys [v_lo[], v_hi[]) are visible (edge: not all).  A group that
      // is not there, or shows no key, has another's place (of two apart).
      auto step = [&](bool edge, const uint32_t (&at)[U], const int (&v_lo)[U], const int (&v_hi)[U]) {
        uint32_t kb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) kb[u] = smem_u32(ring + at[u] * C::kStageBytes);
        auto visible = [&](int u, int key) { return key >= v_lo[u] && key < v_hi[u]; };
        auto none = [&](int u) { return v_lo[u] >= 16 || v_hi[u] <= 0; };
        float x[U][NT][4] = {};
#pragma unroll
        for (int j = 0; j < D / 16; j += 2)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            uint32_t r[4], a[4];
            ldmatrix_x4(r, kb[u] + lane_row[u] + ((j ^ lane_sw[u]) << 4));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              codes_f16<kInt8>(r[2 * k], a[0], a[2]);
              codes_f16<kInt8>(r[2 * k + 1], a[1], a[3]);
              uint2 b[NT];
              q_of(j + k, b);
#pragma unroll
              for (int t8 = 0; t8 < NT; ++t8) mma_f16_16816(x[u][t8], a, b[t8].x, b[t8].y);
            }
          }
        // ---- scores less their base; weights of the value scales relative to the largest met
        float rel[U], most = 0.f;
        float highest = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float2 sc = scales[at[u]][group_of(u)];
          rel[u] = sc.y;
#pragma unroll
          for (int t8 = 0; t8 < NT; ++t8) {
            const uint64_t f = f2_mul(f2_pack(unit_log2[t8][0], unit_log2[t8][1]), f2_pack(sc.x, sc.x));
            const uint64_t low = f2_pack(lower[t8][0], lower[t8][1]);
#pragma unroll
            for (int k = 0; k < 4; k += 2) f2_unpack(f2_fma(f2_pack(x[u][t8][k], x[u][t8][k + 1]), f, low), x[u][t8][k], x[u][t8][k + 1]);
          }
        }
        if (edge) {
          // Keys that are not visible have no score, and their value codes, which may be anything, are cleared: 0 * NaN
          // is NaN.  (Nothing was written for a group without a visible key.)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (none(u)) rel[u] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int t8 = 0; t8 < NT; ++t8)
                x[u][t8][k] = visible(u, g + 8 * (k >> 1)) ? x[u][t8][k] : -INFINITY;
          }
#pragma unroll
          for (int u = 0; u < (C::kApart ? U : 1); ++u) {  // (groups of one tile are rows one behind the other)
            if (C::kApart && none(u)) continue;
            const uint32_t rows_at = kb[u] + C::kTileBytes + group_of(u) * 16 * D;
#pragma unroll 1
            for (int i = lane; i < (C::kApart ? 1 : U) * D; i += 32) {  // (a row's 16-byte chunks change places within its line)
              const int line = i / 8, chunk = (i & 7) ^ (line & 7);
              if (!visible(u, D == 128 ? line : 2 * line + (chunk >> 2))) st_shared_zero16(rows_at + i * 16);
            }
          }
          __syncwarp();
          fence_proxy_async_smem();  // the ring's next copy into this place comes behind these stores
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          most = fmaxf(most, fabsf(rel[u]));
#pragma unroll
          for (int t8 = 0; t8 < NT; ++t8)
            highest = fmaxf(fmaxf(highest, fmaxf(x[u][t8][0], x[u][t8][1])), fmaxf(x[u][t8][2], x[u][t8][3]));
        }
        constexpr unsigned kAll = (1u << (2 * NT)) - 1u;
        if (__any_sync(0xffffffffu, highest > 8.f || started != kAll || most > ref)) {
          float grow = 1.f;
          if (most > ref) {
            grow = ref / most;
            ref = most;
            inv_ref = 1.f / most;
          }
#pragma unroll
          for (int t8 = 0; t8 < NT; ++t8) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float m = -INFINITY;
#pragma unroll
              for (int u = 0; u < U; ++u) m = fmaxf(m, fmaxf(x[u][t8][k], x[u][t8][k + 2]));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              const unsigned bit = 1u << (2 * t8 + k);
              if (started & bit) {
                m = fmaxf(m, 0.f);
              } else if (m == -INFINITY) {
                m = 0.f;
              } else {
                started |= bit;
              }
              const float lowered = lower[t8][k] - m;
              m = lower[t8][k] - lowered;  // as later scores will find it
              lower[t8][k] = lowered;
              f[k] = ex2_approx(-m);
              f[k] = f[k] == INFINITY ? 1.f : f[k];  // (what is not started holds zeros)
              sum[t8][k] *= f[k];
              f[k] *= grow;
#pragma unroll
              for (int u = 0; u < U; ++u) {
                x[u][t8][k] -= m;
                x[u][t8][k + 2] -= m;
              }
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[j][t8][0] *= f[0];
              o[j][t8][1] *= f[1];
              o[j][t8][2] *= f[0];
              o[j][t8][3] *= f[1];
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) rel[u] = rel[u] * inv_ref * 128.f;
        uint32_t pb[U][NT][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t8 = 0; t8 < NT; ++t8)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const uint64_t y = f2_pack(ex2_approx(x[u][t8][k]), ex2_approx(x[u][t8][k + 1]));
              f2_unpack(f2_add(f2_pack(sum[t8][0], sum[t8][1]), y), sum[t8][0], sum[t8][1]);
              f2_unpack(f2_mul(y, f2_pack(rel[u], rel[u])), x[u][t8][k], x[u][t8][k + 1]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t8 = 0; t8 < NT; ++t8) {
            pb[u][t8][0] = movmatrix_trans(pack_f16x2(x[u][t8][0], x[u][t8][1]));
            pb[u][t8][1] = movmatrix_trans(pack_f16x2(x[u][t8][2], x[u][t8][3]));
          }
#pragma unroll
        for (int j = 0; j < D / 16; j += 2)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            uint32_t r[4], a[4];  // (keys 2c, 2c + 1) x (columns 2g, 2g + 1): keys side by side after the exchange
            ldmatrix_x4_trans(r, kb[u] + C::kTileBytes + lane_row[u] + ((j ^ lane_sw[u]) << 4));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              codes_f16<kInt8>(__byte_perm(r[2 * k], 0, 0x3120), a[0], a[1]);
              codes_f16<kInt8>(__byte_perm(r[2 * k + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
              for (int t8 = 0; t8 < NT; ++t8) mma_f16_16816(o[j + k][t8], a, pb[u][t8][0], pb[u][t8][1]);
            }
          }
      };

      auto next_stage = [&](uint32_t& stage, uint32_t& phase) {
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      };
      const int tiles = int(end - first);
      for (int i = int(t - first); i < tiles;) {
        const bool two = C::kApart && i + 1 < tiles;
        uint32_t e1 = e, ph1 = ph;  // the stage of the second tile
        if (two) next_stage(e1, ph1);
        int j0, v_lo[U], v_hi[U];
        keys_of(i, j0, v_lo[0], v_hi[0]);
        v_lo[0] -= j0 + group_of(0) * 16;
        v_hi[0] -= j0 + group_of(0) * 16;
        if (two) {
          keys_of(i + 1, j0, v_lo[U - 1], v_hi[U - 1]);
          v_lo[U - 1] -= j0 + group_of(U - 1) * 16;
          v_hi[U - 1] -= j0 + group_of(U - 1) * 16;
        } else if (U == 2) {
          v_lo[U - 1] = C::kApart ? 0 : v_lo[0] - 16;
          v_hi[U - 1] = C::kApart ? 0 : v_hi[0] - 16;
        }
        bool seen[U], any = false, all = true;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          seen[u] = v_lo[u] < 16 && v_hi[u] > 0;
          any |= seen[u];
          all &= v_lo[u] <= 0 && v_hi[u] >= 16;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&full[e], ph, abort_flag, kWaitTimeoutNs));
        if (two && ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[e1], ph1, abort_flag, kWaitTimeoutNs));
        if (!ok) break;
        if (any) {
          uint32_t at[U];
#pragma unroll
          for (int u = 0; u < U; ++u) at[u] = C::kApart && seen[U - 1] && (u == 1 || !seen[0]) ? e1 : e;
          step(!all, at, v_lo, v_hi);
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&empty[e]);
          if (two) mbar_arrive(&empty[e1]);
        }
        e = e1;
        ph = ph1;
        next_stage(e, ph);
        i += two ? 2 : 1;
      }
      t = end;
      // ---- join the warps' rows through shared memory, 32 columns at a time.  The warps first agree on
      //      whether every wait came through: a warp that left alone would leave the others at a barrier.
      ok = named_bar_and(1, kThreads, ok);
      if (!ok) break;
      const bool whole = seg0 == first && end == w.unit0 + w.s.n;
      float* part_rows = slot_of(blockIdx.x, t0 < w.unit0);
      // each warp's maximum and sum of a row become its weight in the joined row
#pragma unroll
      for (int t8 = 0; t8 < NT; ++t8)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float l = sum[t8][k];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          sum[t8][k] = l;
          if (g == 0) weights[warp * C::kHeads + t8 * 8 + 2 * c + k] = make_float2(l == 0.f ? -INFINITY : -lower[t8][k], l);
        }
      named_bar_sync(1, kThreads);
      if (tid < rows) {
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < C::kWarps; ++k) m = fmaxf(m, weights[k * C::kHeads + tid].x);
        const float u = m == -INFINITY ? 0.f : m;
        float f[C::kWarps];
#pragma unroll
        for (int k = 0; k < C::kWarps; ++k) {
          f[k] = ex2_approx(weights[k * C::kHeads + tid].x - u);
          l += f[k] * weights[k * C::kHeads + tid].y;
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int k = 0; k < C::kWarps; ++k) weights[k * C::kHeads + tid].x = f[k] * inv;
        if (whole) {
          p.lse[int64_t(h0 + tid) * p.B + w.b] = l != 0.f ? (u + log2f(l)) * kLn2 : -INFINITY;
        } else {
          *reinterpret_cast<float2*>(part_rows + tid * kPitch + D) = make_float2(m, l);
        }
      }
      named_bar_sync(1, kThreads);
      // (O^T holds sums of up to 2^15 n codes, so that next to the smallest ref its factor is too small for a float: there
      // the factor is 2^60 times as large until it has been applied)
      const float up = ref < 8.6736174e-19f ? 1.1529215e18f : 1.f, down = ref < 8.6736174e-19f ? 8.6736174e-19f : 1.f;
      float out_f[NT][2];
#pragma unroll
      for (int t8 = 0; t8 < NT; ++t8)
#pragma unroll
        for (int k = 0; k < 2; ++k) out_f[t8][k] = weights[warp * C::kHeads + t8 * 8 + 2 * c + k].x * up * ref * (1.f / 128.f);
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        named_bar_sync(1, kThreads);  // the weights, or the previous columns, have been read
#pragma unroll
        for (int t8 = 0; t8 < NT; ++t8)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float* row = join + (warp * C::kHeads + t8 * 8 + 2 * c + k) * kQJoinPitch;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float* v = o[c0 / 16 + j][t8];
              *reinterpret_cast<float2*>(row + 16 * j + 2 * g) = make_float2(v[k] * out_f[t8][k] * down, v[2 + k] * out_f[t8][k] * down);
            }
          }
        named_bar_sync(1, kThreads);
#pragma unroll 1
        for (int i = tid; i < rows * 8; i += kThreads) {
          const int r = i >> 3, col = (i & 7) * 4;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < C::kWarps; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(join + (k * C::kHeads + r) * kQJoinPitch + col);
            x.x += v.x;
            x.y += v.y;
            x.z += v.z;
            x.w += v.w;
          }
          if (whole) {
            *reinterpret_cast<uint2*>(p.out + (int64_t(w.b) * p.H + h0 + r) * D + c0 + col) =
                make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
          } else {
            *reinterpret_cast<float4*>(part_rows + r * kPitch + c0 + col) = x;
          }
        }
      }
      if (whole) continue;
      // ---- the unit's last CTA to arrive joins the partial rows of all, in CTA order; of many, the last of each
      //      group joins the group's first (one CTA alone would read 304 partials of 16 rows: 2.5 MB)
      xa = cta_of(total, first, ctas);
      count = cta_of(total, w.unit0 + w.s.n - 1, ctas) - xa + 1;
      later = first_tile(total, xa, ctas) < w.unit0;  // of the first CTA; the others start in the unit
    }
    const int64_t unit = (int64_t(w.b) * p.Hkv + w.hk) * p.RB + w.rb;
    auto last_of = [&](unsigned* counter, unsigned count) {  // whether this CTA is the last of `count` to get here
      named_bar_sync(1, kThreads);
      if (tid == 0) {
        __threadfence();
        is_last = atomicAdd(counter, 1u) == count - 1;
        if (is_last) {
          __threadfence();
          *counter = 0;
        }
      }
      named_bar_sync(1, kThreads);
      return is_last != 0;
    };
    const int stride = count > 2 * kJoinGroup ? kJoinGroup : 1;
    // a group's members (first round, where there are groups) or their firsts
    bool in_group = stride > 1;
#pragma unroll 1
    for (;; in_group = false) {
      const int from = in_group ? xa + (int(blockIdx.x) - xa) / stride * stride : xa;
      const int members = in_group ? min(stride, xa + count - from) : (count + stride - 1) / stride, step = in_group ? 1 : stride;
      const bool from_later = from == xa && later;
      if (!rehearsal && !last_of(in_group ? p.grouped + 2 * int64_t(from) + from_later : p.arrived + unit, members)) break;
      float* into = slot_of(from, from_later);
      join_slots<D, kThreads, kJoinAhead, kJoinItems>(
          weights, rows, members, tid, [&](int s) { return slot_of(from + s * step, s == 0 && from_later); },
          [&](int r, int col, const float4& x, const float2& ml) {
            if (rehearsal) return;
            if (in_group) {  // (each thread overwrites what it alone has read; the maxima and sums have been)
              *reinterpret_cast<float4*>(into + r * kPitch + col) = x;
              if (col == 0) *reinterpret_cast<float2*>(into + r * kPitch + D) = ml;
            } else {
              *reinterpret_cast<uint2*>(p.out + (int64_t(w.b) * p.H + h0 + r) * D + col) =
                  make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
              if (col == 0)
                p.lse[int64_t(h0 + r) * p.B + w.b] =
                    ml.y != 0.f ? ((ml.x == -INFINITY ? 0.f : ml.x) + log2f(ml.y)) * kLn2 : -INFINITY;
            }
          });
      if (!in_group) break;
    }
  }
  if (!ok && lane == 0) {
    raise_status(p.status, JFA_ERR_TIMEOUT);
    *p.counters_used = 1;  // units that this CTA leaves undone keep their counts
  }
}

template <int D, bool kInt8, int NT>
cudaError_t launch_qattn_t(const CUtensorMap& km, const CUtensorMap& vm, const QAttnParams& p, int num_sms,
                           cudaStream_t stream) {
  using C = QCfg<D, NT>;
  auto kern = qcache_attention_kernel<D, kInt8, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e == cudaSuccess && C::kSplitRegs) e = check_launch_registers_of<qcache_attention_kernel<D, kInt8, NT>>(kQLaunchRegs);
  if (e != cudaSuccess) return e;
  constexpr int kMost = kMaxAttnCtas * 16 / (C::kHeads > 16 ? C::kHeads : 16);  // the partial rows' room
  int grid = C::kCtasPerSm * num_sms;
  if (grid > kMost) grid = kMost;
  return launch_pdl(kern, dim3(grid), dim3(C::kThreads), C::kSmemBytes, stream, km, vm, p);
}

template <int D, bool kInt8>
cudaError_t launch_qattn(const CUtensorMap& km, const CUtensorMap& vm, QAttnParams& p, int num_sms, cudaStream_t stream) {
  const int block = p.G <= 8 ? 8 : p.G <= 16 ? 16 : 32;  // query heads that share a key's reading
  p.RB = (p.G + block - 1) / block;
  p.rows = p.G < block ? p.G : block;
  if (block == 8) return launch_qattn_t<D, kInt8, 1>(km, vm, p, num_sms, stream);
  if (block == 16) return launch_qattn_t<D, kInt8, 2>(km, vm, p, num_sms, stream);
  return launch_qattn_t<D, kInt8, 4>(km, vm, p, num_sms, stream);
}

}  // namespace

cudaError_t launch_qcache_attention(const jfa_qcache& qc, const CUtensorMap& km, const CUtensorMap& vm, const void* q, int H,
                                    int window, int sinks, float scale, void* out, float* lse, void* ws, int num_sms,
                                    cudaStream_t stream) {
  const jfa_cache& c = qc.cache;
  uint8_t* w = static_cast<uint8_t*>(ws);
  QAttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.page_table = c.page_table;
  p.lengths = c.lengths;
  p.k_scale = qc.k_scale;
  p.v_scale = qc.v_scale;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.num_pages = c.num_pages;
  p.B = c.B;
  p.H = H;
  p.Hkv = c.H_kv;
  p.G = H / c.H_kv;
  p.page_size = c.page_size;
  p.max_pages = c.max_pages;
  p.lb = log2_of(qc.block);
  p.blocks_per_page = c.page_size / qc.block;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = scale * kLog2e;
  p.status = &reinterpret_cast<WsHeader*>(w)->status;
  p.counters_used = &reinterpret_cast<WsHeader*>(w)->counters_used;
  p.arrived = reinterpret_cast<unsigned*>(w + kArrivedAt);
  p.grouped = reinterpret_cast<unsigned*>(w + kGroupAt);
  p.partial = reinterpret_cast<float*>(w + kPartialAt);
  const bool int8 = qc.kind == JFA_CODES_INT8;
  if (c.d == 128) return int8 ? launch_qattn<128, true>(km, vm, p, num_sms, stream) : launch_qattn<128, false>(km, vm, p, num_sms, stream);
  return int8 ? launch_qattn<64, true>(km, vm, p, num_sms, stream) : launch_qattn<64, false>(km, vm, p, num_sms, stream);
}

// The whole cache as lines of 128 bytes (two rows of d = 64): boxes of 16 or 32 rows of one page.
int qcache_box_rows(int page_size) { return page_size < 32 ? 16 : 32; }

}  // namespace jfa
