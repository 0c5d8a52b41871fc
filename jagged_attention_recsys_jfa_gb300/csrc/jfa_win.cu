// Windowed jagged attention forward for sm_103a: causal, a sliding window plus a sequence's
// first keys (sinks), query heads sharing key/value heads (include/jfa.h).
//
//   out_i = sum_j exp(s_ij - lse_i) v_j  over the keys j that query i sees, s = scale q.k
//
// A query tile of 128 rows meets only (window + 127) keys, so an item is a few short steps and
// what counts is how quickly tiles follow one another, not the steady state of a long key loop.
// Hence two CTAs per SM, each working on one query tile at a time with half of the SM's shared
// memory and tensor memory: while one CTA waits (for its next query tile, for a product, for its
// rows to be written) the other one computes.
//
// A step takes 64 keys: first the sinks', then those of the window part (win_seq), in steps that
// follow the window's two edges closer than 128 would (a window of 255: 5.9 steps of 64 per
// query tile against 3.3 of 128).  Masks are applied only in steps that the edge of some row's
// window crosses, and a warp whose 32 rows see none of a step's keys skips its arithmetic.
//
//   warp 0     K/V producer (TMA into two rings of 64-key tiles)
//   warp 1     issues the products PV(j)
//   warp 2     loads the query tile and issues the scores S(j), up to kBufs steps ahead
//   warp 3     scheduler (claims items, publishes their metadata)
//   warps 4-7  softmax: one TMEM lane = one query row per thread
// TMEM (256 of the 512 columns): O [0, d), then kBufs score buffers of 64 columns (P, bf16,
// overwrites the first 32 of its buffer).  With the next steps' scores computed ahead, the chain
// of a step is its softmax alone; the products' latency (about 1300 cycles per step otherwise) is
// off it.  Scores and products have an issuing warp each: a short step's MMAs take less time than
// the waits and commits around them take one warp: one issuer for both took 120 us where two and
// metadata worked out by the scheduler take 115 (128 sequences of 1 to 2048 tokens, d = 64, 4 query
// and 2 key/value heads, window 255, 4 sinks), and 172 where they take 159 (64 long-tailed sequences
// of up to 16384 tokens, d = 128, 8 heads, window 1024, 4 sinks).  With the window's grid aligned
// (win_seq) and a sequence's partial tiles through its own maps the two take 103 and 153 (floors 30
// and 64): neither memory (16% and 46%) nor the tensor pipe (17% and 41%) sets the pace, but the
// steps' hand-offs.  By timing copies that leave work out, the softmax arithmetic is about 35 us of
// the first, half of the score products 5.
//
// P is rounded to bf16 for its product (at most 2^-8 relative a term); scores, maximum, sum and O are fp32.
#include "jfa_win.cuh"

namespace jfa {
namespace {

// The reference maximum is raised, and O rescaled, only when a row outgrows it by this much (log2
// units): until then P is at most 2^16, which bf16 and the fp32 sums hold with the same relative
// precision.  A rescale stalls its CTA for about 2000 cycles; at 2^8 a tile whose first step is a
// few sinks met one now and then.
constexpr float kRescaleThreshold = 16.0f;

struct WinFwdParams {
  const int64_t* q_off;
  const int64_t* kv_off;
  int H, group;  // group: query heads per key/value head
  int64_t total_q;
  float scale_log2;  // scale * log2(e), > 0
  WindowSpec win;
  bool whole;                // the tensors' own maps serve whole tiles (row numbers fit 31 bits)
  const CUtensorMap* maps;   // [B][kNumMapSlots]: Q, and K / V of the window part
  const CUtensorMap* smaps;  // K / V of the sinks
  int sink_box;              // rows of their boxes (16 .. 64)
  const WorkItem* items;
  const int* n_items;
  int* claim;
  int* status;
  const uint64_t* wait_ns;
  __nv_bfloat16* out;
  float* lse;
  bool wide_out;  // out is 32-byte aligned
  TraceBuf trace;
};

template <int D>
struct WinCfg {
  static constexpr int kQBytes = kBM * D * 2;
  static constexpr int kTileBytes = kWinKeys * D * 2;
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kWinKeys * 128;  // one 64-column box of a K or V tile
  static constexpr int kStages = D == 128 ? 2 : 4;  // tiles of the K ring, and of the V ring
  static constexpr int kBufs = D == 128 ? 2 : 3;    // score buffers
  static constexpr int kSmemBytes = kQBytes + 2 * kStages * kTileBytes + 1024;
  static constexpr uint32_t kColO = 0, kColS = D;
  static_assert(kColS + kBufs * kWinKeys <= kWinTmemCols, "TMEM columns");
  // v_empty of step j is what S(j + kBufs) waits for: it must not have gone round again by then
  static_assert(kStages >= kBufs, "V ring");
  static_assert(2 * (kSmemBytes + 2048) <= 233472, "two CTAs per SM");
};

template <int D>
__global__ void __launch_bounds__(kWinThreads, 2)
    win_fwd_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const __grid_constant__ WinFwdParams p) {
  using C = WinCfg<D>;
  constexpr int R = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kQBytes;
  uint8_t* sV = sK + R * C::kTileBytes;

  __shared__ uint64_t q_full, q_empty, o_full, pv_done, s_done;
  __shared__ uint64_t k_full[R], k_empty[R], v_full[R], v_empty[R], s_full[C::kBufs], p_full[C::kBufs];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ TileRing tiles;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&o_full, 1);
    mbar_init(&pv_done, 1);
    mbar_init(&s_done, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 32 * kSoftmaxWarps);
    }
    for (int i = 0; i < kMetaSlots; ++i) {
      mbar_init(&tiles.full[i], 1);
      mbar_init(&tiles.empty[i], kWinConsumers);
    }
    tiles.wait_ns = p.wait_ns;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, kWinTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();  // the planner's lists and maps, the previous kernels' outputs
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_flag = &abort_sh;

  if (warp < kFirstComputeWarp) {
   if (warp == 0) {
    // ------------------------------------------------------------ K/V producer
    if (lane == 0) {
      Ring<R> kr, vr;
      uint32_t n_k = 0, n_v = 0, tn = 0;  // tiles loaded
      bool ok = true;
      if (p.whole) {
        tmap_prefetch(&k_map);
        tmap_prefetch(&v_map);
      }
      const CUtensorMap* const whole_k = p.whole ? &k_map : nullptr;
      const CUtensorMap* const whole_v = p.whole ? &v_map : nullptr;
      for (uint32_t k = 0; ok; ++k) {
        if (!tile_wait(tiles, k, abort_flag)) { ok = false; break; }
        const WinTile& w = tiles.e[k % kMetaSlots];
        if (w.b < 0) break;  // end of this CTA's items
        const int col = w.h / p.group * D;  // first column of the key/value head
        auto fill = [&](int slot, int j, Ring<R>& r, uint64_t* full, uint64_t* empty, uint8_t* smem_tiles) {
          const bool sink = j < w.nz;
          const TileMap m =
              sink ? win_tile_map(nullptr, p.smaps, slot, w.b, 0, j, 0, kWinKeys, 0)
                   : win_tile_map(slot == kMapK ? whole_k : whole_v, p.maps, slot, w.b, w.ko, w.a + j - w.nz, w.Lk,
                                  kWinKeys, w.skip);
          if (m.tail) tmap_acquire(m.map);
          if (!mbar_wait(&empty[r.e], r.ph ^ 1, abort_flag, kWaitTimeoutNs)) return false;
          trace_event(p.trace, kTraceProducer, tn, slot);
          mbar_arrive_expect_tx(&full[r.e], uint32_t(sink ? p.sink_box : kWinKeys) * D * 2);
#pragma unroll
          for (int c = 0; c < C::kBoxes; ++c)
            tma_load_2d(smem_tiles + r.e * C::kTileBytes + c * C::kBoxBytes, m.map, &full[r.e], col + c * 64, m.y);
          r.next();
          return true;
        };
        auto fill_k = [&](int j) { return ++n_k, fill(kMapK, j, kr, k_full, k_empty, sK); };
        auto fill_v = [&](int j) { return ++n_v, fill(kMapV, j, vr, v_full, v_empty, sV); };
        for (int j = 0; j < min(C::kBufs, w.n) && ok; ++j) ok = fill_k(j);
        for (int j = 0; j < w.n && ok; ++j) {
          ok = fill_v(j);
          if (ok && j + C::kBufs < w.n) ok = fill_k(j + C::kBufs);
        }
        if (ok) mbar_arrive(&tiles.empty[k % kMetaSlots]);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      // every copy this thread started has landed before the CTA can exit
      for (uint32_t n = n_k > R ? n_k - R : 0; n < n_k; ++n) drain_wait(&k_full[n % R], (n / R) & 1);
      for (uint32_t n = n_v > R ? n_v - R : 0; n < n_v; ++n) drain_wait(&v_full[n % R], (n / R) & 1);
    }
   } else if (warp == 1) {
    // ------------------------------------------------------------ products P V
    // the whole warp walks the schedule; one elected lane issues the tcgen05 instructions
    constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, false, true);
    const uint64_t vd0 = sdesc_sw128(smem_u32(sV), C::kBoxBytes, 1024);
    uint32_t tn = 0;
    Ring<R> vr;
    Ring<C::kBufs> pr;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!tile_wait_warp(tiles, k, abort_flag)) { ok = false; break; }
      const int n = tiles.e[k % kMetaSlots].n, nz = tiles.e[k % kMetaSlots].nz;
      const bool end = tiles.e[k % kMetaSlots].b < 0;
      tile_release_warp(tiles, k);  // all it needs is in registers
      if (end) break;
      for (int j = 0; j < n; ++j) {
        if (!warp_wait(&v_full[vr.e], vr.ph, abort_flag) || !warp_wait(&p_full[pr.e], pr.ph, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) trace_event(p.trace, kTraceMma, tn, 12);
        const uint64_t vd = vd0 + vr.e * uint32_t(C::kTileBytes >> 4);
        const uint32_t col = tmem + C::kColS + pr.e * kWinKeys;
        const int kks = j < nz ? p.sink_box / 16 : kWinKeys / 16;  // 16 keys per product
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kWinKeys / 16; ++kk)
            if (kk < kks)
              umma_ts(tmem + C::kColO, col + kk * 8, vd + uint32_t(kk * 2048 >> 4), kIdPV, j > 0 || kk > 0);
          umma_commit(&v_empty[vr.e]);
          if (j + 1 == n) umma_commit(&o_full);
        }
        vr.next();
        pr.next();
        if (lane == 0) trace_event(p.trace, kTraceMma, tn, 14);
      }
    }
    if (!ok && lane == 0) raise_status(p.status, JFA_ERR_TIMEOUT);
    if (elect_one()) umma_commit(&pv_done);
    drain_wait(&pv_done, 0);
   } else if (warp == 2) {
    // ------------------------------------------------------------ query tile, scores Q K^T
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kWinKeys, false, false);
    const uint32_t id_sink = idesc_bf16_f32(128, p.sink_box, false, false);
    const uint64_t qd = sdesc_sw128(smem_u32(sQ), 16, 1024), kd0 = sdesc_sw128(smem_u32(sK), 16, 1024);
    uint32_t n_q = 0, g = 0, tn = 0;  // query tiles loaded, scores issued
    Ring<R> kr, vr;                   // vr: V tile of the step whose buffer is taken over
    Ring<C::kBufs> sr;
    bool ok = true;
    if (lane == 0 && p.whole) tmap_prefetch(&q_map);
    for (uint32_t k = 0; ok; ++k) {
      if (!tile_wait_warp(tiles, k, abort_flag)) { ok = false; break; }
      const WinTile& w = tiles.e[k % kMetaSlots];
      if (w.b < 0) break;
      const int n = w.n, nz = w.nz;
      if (n == 0) {
        tile_release_warp(tiles, k);
        continue;
      }
      // the last scores of the previous tile have read the buffer
      if (!warp_wait(&q_empty, (n_q & 1) ^ 1, abort_flag)) { ok = false; break; }
      if (lane == 0) {
        const TileMap m = win_tile_map(p.whole ? &q_map : nullptr, p.maps, kMapQ, w.b, w.qo, w.t, w.Lq, kBM, 0);
        if (m.tail) tmap_acquire(m.map);
        trace_event(p.trace, kTraceLoader, tn, 1);
        mbar_arrive_expect_tx(&q_full, C::kQBytes);
#pragma unroll
        for (int c = 0; c < C::kBoxes; ++c) tma_load_2d(sQ + c * 16384, m.map, &q_full, w.h * D + c * 64, m.y);
        // pull the CTA's next query tile into L2 meanwhile, if the scheduler has it already
        const uint32_t kn = k + 1;
        if (p.whole && mbar_test_wait(&tiles.full[kn % kMetaSlots], (kn / kMetaSlots) & 1)) {
          const WinTile& x = tiles.e[kn % kMetaSlots];
          if (x.b >= 0 && x.rows == kBM)
            for (int c = 0; c < C::kBoxes; ++c) tma_prefetch_2d(&q_map, x.h * D + c * 64, int(x.qo) + x.t * kBM);
        }
      }
      tile_release_warp(tiles, k);
      ++n_q;
      if (!warp_wait(&q_full, (n_q - 1) & 1, abort_flag)) { ok = false; break; }
      for (int j = 0; j < n; ++j, ++g) {
        if (!warp_wait(&k_full[kr.e], kr.ph, abort_flag)) { ok = false; break; }
        if (g >= C::kBufs) {  // the buffer's last product has read its P
          if (!warp_wait(&v_empty[vr.e], vr.ph, abort_flag)) { ok = false; break; }
          vr.next();
        }
        tc_fence_after();
        const uint64_t kd = kd0 + kr.e * uint32_t(C::kTileBytes >> 4);
        const uint32_t id = j < nz ? id_sink : kIdS, col = tmem + C::kColS + sr.e * kWinKeys;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_ss(col, qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                    kd + (((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4), id, kk > 0);
          umma_commit(&s_full[sr.e]);
          umma_commit(&k_empty[kr.e]);
          if (j + 1 == n) umma_commit(&q_empty);
        }
        sr.next();
        kr.next();
        if (lane == 0) trace_event(p.trace, kTraceLoader, tn, 16);
      }
    }
    if (!ok && lane == 0) raise_status(p.status, JFA_ERR_TIMEOUT);
    // the query copy and the scores have landed before the CTA can exit
    if (n_q > 0) drain_wait(&q_full, (n_q - 1) & 1);
    if (elect_one()) umma_commit(&s_done);
    drain_wait(&s_done, 0);
   } else {
    // ------------------------------------------------------------ scheduler
    if (lane == 0 && !publish_tiles<kWinKeys>(tiles, p, nullptr, abort_flag))
      raise_status(p.status, JFA_ERR_TIMEOUT);
   }
  } else {
    // ------------------------------------------------------------ softmax warps
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_addr + C::kColO;
    const float sl2 = p.scale_log2;
    uint32_t v_n = 0, o_n = 0, tn = 0;  // v_n: steps before this tile
    Ring<C::kBufs> sr;                  // score buffer of the next step
    const bool leader = quarter == 0 && lane == 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!tile_wait_warp(tiles, k, abort_flag)) { ok = false; break; }
      const WinTile& w = tiles.e[k % kMetaSlots];
      if (w.b < 0) break;
      const int n = w.n, nz = w.nz, ns = w.ns, rows = w.rows;
      const int r0 = quarter * 32, i = r0 + lane;  // the warp's first row, this thread's
      const bool valid = i < rows;
      const int64_t q_row = w.qo + w.t * kBM + i;
      __nv_bfloat16* orow = p.out + (q_row * p.H + w.h) * int64_t(D);
      float* lrow = p.lse + int64_t(w.h) * p.total_q + q_row;
      int hi0 = r0 + w.pos + w.org, last = ns - 1, lo0 = -(1 << 30), pad = 0;     // first step of sinks
      const int hi_win = r0 + w.pos - w.a * kWinKeys, pad_win = w.pad - w.a * kWinKeys;  // first tile of the window part
      tile_release_warp(tiles, k);  // the rest is in registers
      if (n == 0) {
        if (valid) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0, 0, 0, 0);
          *lrow = -INFINITY;
        }
        continue;
      }
      // Row i sees columns [clo, chi] of a step.  The warp's rows see a band: rows r0 and r0 + 31
      // up to hi0 and hi0 + 31 (the sinks' step: `last` at most), row r0 from lo0 and row r0 + 31
      // from lo0 + 31 on.
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        if (j == nz) {  // first key tile of the window part
          hi0 = hi_win;
          last = 1 << 30;
          lo0 = hi0 - p.win.window + 1;
          pad = pad_win;  // columns before it hold no key
        }
        const bool hidden = min(last, hi0 + 31) < 0 || lo0 >= kWinKeys || r0 >= rows;      // from all 32 rows
        const bool whole = min(last, hi0) >= kWinKeys - 1 && lo0 <= -31 && pad <= 0;  // seen by all 32
        const uint32_t tS = tmem + lane_addr + C::kColS + sr.e * kWinKeys;
        if (!warp_wait(&s_full[sr.e], sr.ph, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (leader) trace_event(p.trace, kTraceCompute0, tn, 20);
        uint32_t pk[32];
        if (!hidden) {
          float x[64];
          {
            uint32_t r[2][32];
            tmem_ld32(tS, r[0]);
            tmem_ld32(tS + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = __uint_as_float(r[c >> 5][c & 31]);
          }
          if (!whole) {
            const int chi = min(last, hi0 + lane), clo = max(lo0 + lane, pad);
            const uint32_t bits[2] = {low_bits(chi + 1) & ~low_bits(clo), low_bits(chi - 31) & ~low_bits(clo - 32)};
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(bits[c >> 5] & (1u << (c & 31)))) x[c] = -INFINITY;
          }
          float mx4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float m0 = fmaxf(x[16 * q], x[16 * q + 1]);
#pragma unroll
            for (int c = 2; c < 16; c += 2) m0 = fmax3(m0, x[16 * q + c], x[16 * q + c + 1]);
            mx4[q] = m0;
          }
          const float m_tile = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
          const bool need = m_tile > m + kRescaleThreshold;
          const float m_new = need ? m_tile : m;
          const float alpha = need ? ex2_approx(m - m_new) : 1.f;  // m = -inf gives 0
          const bool rescale = __any_sync(0xffffffffu, need && m != -INFINITY);
          l *= alpha;
          m = m_new;
          const float m_use = m == -INFINITY ? 0.f : m;
          const uint64_t k_scale = f2_pack(sl2, sl2), k_negm = f2_pack(-m_use, -m_use);
          uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c2 = 0; c2 < 32; ++c2) {
            float e0, e1;
            f2_unpack(f2_fma(f2_pack(x[2 * c2], x[2 * c2 + 1]), k_scale, k_negm), e0, e1);
            e0 = ex2_approx(e0);
            e1 = ex2_approx(e1);
            sum2[c2 & 3] = f2_add(sum2[c2 & 3], f2_pack(e0, e1));
            pk[c2] = pack_bf16x2(e0, e1);
          }
          tmem_st32(tS, pk);
          float s0, s1;
          f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), s0, s1);
          l += s0 + s1;
          if (rescale) {
            // O holds earlier steps; the last of their products frees its V tile when done
            const uint32_t n = v_n + j - 1;
            if (!warp_wait(&v_empty[n % R], (n / R) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t r[32];
              tmem_ld32(tO + cc * 32, r);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * alpha);
              tmem_st32(tO + cc * 32, r);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = 0u;
          tmem_st32(tS, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[sr.e]);
        if (leader) trace_event(p.trace, kTraceCompute0, tn, 21);
        sr.next();
        hi0 -= kWinKeys;
        lo0 -= kWinKeys;
        pad -= kWinKeys;
        last -= kWinKeys;
      }
      if (!ok) break;
      v_n += n;
      // ---- epilogue: O / l -> bf16, lse = ln(sum) = (m + log2 l) * ln 2; a NaN among the row's scores is
      // in l and stays in both (only a sum of 0 is a row without keys)
      const bool live = l != 0.f;
      const float inv_l = live ? 1.f / l : 0.f;
      if (valid) *lrow = live ? ((m == -INFINITY ? 0.f : m) + __log2f(l)) * kLn2 : -INFINITY;
      if (!warp_wait(&o_full, o_n & 1, abort_flag)) { ok = false; break; }
      ++o_n;
      tc_fence_after();
      if (leader) trace_event(p.trace, kTraceCompute0, tn, 22);
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 64) {
        uint32_t r[2][32];
        tmem_ld32(tO + c0, r[0]);
        tmem_ld32(tO + c0 + 32, r[1]);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w8[e] = pack_bf16x2(__uint_as_float(r[q >> 1][(q & 1) * 16 + 2 * e]) * inv_l,
                                __uint_as_float(r[q >> 1][(q & 1) * 16 + 2 * e + 1]) * inv_l);
          if (!valid) continue;
          if (p.wide_out) {
            st_global_v8(orow + c0 + q * 16, w8[0], w8[1], w8[2], w8[3], w8[4], w8[5], w8[6], w8[7]);
          } else {
            uint4* o = reinterpret_cast<uint4*>(orow + c0 + q * 16);
            o[0] = make_uint4(w8[0], w8[1], w8[2], w8[3]);
            o[1] = make_uint4(w8[4], w8[5], w8[6], w8[7]);
          }
        }
      }
      tc_fence_before();
      if (leader) trace_event(p.trace, kTraceCompute0, tn, 23);
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kWinTmemCols);
}

template <int D>
cudaError_t launch_win_fwd_t(const PlanMaps& maps, const WinFwdParams& fp, int grid, cudaStream_t stream) {
  auto kern = win_fwd_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, WinCfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kWinThreads), WinCfg<D>::kSmemBytes, stream, maps.tmpl[kMapQ], maps.tmpl[kMapK],
                    maps.tmpl[kMapV], fp);
}

}  // namespace

cudaError_t launch_win_forward(const Problem& pr, const PlanMaps& maps, void* ws, const WsLayout& L, void* out,
                               float* lse, int num_sms, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  WinFwdParams fp;
  fp.q_off = pr.q_off;
  fp.kv_off = pr.kv_off;
  fp.H = pr.H;
  fp.group = pr.H / pr.win.H_kv;
  fp.total_q = pr.total_q;
  fp.scale_log2 = pr.scale * kLog2e;
  fp.win = pr.win;
  fp.whole = pr.total_q < (int64_t(1) << 31) && pr.total_kv < (int64_t(1) << 31);
  fp.maps = reinterpret_cast<const CUtensorMap*>(w + L.maps);
  fp.smaps = reinterpret_cast<const CUtensorMap*>(w + L.smaps);
  fp.sink_box = win_sink_box(pr.win.sinks);
  fp.items = reinterpret_cast<const WorkItem*>(w + L.fwd);
  fp.n_items = &reinterpret_cast<const WsHeader*>(w)->n_fwd;
  fp.claim = &reinterpret_cast<WsHeader*>(w)->claim_fwd;
  fp.status = &reinterpret_cast<WsHeader*>(w)->status;
  fp.wait_ns = &reinterpret_cast<const WsHeader*>(w)->wait_ns[0];
  fp.out = static_cast<__nv_bfloat16*>(out);
  fp.lse = lse;
  fp.wide_out = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  fp.trace = pr.trace[JFA_KERNEL_FORWARD];
  const int grid = kWinCtasPerSm * num_sms;
  return pr.d == 128 ? launch_win_fwd_t<128>(maps, fp, grid, stream) : launch_win_fwd_t<64>(maps, fp, grid, stream);
}

}  // namespace jfa
