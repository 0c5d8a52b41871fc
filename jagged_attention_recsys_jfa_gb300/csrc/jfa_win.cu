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
//   warps 0-3  softmax: one TMEM lane = one query row per thread
//   warp 4     K/V producer (TMA into a ring of 64-key tiles)
//   warp 5     MMA issuer: the first scores, then for each step PV(j), S(j + kBufs)
//   warp 6     query tile loader
//   warp 7     scheduler (claims items, publishes their metadata)
// TMEM (256 of the 512 columns): O [0, d), then kBufs score buffers of 64 columns (P, bf16,
// overwrites the first 32 of its buffer).  With the next steps' scores computed ahead, the chain
// of a step is its softmax alone; the products' latency (about 1300 cycles per step otherwise) is
// off it.
#include <cuda_bf16.h>

#include "jfa_internal.h"
#include "sm100_ptx.cuh"
#include "jfa_sched.cuh"

namespace jfa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kWinThreads = 256;
constexpr int kSoftmaxWarps = 4;
constexpr int kWinConsumers = 3 + kSoftmaxWarps;  // of a metadata entry
constexpr uint32_t kWinTmemCols = 256;

struct WinFwdParams {
  const int64_t* q_off;
  const int64_t* kv_off;
  int B, H, group;  // group: query heads per key/value head
  int64_t total_q, total_kv;
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
  TraceBuf trace;
};

template <int D>
struct WinCfg {
  static constexpr int kQBytes = kBM * D * 2;
  static constexpr int kTileBytes = kWinKeys * D * 2;
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kWinKeys * 128;  // one 64-column box of a K or V tile
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kBufs = D == 128 ? 2 : 3;    // score buffers
  static constexpr int kSmemBytes = kQBytes + kStages * kTileBytes + 1024;
  static constexpr uint32_t kColO = 0, kColS = D;
  static_assert(kColS + kBufs * kWinKeys <= kWinTmemCols, "TMEM columns");
  static_assert(2 * (kSmemBytes + 2048) <= 233472, "two CTAs per SM");
};

// A query tile's steps: nz of sinks, then the window part's 64-key tiles from a on; n in all.
struct TileSteps {
  int nz, a, n;
};
__device__ __forceinline__ TileSteps tile_steps(const ItemMeta& m, int t, int window) {
  const WinSeq ws = meta_win(m);
  TileSteps r;
  int e;
  win_kv_tiles(t, m.Lq, m.Lk, window, &r.a, &e, kWinKeys);
  r.nz = win_sees_sinks(t, m.Lq, ws) ? (ws.ns + kWinKeys - 1) / kWinKeys : 0;
  r.n = r.nz + e - r.a;
  return r;
}
// Order of a tile's loads, which is the order the products need them in: the scores run kBufs
// steps ahead, so K0 .. K(kBufs-1), then V0, K(kBufs), V1, ..
template <int kBufs>
__device__ __forceinline__ uint32_t k_pos(int j) { return j < kBufs ? j : 2 * j - kBufs + 1; }
template <int kBufs>
__device__ __forceinline__ uint32_t v_pos(int j, int n) {
  return min(j + kBufs, n) + j;  // the V tiles before it, and the K tiles of steps < j + kBufs
}

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

template <int D>
__global__ void __launch_bounds__(kWinThreads, 2)
    win_fwd_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const __grid_constant__ WinFwdParams p) {
  using C = WinCfg<D>;
  constexpr int R = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::kQBytes;

  __shared__ uint64_t q_full, q_empty, o_full, mma_done;
  __shared__ uint64_t kv_full[R], kv_empty[R], s_full[C::kBufs], p_full[C::kBufs];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ MetaRing meta;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&o_full, 1);
    mbar_init(&mma_done, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 32 * kSoftmaxWarps);
    }
    meta_init(meta, p.wait_ns, kWinConsumers);
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&tmem_base_sh, kWinTmemCols);
    tmem_relinquish();
  }
  grid_dependency_wait();  // the planner's lists and maps, the previous kernels' outputs
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_flag = &abort_sh;

  if (warp >= kSoftmaxWarps) {
   if (warp == 4) {
    // ------------------------------------------------------------ K/V producer
    if (lane == 0) {
      uint32_t ring_n = 0, tn = 0;
      bool ok = true;
      if (p.whole) {
        tmap_prefetch(&k_map);
        tmap_prefetch(&v_map);
      }
      const CUtensorMap* const whole_k = p.whole ? &k_map : nullptr;
      const CUtensorMap* const whole_v = p.whole ? &v_map : nullptr;
      for (uint32_t k = 0; ok; ++k) {
        if (!meta_wait(meta, k, abort_flag)) { ok = false; break; }
        const ItemMeta& wi = meta.e[k % kMetaSlots];  // read in place, freed after the item
        if (wi.b < 0) break;  // end of this CTA's items
        const WinSeq ws = meta_win(wi);
        const int col = wi.h / p.group * D;  // first column of the key/value head
        for (int t = wi.u0; t < wi.u1 && ok; ++t) {
          const TileSteps st = tile_steps(wi, t, p.win.window);
          if (st.n == 0) continue;
          auto fill = [&](int slot, int j) {
            const bool sink = j < st.nz;
            const TileMap m =
                sink ? tile_map(nullptr, p.smaps, p.B, slot, wi.b, wi.ko - ws.org, j, ws.ns, p.total_kv, kWinKeys)
                     : tile_map(slot == kMapK ? whole_k : whole_v, p.maps, p.B, slot, wi.b, wi.ko, st.a + j - st.nz, wi.Lk,
                                p.total_kv, kWinKeys);
            const uint32_t e = ring_n % R, ph = (ring_n / R) & 1;
            if (m.tail) tmap_acquire(m.map);
            if (!mbar_wait(&kv_empty[e], ph ^ 1, abort_flag, kWaitTimeoutNs)) return false;
            trace_event(p.trace, kTraceProducer, tn, 2);
            mbar_arrive_expect_tx(&kv_full[e], uint32_t(sink ? p.sink_box : kWinKeys) * D * 2);
#pragma unroll
            for (int c = 0; c < C::kBoxes; ++c)
              tma_load_2d(sRing + e * C::kTileBytes + c * C::kBoxBytes, m.map, &kv_full[e], col + c * 64, m.y);
            ++ring_n;
            return true;
          };
          for (int j = 0; j < min(C::kBufs, st.n) && ok; ++j) ok = fill(kMapK, j);
          for (int j = 0; j < st.n && ok; ++j) {
            ok = fill(kMapV, j);
            if (ok && j + C::kBufs < st.n) ok = fill(kMapK, j + C::kBufs);
          }
        }
        if (ok) meta_release(meta, k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      // every copy this thread started has landed before the CTA can exit
      const uint32_t first = ring_n > uint32_t(R) ? ring_n - R : 0;
      for (uint32_t n = first; n < ring_n; ++n) drain_wait(&kv_full[n % R], (n / R) & 1);
    }
   } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    // the whole warp walks the schedule; one elected lane issues the tcgen05 instructions
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kWinKeys, false, false);
    constexpr uint32_t kIdPV = idesc_bf16_f32(128, D, false, true);
    const uint32_t id_sink = idesc_bf16_f32(128, p.sink_box, false, false);
    const uint32_t aQ = smem_u32(sQ), aR = smem_u32(sRing);
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
    };
    uint32_t ring_n = 0, item_n = 0, tn = 0;
    uint32_t sb = 0, pb = 0, p_par = 0;  // score buffers of the next S and PV, parity of the latter's P
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
      const bool r = warp_wait(bar, par, abort_flag);
      tc_fence_after();
      return r;
    };
    for (uint32_t k = 0; ok; ++k) {
      if (!meta_wait_warp(meta, k, abort_flag)) { ok = false; break; }
      const ItemMeta& wi = meta.e[k % kMetaSlots];
      if (wi.b < 0) break;
      for (int t = wi.u0; t < wi.u1 && ok; ++t) {
        const TileSteps st = tile_steps(wi, t, p.win.window);
        if (st.n == 0) continue;
        if (!wait(&q_full, item_n & 1)) { ok = false; break; }
        ++item_n;
        if (lane == 0) trace_event(p.trace, kTraceMma, tn, 10);
        const uint32_t n0 = ring_n;
        auto issue_S = [&](int j) -> bool {
          const uint32_t n = n0 + k_pos<C::kBufs>(j), e = n % R;
          if (!wait(&kv_full[e], (n / R) & 1)) return false;
          const uint64_t qd = sdesc_sw128(aQ, 16, 1024), kd = sdesc_sw128(aR + e * C::kTileBytes, 16, 1024);
          const uint32_t id = j < st.nz ? id_sink : kIdS, col = tmem + C::kColS + sb * kWinKeys;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ss(col, qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                      kd + (((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4), id, kk > 0);
            umma_commit(&s_full[sb]);
            umma_commit(&kv_empty[e]);
            if (j + 1 == st.n) umma_commit(&q_empty);
          }
          sb = sb + 1 == C::kBufs ? 0 : sb + 1;
          if (lane == 0) trace_event(p.trace, kTraceMma, tn, 16);
          return true;
        };
        for (int j = 0; j < min(C::kBufs, st.n) && ok; ++j) ok = issue_S(j);
        for (int j = 0; j < st.n && ok; ++j) {
          const uint32_t n = n0 + v_pos<C::kBufs>(j, st.n), e = n % R;
          if (!wait(&kv_full[e], (n / R) & 1) || !wait(&p_full[pb], p_par)) { ok = false; break; }
          if (lane == 0) trace_event(p.trace, kTraceMma, tn, 12);
          const uint64_t vd = sdesc_sw128(aR + e * C::kTileBytes, C::kBoxBytes, 1024);
          const uint32_t col = tmem + C::kColS + pb * kWinKeys;
          const int kks = j < st.nz ? p.sink_box / 16 : kWinKeys / 16;  // 16 keys per product
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kWinKeys / 16; ++kk)
              if (kk < kks)
                umma_ts(tmem + C::kColO, col + kk * 8, vd + uint32_t(kk * 2048 >> 4), kIdPV, j > 0 || kk > 0);
            umma_commit(&kv_empty[e]);
            if (j + 1 == st.n) umma_commit(&o_full);
          }
          if (++pb == C::kBufs) {
            pb = 0;
            p_par ^= 1;
          }
          if (lane == 0) trace_event(p.trace, kTraceMma, tn, 14);
          if (j + C::kBufs < st.n) ok = issue_S(j + C::kBufs);
        }
        ring_n = n0 + 2 * st.n;
      }
      if (ok) meta_release_warp(meta, k);
    }
    if (!ok && lane == 0) raise_status(p.status, JFA_ERR_TIMEOUT);
    commit(&mma_done);
    drain_wait(&mma_done, 0);
   } else if (warp == 6) {
    // ------------------------------------------------------------ query tile loader
    if (lane == 0) {
      uint32_t item_n = 0, tn = 0;
      bool ok = true;
      if (p.whole) tmap_prefetch(&q_map);
      for (uint32_t k = 0; ok; ++k) {
        if (!meta_wait(meta, k, abort_flag)) { ok = false; break; }
        const ItemMeta& wi = meta.e[k % kMetaSlots];
        if (wi.b < 0) break;
        for (int t = wi.u0; t < wi.u1 && ok; ++t) {
          if (tile_steps(wi, t, p.win.window).n == 0) continue;
          const TileMap m = tile_map(p.whole ? &q_map : nullptr, p.maps, p.B, kMapQ, wi.b, wi.qo, t, wi.Lq, p.total_q);
          if (m.tail) tmap_acquire(m.map);
          if (!mbar_wait(&q_empty, (item_n & 1) ^ 1, abort_flag, kWaitTimeoutNs)) { ok = false; break; }
          trace_event(p.trace, kTraceLoader, tn, 1);
          mbar_arrive_expect_tx(&q_full, C::kQBytes);
#pragma unroll
          for (int c = 0; c < C::kBoxes; ++c) tma_load_2d(sQ + c * 16384, m.map, &q_full, wi.h * D + c * 64, m.y);
          ++item_n;
          // pull the next query tile into L2 meanwhile: the next of this range, else the first
          // of this CTA's next item
          const ItemMeta* nx = t + 1 < wi.u1 ? &wi : meta_peek_next(meta, k);
          if (nx && p.whole) {
            const int nt = t + 1 < wi.u1 ? t + 1 : nx->u0;
            if ((nt + 1) * kBM <= nx->Lq)
              for (int c = 0; c < C::kBoxes; ++c)
                tma_prefetch_2d(&q_map, nx->h * D + c * 64, int(nx->qo) + nt * kBM);
          }
        }
        if (ok) meta_release(meta, k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      if (item_n > 0) drain_wait(&q_full, (item_n - 1) & 1);
    }
   } else {
    // ------------------------------------------------------------ scheduler
    if (lane == 0 && !meta_publish<true>(meta, p.items, *p.n_items, p.claim, p.q_off, p.kv_off, nullptr, nullptr,
                                         abort_flag, p.win.window, p.win.sinks))
      raise_status(p.status, JFA_ERR_TIMEOUT);
   }
  } else {
    // ------------------------------------------------------------ softmax warps
    const uint32_t lane_addr = uint32_t(warp * 32) << 16;
    const uint32_t tO = tmem + lane_addr + C::kColO;
    const float sl2 = p.scale_log2;
    uint32_t ring_n = 0, b = 0, s_par = 0, o_n = 0, tn = 0;  // b: score buffer of the next step
    const bool leader = threadIdx.x == 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!meta_wait_warp(meta, k, abort_flag)) { ok = false; break; }
      const ItemMeta& wi = meta.e[k % kMetaSlots];
      if (wi.b < 0) break;
      const WinSeq ws = meta_win(wi);
      const int Lq = wi.Lq, diag = wi.Lk - Lq;
      for (int t = wi.u0; t < wi.u1 && ok; ++t) {
        const TileSteps st = tile_steps(wi, t, p.win.window);
        const int r0 = t * kBM + warp * 32, i = r0 + lane;  // the warp's first row, this thread's
        const bool valid = i < Lq;
        __nv_bfloat16* orow = p.out + ((wi.qo + i) * p.H + wi.h) * int64_t(D);
        float* lrow = p.lse + int64_t(wi.h) * p.total_q + wi.qo + i;
        if (st.n == 0) {
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
        int hi0 = r0 + diag + ws.org, last = ws.ns - 1, lo0 = -(1 << 30);  // first step of sinks
        for (int j = 0; j < st.n; ++j) {
          if (j == st.nz) {  // first key tile of the window part
            hi0 = r0 + diag - st.a * kWinKeys;
            last = 1 << 30;
            lo0 = hi0 - p.win.window + 1;
          }
          const bool hidden = min(last, hi0 + 31) < 0 || lo0 >= kWinKeys || r0 >= Lq;  // from all 32 rows
          const bool whole = min(last, hi0) >= kWinKeys - 1 && lo0 <= -31;             // seen by all 32
          const uint32_t tS = tmem + lane_addr + C::kColS + b * kWinKeys;
          if (!warp_wait(&s_full[b], s_par, abort_flag)) { ok = false; break; }
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
              const int chi = min(last, hi0 + lane), clo = lo0 + lane;
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
            // raise the reference maximum only when it grows by more than 2^8
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
              const uint32_t n = ring_n + v_pos<C::kBufs>(j - 1, st.n);
              if (!warp_wait(&kv_empty[n % R], (n / R) & 1, abort_flag)) { ok = false; break; }
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
          mbar_arrive(&p_full[b]);
          if (leader) trace_event(p.trace, kTraceCompute0, tn, 21);
          if (++b == C::kBufs) {
            b = 0;
            s_par ^= 1;
          }
          hi0 -= kWinKeys;
          lo0 -= kWinKeys;
          last -= kWinKeys;
        }
        if (!ok) break;
        ring_n += 2 * st.n;
        // ---- epilogue: O / l -> bf16, lse = ln(sum) = (m + log2 l) * ln 2
        if (!warp_wait(&o_full, o_n & 1, abort_flag)) { ok = false; break; }
        ++o_n;
        tc_fence_after();
        if (leader) trace_event(p.trace, kTraceCompute0, tn, 22);
        const bool live = l > 0.f;
        const float inv_l = live ? 1.f / l : 0.f;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 64) {
          uint32_t r[2][32];
          tmem_ld32(tO + c0, r[0]);
          tmem_ld32(tO + c0 + 32, r[1]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[e] = pack_bf16x2(__uint_as_float(r[q >> 1][(q & 1) * 16 + 2 * e]) * inv_l,
                                 __uint_as_float(r[q >> 1][(q & 1) * 16 + 2 * e + 1]) * inv_l);
            if (valid) st_global_v8(orow + c0 + q * 16, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
          }
        }
        if (valid) *lrow = live ? ((m == -INFINITY ? 0.f : m) + __log2f(l)) * kLn2 : -INFINITY;
        tc_fence_before();
        if (leader) trace_event(p.trace, kTraceCompute0, tn, 23);
      }
      if (ok) meta_release_warp(meta, k);
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kWinTmemCols);
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

cudaError_t launch_win_forward(const Problem& pr, const PlanMaps& maps, void* ws, const WsLayout& L, void* out, float* lse, int num_sms,
                               cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  WinFwdParams fp;
  fp.q_off = pr.q_off;
  fp.kv_off = pr.kv_off;
  fp.B = pr.B;
  fp.H = pr.H;
  fp.group = pr.H / pr.win.H_kv;
  fp.total_q = pr.total_q;
  fp.total_kv = pr.total_kv;
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
  fp.trace = pr.trace[JFA_KERNEL_FORWARD];
  const int grid = kWinCtasPerSm * num_sms;
  return pr.d == 128 ? launch_win_fwd_t<128>(maps, fp, grid, stream) : launch_win_fwd_t<64>(maps, fp, grid, stream);
}

}  // namespace jfa
