// The windowed backward's dQ pass for d = 64 (the formulas: jfa_win_bwd.cu).  One item per (sequence,
// query head, query tile):  S = Q K^T, P = exp(S - lse), dP = dO V^T, dS = P o (dP - D), dQ += dS K
// over the sinks and the window part in steps of 64 keys.
//
// Built like the windowed forward (jfa_win.cu), for the same reason: an item is a few short steps
// whose hand-offs, not their products, set the pace, so two CTAs share an SM, each with half of its
// shared and tensor memory.  (At d = 128 Q, dO and one stage of K and V take 97 of the 112 KB that a
// CTA would have: room for no second stage, and not tried.)
// 62 us (64 sequences of up to 2048 tokens, 4 query and 2 key/value heads, window 256, 4 sinks), with
// every tile through its sequence's maps 86; one CTA per SM with 128-key steps took 93.  2048
// sequences of up to 96 tokens: 157 us instead of 282.
//
//   warp 0     K/V producer (two rings of 64-key tiles)
//   warp 1     issues the products dQ(j)
//   warp 2     loads the tile's Q and dO, issues S(j) and dP(j)
//   warp 3     scheduler
//   warps 4-7  P and dS: one TMEM lane = one query row per thread
// TMEM (256 columns): dQ [0, 64), then three buffers of 64 columns that S(0), dP(0), S(1), dP(1), ...
// take in turn: S(j)'s is free as soon as its scores are in registers, and dP(j)'s, which dS(j)
// (bf16) overwrites, once dQ(j) has read it.  So S(j + 1) is there before step j is done.
#include "jfa_win.cuh"

namespace jfa {
namespace {

struct WinDqParams {
  const int64_t *q_off, *kv_off, *qpad;
  int H, group;
  float scale, scale_log2;
  WindowSpec win;
  bool whole;  // the tensors' own maps serve whole tiles (row numbers fit 31 bits)
  const CUtensorMap *maps, *smaps;
  int sink_box;
  const WorkItem* items;
  const int* n_items;
  int* claim;
  int* status;
  const uint64_t* wait_ns;
  const float *lse2, *delta;  // -lse log2 e and -D of the padded query rows
  int64_t qpad_cap;
  __nv_bfloat16* dq;
  bool wide_out;  // dq is 32-byte aligned
};

constexpr int kD = 64;
constexpr int kQBytes = kBM * kD * 2, kKeyBytes = kWinKeys * kD * 2;
constexpr int kStages = 4;  // tiles of the K ring, and of the V ring
constexpr int kDqSmemBytes = 2 * kQBytes + 2 * kStages * kKeyBytes + 1024;
constexpr uint32_t kColDq = 0, kColBuf = kD;
static_assert(kColBuf + 3 * kWinKeys <= kWinTmemCols, "TMEM columns");
static_assert(2 * (kDqSmemBytes + 2048) <= 233472, "two CTAs per SM");

__global__ void __launch_bounds__(kWinThreads, 2)
    win_dq64_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap do_map,
                    const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                    const __grid_constant__ WinDqParams p) {
  constexpr int R = kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sDO = smem + kQBytes;
  uint8_t* sK = smem + 2 * kQBytes;
  uint8_t* sV = sK + R * kKeyBytes;

  // barriers of step g at index g & 1: a step is at most one ahead of the previous one's last use
  __shared__ uint64_t q_full, q_empty, o_full, dq_done, s_done;
  __shared__ uint64_t k_full[R], k_empty[R], v_full[R], v_empty[R], s_full[2], s_free[2], dp_full[2], ds_full[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ TileRing tiles;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&o_full, 1);
    mbar_init(&dq_done, 1);
    mbar_init(&s_done, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 32 * kSoftmaxWarps);
      mbar_init(&dp_full[i], 1);
      mbar_init(&ds_full[i], 32 * kSoftmaxWarps);
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
      uint32_t n = 0;  // tiles loaded into each ring
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
        const int col = w.h / p.group * kD;
        auto fill = [&](int slot, int j, Ring<R>& r, uint64_t* full, uint64_t* empty, uint8_t* smem_tiles) {
          const bool sink = j < w.nz;
          const TileMap m = sink ? win_tile_map(p.smaps, slot, w.b, j, kWinKeys, 0)
                                 : win_tile_map(slot == kMapK ? whole_k : whole_v, p.maps, slot, w.b, w.ko,
                                                w.a + j - w.nz, w.Lk, kWinKeys, w.skip);
          if (sink || m.tail) tmap_acquire(m.map);
          if (!mbar_wait(&empty[r.e], r.ph ^ 1, abort_flag, kWaitTimeoutNs)) return false;
          mbar_arrive_expect_tx(&full[r.e], uint32_t(sink ? p.sink_box : kWinKeys) * kD * 2);
          tma_load_2d(smem_tiles + r.e * kKeyBytes, m.map, &full[r.e], col, m.y);
          r.next();
          return true;
        };
        for (int j = 0; j < w.n && ok; ++j) {
          if (!fill(kMapK, j, kr, k_full, k_empty, sK)) { ok = false; break; }
          if (!fill(kMapV, j, vr, v_full, v_empty, sV)) {
            ok = false;
            drain_wait(&k_full[n % R], (n / R) & 1);
            break;
          }
          ++n;
        }
        if (ok) mbar_arrive(&tiles.empty[k % kMetaSlots]);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      // every copy this thread started has landed before the CTA can exit
      for (uint32_t i = n > R ? n - R : 0; i < n; ++i) {
        drain_wait(&k_full[i % R], (i / R) & 1);
        drain_wait(&v_full[i % R], (i / R) & 1);
      }
    }
   } else if (warp == 1) {
    // ------------------------------------------------------------ products dS K
    constexpr uint32_t kIdDq = idesc_bf16_f32(128, kD, false, true);
    const uint64_t kd0 = sdesc_sw128(smem_u32(sK), kKeyBytes, 1024);
    Ring<R> kr;
    Ring<3> br;  // buffer of dP(g)
    br.next();
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!tile_wait_warp(tiles, k, abort_flag)) { ok = false; break; }
      const int n = tiles.e[k % kMetaSlots].n, nz = tiles.e[k % kMetaSlots].nz;
      const bool end = tiles.e[k % kMetaSlots].b < 0;
      tile_release_warp(tiles, k);  // all it needs is in registers
      if (end) break;
      for (int j = 0; j < n; ++j, ++g) {
        if (!warp_wait(&k_full[kr.e], kr.ph, abort_flag) || !warp_wait(&ds_full[g & 1], (g >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t kd = kd0 + kr.e * uint32_t(kKeyBytes >> 4);
        const uint32_t col = tmem + kColBuf + br.e * kWinKeys;
        const int kks = j < nz ? p.sink_box / 16 : kWinKeys / 16;  // 16 keys per product
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kWinKeys / 16; ++kk)
            if (kk < kks)
              umma_ts(tmem + kColDq, col + kk * 8, kd + uint32_t(kk * 2048 >> 4), kIdDq, j > 0 || kk > 0);
          umma_commit(&k_empty[kr.e]);
          if (j + 1 == n) umma_commit(&o_full);
        }
        kr.next();
        br.next();
        br.next();
      }
    }
    if (!ok && lane == 0) raise_status(p.status, JFA_ERR_TIMEOUT);
    if (elect_one()) umma_commit(&dq_done);
    drain_wait(&dq_done, 0);
   } else if (warp == 2) {
    // ------------------------------------------------------------ Q and dO, products Q K^T and dO V^T
    constexpr uint32_t kIdS = idesc_bf16_f32(128, kWinKeys, false, false);
    const uint32_t id_sink = idesc_bf16_f32(128, p.sink_box, false, false);
    const uint64_t qd = sdesc_sw128(smem_u32(sQ), 16, 1024), dod = sdesc_sw128(smem_u32(sDO), 16, 1024);
    const uint64_t kd0 = sdesc_sw128(smem_u32(sK), 16, 1024), vd0 = sdesc_sw128(smem_u32(sV), 16, 1024);
    uint32_t n_q = 0, g = 0;  // query tiles loaded, steps issued
    Ring<R> kr, vr, fr;       // fr: K tile of step g - 2, whose dQ frees the buffer of S(g)
    Ring<3> br;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!tile_wait_warp(tiles, k, abort_flag)) { ok = false; break; }
      const WinTile& w = tiles.e[k % kMetaSlots];
      if (w.b < 0) break;
      const int n = w.n, nz = w.nz;
      if (n == 0) {
        tile_release_warp(tiles, k);
        continue;
      }
      // the last products of the previous tile have read the buffers
      if (!warp_wait(&q_empty, (n_q & 1) ^ 1, abort_flag)) { ok = false; break; }
      if (lane == 0) {
        const TileMap mq = win_tile_map(p.whole ? &q_map : nullptr, p.maps, kMapQ, w.b, w.qo, w.t, w.Lq, kBM, 0);
        const TileMap md = win_tile_map(p.whole ? &do_map : nullptr, p.maps, kMapDO, w.b, w.qo, w.t, w.Lq, kBM, 0);
        if (mq.tail) {
          tmap_acquire(mq.map);
          tmap_acquire(md.map);
        }
        mbar_arrive_expect_tx(&q_full, 2 * kQBytes);
        tma_load_2d(sQ, mq.map, &q_full, w.h * kD, mq.y);
        tma_load_2d(sDO, md.map, &q_full, w.h * kD, md.y);
        // pull the CTA's next query tile into L2 meanwhile, if the scheduler has it already
        const uint32_t kn = k + 1;
        if (p.whole && mbar_test_wait(&tiles.full[kn % kMetaSlots], (kn / kMetaSlots) & 1)) {
          const WinTile& x = tiles.e[kn % kMetaSlots];
          if (x.b >= 0 && x.rows == kBM) {
            tma_prefetch_2d(&q_map, x.h * kD, int(x.qo) + x.t * kBM);
            tma_prefetch_2d(&do_map, x.h * kD, int(x.qo) + x.t * kBM);
          }
        }
      }
      tile_release_warp(tiles, k);
      ++n_q;
      if (!warp_wait(&q_full, (n_q - 1) & 1, abort_flag)) { ok = false; break; }
      for (int j = 0; j < n; ++j, ++g) {
        const uint32_t id = j < nz ? id_sink : kIdS;
        if (!warp_wait(&k_full[kr.e], kr.ph, abort_flag)) { ok = false; break; }
        if (g >= 2) {
          if (!warp_wait(&k_empty[fr.e], fr.ph, abort_flag)) { ok = false; break; }
          fr.next();
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kd = kd0 + kr.e * uint32_t(kKeyBytes >> 4);
          const uint32_t col = tmem + kColBuf + br.e * kWinKeys;
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) umma_ss(col, qd + (kk * 32 >> 4), kd + (kk * 32 >> 4), id, kk > 0);
          umma_commit(&s_full[g & 1]);
        }
        kr.next();
        br.next();
        if (!warp_wait(&v_full[vr.e], vr.ph, abort_flag)) { ok = false; break; }
        if (g >= 1 && !warp_wait(&s_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = vd0 + vr.e * uint32_t(kKeyBytes >> 4);
          const uint32_t col = tmem + kColBuf + br.e * kWinKeys;
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) umma_ss(col, dod + (kk * 32 >> 4), vd + (kk * 32 >> 4), id, kk > 0);
          umma_commit(&dp_full[g & 1]);
          umma_commit(&v_empty[vr.e]);
          if (j + 1 == n) umma_commit(&q_empty);
        }
        vr.next();
        br.next();
      }
    }
    if (!ok && lane == 0) raise_status(p.status, JFA_ERR_TIMEOUT);
    // the query copies and the products have landed before the CTA can exit
    if (n_q > 0) drain_wait(&q_full, (n_q - 1) & 1);
    if (elect_one()) umma_commit(&s_done);
    drain_wait(&s_done, 0);
   } else {
    // ------------------------------------------------------------ scheduler (maps laid out for 128-key tiles)
    if (lane == 0 && !publish_tiles<kBN>(tiles, p, p.qpad, abort_flag)) raise_status(p.status, JFA_ERR_TIMEOUT);
   }
  } else {
    // ------------------------------------------------------------ P and dS
    const int quarter = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
    const uint32_t tQ = tmem + lane_addr + kColDq, tB = tmem + lane_addr + kColBuf;
    const uint64_t k_sl2 = f2_pack(p.scale_log2, p.scale_log2);
    uint32_t g = 0, o_n = 0;
    Ring<3> br;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!tile_wait_warp(tiles, k, abort_flag)) { ok = false; break; }
      const WinTile& w = tiles.e[k % kMetaSlots];
      if (w.b < 0) break;
      const int n = w.n, nz = w.nz, ns = w.ns, rows = w.rows;
      const int r0 = quarter * 32, i = r0 + lane;
      const bool valid = i < rows;
      __nv_bfloat16* orow = p.dq + ((w.qo + w.t * kBM + i) * p.H + w.h) * int64_t(kD);
      const int64_t vec = int64_t(w.h) * p.qpad_cap + w.qp + w.t * kBM + i;
      int hi0 = r0 + w.pos + w.org, last = ns - 1, lo0 = -(1 << 30), pad = 0;            // first step of sinks
      const int hi_win = r0 + w.pos - w.a * kWinKeys, pad_win = w.pad - w.a * kWinKeys;  // first tile of the window part
      tile_release_warp(tiles, k);  // the rest is in registers
      if (n == 0) {
        if (valid) {
#pragma unroll
          for (int c = 0; c < kD / 8; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      const float nl = __ldg(p.lse2 + vec), nd = __ldg(p.delta + vec);
      const uint64_t k_nl = f2_pack(nl, nl), k_nd = f2_pack(nd, nd);
      // masks as in the forward: row i sees columns [clo, chi] of a step
      for (int j = 0; j < n; ++j, ++g) {
        if (j == nz) {  // first key tile of the window part
          hi0 = hi_win;
          last = 1 << 30;
          lo0 = hi0 - p.win.window + 1;
          pad = pad_win;
        }
        const bool hidden = min(last, hi0 + 31) < 0 || lo0 >= kWinKeys || r0 >= rows;
        const bool whole = min(last, hi0) >= kWinKeys - 1 && lo0 <= -31 && pad <= 0;
        const uint32_t tS = tB + br.e * kWinKeys;
        br.next();
        const uint32_t tP = tB + br.e * kWinKeys;
        br.next();
        if (!warp_wait(&s_full[g & 1], (g >> 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
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
          tc_fence_before();
          mbar_arrive(&s_free[g & 1]);
          if (!whole) {
            const int chi = min(last, hi0 + lane), clo = max(lo0 + lane, pad);
            const uint32_t bits[2] = {low_bits(chi + 1) & ~low_bits(clo), low_bits(chi - 31) & ~low_bits(clo - 32)};
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(bits[c >> 5] & (1u << (c & 31)))) x[c] = -INFINITY;
          }
#pragma unroll
          for (int c2 = 0; c2 < 32; ++c2) {
            f2_unpack(f2_fma(f2_pack(x[2 * c2], x[2 * c2 + 1]), k_sl2, k_nl), x[2 * c2], x[2 * c2 + 1]);
            x[2 * c2] = ex2_approx(x[2 * c2]);
            x[2 * c2 + 1] = ex2_approx(x[2 * c2 + 1]);
          }
          if (!warp_wait(&dp_full[g & 1], (g >> 1) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t r[32];
            tmem_ld32(tP + 32 * half, r);
            tmem_ld_wait();
#pragma unroll
            for (int c2 = 0; c2 < 16; ++c2) {  // dS = P o (dP - D)
              const int c = 32 * half + 2 * c2;
              float d0, d1;
              f2_unpack(f2_mul(f2_pack(x[c], x[c + 1]),
                               f2_add(f2_pack(__uint_as_float(r[2 * c2]), __uint_as_float(r[2 * c2 + 1])), k_nd)),
                        d0, d1);
              pk[c >> 1] = pack_bf16x2(d0, d1);
            }
          }
        } else {
          mbar_arrive(&s_free[g & 1]);
          if (!warp_wait(&dp_full[g & 1], (g >> 1) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = 0u;
        }
        tmem_st32(tP, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ds_full[g & 1]);
        hi0 -= kWinKeys;
        lo0 -= kWinKeys;
        pad -= kWinKeys;
        last -= kWinKeys;
      }
      if (!ok) break;
      if (!warp_wait(&o_full, o_n & 1, abort_flag)) { ok = false; break; }
      ++o_n;
      tc_fence_after();
      uint32_t r[2][32];
      tmem_ld32(tQ, r[0]);
      tmem_ld32(tQ + 32, r[1]);
      tmem_ld_wait();
      tc_fence_before();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w8[e] = pack_bf16x2(__uint_as_float(r[q >> 1][(q & 1) * 16 + 2 * e]) * p.scale,
                              __uint_as_float(r[q >> 1][(q & 1) * 16 + 2 * e + 1]) * p.scale);
        if (!valid) continue;
        if (p.wide_out) {
          st_global_v8(orow + q * 16, w8[0], w8[1], w8[2], w8[3], w8[4], w8[5], w8[6], w8[7]);
        } else {
          uint4* o = reinterpret_cast<uint4*>(orow + q * 16);
          o[0] = make_uint4(w8[0], w8[1], w8[2], w8[3]);
          o[1] = make_uint4(w8[4], w8[5], w8[6], w8[7]);
        }
      }
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kWinTmemCols);
}

}  // namespace

cudaError_t launch_win_dq64(const Problem& pr, const WinPlanMaps& maps, void* ws, const WsLayout& L, void* dq,
                            int num_sms, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(w);
  WinDqParams p;
  p.q_off = pr.q_off;
  p.kv_off = pr.kv_off;
  p.qpad = reinterpret_cast<const int64_t*>(w + L.qpad);
  p.H = pr.H;
  p.group = pr.H / pr.win.H_kv;
  p.scale = pr.scale;
  p.scale_log2 = pr.scale * kLog2e;
  p.win = pr.win;
  p.whole = pr.total_q < (int64_t(1) << 31) && pr.total_kv < (int64_t(1) << 31);
  p.maps = reinterpret_cast<const CUtensorMap*>(w + L.maps);
  p.smaps = reinterpret_cast<const CUtensorMap*>(w + L.smaps);
  p.sink_box = win_sink_box(pr.win.sinks);
  p.items = reinterpret_cast<const WorkItem*>(w + L.dq);
  p.n_items = &hdr->n_dq;
  p.claim = &hdr->claim_dq;
  p.status = &hdr->status;
  p.wait_ns = &hdr->wait_ns[1];
  p.lse2 = reinterpret_cast<const float*>(w + L.lse2);
  p.delta = reinterpret_cast<const float*>(w + L.delta);
  p.qpad_cap = L.qpad_cap;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.wide_out = (reinterpret_cast<uintptr_t>(dq) & 31u) == 0;
  const cudaError_t e = cudaFuncSetAttribute(win_dq64_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDqSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(win_dq64_kernel, dim3(kWinCtasPerSm * num_sms), dim3(kWinThreads), kDqSmemBytes, stream, maps.tmpl[kMapQ],
                    maps.tmpl[kMapDO], maps.tmpl[kMapK], maps.tmpl[kMapV], p);
}

}  // namespace jfa
