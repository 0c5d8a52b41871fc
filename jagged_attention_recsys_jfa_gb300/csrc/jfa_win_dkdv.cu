// The windowed backward's dK/dV pass for d = 64 (the formulas, items and partial sums of the sinks:
// jfa_win_bwd.cu).  Two CTAs per SM, each with half of its shared and tensor memory, as in the dQ pass
// (jfa_win_dq.cu): while one waits for its next key tile, a product or its rows, the other computes.
//
// 88 us (64 sequences of up to 2048 tokens, 4 query and 2 key/value heads, window 256, 4 sinks); one
// CTA per SM with 128-query steps took 108, and 333 instead of 249 on 2048 sequences of up to 96
// tokens.  The tensor pipe is busy 27% of it, memory 17%: the hand-offs and every warp's own work
// per step set the pace (eight warps of 32 queries each took 113; vectors read 16 bytes at a time and
// the next key tile pulled into L2 changed nothing).
//
// A step takes 64 queries of one query head against the item's 128 keys; of a query tile's two
// halves only those are taken that a key's window reaches.
//
//   warp 0     producer of the query tiles: Q, dO, -lse log2 e and -D of 128 rows, two stages
//   warp 1     issues the products:  S^T(g + 1) behind dV(g), dP^T(g + 1) behind dK(g)
//   warp 2     K/V loader
//   warp 3     scheduler
//   warps 4-7  P^T and dS^T, one TMEM lane = one key per thread; and the finished rows
// TMEM (256 columns): dK [0, 64), dV [64, 128), S^T [128, 192), dP^T [192, 256); P^T and dS^T (bf16)
// overwrite the first halves of theirs.  The tensor pipe takes products in order, so S^T(g + 1) may be
// issued behind the dV(g) that reads P^T(g): it is there when the warps have done dS^T(g).
#include "jfa_win.cuh"

namespace jfa {
namespace {

struct WinDkdvParams {
  const int64_t *q_off, *kv_off, *qpad;
  int H, group;
  float scale, scale_log2;
  WindowSpec win;
  bool whole;  // the tensors' own maps serve whole tiles (row numbers fit 31 bits)
  const CUtensorMap *maps, *smaps;
  int sink_rows;  // of the sinks' tile, in boxes of up to kWinKeys
  const WorkItem* items;
  const int* n_items;
  int* claim;
  int* status;
  const uint64_t* wait_ns;
  const float *lse2, *delta;  // -lse log2 e and -D of the padded query rows
  int64_t qpad_cap;
  __nv_bfloat16 *dk, *dv;
  float* spart;  // partial dK, dV of the sinks: [slot][2][sinks][64]
};

constexpr int kD = 64;
constexpr int kTileBytes = 128 * kD * 2;     // a tile of 128 rows
constexpr int kHalfBytes = kTileBytes / 2;   // 64 rows of it
constexpr int kStages = 2;                   // query tiles under way
constexpr int kVecFloats = 2 * kBM;          // -lse log2 e and -D of a query tile
constexpr int kDkdvSmemBytes = 2 * kTileBytes + kStages * (2 * kTileBytes + kVecFloats * 4) + 1024;
constexpr uint32_t kColDk = 0, kColDv = 64, kColS = 128, kColP = 192;
static_assert(kColP + 64 <= kWinTmemCols, "TMEM columns");
static_assert(2 * (kDkdvSmemBytes + 2048) <= 233472, "two CTAs per SM");

// A unit's steps: its pairs of query head and query tile in order, and of each tile the halves that
// see any of its keys.  (Counted on, not divided out of the pair's number, which costs every warp
// some hundred instructions a step.)
struct StepWalk {
  int left;         // pairs not done yet
  int t, half;      // query tile, its half
  int first, end;   // tiles of one head
  int lo, hi;       // queries outside [lo, hi] see no key
  __device__ __forceinline__ StepWalk(const WinKeyUnit& u)
      : left(u.r1 - u.r0), t(u.first + u.r0 % u.n), first(u.first), end(u.first + u.n), lo(u.lo), hi(u.hi) {
    half = first_half();
  }
  __device__ __forceinline__ bool live() const { return left > 0; }
  __device__ __forceinline__ bool final() const { return left == 1 && last_half(); }
  __device__ __forceinline__ int first_half() const { return t * kBM + 63 >= lo ? 0 : 1; }
  __device__ __forceinline__ bool last_half() const { return half == 1 || t * kBM + 64 > hi; }
  __device__ __forceinline__ void next() {
    if (!last_half()) {
      half = 1;
    } else {
      --left;
      t = t + 1 == end ? first : t + 1;
      half = first_half();
    }
  }
};

__device__ __forceinline__ void store_row(const uint32_t (&r)[32], float mul, __nv_bfloat16* dst) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    reinterpret_cast<uint4*>(dst)[c] =
        make_uint4(pack_bf16x2(__uint_as_float(r[8 * c]) * mul, __uint_as_float(r[8 * c + 1]) * mul),
                   pack_bf16x2(__uint_as_float(r[8 * c + 2]) * mul, __uint_as_float(r[8 * c + 3]) * mul),
                   pack_bf16x2(__uint_as_float(r[8 * c + 4]) * mul, __uint_as_float(r[8 * c + 5]) * mul),
                   pack_bf16x2(__uint_as_float(r[8 * c + 6]) * mul, __uint_as_float(r[8 * c + 7]) * mul));
}

__global__ void __launch_bounds__(kWinThreads, 2)
    win_dkdv64_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap do_map,
                      const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                      const __grid_constant__ WinDkdvParams p) {
  constexpr int R = kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + kTileBytes;
  uint8_t* sQ = smem + 2 * kTileBytes;           // [stage]
  uint8_t* sDO = sQ + R * kTileBytes;            // [stage]
  float* sVec = reinterpret_cast<float*>(sDO + R * kTileBytes);  // [stage][2][128]

  __shared__ uint64_t kv_full, kv_empty, s_full, dp_full, p_full, ds_full, acc_full, mma_done;
  __shared__ uint64_t ring_full[R], ring_empty[R];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ MetaRing meta;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    mbar_init(&kv_full, 1);
    mbar_init(&kv_empty, 1);
    mbar_init(&s_full, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&p_full, 32 * kSoftmaxWarps);
    mbar_init(&ds_full, 32 * kSoftmaxWarps);
    mbar_init(&acc_full, 1);
    mbar_init(&mma_done, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(&ring_full[i], 1);
      mbar_init(&ring_empty[i], 1);
    }
    meta_init(meta, p.wait_ns, kWinConsumers);
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
  auto unit_of = [&](const ItemMeta& m) { return win_key_unit(m.u0, m.Lq, meta_win(m), p.win.window, p.group); };

  if (warp < kFirstComputeWarp) {
   if (warp == 0) {
    // ------------------------------------------------------------ query tiles
    if (lane == 0) {
      Ring<R> r;
      uint32_t n = 0;
      bool ok = true;
      if (p.whole) {
        tmap_prefetch(&q_map);
        tmap_prefetch(&do_map);
      }
      for (uint32_t k = 0; ok; ++k) {
        if (!meta_wait(meta, k, abort_flag)) { ok = false; break; }
        const ItemMeta& wi = meta.e[k % kMetaSlots];  // read in place, freed after the item
        if (wi.b < 0) break;  // end of this CTA's items
        const WinKeyUnit u = unit_of(wi);
        int t = u.first + u.r0 % u.n, h = wi.h * p.group + u.r0 / u.n;
        for (int i = u.r0; i < u.r1; ++i) {
          const TileMap mq = win_tile_map(p.whole ? &q_map : nullptr, p.maps, kMapQ, wi.b, wi.qo, t, wi.Lq, kBM, 0);
          const TileMap md = win_tile_map(p.whole ? &do_map : nullptr, p.maps, kMapDO, wi.b, wi.qo, t, wi.Lq, kBM, 0);
          if (mq.tail) {
            tmap_acquire(mq.map);
            tmap_acquire(md.map);
          }
          if (!mbar_wait(&ring_empty[r.e], r.ph ^ 1, abort_flag, kWaitTimeoutNs)) { ok = false; break; }
          mbar_arrive_expect_tx(&ring_full[r.e], 2 * kTileBytes + kVecFloats * 4);
          tma_load_2d(sQ + r.e * kTileBytes, mq.map, &ring_full[r.e], h * kD, mq.y);
          tma_load_2d(sDO + r.e * kTileBytes, md.map, &ring_full[r.e], h * kD, md.y);
          const int64_t vec = int64_t(h) * p.qpad_cap + wi.qp + t * kBM;
          float* v = sVec + r.e * kVecFloats;
          bulk_load(v, p.lse2 + vec, kBM * 4, &ring_full[r.e]);
          bulk_load(v + kBM, p.delta + vec, kBM * 4, &ring_full[r.e]);
          r.next();
          ++n;
          if (++t == u.first + u.n) {  // the group's next query head
            t = u.first;
            ++h;
          }
        }
        if (ok) meta_release(meta, k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      // every copy this thread started has landed before the CTA can exit
      for (uint32_t i = n > R ? n - R : 0; i < n; ++i) drain_wait(&ring_full[i % R], (i / R) & 1);
    }
   } else if (warp == 1) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kIdS = idesc_bf16_f32(128, 64, false, false), kIdAcc = idesc_bf16_f32(128, kD, false, true);
    const uint64_t kd = sdesc_sw128(smem_u32(sK), 16, 1024), vd = sdesc_sw128(smem_u32(sV), 16, 1024);
    const uint32_t aQ = smem_u32(sQ), aDO = smem_u32(sDO);
    Ring<R> cur;             // stage of the current step
    uint32_t item_n = 0, g = 0;
    bool ok = true;
    // S^T (keys K, Q rows at b) or dP^T (V, dO): 128 keys x 64 queries
    auto mma_nt = [&](uint32_t col, uint64_t a, uint32_t b) {
      const uint64_t bd = sdesc_sw128(b, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < kD / 16; ++kk) umma_ss(tmem + col, a + (kk * 32 >> 4), bd + (kk * 32 >> 4), kIdS, kk > 0);
    };
    // acc (keys x 64) += X^T (TMEM bf16, keys x 64 queries) * rows at b (queries x 64)
    auto mma_acc = [&](uint32_t acc, uint32_t x, uint32_t b, bool add) {
      const uint64_t bd = sdesc_sw128(b, kHalfBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_ts(tmem + acc, tmem + x + kk * 8, bd + uint32_t(kk * 2048 >> 4), kIdAcc, add || kk > 0);
    };
    for (uint32_t k = 0; ok; ++k) {
      if (!meta_wait_warp(meta, k, abort_flag)) { ok = false; break; }
      const ItemMeta& wi = meta.e[k % kMetaSlots];
      if (wi.b < 0) break;
      const WinKeyUnit u = unit_of(wi);
      meta_release_warp(meta, k);  // the rest is in registers
      if (u.r1 <= u.r0) continue;
      StepWalk w(u);
      if (!warp_wait(&kv_full, item_n & 1, abort_flag) || !warp_wait(&ring_full[cur.e], cur.ph, abort_flag)) {
        ok = false;
        break;
      }
      ++item_n;
      tc_fence_after();
      {
        const uint32_t at = cur.e * kTileBytes + w.half * kHalfBytes;
        if (elect_one()) {
          mma_nt(kColS, kd, aQ + at);
          umma_commit(&s_full);
          mma_nt(kColP, vd, aDO + at);
          umma_commit(&dp_full);
          if (w.final()) umma_commit(&kv_empty);
        }
      }
      bool first = true;
      while (w.live()) {
        const uint32_t at = cur.e * kTileBytes + w.half * kHalfBytes, e = cur.e;
        const bool pair_done = w.last_half();
        StepWalk nx = w;
        nx.next();
        const bool more = nx.live();
        if (pair_done) cur.next();
        const uint32_t at_next = cur.e * kTileBytes + nx.half * kHalfBytes;
        if (!warp_wait(&p_full, g & 1, abort_flag)) { ok = false; break; }
        if (more && pair_done && !warp_wait(&ring_full[cur.e], cur.ph, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          mma_acc(kColDv, kColS, aDO + at, !first);  // dV += P^T dO
          if (more) {
            mma_nt(kColS, kd, aQ + at_next);
            umma_commit(&s_full);
          }
        }
        if (!warp_wait(&ds_full, g & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          mma_acc(kColDk, kColP, aQ + at, !first);  // dK += dS^T Q
          if (pair_done) umma_commit(&ring_empty[e]);
          if (more) {
            mma_nt(kColP, vd, aDO + at_next);
            umma_commit(&dp_full);
            if (nx.final()) umma_commit(&kv_empty);  // the last to read K and V
          } else {
            umma_commit(&acc_full);
          }
        }
        first = false;
        ++g;
        w = nx;
      }
    }
    if (!ok && lane == 0) raise_status(p.status, JFA_ERR_TIMEOUT);
    if (elect_one()) umma_commit(&mma_done);
    drain_wait(&mma_done, 0);
   } else if (warp == 2) {
    // ------------------------------------------------------------ K/V loader
    if (lane == 0) {
      uint32_t item_n = 0;
      bool ok = true;
      if (p.whole) {
        tmap_prefetch(&k_map);
        tmap_prefetch(&v_map);
      }
      for (uint32_t k = 0; ok; ++k) {
        if (!meta_wait(meta, k, abort_flag)) { ok = false; break; }
        const ItemMeta& wi = meta.e[k % kMetaSlots];
        if (wi.b < 0) break;
        const WinKeyUnit u = unit_of(wi);
        if (u.r1 > u.r0) {
          const bool sink = u.chunk >= 0, half = sink && p.sink_rows <= kWinKeys;  // one box of the two
          auto map_of = [&](int slot, const CUtensorMap* whole) {
            return sink ? win_tile_map(p.smaps, slot, wi.b, 0, kBN, 0)
                        : win_tile_map(p.whole ? whole : nullptr, p.maps, slot, wi.b, wi.ko, wi.u0, wi.Lk, kBN,
                                       meta_win(wi).skip);
          };
          const TileMap mk = map_of(kMapK, &k_map), mv = map_of(kMapV, &v_map);
          if (sink || mk.tail) {
            tmap_acquire(mk.map);
            tmap_acquire(mv.map);
          }
          if (!mbar_wait(&kv_empty, (item_n & 1) ^ 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
          mbar_arrive_expect_tx(&kv_full, half ? uint32_t(p.sink_rows) * kD * 4 : 2u * kTileBytes);
          const int col = wi.h * kD;
          tma_load_2d(sK, mk.map, &kv_full, col, mk.y);
          tma_load_2d(sV, mv.map, &kv_full, col, mv.y);
          if (!half) {
            tma_load_2d(sK + kHalfBytes, mk.map, &kv_full, col, mk.y + kWinKeys);
            tma_load_2d(sV + kHalfBytes, mv.map, &kv_full, col, mv.y + kWinKeys);
          }
          ++item_n;
        }
        if (ok) meta_release(meta, k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      if (item_n > 0) drain_wait(&kv_full, (item_n - 1) & 1);
    }
   } else {
    // ------------------------------------------------------------ scheduler
    if (lane == 0 && !meta_publish<true>(meta, p.items, *p.n_items, p.claim, p.q_off, p.kv_off, p.qpad, nullptr,
                                         abort_flag, p.win.window, p.win.sinks, p.win.H_kv))
      raise_status(p.status, JFA_ERR_TIMEOUT);
   }
  } else {
    // ------------------------------------------------------------ P^T and dS^T
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // key row of the tile
    const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_addr + kColS, tP = tmem + lane_addr + kColP;
    const uint64_t k_sl2 = f2_pack(p.scale_log2, p.scale_log2);
    Ring<R> cur;
    uint32_t g = 0, acc_n = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      if (!meta_wait_warp(meta, k, abort_flag)) { ok = false; break; }
      const ItemMeta& it = meta.e[k % kMetaSlots];
      if (it.b < 0) break;
      const WinKeyUnit u = unit_of(it);
      const bool sink = u.chunk >= 0;
      const int chunk = u.chunk;
      const int j = sink ? row - meta_win(it).org : it.u0 * kBN + row;  // local key index (sinks: behind org)
      // (the entry is read in place, also at the end: fewer values live through the steps)
      auto valid = [&] { return sink ? row < meta_win(it).ns : j < it.Lk && j >= meta_win(it).pad; };
      auto row_of = [&](__nv_bfloat16* base) { return base + ((it.ko + j) * p.win.H_kv + it.h) * int64_t(kD); };
      if (u.r1 <= u.r0) {  // no query sees these keys
        if (valid()) {
          __nv_bfloat16 *dk_row = row_of(p.dk), *dv_row = row_of(p.dv);
#pragma unroll
          for (int c = 0; c < kD / 8; ++c) {
            reinterpret_cast<uint4*>(dk_row)[c] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(dv_row)[c] = make_uint4(0, 0, 0, 0);
          }
        }
        meta_release_warp(meta, k);
        continue;
      }
      const bool no_key = quarter * 32 >= (sink ? meta_win(it).ns : it.Lk - it.u0 * kBN);  // of the warp's
      const int j_diag = j - (it.Lk - it.Lq);  // first query that sees this thread's key
      for (StepWalk w(u); w.live(); w.next(), ++g) {
        const int i0 = w.t * kBM + 64 * w.half;  // local query index of column 0
        const bool pair_done = w.last_half();
        // the stage's vectors
        if (!warp_wait(&ring_full[cur.e], cur.ph, abort_flag)) { ok = false; break; }
        const float* vec = sVec + cur.e * kVecFloats + 64 * w.half;
        if (pair_done) cur.next();
        if (!warp_wait(&s_full, g & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        // columns [clo, chi] see this thread's key; the warp's lanes move both by one each
        const int clo = j_diag - i0, chi = sink ? 1 << 30 : clo + p.win.window - 1;
        const int clo0 = clo - lane, chi0 = sink ? 1 << 30 : chi - lane;  // lane 0's
        const bool hidden = no_key || clo0 > 63 || (!sink && chi0 + 31 < 0);
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
          if (clo0 + 31 > 0 || chi0 < 63) {
            const uint32_t bits[2] = {low_bits(chi + 1) & ~low_bits(clo), low_bits(chi - 31) & ~low_bits(clo - 32)};
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(bits[c >> 5] & (1u << (c & 31)))) x[c] = -INFINITY;
          }
          const uint64_t* nl = reinterpret_cast<const uint64_t*>(vec);
#pragma unroll
          for (int c2 = 0; c2 < 32; ++c2) {
            f2_unpack(f2_fma(f2_pack(x[2 * c2], x[2 * c2 + 1]), k_sl2, nl[c2]), x[2 * c2], x[2 * c2 + 1]);
            x[2 * c2] = ex2_approx(x[2 * c2]);
            x[2 * c2 + 1] = ex2_approx(x[2 * c2 + 1]);
            pk[c2] = pack_bf16x2(x[2 * c2], x[2 * c2 + 1]);
          }
          tmem_st32(tS, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full);
          if (!warp_wait(&dp_full, g & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint64_t* nd = reinterpret_cast<const uint64_t*>(vec + kBM);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t r[32];
            tmem_ld32(tP + 32 * half, r);
            tmem_ld_wait();
#pragma unroll
            for (int c2 = 0; c2 < 16; ++c2) {  // dS^T = P^T o (dP^T - D)
              const int c = 32 * half + 2 * c2;
              float d0, d1;
              f2_unpack(f2_mul(f2_pack(x[c], x[c + 1]),
                               f2_add(f2_pack(__uint_as_float(r[2 * c2]), __uint_as_float(r[2 * c2 + 1])), nd[c >> 1])),
                        d0, d1);
              pk[c >> 1] = pack_bf16x2(d0, d1);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = 0u;
          tmem_st32(tS, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full);
          if (!warp_wait(&dp_full, g & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
        }
        tmem_st32(tP, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ds_full);
      }
      if (!ok) break;
      // ---- the finished rows: dV, then dK
      if (!warp_wait(&acc_full, acc_n & 1, abort_flag)) { ok = false; break; }
      ++acc_n;
      tc_fence_after();
      const bool stored = valid();
      float* part = nullptr;
      if (sink)
        part = p.spart + ((sink_slot0(it.qp / kBM, it.b, p.group) * p.win.H_kv +
                           int64_t(it.h) * win_sink_chunks(it.Lq, meta_win(it), p.group) + chunk) *
                              2 * p.win.sinks + row) * int64_t(kD);
      __nv_bfloat16 *dk_row = row_of(p.dk), *dv_row = row_of(p.dv);
      meta_release_warp(meta, k);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int c0 = 0; c0 < kD; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(tmem + lane_addr + (t ? kColDk : kColDv) + c0, r);
          tmem_ld_wait();
          if (!stored) continue;
          if (sink) {  // fp32 partial sums, dK in front of dV
            uint4* o = reinterpret_cast<uint4*>(part + (t ? 0 : p.win.sinks * kD) + c0);
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c] = make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
          } else {
            store_row(r, t ? p.scale : 1.f, (t ? dk_row : dv_row) + c0);
          }
        }
      }
      tc_fence_before();
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kWinTmemCols);
}

}  // namespace

cudaError_t launch_win_dkdv64(const Problem& pr, const WinPlanMaps& maps, void* ws, const WsLayout& L, void* dk, void* dv,
                              int num_sms, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(w);
  WinDkdvParams p;
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
  p.sink_rows = sink_rows(pr.win.sinks);
  p.items = reinterpret_cast<const WorkItem*>(w + L.dkv);
  p.n_items = &hdr->n_dkv;
  p.claim = &hdr->claim_dkv;
  p.status = &hdr->status;
  p.wait_ns = &hdr->wait_ns[2];
  p.lse2 = reinterpret_cast<const float*>(w + L.lse2);
  p.delta = reinterpret_cast<const float*>(w + L.delta);
  p.qpad_cap = L.qpad_cap;
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.spart = reinterpret_cast<float*>(w + L.spart);
  const cudaError_t e = cudaFuncSetAttribute(win_dkdv64_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDkdvSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(win_dkdv64_kernel, dim3(kWinCtasPerSm * num_sms), dim3(kWinThreads), kDkdvSmemBytes, stream,
                    maps.tmpl[kMapQ], maps.tmpl[kMapDO], maps.tmpl[kMapK], maps.tmpl[kMapV], p);
}

}  // namespace jfa
