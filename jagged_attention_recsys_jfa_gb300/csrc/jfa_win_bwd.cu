// Windowed jagged attention backward for sm_103a: the gradients of the windowed call (jfa_win.cu,
// include/jfa.h) in the split scheme of the plain call's (jfa_bwd.cu), whose formulas, warp roles,
// memory plan and pipelines the two passes here share (d = 128; the passes for d = 64, with the same
// items, are kernels of two CTAs per SM: jfa_win_dkdv.cu, jfa_win_dq.cu):
//
//   dK/dV pass   one item per (sequence, key/value head, key tile of the window part), summed over
//                the query tiles that its keys' windows reach, of every query head of the group;
//                further items take the sinks, 16 query tiles each, and leave fp32 partial sums
//   dQ pass      one item per (sequence, query head, query tile): the sinks, then the key tiles
//                of the window part that its rows' windows reach
//   join         adds up the sinks' partial sums in a fixed order
//
// Kernels of their own, not variants of the plain passes' source: apart, the windowed training step
// takes 773 us, 13 less (64 long-tailed sequences of up to 16384 tokens, d = 128, 8 query and
// 4 key/value heads, window 512, 16 sinks) and the plain dK/dV pass keeps its 0.699 ms (0.714 with
// the window's branches in the code it shared).  Of the 773 the dK/dV pass is 298, dQ 235, forward
// 154, preprocess 50, join 10; the floor of the step's products is 190.
// P and dS are rounded to bf16 as operands (at most 2^-8 relative a term), and D = rowsum(dO o out) is
// formed from the bf16 out that the forward wrote, as in the plain call; sums are fp32.
// Bound by the tensor pipe with its operands and results in TMEM (4150 cycles per 128 x 128 pair of
// the dK/dV pass, as in the plain call).
#include <cuda_bf16.h>

#include "jfa_bwd.cuh"

namespace jfa {
namespace {

// The D accumulator columns of this thread's TMEM lane as fp32 to its own row (16-byte
// aligned); arrives on `empty` as soon as the last columns are in registers.
template <int D>
__device__ __forceinline__ void drain_row_f32(uint32_t taddr, float* dst, bool valid, uint64_t* empty) {
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + c0, r);
    tmem_ld_wait();
    if (c0 + 32 == D) {
      tc_fence_before();
      mbar_arrive(empty);
    }
    if (valid) {
#pragma unroll
      for (int c = 0; c < 32; c += 4)
        *reinterpret_cast<uint4*>(dst + c0 + c) = make_uint4(r[c], r[c + 1], r[c + 2], r[c + 3]);
    }
  }
}

// ================================================================== dK / dV pass
// Ring of single tiles, filled dO_i, Q_i per query tile in the order of the item's pairs (query
// head by query head); K and V, or the sinks' rows of them, stay for the whole item.
__device__ __forceinline__ WinKeyUnit key_unit(const BwdParams& p, const ItemMeta& m, int kt) {
  return win_key_unit(kt, m.Lq, meta_win(m), p.win.window, p.group);
}
__device__ __forceinline__ int count_of(const WinKeyUnit& u) { return u.r1 - u.r0; }
__global__ void __launch_bounds__(kThreadsDkdv, 1) win_dkdv_kernel(const BwdParams p) {
  constexpr int D = 128;
  using C = BwdCfg<D>;
  constexpr int R = C::kRingDkdv;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTileBytes;
  uint8_t* sRing = smem + 2 * C::kTileBytes;
  float* sVec = reinterpret_cast<float*>(sRing + R * C::kTileBytes);  // [kVecSlots][2][128]: lse2, D

  // dV and dK hand over to the epilogue separately: dV(last) completes one MMA group
  // before dK(last), and the next key tile's dV(0) only needs dV stored, not dK.
  __shared__ uint64_t kv_full, kv_empty, st_full, dpt_full, p_full, ds_full, mma_done;
  __shared__ uint64_t dv_full, dv_empty, dk_full, dk_empty;
  __shared__ uint64_t ring_full[R], ring_empty[R];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ MetaRing meta;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    mbar_init(&kv_full, 1);
    mbar_init(&kv_empty, 1);
    mbar_init(&st_full, 1);
    mbar_init(&dpt_full, 1);
    mbar_init(&p_full, 256);
    mbar_init(&ds_full, 256);
    mbar_init(&dv_full, 1);
    mbar_init(&dv_empty, 128);
    mbar_init(&dk_full, 1);
    mbar_init(&dk_empty, 128);
    mbar_init(&mma_done, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(&ring_full[i], 1);
      mbar_init(&ring_empty[i], 1);
    }
    meta_init(meta, p.wait_ns, 3 + (kThreadsDkdv / 32 - kFirstComputeWarp));
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();  // the planner's lists and maps, the previous kernels' outputs
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int n_items = *p.n_items;
  volatile int* abort_flag = &abort_sh;

  if (warp < kFirstComputeWarp) {
   setmaxnreg_dec<kRegsLoadDkdv>();
   if (warp == 2) {
    // ------------------------------------------------------------ K/V loader
    // Its own warp, so a key tile's K/V load starts as soon as the previous tile's last
    // dP^T MMA frees the buffers, whatever the ring producer is waiting on.
    if (lane == 0) {
      uint32_t item_n = 0, tn = 0;
      int acq_b = -1, acq_s = -1;  // sequences whose maps (sink maps) this thread has acquired
      bool ok = true;
      uint32_t item_k = 0;
      for (; ok; ++item_k) {
        if (!meta_wait(meta, item_k, abort_flag)) { ok = false; break; }
        const ItemMeta& wi = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
        if (wi.b < 0) break;  // end of this CTA's items
        acquire_seq_maps(p.maps, wi.b, kMapK, kMapV, acq_b, false);
        if (p.win.sinks > 0) acquire_seq_maps(p.smaps, wi.b, kMapK, kMapV, acq_s, false);
        for (int kt = wi.u0; kt < wi.u1 && ok; ++kt) {
          const WinKeyUnit ku = key_unit(p, wi, kt);
          if (count_of(ku) == 0) continue;
          const bool sink = ku.chunk >= 0;
          const CUtensorMap* maps = sink ? p.smaps : p.maps;
          const int skip = !sink ? meta_win(wi).skip : 0;
          const TileMap mk = win_tile_map(maps, kMapK, wi.b, sink ? 0 : kt, kBN, skip);
          const TileMap mv = win_tile_map(maps, kMapV, wi.b, sink ? 0 : kt, kBN, skip);
          if (!mbar_wait(&kv_empty, (item_n & 1) ^ 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
          trace_event(p.trace, kTraceLoader, tn, 1);
          mbar_arrive_expect_tx(&kv_full, sink ? uint32_t(p.sink_rows) * D * 4 : 2u * C::kTileBytes);
          load_tile<D>(sK, mk.map, &kv_full, wi.h * D, mk.y);
          load_tile<D>(sV, mv.map, &kv_full, wi.h * D, mv.y);
          ++item_n;
          // the key tile of this CTA's next item into L2 meanwhile (at d = 128, long-tailed batch:
          // 342 -> 334 us)
          {
            const ItemMeta* wn = meta_peek_next(meta, item_k);
            if (wn && wn->u0 * kBN < wn->Lk) {
              acquire_seq_maps(p.maps, wn->b, kMapK, kMapV, acq_b, true);
              win_prefetch_tile<D / 64>(p.maps, kMapK, wn->b, wn->u0, wn->h * D, meta_win(*wn).skip);
              win_prefetch_tile<D / 64>(p.maps, kMapV, wn->b, wn->u0, wn->h * D, meta_win(*wn).skip);
            }
          }
        }
        if (ok) meta_release(meta, item_k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      if (item_n > 0) drain_wait(&kv_full, (item_n - 1) & 1);
    }
   } else if (warp == 0) {
    // ------------------------------------------------------------ dO / Q ring producer
    if (lane == 0) {
      uint32_t ring_n = 0, qtile_n = 0, tn = 0;
      int acq_b = -1;  // sequence whose maps this thread has acquired
      bool ok = true;
      auto fill = [&](const TileMap& m, int col, const float* l2src, const float* dsrc) {
        const uint32_t e = ring_n % R, ph = (ring_n / R) & 1;
        if (!mbar_wait(&ring_empty[e], ph ^ 1, abort_flag, kWaitTimeoutNs)) return false;
        trace_event(p.trace, kTraceProducer, tn, 2);
        mbar_arrive_expect_tx(&ring_full[e], C::kTileBytes + (l2src ? 2 * kBM * 4 : 0));
        load_tile<D>(sRing + e * C::kTileBytes, m.map, &ring_full[e], col, m.y);
        if (l2src) {
          float* v = sVec + (qtile_n % C::kVecSlots) * 256;
          bulk_load(v, l2src, kBM * 4, &ring_full[e]);
          bulk_load(v + 128, dsrc, kBM * 4, &ring_full[e]);
        }
        ++ring_n;
        return true;
      };
      uint32_t item_k = 0;
      for (; ok; ++item_k) {
        if (!meta_wait(meta, item_k, abort_flag)) { ok = false; break; }
        const ItemMeta& wi = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
        if (wi.b < 0) break;  // end of this CTA's items
        acquire_seq_maps(p.maps, wi.b, kMapQ, kMapDO, acq_b, false);
        for (int kt = wi.u0; kt < wi.u1 && ok; ++kt) {
          const WinKeyUnit ku = key_unit(p, wi, kt);
          if (const ItemMeta* wnp = meta_peek_next(meta, item_k)) {
            // the first query tiles of this CTA's next item into L2 meanwhile
            const WinKeyUnit nu = key_unit(p, *wnp, wnp->u0);
            acquire_seq_maps(p.maps, wnp->b, kMapQ, kMapDO, acq_b, true);
            for (int r = 0; r < min(count_of(nu), 2); ++r) {
              const int t = nu.first + (nu.r0 + r) % nu.n, col = (wnp->h * p.group + (nu.r0 + r) / nu.n) * D;
              win_prefetch_tile<D / 64>(p.maps, kMapDO, wnp->b, t, col, 0);
              win_prefetch_tile<D / 64>(p.maps, kMapQ, wnp->b, t, col, 0);
            }
          }
          for (int i = 0; i < count_of(ku) && ok; ++i) {
            const int qt = ku.first + (ku.r0 + i) % ku.n, qh = wi.h * p.group + (ku.r0 + i) / ku.n;
            const int64_t vec0 = int64_t(qh) * p.qpad_cap + wi.qp;
            const TileMap mdo = win_tile_map(p.maps, kMapDO, wi.b, qt, kBM, 0);
            const TileMap mq = win_tile_map(p.maps, kMapQ, wi.b, qt, kBM, 0);
            if (!fill(mdo, qh * D, nullptr, nullptr)) { ok = false; break; }
            if (!fill(mq, qh * D, p.lse2 + vec0 + qt * kBM, p.delta + vec0 + qt * kBM)) {
              ok = false;
              break;
            }
            ++qtile_n;
          }
        }
        if (ok) meta_release(meta, item_k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      const uint32_t f = ring_n > uint32_t(R) ? ring_n - R : 0;
      for (uint32_t n = f; n < ring_n; ++n) drain_wait(&ring_full[n % R], (n / R) & 1);
    }
   } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdAcc = idesc_bf16_f32(128, D, false, true);
      const uint32_t aK = smem_u32(sK), aV = smem_u32(sV), aR = smem_u32(sRing);
      uint32_t ring_n = 0, item_n = 0, tile_n = 0, acc_n = 0, tn = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        if (!mbar_wait(bar, par, abort_flag, kWaitTimeoutNs)) return false;
        tc_fence_after();
        return true;
      };
      auto wait_ring = [&](uint32_t n) { return wait(&ring_full[n % R], (n / R) & 1); };
      auto ra = [&](uint32_t n) { return aR + (n % R) * C::kTileBytes; };
      // S^T (or dP^T) = A_tile(keys x D) * B_tile(queries x D)^T, both K-major
      auto mma_nt = [&](uint32_t dcol, uint32_t a, uint32_t b) {
        const uint64_t ad = sdesc_sw128(a, 16, 1024), bd = sdesc_sw128(b, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_ss(tmem + dcol, ad + o, bd + o, kIdS, kk > 0);
        }
      };
      // acc(keys x D) += X^T (TMEM bf16, keys x 128 queries, two halves kXHalf columns apart) * B(queries x D, MN-major)
      auto mma_acc = [&](uint32_t dcol, uint32_t xcol, uint32_t b, bool acc) {
        const uint64_t bd = sdesc_sw128(b, 16384, 1024);
#pragma unroll
        for (int kk = 0; kk < kBM / 16; ++kk)
          umma_ts(tmem + dcol, tmem + xcol + (kk >> 2) * C::kXHalf + (kk & 3) * 8, bd + uint32_t(kk * 2048 >> 4),
                  kIdAcc, (acc || kk > 0) ? 1u : 0u);
      };
      uint32_t item_k = 0;
      for (; ok; ++item_k) {
       if (!meta_wait(meta, item_k, abort_flag)) { ok = false; break; }
       const ItemMeta& wi = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
       if (wi.b < 0) break;  // end of this CTA's items
       for (int kt = wi.u0; kt < wi.u1 && ok; ++kt) {
        const int count = count_of(key_unit(p, wi, kt));
        if (count == 0) continue;
        if (!wait(&kv_full, item_n & 1)) { ok = false; break; }
        ++item_n;
        trace_event(p.trace, kTraceMma, tn, 10);
        const uint32_t n0 = ring_n;  // dO_i at n0 + 2i, Q_i at n0 + 2i + 1
        if (!wait_ring(n0 + 1)) { ok = false; break; }
        mma_nt(C::kColS, aK, ra(n0 + 1));
        umma_commit(&st_full);
        if (!wait_ring(n0)) { ok = false; break; }
        mma_nt(C::kColP, aV, ra(n0));
        umma_commit(&dpt_full);
        // K and V are read only by S^T and dP^T: once the last dP^T is issued the loader
        // may bring in the next key tile while dV / dK of this one still run
        if (count == 1) umma_commit(&kv_empty);
        for (int i = 0; i < count && ok; ++i) {
          const uint32_t nd = n0 + 2 * i, nq = nd + 1;
          if (!wait(&p_full, tile_n & 1)) { ok = false; break; }
          trace_event(p.trace, kTraceMma, tn, 11);
          if (i == 0 && !wait(&dv_empty, (acc_n & 1) ^ 1)) { ok = false; break; }
          mma_acc(C::kColA1, C::kColPT, ra(nd), i > 0);  // dV += P^T dO
          umma_commit(&ring_empty[nd % R]);
          if (i + 1 == count) umma_commit(&dv_full);
          trace_event(p.trace, kTraceMma, tn, 12);
          if (i + 1 < count) {
            if (!wait_ring(nq + 2)) { ok = false; break; }
            mma_nt(C::kColS, aK, ra(nq + 2));
            umma_commit(&st_full);
            trace_event(p.trace, kTraceMma, tn, 13);
          }
          if (!wait(&ds_full, tile_n & 1)) { ok = false; break; }
          trace_event(p.trace, kTraceMma, tn, 14);
          ++tile_n;
          if (i == 0 && !wait(&dk_empty, (acc_n & 1) ^ 1)) { ok = false; break; }
          mma_acc(C::kColA0, C::kColDST, ra(nq), i > 0);  // dK += dS^T Q
          umma_commit(&ring_empty[nq % R]);
          trace_event(p.trace, kTraceMma, tn, 15);
          if (i + 1 < count) {
            if (!wait_ring(nd + 2)) { ok = false; break; }
            mma_nt(C::kColP, aV, ra(nd + 2));
            umma_commit(&dpt_full);
            if (i + 2 == count) umma_commit(&kv_empty);
            trace_event(p.trace, kTraceMma, tn, 16);
          }
        }
        if (!ok) break;
        ring_n = n0 + 2 * count;
        ++acc_n;
        umma_commit(&dk_full);
       }
       if (ok) meta_release(meta, item_k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      umma_commit(&mma_done);
      drain_wait(&mma_done, 0);
    }
   } else if (warp == 3) {
    // ------------------------------------------------------------ scheduler
    if (lane == 0 && !meta_publish<true>(meta, p.items, n_items, p.claim, p.q_off, p.kv_off, p.qpad, nullptr, abort_flag,
                                         p.win.window, p.win.sinks, p.win.H_kv))
      raise_status(p.status, JFA_ERR_TIMEOUT);
   }
  } else if (warp < kFirstEpilogueWarp) {
    setmaxnreg_inc<kRegsComputeDkdv>();
    // ------------------------------------------------------------ compute warpgroups
    const int w = (warp - kFirstComputeWarp) >> 2;  // column half owned: queries [64w, 64w+64)
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // key row within the tile
    const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_addr + C::kColS + 64 * w;
    const uint32_t tP = tmem + lane_addr + C::kColP + 64 * w;
    const uint32_t tPT = tmem + lane_addr + C::kColPT + C::kXHalf * w;    // P^T, bf16
    const uint32_t tDST = tmem + lane_addr + C::kColDST + C::kXHalf * w;  // dS^T, bf16
    const float sl2 = p.scale_log2;
    uint32_t ring_n = 0, tile_n = 0, qtile_n = 0, tn = 0;
    const bool leader = (warp & 3) == 0 && lane == 0;
    bool ok = true;
    uint32_t item_k = 0;
    for (; ok; ++item_k) {
     if (!meta_wait_warp(meta, item_k, abort_flag)) { ok = false; break; }
     const ItemMeta& it = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
     if (it.b < 0) break;  // end of this CTA's items
     const int Lq = it.Lq, Lk = it.Lk;
     for (int kt = it.u0; kt < it.u1 && ok; ++kt) {
      const WinKeyUnit ku = key_unit(p, it, kt);
      const int count = count_of(ku);
      const bool sink = ku.chunk >= 0;
      const int j = sink ? row - meta_win(it).org : kt * kBN + row;  // local key index (sinks: behind org)
      if (count == 0) continue;  // rows of zeros: written by the epilogue warpgroup
      const int diag = Lk - Lq;  // key j visible to query i iff i >= j - diag
      for (int i = 0; i < count && ok; ++i) {
        const int qt = ku.first + (ku.r0 + i) % ku.n;
        // Q_i's ring slot carries this tile's lse2 / D vectors: wait for it
        const uint32_t nq = ring_n + 1;
        if (!mbar_wait(&ring_full[nq % R], (nq / R) & 1, abort_flag, kWaitTimeoutNs)) { ok = false; break; }
        ring_n += 2;
        const float* vec = sVec + (qtile_n % C::kVecSlots) * 256;
        ++qtile_n;
        const uint64_t* nlse2 = reinterpret_cast<const uint64_t*>(vec + 64 * w);  // -lse2 pairs
        const uint64_t* ndvec = reinterpret_cast<const uint64_t*>(vec + 128 + 64 * w);  // -D pairs
        if (!mbar_wait(&st_full, tile_n & 1, abort_flag, kWaitTimeoutNs)) { ok = false; break; }
        tc_fence_after();
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 20);
        const int i0 = qt * kBM + 64 * w;  // local query index of column 0 of this half
        float x[64];
        ld_cols64(tS, x);
        {
          const uint64_t k_sl2 = f2_pack(sl2, sl2);
#pragma unroll
          for (int c2 = 0; c2 < 32; ++c2)
            f2_unpack(f2_fma(f2_pack(x[2 * c2], x[2 * c2 + 1]), k_sl2, nlse2[c2]), x[2 * c2], x[2 * c2 + 1]);
        }
        const int lim = j - diag - i0;  // columns c < lim are hidden
        if (lim > 0) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < lim) x[c] = -INFINITY;
        }
        if (!sink) {
          const int hi = lim + p.win.window - 1;  // columns c > hi have moved past the key
          if (hi < 63) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c > hi) x[c] = -INFINITY;
          }
        }
#pragma unroll
        for (int c = 0; c < 64; ++c) x[c] = ex2_approx(x[c]);  // P^T
        st_bf16_64(tPT, x);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full);
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 21);
        if (!mbar_wait(&dpt_full, tile_n & 1, abort_flag, kWaitTimeoutNs)) { ok = false; break; }
        ++tile_n;
        tc_fence_after();
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 22);
        float dp[64];
        ld_cols64(tP, dp);
#pragma unroll
        for (int c2 = 0; c2 < 32; ++c2)  // dS^T = P^T o (dP^T - D)
          f2_unpack(f2_mul(f2_pack(x[2 * c2], x[2 * c2 + 1]), f2_add(f2_pack(dp[2 * c2], dp[2 * c2 + 1]), ndvec[c2])),
                    dp[2 * c2], dp[2 * c2 + 1]);
        st_bf16_64(tDST, dp);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ds_full);
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 23);
      }
      if (!ok) break;
     }
     if (__all_sync(0xffffffffu, ok)) meta_release_warp(meta, item_k);
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  } else {
    setmaxnreg_dec<kRegsEpiDkdv>();
    // ------------------------------------------------------------ epilogue warpgroup
    // Writes each key tile's dV and dK rows (this thread's TMEM lane = one key row, all D
    // columns, 32 at a time) while the compute warpgroups go on with the next key tile;
    // an accumulator is released as soon as its last columns are in registers.
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
    uint32_t acc_n = 0;
    bool ok = true;
    uint32_t item_k = 0;
    for (; ok; ++item_k) {
     if (!meta_wait_warp(meta, item_k, abort_flag)) { ok = false; break; }
     const ItemMeta& it = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
     if (it.b < 0) break;  // end of this CTA's items
     const int64_t ko = it.ko;
     const int Lq = it.Lq, Lk = it.Lk;
     for (int kt = it.u0; kt < it.u1 && ok; ++kt) {
      const WinKeyUnit ku = key_unit(p, it, kt);
      const int count = count_of(ku);
      const int j = kt * kBN + row;  // local key index
      const bool valid = j < Lk && j >= meta_win(it).pad;
      const int heads = p.win.H_kv;
      __nv_bfloat16* dk_row = p.g0 + ((ko + j) * heads + it.h) * int64_t(D);
      __nv_bfloat16* dv_row = p.g1 + ((ko + j) * heads + it.h) * int64_t(D);
      if (ku.chunk >= 0) {  // a chunk of the sinks: fp32 partial sums
        const WinSeq ws = meta_win(it);
        const int64_t slot = sink_slot0(it.qp / kBM, it.b, p.group) * p.win.H_kv +
                             int64_t(it.h) * win_sink_chunks(Lq, ws, p.group) + ku.chunk;
        float* part = p.spart + (slot * 2 * p.win.sinks + row) * int64_t(D);
        if (!mbar_wait(&dv_full, acc_n & 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
        tc_fence_after();
        drain_row_f32<D>(tmem + lane_addr + C::kColA1, part + p.win.sinks * int64_t(D), row < ws.ns, &dv_empty);
        if (!mbar_wait(&dk_full, acc_n & 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
        ++acc_n;
        tc_fence_after();
        drain_row_f32<D>(tmem + lane_addr + C::kColA0, part, row < ws.ns, &dk_empty);
        continue;
      }
      if (count == 0) {  // no query sees these keys
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          store_acc_row<32>(0, 0.f, dk_row + c0, valid, true);
          store_acc_row<32>(0, 0.f, dv_row + c0, valid, true);
        }
        continue;
      }
      if (!mbar_wait(&dv_full, acc_n & 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
      tc_fence_after();
      drain_acc_rows<D>(tmem + lane_addr + C::kColA1, 1.f, dv_row, valid, &dv_empty);
      if (!mbar_wait(&dk_full, acc_n & 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
      ++acc_n;
      tc_fence_after();
      drain_acc_rows<D>(tmem + lane_addr + C::kColA0, p.scale, dk_row, valid, &dk_empty);
     }
     if (__all_sync(0xffffffffu, ok)) meta_release_warp(meta, item_k);
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ================================================================== dQ pass
// Ring of single tiles, filled V_j, K_j per step.  The first step may be the sinks' (nz = 1), whose
// products have sink_rows keys; the others are the window part's key tiles from a on.
struct QueryUnit {
  int a, nz, nkv;
};
__device__ __forceinline__ QueryUnit query_unit(const BwdParams& p, const ItemMeta& m, int qt) {
  QueryUnit u;
  int e;
  win_kv_tiles(qt, m.Lq, meta_win(m), p.win.window, &u.a, &e);
  u.nz = win_sees_sinks(qt, m.Lq, meta_win(m)) ? 1 : 0;
  u.nkv = e - u.a + u.nz;
  return u;
}

__global__ void __launch_bounds__(kThreadsDkdv, 1) win_dq_kernel(const BwdParams p) {
  constexpr int D = 128;
  using C = BwdCfg<D>;
  constexpr int R = C::kRingDq;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sDO = smem + C::kTileBytes;
  uint8_t* sRing = smem + 2 * C::kTileBytes;

  __shared__ uint64_t qdo_full, qdo_empty, s_full, s_free, acc_full, acc_empty, mma_done;
  // dp_full / ds_full of global tile g live at index g & 1: dP(g+1) is issued before dQ(g)
  // waits for dS(g), so one warpgroup may finish tile g+1 while the other still works on
  // tile g (never further: S(g+2) waits for both warpgroups' s_free(g+1)); separate
  // barriers per tile parity keep their arrivals apart.
  __shared__ uint64_t dp_full[2], ds_full[2];
  __shared__ uint64_t ring_full[R], ring_empty[R];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ MetaRing meta;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_sh = 0;
    mbar_init(&qdo_full, 1);
    mbar_init(&qdo_empty, 1);
    mbar_init(&s_full, 1);
    mbar_init(&s_free, 256);
    mbar_init(&dp_full[0], 1);
    mbar_init(&dp_full[1], 1);
    mbar_init(&ds_full[0], 256);
    mbar_init(&ds_full[1], 256);
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, 128);
    mbar_init(&mma_done, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(&ring_full[i], 1);
      mbar_init(&ring_empty[i], 1);
    }
    meta_init(meta, p.wait_ns, 3 + (kThreadsDkdv / 32 - kFirstComputeWarp));
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();  // the planner's lists and maps, the previous kernels' outputs
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int n_items = *p.n_items;
  volatile int* abort_flag = &abort_sh;
  auto colP = [](uint32_t g) { return (g & 1) ? C::kColP1 : C::kColP; };

  if (warp < kFirstComputeWarp) {
   setmaxnreg_dec<kRegsLoadDkdv>();
   if (warp == 2) {
    // ------------------------------------------------------------ Q / dO loader
    if (lane == 0) {
      uint32_t item_n = 0, tn = 0;
      int acq_b = -1;  // sequence whose maps this thread has acquired
      bool ok = true;
      uint32_t item_k = 0;
      for (; ok; ++item_k) {
       if (!meta_wait(meta, item_k, abort_flag)) { ok = false; break; }
       const ItemMeta& wi = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
       if (wi.b < 0) break;  // end of this CTA's items
       acquire_seq_maps(p.maps, wi.b, kMapQ, kMapDO, acq_b, false);
       for (int qt = wi.u0; qt < wi.u1 && ok; ++qt) {
        if (query_unit(p, wi, qt).nkv == 0) continue;
        const TileMap mq = win_tile_map(p.maps, kMapQ, wi.b, qt, kBM, 0);
        const TileMap mdo = win_tile_map(p.maps, kMapDO, wi.b, qt, kBM, 0);
        if (!mbar_wait(&qdo_empty, (item_n & 1) ^ 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
        trace_event(p.trace, kTraceLoader, tn, 1);
        mbar_arrive_expect_tx(&qdo_full, 2 * C::kTileBytes);
        load_tile<D>(sQ, mq.map, &qdo_full, wi.h * D, mq.y);
        load_tile<D>(sDO, mdo.map, &qdo_full, wi.h * D, mdo.y);
        ++item_n;
        // pull the next query tile into L2 meanwhile: the next of this range, else the first
        // of this CTA's next item
        {
          int nb = -1, nh = 0, nt = 0;
          if (qt + 1 < wi.u1) {
            nb = wi.b, nh = wi.h, nt = qt + 1;
          } else if (const ItemMeta* wn = meta_peek_next(meta, item_k)) {
            nb = wn->b, nh = wn->h, nt = wn->u0;
          }
          if (nb >= 0) {
            const int64_t nqo = p.q_off[nb];
            acquire_seq_maps(p.maps, nb, kMapQ, kMapDO, acq_b, true);
            if (nt * kBM < int(p.q_off[nb + 1] - nqo)) {
              win_prefetch_tile<D / 64>(p.maps, kMapQ, nb, nt, nh * D, 0);
              win_prefetch_tile<D / 64>(p.maps, kMapDO, nb, nt, nh * D, 0);
            }
          }
        }
       }
       if (ok) meta_release(meta, item_k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      if (item_n > 0) drain_wait(&qdo_full, (item_n - 1) & 1);
    }
   } else if (warp == 0) {
    // ------------------------------------------------------------ V / K ring producer
    if (lane == 0) {
      uint32_t ring_n = 0, tn = 0;
      int acq_b = -1, acq_s = -1;  // sequences whose maps (sink maps) this thread has acquired
      bool ok = true;
      auto fill = [&](const TileMap& m, int col, uint32_t bytes) {
        const uint32_t e = ring_n % R, ph = (ring_n / R) & 1;
        if (!mbar_wait(&ring_empty[e], ph ^ 1, abort_flag, kWaitTimeoutNs)) return false;
        trace_event(p.trace, kTraceProducer, tn, 2);
        mbar_arrive_expect_tx(&ring_full[e], bytes);
        load_tile<D>(sRing + e * C::kTileBytes, m.map, &ring_full[e], col, m.y);
        ++ring_n;
        return true;
      };
      uint32_t item_k = 0;
      for (; ok; ++item_k) {
       if (!meta_wait(meta, item_k, abort_flag)) { ok = false; break; }
       const ItemMeta& wi = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
       if (wi.b < 0) break;  // end of this CTA's items
       const int col = wi.h / p.group * D;  // first column of the key/value head
       acquire_seq_maps(p.maps, wi.b, kMapK, kMapV, acq_b, false);
       if (p.win.sinks > 0) acquire_seq_maps(p.smaps, wi.b, kMapK, kMapV, acq_s, false);
       for (int qt = wi.u0; qt < wi.u1 && ok; ++qt) {
        const QueryUnit qu = query_unit(p, wi, qt);
        const int nkv = qu.nkv;
        if (const ItemMeta* wnp = meta_peek_next(meta, item_k)) {
          // the first key tiles of this CTA's next item into L2 meanwhile
          const QueryUnit nu = query_unit(p, *wnp, wnp->u0);
          const int skip = meta_win(*wnp).skip;
          acquire_seq_maps(p.maps, wnp->b, kMapK, kMapV, acq_b, true);
          for (int t = nu.a; t < nu.a + 2 && t * kBN < wnp->Lk; ++t) {
            win_prefetch_tile<D / 64>(p.maps, kMapV, wnp->b, t, wnp->h / p.group * D, skip);
            win_prefetch_tile<D / 64>(p.maps, kMapK, wnp->b, t, wnp->h / p.group * D, skip);
          }
        }
        for (int jt = 0; jt < nkv && ok; ++jt) {
          const bool sink = jt < qu.nz;
          const CUtensorMap* maps = sink ? p.smaps : p.maps;
          const int kt = sink ? 0 : qu.a + jt - qu.nz;
          const int skip = !sink ? meta_win(wi).skip : 0;
          const TileMap mv = win_tile_map(maps, kMapV, wi.b, kt, kBN, skip);
          const TileMap mk = win_tile_map(maps, kMapK, wi.b, kt, kBN, skip);
          const uint32_t bytes = sink ? uint32_t(p.sink_rows) * D * 2 : uint32_t(C::kTileBytes);
          if (!fill(mv, col, bytes) || !fill(mk, col, bytes)) { ok = false; break; }
        }
       }
       if (ok) meta_release(meta, item_k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      const uint32_t f = ring_n > uint32_t(R) ? ring_n - R : 0;
      for (uint32_t n = f; n < ring_n; ++n) drain_wait(&ring_full[n % R], (n / R) & 1);
    }
   } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdAcc = idesc_bf16_f32(128, D, false, true);
      const uint32_t aQ = smem_u32(sQ), aDO = smem_u32(sDO), aR = smem_u32(sRing);
      uint32_t ring_n = 0, item_n = 0, tile_n = 0, acc_n = 0, tn = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        if (!mbar_wait(bar, par, abort_flag, kWaitTimeoutNs)) return false;
        tc_fence_after();
        return true;
      };
      auto wait_ring = [&](uint32_t n) { return wait(&ring_full[n % R], (n / R) & 1); };
      auto ra = [&](uint32_t n) { return aR + (n % R) * C::kTileBytes; };
      // S (dp = false: Q K^T) or dP (dp = true: dO V^T) of a query tile and the key tile at b
      auto mma_nt = [&](uint32_t dcol, bool dp, uint32_t b, uint32_t id) {
        const uint64_t ad = sdesc_sw128(dp ? aDO : aQ, 16, 1024), bd = sdesc_sw128(b, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_ss(tmem + dcol, ad + o, bd + o, id, kk > 0);
        }
      };
      uint32_t item_k = 0;
      for (; ok; ++item_k) {
       if (!meta_wait(meta, item_k, abort_flag)) { ok = false; break; }
       const ItemMeta& wi = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
       if (wi.b < 0) break;  // end of this CTA's items
       for (int qt = wi.u0; qt < wi.u1 && ok; ++qt) {
        const QueryUnit qu = query_unit(p, wi, qt);
        const int nkv = qu.nkv;
        if (nkv == 0) continue;
        const uint32_t id0 = qu.nz ? idesc_bf16_f32(128, p.sink_rows, false, false) : kIdS;  // the first step's
        if (!wait(&qdo_full, item_n & 1)) { ok = false; break; }
        ++item_n;
        trace_event(p.trace, kTraceMma, tn, 10);
        const uint32_t n0 = ring_n;  // V_j at n0 + 2j, K_j at n0 + 2j + 1
        if (!wait_ring(n0 + 1)) { ok = false; break; }
        mma_nt(C::kColS, false, ra(n0 + 1), id0);
        umma_commit(&s_full);
        if (!wait_ring(n0)) { ok = false; break; }
        mma_nt(colP(tile_n), true, ra(n0), id0);
        umma_commit(&dp_full[tile_n & 1]);
        umma_commit(&ring_empty[n0 % R]);
        // Q and dO are read only by S and dP: once the last dP is issued the loader may
        // bring in the next query tile while dQ of this one still runs (at d = 64 the compute
        // warpgroups free them after copying them into TMEM)
        if (nkv == 1) umma_commit(&qdo_empty);
        for (int jt = 0; jt < nkv && ok; ++jt) {
          const uint32_t g = tile_n;  // global tile index
          const uint32_t nv = n0 + 2 * jt, nk = nv + 1;
          if (jt + 1 < nkv) {
            // next S once the warpgroups hold this S in registers; next dP into the
            // other buffer (its dS was consumed by the dQ MMA issued before)
            if (!wait(&s_free, g & 1)) { ok = false; break; }
            trace_event(p.trace, kTraceMma, tn, 11);
            if (!wait_ring(nk + 2)) { ok = false; break; }
            mma_nt(C::kColS, false, ra(nk + 2), kIdS);
            umma_commit(&s_full);
            trace_event(p.trace, kTraceMma, tn, 12);
            if (!wait_ring(nv + 2)) { ok = false; break; }
            mma_nt(colP(g + 1), true, ra(nv + 2), kIdS);
            umma_commit(&dp_full[(g + 1) & 1]);
            umma_commit(&ring_empty[(nv + 2) % R]);
            if (jt + 2 == nkv) umma_commit(&qdo_empty);
            trace_event(p.trace, kTraceMma, tn, 13);
          }
          if (!wait(&ds_full[g & 1], (g >> 1) & 1)) { ok = false; break; }
          trace_event(p.trace, kTraceMma, tn, 14);
          ++tile_n;
          if (jt == 0 && !wait(&acc_empty, (acc_n & 1) ^ 1)) { ok = false; break; }
          // dQ += dS (TMEM, queries x keys) * K (keys x D, MN-major)
          const uint64_t kd = sdesc_sw128(ra(nk), 16384, 1024);
          if (jt < qu.nz) {
#pragma unroll 1
            for (int kk = 0; kk < p.sink_rows / 16; ++kk)
              umma_ts(tmem + C::kColDQ, tmem + colP(g) + (kk >> 2) * 64 + (kk & 3) * 8, kd + uint32_t(kk * 2048 >> 4),
                      kIdAcc, kk > 0 ? 1u : 0u);
          } else
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            umma_ts(tmem + C::kColDQ, tmem + colP(g) + (kk >> 2) * 64 + (kk & 3) * 8, kd + uint32_t(kk * 2048 >> 4),
                    kIdAcc, (jt > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&ring_empty[nk % R]);
          trace_event(p.trace, kTraceMma, tn, 15);
        }
        if (!ok) break;
        // the last tile's s_free arrival has no consumer above: take it here
        if (!wait(&s_free, (tile_n - 1) & 1)) { ok = false; break; }
        ring_n = n0 + 2 * nkv;
        ++acc_n;
        umma_commit(&acc_full);
       }
       if (ok) meta_release(meta, item_k);
      }
      if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
      umma_commit(&mma_done);
      drain_wait(&mma_done, 0);
    }
   } else if (warp == 3) {
    // ------------------------------------------------------------ scheduler
    if (lane == 0 && !meta_publish<true>(meta, p.items, n_items, p.claim, p.q_off, p.kv_off, p.qpad, nullptr, abort_flag,
                                         p.win.window, p.win.sinks, p.H))
      raise_status(p.status, JFA_ERR_TIMEOUT);
   }
  } else if (warp < kFirstEpilogueWarp) {
    setmaxnreg_inc<kRegsComputeDkdv>();
    const int w = (warp - kFirstComputeWarp) >> 2;  // key columns [64w, 64w+64)
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_addr + C::kColS + 64 * w;
    const float sl2 = p.scale_log2;
    uint32_t tile_n = 0, tn = 0;
    const bool leader = (warp & 3) == 0 && lane == 0;
    bool ok = true;
    uint32_t item_k = 0;
    for (; ok; ++item_k) {
     if (!meta_wait_warp(meta, item_k, abort_flag)) { ok = false; break; }
     const ItemMeta& it = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
     if (it.b < 0) break;  // end of this CTA's items
     const int Lq = it.Lq, Lk = it.Lk;
     const int64_t vec0 = int64_t(it.h) * p.qpad_cap + it.qp;
     for (int qt = it.u0; qt < it.u1 && ok; ++qt) {
      const QueryUnit qu = query_unit(p, it, qt);
      const int nkv = qu.nkv;
      const int i = qt * kBM + row;
      if (nkv == 0) continue;  // rows of zeros: written by the epilogue warpgroup
      // padded per-query vectors (stored negated): 0 past the sequence end, -inf for rows
      // that see no key
      const float nl2 = __ldg(p.lse2 + vec0 + i);
      const uint64_t k_nl2 = f2_pack(nl2, nl2);
      const float nd = __ldg(p.delta + vec0 + i);
      const uint64_t k_nd = f2_pack(nd, nd);
      const int diag = Lk - Lq;
      for (int jt = 0; jt < nkv && ok; ++jt) {
        if (!mbar_wait(&s_full, tile_n & 1, abort_flag, kWaitTimeoutNs)) { ok = false; break; }
        tc_fence_after();
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 20);
        const bool sink = jt < qu.nz;
        // local key index of column 0 of this half (sinks: behind org)
        const int j0 = (sink ? -meta_win(it).org : (qu.a + jt - qu.nz) * kBN) + 64 * w;
        const int n_real = sink ? meta_win(it).ns - 64 * w : Lk - j0;  // columns >= n_real hold no key
        float x[64];
        ld_cols64(tS, x);
        tc_fence_before();
        mbar_arrive(&s_free);
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 21);
        {
          const uint64_t k_sl2 = f2_pack(sl2, sl2);
#pragma unroll
          for (int c2 = 0; c2 < 32; ++c2)
            f2_unpack(f2_fma(f2_pack(x[2 * c2], x[2 * c2 + 1]), k_sl2, k_nl2), x[2 * c2], x[2 * c2 + 1]);
        }
        const int lim = i + diag - j0;  // columns c > lim are hidden
        if (lim < 63) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > lim) x[c] = -INFINITY;
        }
        if (!sink) {
          // columns c < clo are behind the window, or hold no key
          const int clo = max(lim - p.win.window + 1, meta_win(it).pad - j0);
          if (clo > 0) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c < clo) x[c] = -INFINITY;
          }
        }
        if (n_real < 64) {
          // padded keys (zero rows) would score exp2(-lse): keep them out of dS so it stays finite
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= n_real) x[c] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 64; ++c) x[c] = ex2_approx(x[c]);  // P
        const uint32_t g = tile_n;
        const uint32_t tP = tmem + lane_addr + colP(g) + 64 * w;
        if (!mbar_wait(&dp_full[g & 1], (g >> 1) & 1, abort_flag, kWaitTimeoutNs)) { ok = false; break; }
        ++tile_n;
        tc_fence_after();
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 22);
        float dp[64];
        ld_cols64(tP, dp);
#pragma unroll
        for (int c2 = 0; c2 < 32; ++c2)  // dS = P o (dP - D)
          f2_unpack(f2_mul(f2_pack(x[2 * c2], x[2 * c2 + 1]), f2_add(f2_pack(dp[2 * c2], dp[2 * c2 + 1]), k_nd)),
                    dp[2 * c2], dp[2 * c2 + 1]);
        st_bf16_64(tP, dp);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ds_full[g & 1]);
        if (leader) trace_event(p.trace, kTraceCompute0 + w, tn, 23);
      }
      if (!ok) break;
     }
     if (__all_sync(0xffffffffu, ok)) meta_release_warp(meta, item_k);
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  } else {
    setmaxnreg_dec<kRegsEpiDkdv>();
    // ------------------------------------------------------------ epilogue warpgroup
    // Writes each query tile's dQ rows (this thread's TMEM lane = one query row, all D
    // columns, 32 at a time) while warpgroups 1 and 2 start the next query tile; the
    // accumulator is released as soon as its last columns are in registers.
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
    uint32_t acc_n = 0;
    bool ok = true;
    uint32_t item_k = 0;
    for (; ok; ++item_k) {
     if (!meta_wait_warp(meta, item_k, abort_flag)) { ok = false; break; }
     const ItemMeta& it = meta.e[item_k % kMetaSlots];  // read in place, freed after the item
     if (it.b < 0) break;  // end of this CTA's items
     const int Lq = it.Lq;
     for (int qt = it.u0; qt < it.u1 && ok; ++qt) {
      const int i = qt * kBM + row;
      const bool valid = i < Lq;
      __nv_bfloat16* dq_row = p.g0 + ((it.qo + i) * p.H + it.h) * int64_t(D);
      if (query_unit(p, it, qt).nkv == 0) {  // the query tile sees no key
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) store_acc_row<32>(0, 0.f, dq_row + c0, valid, true);
        continue;
      }
      if (!mbar_wait(&acc_full, acc_n & 1, abort_flag, meta.wait_ns, kWaitTimeoutNs)) { ok = false; break; }
      ++acc_n;
      tc_fence_after();
      drain_acc_rows<D>(tmem + lane_addr + C::kColDQ, p.scale, dq_row, valid, &acc_empty);
     }
     if (__all_sync(0xffffffffu, ok)) meta_release_warp(meta, item_k);
    }
    if (!ok) raise_status(p.status, JFA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ================================================================== the sinks' gradients (window)
// dK and dV of each sequence's sinks from the dK/dV pass's partial sums, added in chunk order,
// and zero rows for the keys between the sinks and the window part, which no query sees.
// Memory bound and small: the partials are sinks x d x 2 floats per 16 query tiles.  Every
// sequence gets the same number of warps.
struct JoinParams {
  const int64_t *q_off, *kv_off, *qpad;
  const int* planned;  // 0 with malformed offsets: nothing to do
  const float* spart;
  int B, group;
  WindowSpec win;
  float scale;
  __nv_bfloat16 *dk, *dv;
};

template <int D>
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (*p.planned == 0) return;
  const int lane = threadIdx.x & 31;
  const int warps = int(gridDim.x * blockDim.x) >> 5, warp = int(blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int per_seq = warps / p.B > 0 ? warps / p.B : 1;
  const int Hkv = p.win.H_kv;
  for (int b = warp / per_seq; b < p.B; b += warps / per_seq) {
    const int Lq = int(p.q_off[b + 1] - p.q_off[b]);
    const int64_t ko = p.kv_off[b];
    const WinSeq ws = win_seq(Lq, int(p.kv_off[b + 1] - ko), p.win.window, p.win.sinks, kBN);
    const int chunks = win_sink_chunks(Lq, ws, p.group);
    const int64_t slot0 = sink_slot0(p.qpad[b] / kBM, b, p.group) * Hkv;
    const int64_t row_vecs = int64_t(Hkv) * D / 8;  // 16-byte pieces of a key row, all heads
    const int64_t first = int64_t(warp % per_seq) * 32 + lane, step = int64_t(per_seq) * 32;
    uint4* dk = reinterpret_cast<uint4*>(p.dk + ko * Hkv * D);
    uint4* dv = reinterpret_cast<uint4*>(p.dv + ko * Hkv * D);
    for (int64_t i = first; i < ws.ns * row_vecs; i += step) {
      const int j = int(i / row_vecs), h = int(i % row_vecs) / (D / 8), c = int(i % (D / 8)) * 8;
      const float* part = p.spart + ((slot0 + int64_t(h) * chunks) * 2 * p.win.sinks + j) * D + c;
      float sk[8] = {}, sv[8] = {};
      for (int k = 0; k < chunks; ++k, part += int64_t(2) * p.win.sinks * D) {
        const float* pv = part + int64_t(p.win.sinks) * D;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 a = __ldg(reinterpret_cast<const float4*>(part) + q), v = __ldg(reinterpret_cast<const float4*>(pv) + q);
          sk[4 * q] += a.x;
          sk[4 * q + 1] += a.y;
          sk[4 * q + 2] += a.z;
          sk[4 * q + 3] += a.w;
          sv[4 * q] += v.x;
          sv[4 * q + 1] += v.y;
          sv[4 * q + 2] += v.z;
          sv[4 * q + 3] += v.w;
        }
      }
      dk[i] = make_uint4(pack_bf16x2(sk[0] * p.scale, sk[1] * p.scale), pack_bf16x2(sk[2] * p.scale, sk[3] * p.scale),
                         pack_bf16x2(sk[4] * p.scale, sk[5] * p.scale), pack_bf16x2(sk[6] * p.scale, sk[7] * p.scale));
      dv[i] = make_uint4(pack_bf16x2(sv[0], sv[1]), pack_bf16x2(sv[2], sv[3]), pack_bf16x2(sv[4], sv[5]),
                         pack_bf16x2(sv[6], sv[7]));
    }
    for (int64_t i = ws.ns * row_vecs + first; i < (ws.org + ws.pad) * row_vecs; i += step) {
      dk[i] = make_uint4(0, 0, 0, 0);
      dv[i] = make_uint4(0, 0, 0, 0);
    }
  }
}

}  // namespace

cudaError_t launch_win_dkdv(const Problem& pr, const WinPlanMaps& maps, void* ws, const WsLayout& L, void* dk, void* dv,
                            int num_sms, cudaStream_t stream) {
  if (pr.d == 64) return launch_win_dkdv64(pr, maps, ws, L, dk, dv, num_sms, stream);
  BwdParams bp = make_params(pr, nullptr, ws, L, kPassDkdv);
  bp.g0 = static_cast<__nv_bfloat16*>(dk);
  bp.g1 = static_cast<__nv_bfloat16*>(dv);
  return launch_dkdv_k(win_dkdv_kernel, BwdCfg<128>::kSmemDkdv, num_sms, bp, stream);
}

cudaError_t launch_win_dq(const Problem& pr, const WinPlanMaps& maps, void* ws, const WsLayout& L, void* dq, int num_sms,
                          cudaStream_t stream) {
  if (pr.d == 64) return launch_win_dq64(pr, maps, ws, L, dq, num_sms, stream);
  BwdParams bp = make_params(pr, nullptr, ws, L, kPassDq);
  bp.g0 = static_cast<__nv_bfloat16*>(dq);
  return launch_dkdv_k(win_dq_kernel, BwdCfg<128>::kSmemDq, num_sms, bp, stream);
}

cudaError_t launch_win_join(const Problem& pr, void* ws, const WsLayout& L, void* dk, void* dv, int num_sms,
                            cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  JoinParams jp;
  jp.q_off = pr.q_off;
  jp.kv_off = pr.kv_off;
  jp.qpad = reinterpret_cast<const int64_t*>(w + L.qpad);
  jp.planned = &reinterpret_cast<const WsHeader*>(w)->planned;
  jp.spart = reinterpret_cast<const float*>(w + L.spart);
  jp.B = pr.B;
  jp.group = pr.H / pr.win.H_kv;
  jp.win = pr.win;
  jp.scale = pr.scale;
  jp.dk = static_cast<__nv_bfloat16*>(dk);
  jp.dv = static_cast<__nv_bfloat16*>(dv);
  return pr.d == 128 ? launch_pdl(join_kernel<128>, dim3(2 * num_sms), dim3(256), 0, stream, jp)
                     : launch_pdl(join_kernel<64>, dim3(2 * num_sms), dim3(256), 0, stream, jp);
}

}  // namespace jfa
