// The paged key/value cache: appending (with the position rotation applied on the way) and
// the attention of one new token per sequence over it.
//
// Layout.  k and v are bf16 [num_pages][H_kv][page_size][d]: the page_size rows of one
// (page, head) are contiguous, so a tile of one head is a few whole TMA boxes.  Token p of
// sequence b lives in row p % page_size of page page_table[b][p / page_size].
#include <cuda_bf16.h>

#include "jfa_internal.h"
#include "sm100_ptx.cuh"

namespace jfa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void raise_status(int* status, int code) { atomicCAS(status, 0, code); }

// ================================================================== append
// Pair i of a rotated head turns by p * f_i radians at position p:
//   half split   (x_i, x_{i + r/2})  ->  (x_i cos - x_{i+r/2} sin, x_{i+r/2} cos + x_i sin)
//   interleaved  (x_2i, x_2i+1) likewise
// The angle is kept as a fraction of a turn in 64-bit fixed point, turn_i = f_i / 2 pi mod 1
// in units of 2^-64 (on the host, in twice double precision, to one unit for |f_i| up to 2^20):
// p * turn_i wraps modulo one turn exactly and is off by 2^-33 of a turn at p = 2^31.  Its
// distance to the nearest quarter turn is what becomes fp32, so that a sine or cosine next to
// zero keeps its relative precision: both are good to 2^-22 of their value and 2^-32 of a turn.
// (In fp32 the product p * f_i alone is off by 0.06 rad at p = 10^6.)  Memory bound: every row
// is read once and written once.
struct AppendParams {
  const __nv_bfloat16 *k, *v, *q;              // new rows; q may be nullptr
  int64_t k_stride, v_stride, q_stride;        // elements between tokens
  const int64_t* offsets;                      // [B+1]
  int64_t total;                               // rows of k, v (and q)
  __nv_bfloat16 *k_cache, *v_cache;
  const int32_t* page_table;
  const int32_t* lengths;                      // tokens cached before the call
  int32_t* lengths_out;                        // nullptr, or tokens cached after it (may be `lengths`)
  __nv_bfloat16 *q_out, *k_out;                // rotated rows, contiguous; k_out may be nullptr
  int64_t num_pages;
  int B, H, Hkv, page_size, max_pages;         // H: query heads, 0 without q
  int rot;                                     // leading dims of each head that are rotated (0: none)
  int interleaved;
  int warps_per_token;                         // 1, 2, 4 or 8
  int* status;
  unsigned* done;                              // CTAs that have read `lengths` (left at 0)
  uint64_t turn[64];
};

constexpr int kAppendThreads = 256;
// Rows per lane in flight (841 MB of prompts, d = 128: 1 row 168 us, 2 rows 154, 3 rows 158, 6 rows
// 180; with 2, five CTAs per SM 150).
constexpr int kAppendBatch = 2;

// The last b with offsets[b] <= t (offsets non-decreasing, offsets[0] <= t), by the whole
// warp: 32 probes per step, so B = 1024 takes two dependent loads instead of ten.
__device__ __forceinline__ int find_sequence(const int64_t* offsets, int B, int64_t t, int lane) {
  int lo = 0, n = B;  // candidates lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int probe = lo + lane * step;
    const bool le = lane * step < n && __ldg(offsets + probe) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    const int left = n - last * step;
    lo += last * step;
    n = left < step ? left : step;
  }
  return lo;
}

__device__ __forceinline__ uint32_t rot_lo(uint32_t a, uint32_t b, const float2& c0, const float2& c1) {
  return pack_bf16x2(bf16lo(a) * c0.x - bf16lo(b) * c0.y, bf16hi(a) * c1.x - bf16hi(b) * c1.y);
}
__device__ __forceinline__ uint32_t rot_hi(uint32_t a, uint32_t b, const float2& c0, const float2& c1) {
  return pack_bf16x2(bf16lo(b) * c0.x + bf16lo(a) * c0.y, bf16hi(b) * c1.x + bf16hi(a) * c1.y);
}
__device__ __forceinline__ uint32_t rot_pair(uint32_t a, const float2& c) {
  return pack_bf16x2(bf16lo(a) * c.x - bf16hi(a) * c.y, bf16hi(a) * c.x + bf16lo(a) * c.y);
}

// Whether `n` new tokens of sequence b behind its `len` cached ones all have a page.
__device__ __forceinline__ bool stores_all(const AppendParams& p, int b, int len, int64_t n) {
  if (len < 0 || len + n > int64_t(p.max_pages) * p.page_size) return n == 0 && len >= 0;
  for (int64_t pos = len; pos < len + n; pos += p.page_size - pos % p.page_size) {
    const int page = p.page_table[int64_t(b) * p.max_pages + pos / p.page_size];
    if (page < 0 || page >= p.num_pages) return false;
  }
  return true;
}

// A token is one warp's (or, when there are few tokens, split over warps_per_token warps of a
// CTA): D / 16 lanes share a row, and a lane moves two 16-byte chunks of it, chunks c and c + r/16
// where they are a half-split pair's halves, else neighbours, so that both elements of every pair
// meet in one lane.  A lane's pairs are the same in every row of the token, so its 8 sines and
// cosines stay in registers for all heads (read again for every row from shared memory, the call
// took 166 us on 841 MB instead of 150; now 147, 5.7 TB/s).  The first rows' loads are under way while the
// token's sequence, page and angles are found.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 5) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 16, kSlots = 32 / kLanes;  // lanes per row, rows a warp takes at a time
  constexpr int kWarps = kAppendThreads / 32;
  __shared__ __align__(16) float2 cs_all[kWarps][D / 2];  // cos, sin of each warp's token
  __shared__ bool last_cta, errors;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = (int64_t(blockIdx.x) * kWarps + warp) / p.warps_per_token;
  const int sub = warp % p.warps_per_token;

  if (blockIdx.x == 0) {  // malformed offsets or lengths: every access below stays in bounds all the same
    int bad = 0;
    for (int b = tid; b < p.B; b += kAppendThreads) bad |= p.offsets[b + 1] < p.offsets[b] || p.lengths[b] < 0;
    if (tid == 0) bad |= p.offsets[0] != 0 || p.offsets[p.B] > p.total;
    if (bad) raise_status(p.status, JFA_ERR_BAD_OFFSETS);
  }
  const int64_t first = __ldg(p.offsets), last = __ldg(p.offsets + p.B);
  if (t < p.total && t >= first && t < last) {  // rows of a sequence; others are left alone
    const int c = lane % kLanes;  // this lane's chunk pair
    const int half = p.rot / 16;  // chunks in half of the rotated dims
    const bool split = !p.interleaved && c < half, inter = p.interleaved && 16 * c < p.rot;
    const int a = split ? c : 2 * c, b = split ? c + half : a + 1;
    // rows of the token: H_kv of k, H_kv of v, H of q
    const int rows = 2 * p.Hkv + p.H, step = kSlots * p.warps_per_token;
    const __nv_bfloat16 *kt = p.k + t * p.k_stride, *vt = p.v + t * p.v_stride, *qt = p.q + t * p.q_stride;
    uint4 x[kAppendBatch], y[kAppendBatch];
    auto load = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kAppendBatch; ++u) {
        const int r = r0 + u * step;
        if (r >= rows) break;
        const __nv_bfloat16* src = r < p.Hkv ? kt + r * D : r < 2 * p.Hkv ? vt + (r - p.Hkv) * D : qt + (r - 2 * p.Hkv) * D;
        x[u] = reinterpret_cast<const uint4*>(src)[a];
        y[u] = reinterpret_cast<const uint4*>(src)[b];
      }
    };
    const int r_first = sub * kSlots + lane / kLanes;
    load(r_first);

    // ---- the token's place and angles
    const int seq = find_sequence(p.offsets, p.B, t, lane);
    const int64_t pos = int64_t(p.lengths[seq]) + (t - __ldg(p.offsets + seq));
    const int64_t pg = pos / p.page_size;
    int64_t at = -1;  // element offset of the token's row of head 0 in the cache, -1: not stored
    if (pos >= 0 && pg < p.max_pages) {
      const int page = __ldg(p.page_table + int64_t(seq) * p.max_pages + pg);
      if (page >= 0 && page < p.num_pages)
        at = (int64_t(page) * p.Hkv * p.page_size + (pos - pg * p.page_size)) * D;
    }
    if (at < 0 && lane == 0) raise_status(p.status, pos < 0 ? JFA_ERR_BAD_OFFSETS : JFA_ERR_BAD_PAGES);
    float2* cs = cs_all[warp];
    for (int i = lane; i < p.rot / 2; i += 32) {
      const uint64_t turns = uint64_t(pos) * p.turn[i];
      const uint32_t units = uint32_t((turns + (1ull << 31)) >> 32);  // of 2^-32 turns
      const uint32_t quarter = (units + (1u << 29)) >> 30;             // the nearest quarter turn, 4 being 0
      const int32_t rest = int32_t(units - (quarter << 30));           // behind it, at most an eighth
      float sn, cn;
      sincospif(float(rest) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31: half turns
      const float2 at_0 = make_float2(cn, sn), at_1 = make_float2(-sn, cn);
      const float2 w1 = quarter & 1 ? at_1 : at_0;
      cs[i] = quarter & 2 ? make_float2(-w1.x, -w1.y) : w1;
    }
    __syncwarp();
    float2 w[8];  // this lane's pairs: 8 of a split pair of chunks, 4 + 4 of two interleaved ones
    if (split || inter) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 f = reinterpret_cast<const float4*>(cs + 8 * c)[e];
        w[2 * e] = make_float2(f.x, f.y);
        w[2 * e + 1] = make_float2(f.z, f.w);
      }
    }

    // ---- rotate and store, kAppendBatch rows at a time
    for (int r0 = r_first; r0 < rows; r0 += kAppendBatch * step) {
      if (r0 != r_first) load(r0);
#pragma unroll
      for (int u = 0; u < kAppendBatch; ++u) {
        const int r = r0 + u * step;
        if (r >= rows) break;
        const bool is_k = r < p.Hkv, is_q = r >= 2 * p.Hkv;
        if (is_k || is_q) {
          const uint4 x0 = x[u], y0 = y[u];
          if (inter) {
            x[u] = make_uint4(rot_pair(x0.x, w[0]), rot_pair(x0.y, w[1]), rot_pair(x0.z, w[2]), rot_pair(x0.w, w[3]));
            y[u] = make_uint4(rot_pair(y0.x, w[4]), rot_pair(y0.y, w[5]), rot_pair(y0.z, w[6]), rot_pair(y0.w, w[7]));
          } else if (split) {
            x[u] = make_uint4(rot_lo(x0.x, y0.x, w[0], w[1]), rot_lo(x0.y, y0.y, w[2], w[3]),
                              rot_lo(x0.z, y0.z, w[4], w[5]), rot_lo(x0.w, y0.w, w[6], w[7]));
            y[u] = make_uint4(rot_hi(x0.x, y0.x, w[0], w[1]), rot_hi(x0.y, y0.y, w[2], w[3]),
                              rot_hi(x0.z, y0.z, w[4], w[5]), rot_hi(x0.w, y0.w, w[6], w[7]));
          }
        }
        if (is_q) {
          uint4* o = reinterpret_cast<uint4*>(p.q_out + (t * p.H + r - 2 * p.Hkv) * D);
          o[a] = x[u];
          o[b] = y[u];
        } else {
          const int h = is_k ? r : r - p.Hkv;
          if (at >= 0) {
            uint4* o = reinterpret_cast<uint4*>((is_k ? p.k_cache : p.v_cache) + at + int64_t(h) * p.page_size * D);
            o[a] = x[u];
            o[b] = y[u];
          }
          if (is_k && p.k_out) {
            uint4* o = reinterpret_cast<uint4*>(p.k_out + (t * p.Hkv + h) * D);
            o[a] = x[u];
            o[b] = y[u];
          }
        }
      }
    }
  }

  // lengths after the call, by the last CTA to get here: every CTA has read `lengths` by
  // then, so lengths_out may be `lengths` itself
  if (p.lengths_out) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      last_cta = atomicAdd(p.done, 1u) == gridDim.x - 1;
      if (last_cta) {
        __threadfence();
        // an error of this call (or an earlier one that nobody has asked for) is in *status by now:
        // then each sequence is looked at for tokens that were not stored.  (One thread reads it: the
        // CTA must agree, whoever clears it meanwhile.)
        errors = *static_cast<volatile const int*>(p.status) != 0;
      }
    }
    __syncthreads();
    if (last_cta) {
      bool bad = false;
      if (errors) {
        for (int b = tid; b < p.B; b += kAppendThreads) bad |= p.offsets[b + 1] < p.offsets[b];
        bad |= p.offsets[0] != 0 || p.offsets[p.B] > p.total;
        bad = __syncthreads_or(bad);
      }
      for (int b = tid; b < p.B; b += kAppendThreads) {
        const int len = p.lengths[b];
        const int64_t n = p.offsets[b + 1] - p.offsets[b];
        const bool grows = !errors || (!bad && stores_all(p, b, len, n));
        p.lengths_out[b] = grows ? int32_t(len + n) : len;
      }
      if (tid == 0) *p.done = 0;
    }
  }
}

// ================================================================== attention over the cache
// One query token per sequence, G = H / H_kv query heads per key/value head.  Memory bound: each
// visible key and value row is read once per block of 16 query heads (4 d G flops per 4 d bytes up to
// G = 16; 537 MB of 128 x 8192 tokens of one head: 101 us for 8 query heads, 109 for 16, 185 for 32,
// 332 for 64).  2.35 GB (128 sequences of up to 16384 tokens, 4 heads of d = 128 read by 16, pages
// of 64): 347 us, 6.77 TB/s, the rate of a plain copy; 996 MB of two sequences 162 us; 189 MB in
// pages of 16 41 us.  Not near that rate: few units of many rows, whose joins one CTA each does
// (2 x 400000 tokens of one head, 410 MB: 153 us for 1 query head, 307 for 8, 518 for 16).
//
// Keys are walked in tiles of 64.  A unit is (sequence, kv head, block of 16 query heads);
// the tiles of all units, in order, are dealt out evenly: CTA x of n takes tiles
// [x N / n, (x + 1) N / n).  So every CTA streams the same number of bytes whatever the
// lengths are; a unit whose tiles lie in several CTAs is joined from their partial sums by
// the CTA that finishes it last, in CTA order, so the result does not depend on timing.
//
// In a CTA a producer warp copies K and V tiles into a ring with TMA (one box per page and
// 64 columns, 128-byte swizzle); four warps take 16 keys of each tile each, with the running
// maximum, sum and output rows in registers:  S = Q K^T and O += P V on m16n8k16 products whose
// 16 rows are the query heads (rows past G are zero); P is rounded to bf16 as an operand (at most
// 2^-8 relative a term).  A NaN among a row's scores is in its sum and so in out and lse; only a sum
// of 0 means that no key is seen (lse = -inf).
constexpr int kTileKeys = 64;
constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * (kAttnWarps + 1);
constexpr int kJoinPitch = 34;  // 32 output columns, maximum, sum

struct CacheAttnParams {
  const __nv_bfloat16* q;       // [B][H][d]
  const int32_t* page_table;
  const int32_t* lengths;
  __nv_bfloat16* out;           // [B][H][d]
  float* lse;                   // [H][B]
  int64_t num_pages;
  int B, H, Hkv, G, RB;         // RB: blocks of 16 query heads per kv head
  int page_size, max_pages;
  int window, sinks;
  float scale_log2;
  int rows;                     // query heads of a block that are real at most: min(G, 16)
  int* status;
  int* counters_used;           // nonzero: `arrived` may not be at 0
  unsigned* arrived;            // [units] partial sums written (left at 0)
  float* partial;               // [2 * grid][rows][d + 2]
};

template <int D>
struct CacheCfg {
  static constexpr int kHalf = kTileKeys * 128;           // one 64-column box column of a tile
  static constexpr int kTileBytes = kTileKeys * D * 2;
  static constexpr int kStageBytes = 2 * kTileBytes;      // K, V
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kCtasPerSm = 2;
  static constexpr int kSmemBytes = kStages * kStageBytes + 1024 + kAttnWarps * 16 * kJoinPitch * 4;
  static_assert(kCtasPerSm * (kSmemBytes + 4096) <= 233472, "shared memory per SM (dynamic, static and reserved)");
};

// The keys a sequence of `len` tokens shows its newest: [0, s_end) and [lo, len), as 64-key tiles.
struct SeqTiles {
  int len, lo, s_end, n_sink, n;  // n_sink tiles of the first part, n in all
};
__device__ __forceinline__ SeqTiles seq_tiles(int len, int window, int sinks) {
  SeqTiles s;
  s.len = len;
  s.lo = len > window ? len - window : 0;
  s.s_end = sinks < s.lo ? sinks : s.lo;
  s.n_sink = (s.s_end + kTileKeys - 1) / kTileKeys;
  s.n = s.n_sink + (len + kTileKeys - 1) / kTileKeys - s.lo / kTileKeys;
  if (len <= 0) s.n = 0;
  return s;
}

// A CTA's walk over the tiles dealt to it, one segment (consecutive tiles of one unit) at a time.
struct Walk {
  int b, hk, rb;      // unit
  int64_t unit0;      // first tile of the unit
  SeqTiles s;
};

// Plain loads of `lengths` and of q: the kernel in front, which may still be running when this grid
// becomes resident, may be the append that writes both, and the read-only path is for data that stays
// as it is for the grid's whole life.  (Page tables and offsets are written by no kernel of the library.)
__device__ __forceinline__ int checked_len(const CacheAttnParams& p, int b) {
  const int len = p.lengths[b];
  return len < 0 || len > int64_t(p.max_pages) * p.page_size ? 0 : len;
}

__device__ __forceinline__ void next_unit(const CacheAttnParams& p, Walk& w) {
  w.unit0 += w.s.n;
  if (++w.rb < p.RB) return;
  w.rb = 0;
  if (++w.hk < p.Hkv) return;
  w.hk = 0;
  do {
    ++w.b;
    w.s = seq_tiles(w.b < p.B ? checked_len(p, w.b) : 0, p.window, p.sinks);
  } while (w.b < p.B && w.s.n == 0);
}

__device__ __forceinline__ int64_t first_tile(int64_t total, int cta, int ctas) { return total * cta / ctas; }
// The CTA that holds tile t: the last x with first_tile(x) <= t.
__device__ __forceinline__ int cta_of(int64_t total, int64_t t, int ctas) {
  return int(((t + 1) * ctas - 1) / total);
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads, CacheCfg<D>::kCtasPerSm)
    cache_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                           const CacheAttnParams p) {
  using C = CacheCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* join = reinterpret_cast<float*>(ring + C::kStages * C::kStageBytes);  // [warp][16][kJoinPitch]
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ long long run_end[kAttnThreads];  // tiles of all units before the end of each thread's run of sequences
  __shared__ int abort_sh;
  __shared__ int refused;
  __shared__ int is_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    abort_sh = 0;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kAttnWarps);
    }
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  volatile int* abort_flag = &abort_sh;

  // (one thread reads the word: another CTA whose wait has run out may be writing it)
  if (tid == 0) refused = *static_cast<volatile const int*>(p.counters_used);
  // ---- tiles per run of consecutive sequences, then their running sums
  const int run = (p.B + kAttnThreads - 1) / kAttnThreads;
  {
    long long sum = 0;
    for (int b = tid * run; b < min(p.B, (tid + 1) * run); ++b) {
      const int len = checked_len(p, b);
      if (len != p.lengths[b] && blockIdx.x == 0) raise_status(p.status, JFA_ERR_BAD_OFFSETS);
      sum += seq_tiles(len, p.window, p.sinks).n;
    }
    run_end[tid] = sum * p.Hkv * p.RB;
  }
  __syncthreads();
  if (warp == 0) {
    long long carry = 0;
    for (int c = 0; c < kAttnThreads; c += 32) {
      long long v = run_end[c + lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      run_end[c + lane] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  if (refused) {  // uniform over the CTA, nothing in flight
    if (tid == 0) raise_status(p.status, JFA_ERR_WORKSPACE);
    return;
  }
  const int64_t total = run_end[kAttnThreads - 1];

  // ---- sequences that show no key: out 0, lse -inf
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (checked_len(p, b) > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + int64_t(b) * p.H * D);
    for (int i = tid; i < p.H * D / 8; i += kAttnThreads) o[i] = make_uint4(0, 0, 0, 0);
    for (int h = tid; h < p.H; h += kAttnThreads) p.lse[int64_t(h) * p.B + b] = -INFINITY;
  }

  const int ctas = total < gridDim.x ? int(total) : int(gridDim.x);  // those with tiles: at least one each
  if (int(blockIdx.x) >= ctas) return;  // uniform over the CTA, nothing in flight
  const int64_t t0 = first_tile(total, blockIdx.x, ctas), t1 = first_tile(total, blockIdx.x + 1, ctas);

  // ---- the unit that holds t0
  Walk w;
  {
    int r = 0;  // runs that end at or before t0 (run_end is non-decreasing, run_end[last] = total > t0)
#pragma unroll
    for (int c = 0; c < kAttnThreads; c += 32) r += __popc(__ballot_sync(0xffffffffu, run_end[c + lane] <= t0));
    int64_t at = r ? run_end[r - 1] : 0;
    w.b = r * run;
    w.s = seq_tiles(checked_len(p, w.b), p.window, p.sinks);
    const int per_seq = p.Hkv * p.RB;
    while (at + int64_t(w.s.n) * per_seq <= t0) {
      at += int64_t(w.s.n) * per_seq;
      ++w.b;
      w.s = seq_tiles(checked_len(p, w.b), p.window, p.sinks);
    }
    const int u = int((t0 - at) / w.s.n);
    w.hk = u / p.RB;
    w.rb = u - w.hk * p.RB;
    w.unit0 = at + int64_t(u) * w.s.n;
  }

  if (warp == kAttnWarps) {
    // ------------------------------------------------------------ producer
    // A tile is `boxes` boxes of K and of V, one page's rows each (64 at most).  The warp looks up
    // the pages of 32 boxes at a time, a batch ahead of the copies: lane x holds box x % boxes of
    // the batch's tile x / boxes.  (With one lookup per tile in front of its copies: 43 us instead of
    // 40 on 189 MB in pages of 16, d = 64.)
    const int box = p.page_size < kTileKeys ? p.page_size : kTileKeys;
    const int boxes = kTileKeys / box, batch = 32 / boxes;
    uint32_t n = 0;
    bool ok = true;
    for (int64_t t = t0; t < t1 && ok; next_unit(p, w)) {
      const int64_t end = min(t1, w.unit0 + w.s.n);
      const int32_t* table = p.page_table + int64_t(w.b) * p.max_pages;
      // this lane's box of the batch that starts at tile t: its page (-1: none to copy) and row in it
      auto look_up = [&](int64_t tb, int& page, int& off) {
        const int i = int(tb - w.unit0) + lane / boxes;
        const bool sink = i < w.s.n_sink;
        const int j0 = (sink ? i : w.s.lo / kTileKeys + i - w.s.n_sink) * kTileKeys;
        const int jb = j0 + lane % boxes * box;  // keys [jb, jb + box)
        page = -1;
        off = jb % p.page_size;
        if (tb + lane / boxes < end && jb < (sink ? w.s.s_end : w.s.len) && jb + box > (sink ? 0 : w.s.lo)) {
          page = __ldg(table + jb / p.page_size);
          if (page < 0 || page >= p.num_pages) {
            raise_status(p.status, JFA_ERR_BAD_PAGES);
            page = -1;
          }
        }
      };
      int page, off, page_next = -1, off_next = 0;
      look_up(t, page, off);
      while (t < end && ok) {
        if (t + batch < end) look_up(t + batch, page_next, off_next);
        const unsigned loads = __ballot_sync(0xffffffffu, page >= 0);
        const int row = int((int64_t(page) * p.Hkv + w.hk) * p.page_size + off);  // below 2^31
        for (int x = 0; x < batch && t < end; ++x, ++t, ++n) {
          const uint32_t e = n % C::kStages, ph = (n / C::kStages) & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[e], ph ^ 1, abort_flag, kWaitTimeoutNs));
          if (!ok) break;
          const unsigned group = ((1u << boxes) - 1u) << (x * boxes);
          if (lane == 0) mbar_arrive_expect_tx(&full[e], uint32_t(__popc(loads & group)) * box * D * 4);
          __syncwarp();
          if ((loads & group) >> lane & 1u) {
            uint8_t* dst = ring + e * C::kStageBytes + (lane - x * boxes) * box * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              tma_load_2d(dst + c * C::kHalf, &k_map, &full[e], c * 64, row);
              tma_load_2d(dst + C::kTileBytes + c * C::kHalf, &v_map, &full[e], c * 64, row);
            }
          }
        }
        page = page_next;
        off = off_next;
      }
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
  } else {
    // ------------------------------------------------------------ the four warps
    const int g = lane >> 2, c2 = (lane & 3) * 2;  // accumulator rows g, g + 8; columns c2, c2 + 1
    uint32_t n = 0;
    bool ok = true;
    for (int64_t t = t0; t < t1 && ok; next_unit(p, w)) {
      const int64_t seg0 = t, end = min(t1, w.unit0 + w.s.n);
      const int h0 = w.hk * p.G + w.rb * 16;          // first query head of the block
      const int rows = min(16, p.G - w.rb * 16);
      uint32_t qa[D / 16][4];
      {
        const uint32_t* q0 = reinterpret_cast<const uint32_t*>(p.q + (int64_t(w.b) * p.H + h0 + g) * D + c2);
        const uint32_t* q1 = q0 + 8 * D / 2;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][0] = g < rows ? q0[kk * 8] : 0u;
          qa[kk][1] = g + 8 < rows ? q1[kk * 8] : 0u;
          qa[kk][2] = g < rows ? q0[kk * 8 + 4] : 0u;
          qa[kk][3] = g + 8 < rows ? q1[kk * 8 + 4] : 0u;
        }
      }
      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // log2 units; l per lane until the end
      for (; t < end; ++t, ++n) {
        const int i = int(t - w.unit0);
        const bool sink = i < w.s.n_sink;
        const int j0 = (sink ? i : w.s.lo / kTileKeys + i - w.s.n_sink) * kTileKeys + warp * 16;
        const int v_lo = (sink ? 0 : w.s.lo) - j0, v_hi = (sink ? w.s.s_end : w.s.len) - j0;  // visible: [v_lo, v_hi)
        const uint32_t e = n % C::kStages, ph = (n / C::kStages) & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&full[e], ph, abort_flag, kWaitTimeoutNs));
        if (!ok) break;
        if (v_lo < 16 && v_hi > 0) {
          const uint32_t kb = smem_u32(ring + e * C::kStageBytes) + warp * 16 * 128;
          const uint32_t vb = kb + C::kTileBytes;
          float x[2][4] = {};
          {
            const int r = (lane & 7) + ((lane >> 4) << 3), cq = (lane >> 3) & 1;  // this lane's row and 16-byte chunk
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              uint32_t b4[4];
              ldmatrix_x4(b4, kb + (kk >> 2) * C::kHalf + r * 128 + ((((kk & 3) * 2 + cq) ^ (r & 7)) << 4));
              mma_bf16_16816(x[0], qa[kk], b4[0], b4[1]);
              mma_bf16_16816(x[1], qa[kk], b4[2], b4[3]);
            }
          }
          const bool edge = v_lo > 0 || v_hi < 16;
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int col = a * 8 + c2 + (b & 1);
              x[a][b] *= p.scale_log2;
              if (edge && (col < v_lo || col >= v_hi)) x[a][b] = -INFINITY;
            }
          float a0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
          float a1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
          a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 1));
          a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
          a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 2));
          a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2));
          const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
          const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
          const float f0 = ex2_approx(m0 - u0), f1 = ex2_approx(m1 - u1);  // 0 on the first tile
          m0 = n0;
          m1 = n1;
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            x[a][0] = ex2_approx(x[a][0] - u0);
            x[a][1] = ex2_approx(x[a][1] - u0);
            x[a][2] = ex2_approx(x[a][2] - u1);
            x[a][3] = ex2_approx(x[a][3] - u1);
          }
          l0 = l0 * f0 + ((x[0][0] + x[0][1]) + (x[1][0] + x[1][1]));
          l1 = l1 * f1 + ((x[0][2] + x[0][3]) + (x[1][2] + x[1][3]));
          // P in bf16, as the second product's left operand
          const uint32_t pa[4] = {pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3]),
                                  pack_bf16x2(x[1][0], x[1][1]), pack_bf16x2(x[1][2], x[1][3])};
          if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
            for (int d8 = 0; d8 < D / 8; ++d8) {
              o[d8][0] *= f0;
              o[d8][1] *= f0;
              o[d8][2] *= f1;
              o[d8][3] *= f1;
            }
          }
          // value rows that no key of this tile shows (past the end, before the window, or a
          // page that was not copied) may hold anything, and 0 * NaN is NaN: clear them
          uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;  // keys c2, c2 + 1 and c2 + 8, c2 + 9
          if (edge) {
            auto bits = [&](int key) {
              return (key >= v_lo && key < v_hi ? 0xffffu : 0u) | (key + 1 >= v_lo && key + 1 < v_hi ? 0xffff0000u : 0u);
            };
            keep_lo = bits(c2);
            keep_hi = bits(c2 + 8);
          }
          {
            const int r = (lane & 7) + (((lane >> 3) & 1) << 3), cq = lane >> 4;
#pragma unroll
            for (int dd = 0; dd < D / 16; ++dd) {
              uint32_t b4[4];
              ldmatrix_x4_trans(b4, vb + (dd >> 2) * C::kHalf + r * 128 + ((((dd & 3) * 2 + cq) ^ (r & 7)) << 4));
              mma_bf16_16816(o[2 * dd], pa, b4[0] & keep_lo, b4[1] & keep_hi);
              mma_bf16_16816(o[2 * dd + 1], pa, b4[2] & keep_lo, b4[3] & keep_hi);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[e]);
      }
      // ---- join the four warps' rows through shared memory, 32 columns at a time.  The warps
      //      first agree on whether every wait came through: a warp that left alone would
      //      leave the others at a barrier.
      ok = named_bar_and(1, kAttnWarps * 32, ok);
      if (!ok) break;
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      const bool whole = seg0 == w.unit0 && end == w.unit0 + w.s.n;
      constexpr int kPitch = D + 2;  // a partial row: O, then m and l
      float* part = p.partial + (2 * int64_t(blockIdx.x) + (seg0 == t0 ? 0 : 1)) * p.rows * kPitch;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        if (c0 > 0) named_bar_sync(1, kAttnWarps * 32);  // the previous columns have been read
#pragma unroll
        for (int r2 = 0; r2 < 2; ++r2) {
          const int r = g + 8 * r2;
          if (r < rows) {
            float* row = join + (warp * 16 + r) * kJoinPitch;
#pragma unroll
            for (int d8 = 0; d8 < 4; ++d8)
              *reinterpret_cast<float2*>(row + d8 * 8 + c2) = make_float2(o[c0 / 8 + d8][2 * r2], o[c0 / 8 + d8][2 * r2 + 1]);
            if ((lane & 3) == 0) *reinterpret_cast<float2*>(row + 32) = r2 ? make_float2(m1, l1) : make_float2(m0, l0);
          }
        }
        named_bar_sync(1, kAttnWarps * 32);
        for (int i = tid; i < rows * 16; i += kAttnWarps * 32) {
          const int r = i >> 4, c = (i & 15) * 2;
          float m = -INFINITY, l = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
          for (int k = 0; k < kAttnWarps; ++k) m = fmaxf(m, join[(k * 16 + r) * kJoinPitch + 32]);
          const float u = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int k = 0; k < kAttnWarps; ++k) {
            const float* row = join + (k * 16 + r) * kJoinPitch;
            const float f = ex2_approx(row[32] - u);
            l += f * row[33];
            x0 += f * row[c];
            x1 += f * row[c + 1];
          }
          if (whole) {
            const float inv = l != 0.f ? 1.f / l : 0.f;
            *reinterpret_cast<uint32_t*>(p.out + (int64_t(w.b) * p.H + h0 + r) * D + c0 + c) = pack_bf16x2(x0 * inv, x1 * inv);
            if (c0 + c == 0) p.lse[int64_t(h0 + r) * p.B + w.b] = l != 0.f ? (u + log2f(l)) * kLn2 : -INFINITY;
          } else {
            *reinterpret_cast<float2*>(part + r * kPitch + c0 + c) = make_float2(x0, x1);
            if (c0 + c == 0) *reinterpret_cast<float2*>(part + r * kPitch + D) = make_float2(m, l);
          }
        }
      }
      if (whole) continue;
      // ---- the unit's last CTA to arrive joins the partial rows of all, in CTA order
      const int ca = cta_of(total, w.unit0, ctas), cb = cta_of(total, w.unit0 + w.s.n - 1, ctas);
      const int64_t unit = (int64_t(w.b) * p.Hkv + w.hk) * p.RB + w.rb;
      named_bar_sync(1, kAttnWarps * 32);
      if (tid == 0) {
        __threadfence();
        is_last = atomicAdd(p.arrived + unit, 1u) == unsigned(cb - ca);
        __threadfence();
      }
      named_bar_sync(1, kAttnWarps * 32);
      if (!is_last) continue;
      auto slot = [&](int x) {  // where CTA x put this unit's rows: its first segment, or a later one
        return p.partial + (2 * int64_t(x) + (first_tile(total, x, ctas) >= w.unit0 ? 0 : 1)) * p.rows * kPitch;
      };
      for (int i = tid; i < rows * (D / 2); i += kAttnWarps * 32) {
        const int r = i / (D / 2), c = (i - r * (D / 2)) * 2;
        float m = -INFINITY, l = 0.f, x0 = 0.f, x1 = 0.f;
        for (int x = ca; x <= cb; ++x) {
          const float* row = slot(x) + r * kPitch;
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(row + D));
          const float2 v = __ldcg(reinterpret_cast<const float2*>(row + c));
          const float mn = fmaxf(m, ml.x), u = mn == -INFINITY ? 0.f : mn;
          const float f = ex2_approx(m - u), fx = ex2_approx(ml.x - u);
          m = mn;
          l = l * f + ml.y * fx;
          x0 = x0 * f + v.x * fx;
          x1 = x1 * f + v.y * fx;
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        *reinterpret_cast<uint32_t*>(p.out + (int64_t(w.b) * p.H + h0 + r) * D + c) = pack_bf16x2(x0 * inv, x1 * inv);
        if (c == 0) p.lse[int64_t(h0 + r) * p.B + w.b] = l != 0.f ? ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2 : -INFINITY;
      }
      if (tid == 0) p.arrived[unit] = 0;
    }
    if (!ok && lane == 0) {
      raise_status(p.status, JFA_ERR_TIMEOUT);
      *p.counters_used = 1;  // units that this CTA leaves undone keep their counts
    }
  }
}

template <int D>
cudaError_t launch_attn_t(const CUtensorMap& km, const CUtensorMap& vm, const CacheAttnParams& p, int num_sms,
                          cudaStream_t stream) {
  using C = CacheCfg<D>;
  auto kern = cache_attention_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  int grid = C::kCtasPerSm * num_sms;
  if (grid > kMaxAttnCtas) grid = kMaxAttnCtas;
  return launch_pdl(kern, dim3(grid), dim3(kAttnThreads), C::kSmemBytes, stream, km, vm, p);
}

}  // namespace

size_t cache_workspace_bytes(int B, int H, int Hkv) {
  const int64_t units = int64_t(B) * Hkv * ((H / Hkv + 15) / 16);
  return align_up(kArrivedAt + size_t(units) * sizeof(unsigned), 256);
}

cudaError_t launch_cache_append(const jfa_cache& c, const CacheAppend& a, void* ws, int num_sms, cudaStream_t stream) {
  AppendParams p;
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_stride = a.q_stride;
  p.offsets = a.offsets;
  p.total = a.total;
  p.k_cache = static_cast<__nv_bfloat16*>(c.k);
  p.v_cache = static_cast<__nv_bfloat16*>(c.v);
  p.page_table = c.page_table;
  p.lengths = c.lengths;
  p.lengths_out = a.lengths_out;
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.k_out = static_cast<__nv_bfloat16*>(a.k_out);
  p.num_pages = c.num_pages;
  p.B = c.B;
  p.H = a.H;
  p.Hkv = c.H_kv;
  p.page_size = c.page_size;
  p.max_pages = c.max_pages;
  p.rot = a.rot;
  p.interleaved = a.interleaved;
  p.status = &static_cast<WsHeader*>(ws)->status;
  p.done = &static_cast<WsHeader*>(ws)->append_done;
  for (int i = 0; i < a.rot / 2; ++i) p.turn[i] = a.turn[i];
  for (int i = a.rot / 2; i < 64; ++i) p.turn[i] = 0;
  // few tokens: several warps for each, until the warps fill the card about twice over; then one
  constexpr int kWarps = kAppendThreads / 32;
  p.warps_per_token = kWarps;
  while (p.warps_per_token > 1 && a.total * p.warps_per_token > int64_t(64) * num_sms) p.warps_per_token /= 2;
  const int64_t ctas = (a.total * p.warps_per_token + kWarps - 1) / kWarps;
  const dim3 grid(unsigned(ctas > 0 ? ctas : 1));
  return c.d == 128 ? launch_pdl(append_kernel<128>, grid, dim3(kAppendThreads), 0, stream, p)
                    : launch_pdl(append_kernel<64>, grid, dim3(kAppendThreads), 0, stream, p);
}

cudaError_t launch_cache_attention(const jfa_cache& c, const CUtensorMap& km, const CUtensorMap& vm, const void* q, int H,
                                   int window, int sinks, float scale, void* out, float* lse, void* ws, int num_sms,
                                   cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  CacheAttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.page_table = c.page_table;
  p.lengths = c.lengths;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.num_pages = c.num_pages;
  p.B = c.B;
  p.H = H;
  p.Hkv = c.H_kv;
  p.G = H / c.H_kv;
  p.RB = (p.G + 15) / 16;
  p.rows = p.G < 16 ? p.G : 16;
  p.page_size = c.page_size;
  p.max_pages = c.max_pages;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = scale * kLog2e;
  p.status = &reinterpret_cast<WsHeader*>(w)->status;
  p.counters_used = &reinterpret_cast<WsHeader*>(w)->counters_used;
  p.arrived = reinterpret_cast<unsigned*>(w + kArrivedAt);
  p.partial = reinterpret_cast<float*>(w + kPartialAt);
  return c.d == 128 ? launch_attn_t<128>(km, vm, p, num_sms, stream) : launch_attn_t<64>(km, vm, p, num_sms, stream);
}

}  // namespace jfa
