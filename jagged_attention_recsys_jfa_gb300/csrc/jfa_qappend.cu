// Appending to the paged cache held in 8 bits, with the position rotation and the rounding to codes on the way.
#include "jfa_qcache.cuh"

namespace jfa {
namespace {

// A block's scale is the smallest power of two, 2^-126 at least, that holds its new values: M s >= max |x|,
// M = 448 or 127.  Keys that are rotated are bounded by sqrt(2) times their largest element: a turned pair is
// no longer than its two elements allow, and a scale that does not depend on the sines is defined to the bit.
// Tokens that share the block with new ones behind them have their codes rounded again where the scale grows;
// between powers of two that is exact for e4m3 (but for its smallest values), and of int8 each step halves the
// codes, so that all roundings of a value together stay below one step of the block's last scale.  A new
// value that is not finite makes the block's scale NaN.  Scales of another origin may have any value.
//
// What a power of two costs: of e4m3 nothing but range.  Of int8 a code's step is up to 2, with rotated keys 2 sqrt(2),
// times max |x| / 127, the smallest with which the block's new values fit: the largest of them is 64 steps at least, of
// rotated keys 45 before they are turned.
//
// With bits m of max |x| as bf16 (exponent E = m >> 7, fraction f = m & 127): M s >= c max |x| for
// s = 2^(E - 127 - kBase + (f > kLimit)), M / c = (1 + x) 2^kBase, kLimit = floor(128 x):
//   448 = 1.75 * 2^8, 448 / sqrt(2) = 1.2374 * 2^8, 127 = 1.984375 * 2^6, 127 / sqrt(2) = 1.4031 * 2^6.
struct QAppendParams : AppendParams {
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int lb, lp;           // log2 of the tokens of a block, of a page
  int blocks_per_page;
};

constexpr int kQAppendThreads = 256;

template <bool kInt8>
__device__ __forceinline__ float scale_for(uint32_t m, bool rotated) {
  const uint32_t base = kInt8 ? 6 : 8, limit = kInt8 ? (rotated ? 51 : 126) : (rotated ? 30 : 96);
  const int e = int(m >> 7) - int(base) + ((m & 127u) > limit ? 1 : 0);
  return m >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float(uint32_t(e < 1 ? 1 : e) << 23);
}

// (cos, sin) of an angle given as a 64-bit fraction of a turn.  Only its distance to the nearest quarter turn becomes
// fp32, at most an eighth of a turn: there the Taylor series of sine and cosine to t^9 and t^10 are good to 2^-28
// of their values, and evaluated in fp32 to 2^-22.  (CUDA's function takes its argument modulo two first, which is
// done here: with it 740 MB of prompts took 160 us when this took 147.)
__device__ __forceinline__ float2 turned(uint64_t turns) {
  const uint32_t units = uint32_t((turns + (1ull << 31)) >> 32);  // of 2^-32 turns
  const uint32_t quarter = (units + (1u << 29)) >> 30;             // the nearest quarter turn, 4 being 0
  const float t = float(int32_t(units - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32: radians behind it
  const float t2 = t * t;
  const float sn = fmaf(t * t2, fmaf(t2, fmaf(t2, fmaf(t2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), t);
  const float c8 = fmaf(t2, -1.f / 3628800, 1.f / 40320);
  const float cn = fmaf(t2, fmaf(t2, fmaf(t2, fmaf(t2, c8, -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float x = quarter & 1 ? sn : cn, y = quarter & 1 ? cn : sn;  // a quarter turn further: (-sin, cos)
  return make_float2(((quarter + 1) & 2) ? -x : x, (quarter & 2) ? -y : y);
}

// A CTA takes consecutive blocks (their new tokens: up to 128 rows each) with all heads, or, when there are few
// blocks, with one of gridDim.y shares of them.  16 rows of a head are a warp's: D / 16 lanes share a row, each
// moving two 16-byte chunks of it, chunks c and c + r/16 where they are a half-split pair's halves, else c and the
// one half a row behind it: the lanes' chunks are side by side in either case.  Warps whose 16 rows belong to one
// block are a team that agrees on the largest element; the others take other heads.  Rows are read once, codes and
// rotated queries written once.  Rows are copied to shared memory ahead, across blocks, and looked at there twice,
// for the largest element and for the codes (held in registers in between: 192 us where this takes 139).
//
// Measured: 740 MB of rotated prompts, 4 + 4 + 16 heads of 128, blocks of 32: 139 us, 5300 GB/s, a quarter more
// than the floor: reads and writes together, and the warps' latency (47% of the issue slots are taken).  102 MB of 64-dim
// heads without queries, blocks of 128: 39 us: what bounds it is this form, rows that go through shared memory (5300 clk
// for a warp's head, eight heads one behind the other, 24 warps an SM) and whole blocks to a CTA (640 over 456 CTAs).  64 decoding tokens of 8 heads: 8 us in a replayed graph.
//
// Blocks are numbered without a sum over the sequences: sequence b's are offsets[b] / block + 2 b + i, which leaves
// each at least the (n - 2) / block + 2 that n tokens can touch; other numbers stay empty.
template <int D, bool kInt8, int kStages>  // kStages: heads of a warp under way at most
__global__ void __launch_bounds__(kQAppendThreads, D == 64 ? 3 : 2) qappend_kernel(const __grid_constant__ QAppendParams p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kPasses = 16 / kRows;
  constexpr int kWarps = kQAppendThreads / 32;
  static_assert(kStages == 2 || kStages == 3, "what is waited for");
  extern __shared__ uint4 smem[];
  uint4* rows_in = smem + (threadIdx.x >> 5) * (kStages * kPasses * 64);  // this warp's: [stage][pass][chunk][lane]
  // [row][4][kLanes]: two pairs' cosines, their sines
  float4* cs = reinterpret_cast<float4*>(smem + kWarps * kStages * kPasses * 64);
  __shared__ uint32_t team_max[2][kWarps];
  __shared__ bool last_cta, errors;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_append<kQAppendThreads>(p, tid);

  const int lb = p.lb, block = 1 << lb;
  const int c = lane % kLanes;  // this lane's chunk pair
  const int half = p.interleaved ? 0 : p.rot / 16;  // chunks in half of the dims that are rotated as halves
  const int ca_turned = c < half ? c : c + half, cb_turned = c < half ? c + half : c + kLanes;  // k's and q's; v's: half = 0
  const int heads = 2 * p.Hkv + p.H, pairs = p.rot / 2;
  // this thread's pair in the table of angles, of every kAtOnce-th row; a lane's chunks meet its pairs in order: of
  // halves, 8c + 2e + k; interleaved, four of its first chunk (e < 2), four of its second
  constexpr int kPairs = D / 2, kAtOnce = kQAppendThreads / kPairs;
  const int pair = tid % kPairs;
  const uint64_t pair_turn = p.turn[pair];
  float* pair_cs;
  {
    const int chunk = pair >> 2, in_lane = p.interleaved ? chunk % kLanes : pair >> 3;
    const int e = p.interleaved ? chunk / kLanes * 2 + (pair >> 1 & 1) : pair >> 1 & 3;
    pair_cs = reinterpret_cast<float*>(cs + e * kLanes + in_lane) + (pair & 1);
  }
  // which of the two buffers of maxima a team uses next; the ring's next stage to read, to copy into
  int turn, in_stage = 0, out_stage = 0;

  auto number = [&](int s) { return (__ldg(p.offsets + s) >> lb) + 2 * int64_t(s); };
  const int64_t numbers = (p.total >> lb) + 2 * int64_t(p.B);
  int64_t at = numbers * blockIdx.x / gridDim.x;
  const int64_t at_end = numbers * (blockIdx.x + 1) / gridDim.x;
  for (int b = find_last(number, p.B, at, lane); b < p.B && at < at_end; ++b) {
    const int64_t off = __ldg(p.offsets + b), n = __ldg(p.offsets + b + 1) - off, number0 = (off >> lb) + 2 * int64_t(b);
    const int64_t len = p.lengths[b];
    if (at < number0) at = number0;
    if (n <= 0 || len < 0 || off < 0 || off + n > p.total) continue;
    const int64_t start0 = (len >> lb) << lb;  // the first block's first position
    const int64_t blocks = ((len + n - 1) >> lb) - (len >> lb) + 1;
    int64_t i = at - number0;
    const int64_t i_end = at_end - number0 < blocks ? at_end - number0 : blocks;
    if (i < 0 || i >= i_end) continue;

    // What this warp does of block j: rows [r0, r1) of it are new, its own start at row0, and its heads are hd,
    // hd + step, ...
    struct Share {
      int first_row;   // row of the block's position 0, were it new (below 0 where the block starts before row 0)
      int r0, r1, g0, groups, team_shift, row0, hd, step;
      unsigned real;   // bit u: the lane's row of pass u is a new one
    };
    auto share_of = [&](int64_t j) {
      Share v;
      const int64_t start = start0 + (j << lb);
      v.first_row = int(off + start - len);
      v.r0 = int(len > start ? len - start : 0);
      v.r1 = int(len + n - start < block ? len + n - start : block);
      v.g0 = v.r0 >> 4;
      v.groups = ((v.r1 - 1) >> 4) - v.g0 + 1;  // 16-row groups with new rows
      v.team_shift = v.groups > 4 ? 3 : v.groups > 2 ? 2 : v.groups - 1;
      const int team = warp >> v.team_shift, in_team = warp & ((1 << v.team_shift) - 1);
      v.row0 = 16 * (v.g0 + in_team) + lane / kLanes;
      v.step = gridDim.y * kWarps >> v.team_shift;
      v.hd = (blockIdx.y * kWarps >> v.team_shift) + team;
      v.real = 0;
#pragma unroll
      for (int u = 0; u < kPasses; ++u) v.real |= (v.row0 + u * kRows >= v.r0 && v.row0 + u * kRows < v.r1 ? 1u : 0u) << u;
      return v;
    };
    // Copies run ahead of the work, over the ends of blocks.  A lane copies its own chunks and reads them back alone:
    // nothing to agree on.
    Share ahead = share_of(i);
    int64_t ahead_i = i;
    int under_way = 0;  // copied or being copied, the head at work among them
    auto copy_ahead = [&]() {
      while (under_way < kStages) {
        if (ahead.hd >= heads) {
          if (++ahead_i >= i_end) {
            --ahead_i;
            return;
          }
          ahead = share_of(ahead_i);
          continue;
        }
        int h = ahead.hd, ca = ca_turned, cb = cb_turned;
        const __nv_bfloat16* src = p.k;
        int64_t stride = p.k_stride;
        if (h >= p.Hkv) {
          h -= p.Hkv;
          src = p.v;
          stride = p.v_stride;
          ca = c;
          cb = c + kLanes;
          if (h >= p.Hkv) {
            h -= p.Hkv;
            src = p.q;
            stride = p.q_stride;
            ca = ca_turned;
            cb = cb_turned;
          }
        }
        src += int64_t(ahead.first_row + ahead.row0) * stride + (h * D + 8 * ca);
        const uint32_t to = smem_u32(rows_in + lane) + out_stage * (kPasses * 1024);
#pragma unroll
        for (int u = 0; u < kPasses; ++u, src += kRows * stride) {
          if (ahead.real >> u & 1u) {
            copy16_async(to + u * 1024, src);
            copy16_async(to + u * 1024 + 512, src + 8 * (cb - ca));
          }
        }
        copy_async_commit();
        ahead.hd += ahead.step;
        out_stage = out_stage == kStages - 1 ? 0 : out_stage + 1;
        ++under_way;
      }
    };

    for (; i < i_end; ++i) {
      const Share v = share_of(i);
      const int64_t start = start0 + (i << lb), pg = start >> p.lp;
      const int in_page = int(start) & (p.page_size - 1);
      int64_t page = -1;
      if (pg < p.max_pages) page = __ldg(p.page_table + int64_t(b) * p.max_pages + pg);
      copy_ahead();
      __syncthreads();  // the block in front is done with its angles and maxima
      turn = 0;         // (its teams may have been others, whose warps took different numbers of heads)
      if (pair < pairs) {
        uint64_t turns = uint64_t(start + 16 * v.g0 + tid / kPairs) * pair_turn;
        float* to = pair_cs + (tid / kPairs) * 16 * kLanes;
        for (int r = tid / kPairs; r < v.groups * 16; r += kAtOnce, turns += kAtOnce * pair_turn, to += kAtOnce * 16 * kLanes) {
          const float2 w = turned(turns);
          to[0] = w.x;
          to[2] = w.y;
        }
      }
      const bool stored = page >= 0 && page < p.num_pages;
      if (!stored && tid == 0) raise_status(p.status, JFA_ERR_BAD_PAGES);
      if (pairs > 0) __syncthreads();

      const int r0 = v.r0, row0 = v.row0, team_size = 1 << v.team_shift, team = warp >> v.team_shift, in_team = warp & (team_size - 1);
      const unsigned real = v.real;
      const int64_t my_row = v.first_row + row0, unit0 = page * p.Hkv;  // unit0: (page, head) number of head 0
      const int64_t place = (unit0 * p.page_size + in_page) * D, scale_place = unit0 * p.blocks_per_page + (in_page >> lb);
      const float4* my_cs = cs + (row0 - 16 * v.g0) * 4 * kLanes + c;
      for (int hd = v.hd; hd < heads; hd += v.step, turn ^= 1) {
        copy_ahead();
        if (kStages == 3 && under_way == 3) {
          copy_async_wait<2>();
        } else if (under_way == 2) {
          copy_async_wait<1>();
        } else {
          copy_async_wait<0>();
        }
        const uint4* in = rows_in + in_stage * kPasses * 64 + lane;  // chunks ca, and 32 behind them cb, of each pass
        in_stage = in_stage == kStages - 1 ? 0 : in_stage + 1;
        const bool is_k = hd < p.Hkv, is_q = hd >= 2 * p.Hkv;
        const int h = is_k ? hd : is_q ? hd - 2 * p.Hkv : hd - p.Hkv;
        uint8_t* codes = nullptr;
        float scale = 1.f;
        if (!is_q) {
          codes = (is_k ? p.k_cache : p.v_cache) + place + h * (p.page_size * D);
          float* scale_at = (is_k ? p.k_scale : p.v_scale) + scale_place + h * p.blocks_per_page;
          const bool old = r0 > 0 && stored;
          float s_old = 0.f;
          if (old) s_old = *scale_at;
          uint32_t m2 = 0;  // largest magnitudes, as bits
#pragma unroll
          for (int u = 0; u < kPasses; ++u) {
            if (!(real >> u & 1u)) continue;
            const uint4 x = in[u * 64], y = in[u * 64 + 32];
            const uint32_t kAbs = 0x7fff7fffu;
            m2 = __vimax3_u16x2(m2, x.x & kAbs, x.y & kAbs);
            m2 = __vimax3_u16x2(m2, x.z & kAbs, x.w & kAbs);
            m2 = __vimax3_u16x2(m2, y.x & kAbs, y.y & kAbs);
            m2 = __vimax3_u16x2(m2, y.z & kAbs, y.w & kAbs);
          }
          uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
          if (team_size > 1) {  // (two buffers in turn: a warp writes one again behind the barrier in between)
            if (lane == 0) team_max[turn][warp] = m;
            named_bar_sync(1 + team, team_size * 32);
            m = __reduce_max_sync(0xffffffffu, team_max[turn][(warp & ~(team_size - 1)) + (lane & (team_size - 1))]);
          }
          scale = scale_for<kInt8>(m, is_k && p.rot > 0);
          if (old && (fabsf(s_old) > scale || s_old != s_old)) scale = s_old;  // (a new scale that is NaN stays)
          if (stored) {
            if (old && scale != s_old && scale == scale) {  // earlier rows' codes at the new scale
              const float f = s_old / scale;
#pragma unroll 1
              for (int k = in_team * 32 + lane; k < r0 * (D / 4); k += team_size * 32) {
                uint32_t* at = reinterpret_cast<uint32_t*>(codes) + k;
                uint32_t lo, hi;
                codes_f16<kInt8>(*at, lo, hi);
                const float2 a = f16x2_floats(lo), z = f16x2_floats(hi);
                // (a code of -128, of another origin, by a factor of -1: 127 is the nearest)
                auto top = [](float x) { return kInt8 ? fminf(x, 127.f) : x; };
                *at = to_codes<kInt8>(top(a.x * f), top(a.y * f), top(z.x * f), top(z.y * f));
              }
            }
            if (in_team == 0 && lane == 0) *scale_at = scale;
          }
        }
        // (of a power of two 2^e from its exponent's bits; NaN's and others' are divided for)
        const uint32_t bits = __float_as_uint(scale);
        const float inv = bits << 9 || bits - (1u << 23) >= 253u << 23 ? 1.f / scale : __uint_as_float((254u << 23) - bits);
        const uint64_t inv2 = f2_pack(inv, inv);
        const int out_heads = is_q ? p.H : p.Hkv;
        const int ca = is_k || is_q ? ca_turned : c, cb = is_k || is_q ? cb_turned : c + kLanes;
        uint4* rows_out = is_q || (is_k && p.k_out)
                              ? reinterpret_cast<uint4*>((is_q ? p.q_out : p.k_out) + (my_row * out_heads + h) * D) + ca : nullptr;
        const int out_step = kRows * out_heads * (D / 8);
        const bool turned = (is_k || is_q) && (p.interleaved ? 8 * c < p.rot : c < half), coded = !is_q && stored;
        codes += row0 * D + 8 * ca;
#pragma unroll 1
        for (int u = 0; u < kPasses; ++u) {
          if (!(real >> u & 1u)) continue;
          const uint4 x = in[u * 64], y = in[u * 64 + 32];
          const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
          uint64_t a[4], z[4];  // pairs of elements of chunks ca and cb
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = f2_pack(bf16lo(wx[e]), bf16hi(wx[e]));
            z[e] = f2_pack(bf16lo(wy[e]), bf16hi(wy[e]));
          }
          if (turned) {
            const float4* w4 = my_cs + u * kRows * 4 * kLanes;
            if (!p.interleaved) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 w = w4[e * kLanes];  // cosines of pairs 2e, 2e + 1 of the lane's eight, their sines
                const uint64_t cos2 = f2_pack(w.x, w.y), sin2 = f2_pack(w.z, w.w), a0 = a[e];
                float z0, z1, x0, x1;
                f2_unpack(z[e], z0, z1);
                f2_unpack(f2_mul(a0, cos2), x0, x1);
                a[e] = f2_pack(fmaf(-z0, w.z, x0), fmaf(-z1, w.w, x1));
                z[e] = f2_fma(z[e], cos2, f2_mul(a0, sin2));
              }
            } else {  // four pairs in chunk ca, four (where they are rotated) in cb
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (e >= 2 && 8 * cb >= p.rot) break;
                const float4 w = w4[e * kLanes];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  uint64_t& v = e < 2 ? a[2 * e + k] : z[2 * (e - 2) + k];
                  float v0, v1;
                  f2_unpack(v, v0, v1);
                  const float cn = k ? w.y : w.x, sn = k ? w.w : w.z;
                  v = f2_pack(v0 * cn - v1 * sn, v1 * cn + v0 * sn);
                }
              }
            }
          }
          if (rows_out) {
            uint32_t b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float lo, hi;
              f2_unpack(e < 4 ? a[e] : z[e - 4], lo, hi);
              b[e] = pack_bf16x2(lo, hi);
            }
            uint4* o = rows_out + int64_t(u) * out_step;
            o[0] = make_uint4(b[0], b[1], b[2], b[3]);
            o[cb - ca] = make_uint4(b[4], b[5], b[6], b[7]);
          }
          if (coded) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v0, v1, v2, v3;
              f2_unpack(f2_mul(e < 2 ? a[2 * e] : z[2 * e - 4], inv2), v0, v1);
              f2_unpack(f2_mul(e < 2 ? a[2 * e + 1] : z[2 * e - 3], inv2), v2, v3);
              w[e] = to_codes<kInt8>(v0, v1, v2, v3);
            }
            uint8_t* o = codes + u * kRows * D;
            *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(o + 8 * (cb - ca)) = make_uint2(w[2], w[3]);
          }
        }
        --under_way;
      }
    }
  }
  if (p.lengths_out) write_lengths<kQAppendThreads>(p, tid, gridDim.x * gridDim.y, last_cta, errors);
}

// The rows under way and, for `rows` rotated rows, their angles.
constexpr int qappend_smem(int d, int stages, int rows) {
  return kQAppendThreads / 32 * stages * 16 * d * 2 + rows * (d / 2) * 8;
}
// CTAs of an SM: its shared memory, the kernel's registers.
constexpr int qappend_ctas(int d, int smem) {
  const int fit = 233472 / (smem + 1280), most = d == 64 ? 3 : 2;
  return fit < most ? fit : most;
}

template <int D, bool kInt8, int kStages>
cudaError_t launch_qappend(const QAppendParams& p, int rows, int num_sms, cudaStream_t stream) {
  auto kern = qappend_kernel<D, kInt8, kStages>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, qappend_smem(D, kStages, 128));
  if (e != cudaSuccess) return e;
  const int smem = qappend_smem(D, kStages, rows);
  // A CTA's blocks follow one another, so that it looks for its place once; a few CTAs for each that the card
  // holds, so that they end together.
  const int64_t blocks = (p.total >> p.lb) + 2 * int64_t(p.B), resident = int64_t(num_sms) * qappend_ctas(D, smem);
  const int64_t run = blocks / (4 * resident) > 1 ? blocks / (4 * resident) : 1;
  // few blocks: their heads split over several CTAs, as long as each of the eight warps has one
  const int64_t busy = p.total < (p.total >> p.lb) + p.B ? p.total : (p.total >> p.lb) + p.B;
  const int heads = 2 * p.Hkv + p.H;
  int shares = 1;
  while (busy * shares < 2 * num_sms && shares * 8 < heads) ++shares;
  const dim3 grid{unsigned((blocks + run - 1) / run), unsigned(shares)};
  return launch_pdl(kern, grid, dim3(kQAppendThreads), smem, stream, p);
}

template <int D, bool kInt8>
cudaError_t launch_qappend(const QAppendParams& p, int num_sms, cudaStream_t stream) {
  const int rows = p.rot > 0 ? 1 << p.lb : 0;
  if constexpr (D == 128) {
    // three heads of a warp under way, or two where that lets a second CTA into the SM, as with rotated blocks of 64
    // (3.1 GB: 707 us with three, 564 with two; blocks of 32, where two CTAs fit either way: 139 and 154 on 740 MB)
    if (qappend_ctas(D, qappend_smem(D, 2, rows)) > qappend_ctas(D, qappend_smem(D, 3, rows)))
      return launch_qappend<D, kInt8, 2>(p, rows, num_sms, stream);
  }
  return launch_qappend<D, kInt8, 3>(p, rows, num_sms, stream);
}

}  // namespace

cudaError_t launch_qcache_append(const jfa_qcache& q, const CacheAppend& a, void* ws, int num_sms, cudaStream_t stream) {
  const jfa_cache& c = q.cache;
  QAppendParams p;
  set_append_params(p, c, a, ws);
  p.k_cache = static_cast<uint8_t*>(c.k);
  p.v_cache = static_cast<uint8_t*>(c.v);
  p.k_scale = q.k_scale;
  p.v_scale = q.v_scale;
  p.lb = log2_of(q.block);
  p.lp = log2_of(c.page_size);
  p.blocks_per_page = c.page_size / q.block;
  const bool int8 = q.kind == JFA_CODES_INT8;
  if (c.d == 128) return int8 ? launch_qappend<128, true>(p, num_sms, stream) : launch_qappend<128, false>(p, num_sms, stream);
  return int8 ? launch_qappend<64, true>(p, num_sms, stream) : launch_qappend<64, false>(p, num_sms, stream);
}

}  // namespace jfa
