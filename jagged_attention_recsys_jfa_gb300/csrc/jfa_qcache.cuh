// The 8-bit cache's codes: e4m3 or int8, [num_pages][H_kv][page_size][d]; the `block` tokens of an aligned block
// of a page and head share one fp32 scale, [num_pages][H_kv][page_size / block]; a value is code * scale.
#pragma once
#include "jfa_cache.cuh"

namespace jfa {

// Four codes as f16x2 pairs: codes 0, 1 (lo) and 2, 3 (hi).  Both types are exact in f16: e4m3 has 4
// significant bits and exponents of -9 to 8, int8 needs 8 of f16's 11 bits (1024 + u, u = code + 128, is the
// f16 0x6400 | u, from which 1152 is taken away).
template <bool kInt8>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kInt8) {
    w ^= 0x80808080u;
    lo = sub_f16x2(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
    hi = sub_f16x2(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    lo = e4m3_lo_f16x2(w);
    hi = e4m3_hi_f16x2(w);
  }
}
// Four values as codes, to the nearest, ties to even (int8: -128 <= x <= 127, added to 1.5 * 2^23).
template <bool kInt8>
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
  if (kInt8) {
    auto low = [](float x) { return __float_as_uint(x + 12582912.f); };
    return __byte_perm(__byte_perm(low(a), low(b), 0x0040), __byte_perm(low(c), low(d), 0x0040), 0x5410);
  }
  return pack_e4m3x2(a, b) | pack_e4m3x2(c, d) << 16;
}

// Tokens of a scale's block, and of a page, are powers of two.
inline int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

}  // namespace jfa
