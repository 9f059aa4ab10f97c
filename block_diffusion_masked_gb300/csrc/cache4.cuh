// Paged 4-bit key/value cache: its format, shared by the host (tests) and the
// kernels.
//
// Layout.  k_cache, v_cache: (pages, kv_heads, page_size, headdim / 2) bytes, a 32-bit
// word for eight neighbouring dims of a token, the even ones in its low half, the odd
// ones in its high half, the first in the lowest four bits.  k_scale, v_scale: (pages,
// kv_heads, headdim / 32, page_size) e5m2, the tokens of one group of dims next to
// one another: the kernels want one group of several tokens at a time.  A value is
// (code - 8) times the scale s of its token, head and 32 dims.
//
// Why this format.  A signed scale gives the largest magnitude the code that has
// no counterpart, -8, so that the step is amax / 8 and not amax / 7.  Scales of three
// significant bits cost up to a fourth of a step and make every value a product of
// four bits and three: exact in f16 and bf16, so that neither the attention nor the
// reading back rounds anything.  e5m2 is the upper byte of f16: a scale is decoded by
// moving its byte.  A token's scale depends on the token alone, so nothing is rounded
// twice, whatever is appended to its page later.  The halves of a word are decoded side
// by side, so that neighbouring dims come out as the pairs that products and stores
// take.
#pragma once

#include <stdint.h>

#include "geometry.cuh"
#if defined(__CUDACC__)
#include <cuda_fp16.h>
#endif

namespace dfa {

constexpr int kCache4Group = 32;
// The e5m2 bytes of 2^-14 (the smallest normal one) and 896 = 1.75 * 2^9, the most
// that the attention's decoding (below) can hold; and of a value that is not a number.
constexpr int kCache4MinScale = 0x04, kCache4MaxScale = 0x63, kCache4NanScale = 0x7f;

// The scale's byte of a group with the largest key `top` among its values: a value's
// bf16 bits with the sign moved below the magnitude (2 |x| + sign), so that a
// negative value comes above a positive one of the same magnitude.
DFA_HD int cache4_scale_byte(unsigned top) {
  const unsigned mag = top >> 1;
  if (mag >= 0x7f80u) return kCache4NanScale;
  // up to two bits behind the leading one of seven, exponent: bias 127 -> 15, / 8
  int e = static_cast<int>((mag + 31u) >> 5) - ((127 - 15 + 3) << 2);
  e = e < kCache4MinScale ? kCache4MinScale : e > kCache4MaxScale ? kCache4MaxScale : e;
  return mag != 0 && (top & 1u) == 0 ? e | 0x80 : e;
}

#if defined(__CUDACC__)
// The scale of a byte, as float.
__device__ __forceinline__ float cache4_scale(unsigned byte) {
  const unsigned short h = static_cast<unsigned short>(byte << 8);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// cache4_decode gives a sixteenth of the values: all of its steps are exact then, with
// half of the codes left where they stand.
constexpr float kCache4Unit = 16.f;
// Two scales s as f16x2, prepared for it.
struct Cache4Scale {
  __half2 low, low_bias, high, high_bias;  // s / 16, -64.5 s; s / 256, -4.5 s
};
__device__ __forceinline__ Cache4Scale cache4_prepare(uint32_t s2) {
  const __half2 s = *reinterpret_cast<const __half2*>(&s2);
  return {__hmul2(s, __float2half2_rn(0.0625f)), __hmul2(s, __float2half2_rn(-64.5f)),
          __hmul2(s, __float2half2_rn(0.00390625f)), __hmul2(s, __float2half2_rn(-4.5f))};
}
// Codes 4 i .. 4 i + 3 of the low half of w and of its high half, as four pairs of f16
// values, low half first, each (n - 8) s / 16.  A code n in bits 0 to 3 of f16's 1024 makes
// it 1024 + n: times s / 16 less 1032 s / 16; in bits 4 to 7, 1024 + 16 n: times s / 256
// less 72 s / 16.  The factors are products of s' three bits with powers of two, 129 / 2 and
// 9 / 2, at most 57792 and at least steps of 2^-24: exact in f16, and so are the sums.
__device__ __forceinline__ void cache4_decode(uint32_t w, const Cache4Scale& s, uint32_t (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t from = i < 2 ? w : w >> 8;
    const uint32_t x = (from & (i & 1 ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
    const __half2 n = *reinterpret_cast<const __half2*>(&x);
    const __half2 y = i & 1 ? __hfma2(n, s.high, s.high_bias) : __hfma2(n, s.low, s.low_bias);
    f[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}
#endif

}  // namespace dfa
