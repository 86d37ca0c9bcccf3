// The 4-bit codes of a quantised cache.
//
//   16 neighbouring channels of a token's key or value share a scale
//     s_j = (8 + j % 8) 2^(j / 8 - 23),  j = 0 .. 255  (2^-20 .. 1.875 2^11),
//   the first with 7 s_j >= max |x|, and channel c is held as the integer
//     q_c in -7 .. 7 nearest to x_c / s_j, ties away from zero.
//
// Why this form: an integer below 8 times a scale of four significant bits is
// a bf16 number, so what is held is exact in bf16 and the products over it
// need no rounding of their own; a scale's byte becomes a bf16 with a shift
// and an add; the range needs no calibration.  4.5 bits a channel.  A float
// format of 4 bits would cost the same bits and one more product of rounding.
//
// x is a bf16 number, and so is every tie (n + 1/2) s_j, n < 7: eight bits
// hold (2 n + 1)(8 + j % 8).  So any other x is off a tie by 2^-8 of it or
// more, and a product with (1 + 2^-16) / s_j, its errors of a few 2^-24
// included, rounds to the same integer as the exact quotient does, and a tie
// away from zero.  The same holds for 7 s_j against max |x|.
//
// A 32-bit word holds 8 channels: channel 2 i in bits 4 i .. 4 i + 3, channel
// 2 i + 1 in bits 16 + 4 i .. 16 + 4 i + 3, two's complement, so that one
// shift and one logical operation make neighbours a bf16x2.  A tile is
// min(page_size, 128) tokens of one head: their keys' codes (d / 2 bytes a
// token), values' codes, keys' scales (d / 16 bytes a token) and values'
// scales; it is one contiguous piece, so that a block of keys with its values
// comes with one bulk copy a page.
#pragma once

#include <stdint.h>

#include "hstu_bf16x8.cuh"

namespace hstu {
namespace {

constexpr int kQ4Group = 16;  // channels of a scale

// Bytes of a token in one head: its key and its value.
__host__ __device__ constexpr int q4_token_bytes(int d) { return 2 * (d / 2 + d / kQ4Group); }

// Byte of token row r of a tile: its keys' or values' codes, and scales.
template <int D>
struct Q4Tile {
  static constexpr int CODEB = D / 2, SCALEB = D / kQ4Group;
  static __device__ __forceinline__ int codes(int shift, int which, int r) {
    return (which * CODEB << shift) + r * CODEB;
  }
  static __device__ __forceinline__ int scales(int shift, int which, int r) {
    return ((2 * CODEB + which * SCALEB) << shift) + r * SCALEB;
  }
};

// ---------------------------------------------------------------- from codes
// bf16 bits of 16 s_j, in both halves of a word, for two scales' bytes j, and
// for one.
__device__ __forceinline__ uint32_t q4_scales(uint32_t j_lo, uint32_t j_hi) {
  return j_lo * 0x10u + (j_hi * 0x100000u + (111u << 7) * 0x10001u);
}
__device__ __forceinline__ uint32_t q4_scales(uint32_t j) { return j * 0x100010u + (111u << 7) * 0x10001u; }
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// A scale pair as the products below want it: 16 s and -24 s (exact).
struct Q4Scale {
  uint32_t s16, s24;
};
__device__ __forceinline__ Q4Scale q4_scale_of(uint32_t s) { return Q4Scale{s, mul_bf16x2(s, 0xbfc0bfc0u)}; }
__device__ __forceinline__ Q4Scale q4_scale(uint32_t j_lo, uint32_t j_hi) {
  return q4_scale_of(q4_scales(j_lo, j_hi));
}
__device__ __forceinline__ Q4Scale q4_scale(uint32_t j) { return q4_scale_of(q4_scales(j)); }
// The codes in nibble I of both halves of w: 1 + (8 + q) / 16 as bf16, then
// 16 s (1 + (8 + q) / 16) - 24 s = q s, exact.
template <int I>
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, const Q4Scale& s) {
  const uint32_t at = I == 0 ? w << 3 : w >> (4 * I - 3);
  return fma_bf16x2((at & 0x00780078u) ^ 0x3fc03fc0u, s.s16, s.s24);
}
// A word's 8 channels in their order.
__device__ __forceinline__ uint4 q4_word(uint32_t w, const Q4Scale& s) {
  return make_uint4(q4_pair<0>(w, s), q4_pair<1>(w, s), q4_pair<2>(w, s), q4_pair<3>(w, s));
}

// ------------------------------------------------------------------ to codes
// Two bf16 numbers as they are held at most: +-26880, 7 times the largest scale
// (0x46d2), and NaN as 0.
constexpr uint32_t kQ4Most = 0x46d2u;
__device__ __forceinline__ uint32_t q4_clamp(uint32_t x) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    const uint32_t h = x >> i & 0xffffu, m = h & 0x7fffu;
    r |= (m > 0x7f80u ? 0u : m > kQ4Most ? (h & 0x8000u) | kQ4Most : h) << i;
  }
  return r;
}

// The codes of this lane's half of a group, 8 channels, and the group's scale's
// byte; the other half is the next lane's (or the one's before).  Whole-warp
// call.
__device__ __forceinline__ uint32_t q4_quantise(const uint4& half, uint32_t* scale) {
  uint32_t x[4] = {half.x, half.y, half.z, half.w};
  auto largest = [&x] {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, x[i] & 0x7fff7fffu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m & 0xffffu, m >> 16);
  };
  uint32_t m = largest();
  if (__any_sync(0xffffffffu, m > kQ4Most)) {  // past the largest scale, or not finite
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = q4_clamp(x[i]);
    m = largest();
  }
  // max / 7, less 2^-16 of it, rounded up to four significant bits
  const float seventh = __uint_as_float(m << 16) * (float)((1.0 - 0x1p-16) / 7.0);
  const int j = max((int)((__float_as_uint(seventh) + 0xfffffu) >> 20) - (107 << 3), 0);  // <= 255: m is clamped
  *scale = (uint32_t)j;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(__uint_as_float((uint32_t)(j + (107 << 3)) << 20)));
  inv *= 1.0f + 0x1p-16f;
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the integers in the low bits of 1.5 2^23 + x / s
    const float2 y =
        __ffma2_rn(make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)),
                   make_float2(inv, inv), make_float2(12582912.f, 12582912.f));
    const uint32_t both = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x5410);
    w |= (both & 0x000f000fu) << (4 * i);
  }
  return w;
}

}  // namespace
}  // namespace hstu
