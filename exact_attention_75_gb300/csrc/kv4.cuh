// A key/value cache held in 4 bits: the format of a row and its way back to 16
// bits.
//
// A row of D channels takes 5 D / 8 bytes: D / 2 bytes of codes (channel 2 i in
// the low half of byte i), then for each 32 channels a scale s and a minimum m
// in the cache's 16-bit type T.  A code c in 0..15 stands for m + c s.  The
// quantizer (append4.cu) sets, over the 32 values x of a group,
//   m = min x,  s = RN_T((max x - m) / 15),  c = min(RN((x - m) / s), 15),
// so m is a value of the group and x is off by s / 2 at most, but at the
// largest, where the rounding of s may add 15 half steps of s.  A group with an
// infinity or a NaN, or whose range passes fp32, has s = m = NaN: all of it
// stands for NaN.  Where s rounded up would carry code 15 past the range of T, it is
// the number below.
//
// Values take part in products as RN_T(m + c s), one fused multiply-add of two
// 16-bit values at a time: half a step of T, the error that a 16-bit cache has in the
// first place.  Keys do not: an error of 2^-9 a channel, even
// of 2^-12, shows in the log-sum-exp of a short sequence.  A code's product with a
// query is exact, and so is that of c - 8, which has three significant bits, with a
// scale of 8 bits; so
//   q . k = sum over groups of  s sum q c  +  m sum q
// is taken with s and m in 32 bits (decoding), or as
//           sum over groups of  sum q ((c - 8) s)  +  (m + 8 s) sum q
// with the second part split into 16-bit terms (chunks).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "sm103_ptx.cuh"

namespace attn {

constexpr int kKv4Group = 32;
constexpr int kv4_row(int d) { return d / 2 + d / 8; }  // bytes

#ifdef __CUDACC__

// (w & mask) | bits, as the one instruction that it is (the compiler makes two of
// them where both are constants).
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
  return r;
}

// Two codes (bits 0-3 and 16-19 of w) less ZERO as 16-bit numbers: their bits in
// the mantissa of 2^7 (bf16) or 2^10 (fp16), less that power and ZERO.
template <bool BF16, int ZERO>
__device__ __forceinline__ uint32_t kv4_codes(uint32_t w) {
  uint32_t r;
  if constexpr (BF16)
    asm("sub.rn.bf16x2 %0, %1, %2;"
        : "=r"(r)
        : "r"(and_or(w, 0x000F000Fu, 0x43004300u)), "r"(0x43004300u + 0x10001u * ZERO));
  else
    asm("sub.rn.f16x2 %0, %1, %2;"
        : "=r"(r)
        : "r"(and_or(w, 0x000F000Fu, 0x64006400u)), "r"(0x64006400u + 0x10001u * ZERO));
  return r;
}

// The codes of a word in fp16, nibbles i and i + 4 side by side; those of odd i times
// 16, since their bits are taken where they stand (one shift a word, not three).
__device__ __forceinline__ void kv4_halves(uint32_t w, uint32_t (&v)[4]) {
  const uint32_t x[2] = {w, w >> 8};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("sub.rn.f16x2 %0, %1, %2;"
        : "=r"(v[i])
        : "r"(and_or(x[i / 2], i & 1 ? 0x00F000F0u : 0x000F000Fu, 0x64006400u)),
          "r"(0x64006400u));
}

// What the codes of a word stand for, nibbles i and i + 4 side by side.
template <bool BF16>
__device__ __forceinline__ void kv4_values(uint32_t w, uint32_t s, uint32_t m, uint32_t (&v)[4]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("fma.rn.bf16x2 %0, %1, %2, %3;"
          : "=r"(v[i])
          : "r"(kv4_codes<true, 0>(w >> (4 * i))), "r"(s), "r"(m));
  } else {
    const uint32_t x[2] = {w, w >> 8};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c;
      if (i & 1)  // (1024 + 16 c) / 16 - 64
        asm("fma.rn.f16x2 %0, %1, %2, %3;"
            : "=r"(c)
            : "r"(and_or(x[i / 2], 0x00F000F0u, 0x64006400u)), "r"(0x2C002C00u), "r"(0xD400D400u));
      else
        c = kv4_codes<false, 0>(x[i / 2]);
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(c), "r"(s), "r"(m));
    }
  }
}

// Two 16-bit values in 32 bits.
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// 2^k that takes the finite number of bits `top` (>= 0) to 2^T .. 2^(T + 1), and 2^-k.
// Both are normal numbers; zero is left where it is.  (fp16 has full precision down
// to 2^-14 and steps of 2^-24 below.)
template <int T>
__device__ __forceinline__ float2 to_fp16_range(uint32_t top) {
  const uint32_t e = top == 0u ? 127u + T : top >> 23;
  const uint32_t up = min(254u + T - e, 253u);
  return make_float2(__uint_as_float(up << 23), __uint_as_float((254u - up) << 23));
}

// Bits of |x|, 0 for infinities and NaN: ordered like the numbers.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// A row of queries as the operand that meets kv4_halves: a quad of lanes has the row,
// lane t channels 32 c + 8 t .. of each group in q[c], which become fp16 in channel
// pairs (i, i + 4), scaled into its range by a power of two, those of odd i over 16:
// half a step of fp16's least numbers, 2^-25, is 2^-34 of the row's largest (even i) or
// 2^-30 where that is brought to 2^9, as the sums of an fp16 cache need to stay in range
// (kv4_sum_terms), and 2^-35 where it is brought to 2^14.
// sums: of the scaled row over each group.  Returns the factor that undoes the
// scaling.  All lanes of the warp call this.
template <bool BF16, int C>
__device__ __forceinline__ float kv4_query(uint4 (&q)[C], float* sums) {
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t y[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<BF16>(y[i]);
      top = max(top, max(finite_bits(f.x), finite_bits(f.y)));
    }
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const float2 f = to_fp16_range<BF16 ? 14 : 9>(top);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t y[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
    float z[8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<BF16>(y[i]);
      z[2 * i] = v.x * f.x;
      z[2 * i + 1] = v.y * f.x;
      sum += z[2 * i] + z[2 * i + 1];
    }
    q[c] = make_uint4(pack_f16x2(z[0], z[4]), pack_f16x2(z[1] * 0.0625f, z[5] * 0.0625f),
                      pack_f16x2(z[2], z[6]), pack_f16x2(z[3] * 0.0625f, z[7] * 0.0625f));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sums[c] = sum + __shfl_xor_sync(0xffffffffu, sum, 2);
  }
  return f.y;
}

// What takes a scaled row's products to base 2.  Neither 0 nor infinite, since a masked
// product, -inf, times 0 would be NaN, and so would 0 times infinity.  Products are below
// 2^124 (keys below 2^100), so that one with the least number, 2^-149, counts nothing;
// one that 1e37 is too little for is infinite as an exponent anyway.
__device__ __forceinline__ float kv4_to_base2(float scale_log2, float undo) {
  return fminf(fmaxf(scale_log2 * undo, 0x1p-149f), 1e37f);
}

// What the minima of the groups add to a score, sum over groups of m sum q, as a product
// of its own in the cache's type, 16 deep: the sum of a query over a group is cut into
// three terms, which meet the group's minimum one by one.  Each quad of lanes has a query
// (operand B) and a key (A, both its registers alike); what no term needs is 0 in B.
template <bool BF16, int C>
__device__ __forceinline__ uint2 kv4_sum_terms(const float (&sums)[C], int t) {
  const bool odd = C > 2 && t & 1;  // groups 2 and 3, not 0 and 1
  float a = sums[0], b = sums[1];
  if (odd) {
    a = sums[C > 2 ? 2 : 0];
    b = C > 3 ? sums[C > 3 ? 3 : 0] : 0.f;
  }
  uint32_t term[3];
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    term[n] = BF16 ? pack_bf16x2(a, b) : pack_f16x2(a, b);
    const float2 had = unpack2<BF16>(term[n]);
    a = isfinite(a) ? a - had.x : 0.f;
    b = isfinite(b) ? b - had.y : 0.f;
  }
  if constexpr (C == 2)
    return make_uint2(t == 0 ? term[0] : (t == 1 ? term[1] : (t == 2 ? term[2] : 0u)), 0u);
  return make_uint2(t < 2 ? term[0] : term[1], t < 2 ? term[2] : 0u);
}
// par: s and m of the key's groups.
template <int C>
__device__ __forceinline__ uint32_t kv4_minima(const uint32_t (&par)[C], int t) {
  const uint32_t low = __byte_perm(par[0], par[1], 0x7632);
  if constexpr (C == 2) return low;
  return t & 1 ? __byte_perm(par[C > 2 ? 2 : 0], C > 3 ? par[C > 3 ? 3 : 0] : 0u, 0x7632) : low;
}

// The eight values of a code word, in channel order or (ORDER false) as channels 0, 4,
// 1, 5, 2, 6, 3, 7; par: s and m of its group.
template <bool BF16, bool ORDER = true>
__device__ __forceinline__ uint4 kv4_word(uint32_t w, uint32_t par) {
  const uint32_t s = __byte_perm(par, par, 0x1010), m = __byte_perm(par, par, 0x3232);
  uint32_t v[4];  // channels i and i + 4
  kv4_values<BF16>(w, s, m, v);
  if constexpr (!ORDER) return make_uint4(v[0], v[1], v[2], v[3]);
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                    __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

// The eight codes of a word less 8, times the two s in fp16 (s / 16 in odd), as channels
// 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ uint4 kv4_scaled_word(uint32_t w, uint32_t even, uint32_t odd) {
  const uint32_t x[2] = {w, w >> 8};
  uint32_t v[4];  // channels i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t c;  // times 16 for odd i
    asm("sub.rn.f16x2 %0, %1, %2;"
        : "=r"(c)
        : "r"(and_or(x[i / 2], i & 1 ? 0x00F000F0u : 0x000F000Fu, 0x64006400u)),
          "r"(i & 1 ? 0x64806480u : 0x64086408u));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(c), "r"(i & 1 ? odd : even));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

#endif  // __CUDACC__

}  // namespace attn
