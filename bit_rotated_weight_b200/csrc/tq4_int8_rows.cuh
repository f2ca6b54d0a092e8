// The int8 rounding of a row, shared by the kernels that quantize rows.
#pragma once
#include "tq4_int8.h"

namespace tq4 {

// A row's divisor, 127 / max|x| = recip + lo to 48 bits.  `lift` is a power of
// two that takes rows of tiny or huge values to where both are normal numbers;
// it changes no quotient.
struct RowUnit {
  float top, recip, lo, lift, scale;
  bool finite;
  __device__ __forceinline__ explicit RowUnit(uint32_t top_bits) {
    finite = top_bits < 0x7F800000u;
    const float t = __uint_as_float(top_bits);
    scale = finite ? __fdiv_rn(t, 127.0f) : __uint_as_float(0x7FC00000u);
    lift = t < 1e-18f ? 0x1p64f : t > 1e18f ? 0x1p-64f : 1.0f;
    top = t * lift;
    recip = lo = 0.0f;
    if (finite && t > 0.0f) {
      recip = __fdiv_rn(127.0f, top);
      lo = __fdiv_rn(__fmaf_rn(-recip, top, 127.0f), top);   // (the remainder is exact)
    }
  }
};

// Codes are the low bytes of quotient + 1.5 * 2^23, which rounds to a whole
// number, ties to even.
constexpr float kRound = 12582912.0f;

template <int N>
__device__ __forceinline__ void pack_codes(bool finite, const uint32_t (&r)[N], uint32_t (&bytes)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint32_t b = prmt(prmt(r[i], r[i + 1], 0x0040), prmt(r[i + 2], r[i + 3], 0x0040), 0x5410);
    bytes[i / 4] = finite ? b : 0u;
  }
}

// The codes of N values of a 16-bit type.  x (recip + lo) is the real quotient
// to 2^-47, so its rounding is exact where the quotient is a tie (few bits),
// and any other quotient of two values of at most 11 bits is further from a
// tie than 2^-20 of itself, far above the rounding: no border needs a look.
template <int N>
__device__ __forceinline__ void codes_of_16(const RowUnit& u, const float (&v)[N], uint32_t (&bytes)[N / 4]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    r[i] = __float_as_uint(__fadd_rn(__fmaf_rn(v[i], u.recip, __fmul_rn(v[i], u.lo)), kRound));
  pack_codes<N>(u.finite, r, bytes);
}

// The codes of N fp32 values.  v * recip is within 127 * 2^-23 (1.6e-5) of the
// real quotient (two roundings of relative 2^-24); where it lies within 2e-5
// of a border, 127 v is compared with border * top, both exact in 64 bits (31
// and 32 significant bits).
template <int N>
__device__ __forceinline__ void codes_of_32(const RowUnit& u, const float (&v)[N], uint32_t (&bytes)[N / 4]) {
  uint32_t r[N];
  float worst = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float p = __fmul_rn(v[i], u.recip);
    const float m = __fadd_rn(p, kRound);
    r[i] = __float_as_uint(m);
    worst = fmaxf(worst, fabsf(__fsub_rn(p, __fsub_rn(m, kRound))));
  }
  if (worst > 0.49998f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float q = __uint_as_float(r[i]) - kRound, d = __fmul_rn(v[i], u.recip) - q;
      if (fabsf(d) <= 0.49998f) continue;
      const float border = q + copysignf(0.5f, d);
      const double l = 127.0 * static_cast<double>(v[i]), e = static_cast<double>(border) * static_cast<double>(u.top);
      r[i] = __float_as_uint((l > e ? border + 0.5f : l < e ? border - 0.5f : rintf(border)) + kRound);
    }
  }
  pack_codes<N>(u.finite, r, bytes);   // (0 * inf and NaN end here)
}

// 16 bytes of a row as fp32, and the largest |v| in them, as fp32 bits.  Bits
// without the sign order like the values do, NaN and infinities on top, so the
// maximum of 16-bit types is taken on pairs before any conversion.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint32_t top(const uint4& r) {
    return max(max(r.x & 0x7FFFFFFFu, r.y & 0x7FFFFFFFu), max(r.z & 0x7FFFFFFFu, r.w & 0x7FFFFFFFu));
  }
  static __device__ __forceinline__ uint32_t top_f32(uint32_t t) { return t; }
  static __device__ __forceinline__ void codes(const RowUnit& u, const float (&v)[4], uint32_t (&b)[1]) {
    codes_of_32(u, v, b);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
};
struct Vec16 {
  static constexpr int N = 8;
  static __device__ __forceinline__ void codes(const RowUnit& u, const float (&v)[8], uint32_t (&b)[2]) {
    codes_of_16(u, v, b);
  }
  static __device__ __forceinline__ uint32_t top(const uint4& r) {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t t = __vmaxu2(__vmaxu2(r.x & m, r.y & m), __vmaxu2(r.z & m, r.w & m));
    return max(t & 0xFFFFu, t >> 16);
  }
};
template <>
struct Vec<__nv_bfloat16> : Vec16 {
  static __device__ __forceinline__ uint32_t top_f32(uint32_t t) { return t << 16; }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Vec<__half> : Vec16 {
  static __device__ __forceinline__ uint32_t top_f32(uint32_t t) {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(t))));
  }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};

}  // namespace tq4
