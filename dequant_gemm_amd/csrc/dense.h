// dense.h -- device helpers of the dense products (fp8.hip, gated_ff.hip): e4m3 values, the
// gate's activations and outputs in three types.
#pragma once
#include <type_traits>

#include "act_quant.h"
#include "common.h"

namespace cubic {

constexpr float kE4m3Max = 448.0f;

// The largest magnitudes of 16-bit values by their bits, two at a time: NaN is the largest.
__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t mag8(const u32x4& v, uint32_t a) {
#pragma unroll
  for (int e = 0; e < 4; ++e) a = mag_max(a, v[e] & 0x7fff7fffu);
  return a;
}
// Of LANES neighbouring lanes, in each of them.
template <int LANES>
__device__ __forceinline__ uint32_t mag_lanes(uint32_t v) {
  auto step = [&](auto ctrl_c) {
    v = mag_max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), decltype(ctrl_c)::value, 0xf, 0xf, false)));
  };
  step(std::integral_constant<int, 0xb1>{});     // quad_perm [1, 0, 3, 2]
  step(std::integral_constant<int, 0x4e>{});     // quad_perm [2, 3, 0, 1]
  step(std::integral_constant<int, 0x141>{});    // row_half_mirror
  if constexpr (LANES >= 16) step(std::integral_constant<int, 0x140>{});   // row_mirror
  if constexpr (LANES == 64) {
    v = mag_max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16, 64)));
    v = mag_max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 32, 64)));
  }
  return v;
}
template <bool F16>
__device__ __forceinline__ float mag_value(uint32_t v) {
  const uint32_t m = max(v & 0xffffu, v >> 16);
  return F16 ? static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(m))) : __uint_as_float(m << 16);
}

// Two fp32 values as e4m3 codes in the low or high half of a word, to nearest, ties to even.
template <bool HI>
__device__ __forceinline__ uint32_t fp8_pack2(float a, float b, uint32_t old) {
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a, b, static_cast<int>(old), HI));
}

// A block's scale, fp32(amax / 448), and its reciprocal, both correctly rounded: the quotient as
// below (equal to the division for every 16-bit amax in the range), the reciprocal by one Newton step from
// the hardware's, except where the scale's significand is all ones. A block of zeros has 0 for both.
// sign: the bit that codes take over from their values, none in a block of zeros.
struct Fp8Scale {
  float s, r;
  uint32_t sign;
  bool fast;
};
__device__ __forceinline__ Fp8Scale fp8_scale_of(float amax) {
  Fp8Scale v;
  const float q = amax * (1.0f / kE4m3Max);
  v.s = fmaf(fmaf(-q, kE4m3Max, amax), 1.0f / kE4m3Max, q);
  const float r = __builtin_amdgcn_rcpf(v.s);
  const bool zeros = amax == 0.0f;
  v.r = zeros ? 0.0f : fmaf(fmaf(-v.s, r, 1.0f), r, r);
  const bool in_range = v.s >= 0x1p-80f && v.s <= 0x1p100f;
  v.fast = zeros || (in_range && (__float_as_uint(v.s) & 0x7fffffu) != 0x7fffffu);
  if (!zeros && !in_range) v.s = __fdiv_rn(amax, kE4m3Max);
  v.sign = zeros ? 0u : 0x80000000u;
  return v;
}

// The codes of eight 16-bit values: e4m3(fp32(x / s)), at most 448 in magnitude; s = 0 gives
// zeros, a NaN stays one (the comparisons below pass it on). The quotient without a division:
// q = fl(x r) is within an ulp, its residual x - q s is exact in one fma, and fl(q + residual r)
// is the correctly rounded quotient (Markstein; equal to the division for every pair of
// significands of a scale and a 16-bit value), but for x = -0, whose residual is +0 and whose q that
// makes +0: the sign comes from x. Scales outside [2^-80, 2^100], where the residual
// might not be exact, take the division. Rounding 448 (1 + 2^-24) to e4m3 gives 448 by itself.
// 4096 x 7168 rows: 28.7 us with divisions, 19 us so.
template <bool XF16>
__device__ __forceinline__ uint2 fp8_quant8(const u32x4& v, const Fp8Scale& scale) {
  float f[8];
  unpack8<XF16>(v, f);
  if (scale.fast) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = f[i] * scale.r;
      const float c = fmaf(fmaf(-q, scale.s, f[i]), scale.r, q);
      f[i] = __uint_as_float((__float_as_uint(c) & ~scale.sign) | (__float_as_uint(f[i]) & scale.sign));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float t = scale.s != 0.0f ? __fdiv_rn(f[i], scale.s) : 0.0f;
      t = t > kE4m3Max ? kE4m3Max : t;
      f[i] = t < -kE4m3Max ? -kE4m3Max : t;
    }
  }
  return make_uint2(fp8_pack2<true>(f[2], f[3], fp8_pack2<false>(f[0], f[1], 0u)),
                    fp8_pack2<true>(f[6], f[7], fp8_pack2<false>(f[4], f[5], 0u)));
}

// Eight e4m3 codes as bf16 (exact).
__device__ __forceinline__ bf16x8 e4m3x8_to_bf16(const u32x2& v) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const int lo = static_cast<int>(v.x), hi = static_cast<int>(v.y);
  const bf16x2 a = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
  const bf16x2 b = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
  const bf16x2 c = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
  const bf16x2 d = __builtin_bit_cast(bf16x2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 16 bits of an fp32 value in bf16 or fp16, rounded to nearest even (NaN stays NaN).
template <bool F16>
__device__ __forceinline__ uint32_t bits16(float v) {
  if constexpr (F16) {
    return f16_bits(v);
  } else {
    return v != v ? ((__float_as_uint(v) >> 16) | 0x40u) : bf16_rne_bits(v);
  }
}

// Output element idx in fp32 (0), bf16 (1) or fp16 (2), rounded once.
__device__ __forceinline__ void store_as(void* y, int dt, int64_t idx, float v) {
  if (dt == 0) {
    static_cast<float*>(y)[idx] = v;
  } else {
    static_cast<uint16_t*>(y)[idx] = static_cast<uint16_t>(dt == 2 ? bits16<true>(v) : bits16<false>(v));
  }
}

// The gate's activation and its derivative. With p = 1 / (1 + exp(-z)):
//   SiLU            a = g p,  a' = p (1 + g (1 - p)),  z = g
//   GELU (tanh)     a = g p,  a' = p + g p (1 - p) z',  z = 2 sqrt(2 / pi) (g + 0.044715 g^3)
// (0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)), which keeps the digits of the negative tail).
struct Act {
  float value, slope;
};
// The hardware's exp2 and reciprocal: within |z| 2^-23 + 2^-21 relative, where a 16-bit result
// rounds by 2^-8 or 2^-11 (libm's expf and a division took 9 us of 4096 x 2048 gates, these 4).
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
constexpr float kGeluC = 1.5957691216057308f, kGeluK = 0.044715f;   // 2 sqrt(2 / pi)

__device__ __forceinline__ Act act_of(float g, int gelu) {
  if (gelu) {
    const float g2 = g * g;
    const float z = kGeluC * g * fmaf(kGeluK, g2, 1.0f);
    const float p = logistic(z);
    // p (1 - p) is 0 in fp32 well before g^2 overflows
    const float bend = g2 < 1e4f ? g * p * (1.0f - p) * kGeluC * fmaf(3.0f * kGeluK, g2, 1.0f) : 0.0f;
    return {g * p, p + bend};
  }
  const float p = logistic(g);
  return {g * p, p * fmaf(g, 1.0f - p, 1.0f)};
}

}  // namespace cubic
