// dense.h -- device helpers of the dense products (fp8.hip, gated_ff.hip): e4m3 values, the
// gate's activations and outputs in three types.
#pragma once
#include "act_quant.h"
#include "common.h"

namespace cubic {

constexpr float kE4m3Max = 448.0f;

// A block's scale: fp32(amax / 448), one rounding.
__device__ __forceinline__ float fp8_scale(float amax) { return __fdiv_rn(amax, kE4m3Max); }

// Two fp32 values as e4m3 codes in the low or high half of a word, to nearest, ties to even.
template <bool HI>
__device__ __forceinline__ uint32_t fp8_pack2(float a, float b, uint32_t old) {
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a, b, static_cast<int>(old), HI));
}

// A block's scale with its reciprocal, correctly rounded (one Newton step from the hardware's,
// except where the scale's significand is all ones).
struct Fp8Scale {
  float s, r;
  bool fast;
};
__device__ __forceinline__ Fp8Scale fp8_scale_of(float amax) {
  Fp8Scale v;
  v.s = fp8_scale(amax);
  const float r = __builtin_amdgcn_rcpf(v.s);
  v.r = fmaf(fmaf(-v.s, r, 1.0f), r, r);
  v.fast = v.s >= 0x1p-80f && v.s <= 0x1p100f && (__float_as_uint(v.s) & 0x7fffffu) != 0x7fffffu;
  return v;
}

// The codes of eight 16-bit values: e4m3(fp32(x / s)), at most 448 in magnitude; s = 0 gives
// zeros, a NaN stays one (the comparisons below pass it on). The quotient without a division:
// q = fl(x r) is within an ulp, its residual x - q s is exact in one fma, and fl(q + residual r)
// is the correctly rounded quotient (Markstein; equal to the division for every pair of
// significands of a scale and a 16-bit value). Scales outside [2^-80, 2^100], where the residual
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
      f[i] = fmaf(fmaf(-q, scale.s, f[i]), scale.r, q);
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
