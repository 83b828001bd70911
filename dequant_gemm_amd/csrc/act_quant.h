// act_quant.h -- the per-row INT8 quantiser's arithmetic on eight values at a time,
// shared by act_quant_int8_per_token (basic.hip) and the int8 product that
// quantises its rows itself (w8a8.hip).
#pragma once
#include "common.h"

namespace cubic {

// Per-row INT8 quantisation (the msModelSlim article's per-token dynamic scheme,
// with this library's reading of the A8 scale): sx = fp32(amax / 127) and
// q = clamp(rne(fp32(x / sx)), -127, 127), bit for bit.
//
// The quotient is not formed per element. With r = v_rcp_f32(sx) (1 ulp),
// x * r is within 2^-16 of x / sx for |x| <= amax, and the IEEE quotient within
// 2^-18, so whenever x * r lies more than 2^-14 from every half-integer both
// round to the same integer. One fma against 1.5 * 2^23 rounds x * r to the
// nearest integer n (ties to even) and leaves n in the low byte of its bits;
// a second fma gives the residual x * r - n. Lanes with a residual within 2^-14
// of one half, and rows whose scale lies outside [2^-100, 2^100] (tiny or huge
// rows, where the bound or the reciprocal fails), take the IEEE division.
constexpr float kRneMagic = 12582912.0f;        // 1.5 * 2^23

// A row's scale: fp32(amax / 127) (act_quant_int8_per_token), or with RECIP
// fp32(amax * fp32(1 / 127)) (cubic_linear_w8a8).
template <bool RECIP>
__device__ __forceinline__ float scale_of(float amax) {
  return RECIP ? amax * (1.0f / 127.0f) : __fdiv_rn(amax, 127.0f);
}

// The larger of two magnitudes. RECIP: of their bits, so that a NaN is the largest and
// reaches the row's scale; else a NaN is passed over.
template <bool RECIP>
__device__ __forceinline__ float larger(float a, float b) {
  if constexpr (RECIP) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
  } else {
    return fmaxf(a, b);
  }
}

// Eight bf16 (or, with XF16, fp16) values of one 16-byte vector as fp32 (exact).
template <bool XF16>
__device__ __forceinline__ void unpack8(const u32x4& v, float* xv) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (XF16) {
      xv[2 * q] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(u[q] & 0xffffu)));
      xv[2 * q + 1] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(u[q] >> 16)));
    } else {
      xv[2 * q] = __uint_as_float(u[q] << 16);
      xv[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
    }
  }
}

// Their eight int8 codes.
template <bool XF16>
__device__ __forceinline__ uint2 quant8(const u32x4& v, float sx, float rcp, bool fast) {
  float xv[8];
  unpack8<XF16>(v, xv);
  uint32_t f[8];
  bool exact = !fast;
  if (fast) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = fmaf(xv[e], rcp, kRneMagic);
      const float n = y - kRneMagic;                 // exact: the rounded integer
      const float t = fmaf(xv[e], rcp, -n);          // x * r - n, one rounding
      exact = exact || fabsf(t) > 0.5f - 0x1p-14f;
      f[e] = __float_as_uint(y);                     // low byte: n (two's complement)
    }
  }
  if (exact) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int qi = 0;
      if (sx != 0.0f) {
        float r = rintf(__fdiv_rn(xv[e], sx));
        r = fminf(fmaxf(r, -127.0f), 127.0f);
        qi = static_cast<int>(r);
      }
      f[e] = static_cast<uint32_t>(qi);
    }
  }
  const uint32_t lo = __builtin_amdgcn_perm(f[1], f[0], 0x0c0c0400u) | __builtin_amdgcn_perm(f[3], f[2], 0x04000c0cu);
  const uint32_t hi = __builtin_amdgcn_perm(f[5], f[4], 0x0c0c0400u) | __builtin_amdgcn_perm(f[7], f[6], 0x04000c0cu);
  return make_uint2(lo, hi);
}

template <bool XF16, bool RECIP>
__device__ __forceinline__ float absmax8(const u32x4& v, float a) {
  float xv[8];
  unpack8<XF16>(v, xv);
#pragma unroll
  for (int e = 0; e < 8; ++e) a = larger<RECIP>(a, fabsf(xv[e]));
  return a;
}

// The largest of the wave's magnitudes, in every lane.
template <bool RECIP>
__device__ __forceinline__ float wave_larger(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = larger<RECIP>(v, __shfl_xor(v, o, 64));
  return v;
}

}  // namespace cubic
