// gated_ff.hip -- the gated feed-forward block over 16-bit weights and its backward pass.
//
//   [g | u] = x W^T,  h = act(g) * u;   dg = dh * u * act'(g),  du = dh * act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
#include <type_traits>

#include "common.h"
#include "dense.h"
#include "launch.h"

namespace cubic {
namespace {

// C[m][n] = sum_k A(m, k) B(n, k) for 64 x 64 outputs a workgroup, 32 k a step. A(m, k) is
// a[m * lda + k], or with AT a[k * lda + m]; B likewise.
template <bool F16, bool AT, bool BT>
__global__ __launch_bounds__(256) void k_simple16(const uint16_t* __restrict__ a, int64_t lda, const uint16_t* __restrict__ b,
                                                  int64_t ldb, int64_t M, int64_t N, int64_t K, void* __restrict__ c, int cdt) {
  constexpr int kStride = 40;
  __shared__ __align__(16) uint16_t sa[64 * kStride], sb[64 * kStride];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t tn = (N + 63) / 64, tile = blockIdx.x;
  const int64_t m0 = tile / tn * 64, n0 = tile % tn * 64;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  auto stage = [&](auto t_c, const uint16_t* p, int64_t ld, int64_t row0, int64_t rows, int64_t k0, uint16_t* s) {
    constexpr bool T = decltype(t_c)::value;
    if constexpr (T) {
      const int k = tid >> 3, row = 8 * (tid & 7);
      const bool on = k0 + k < K && row0 + row < rows;   // rows a multiple of 8
      const u32x4 v = on ? *reinterpret_cast<const u32x4*>(p + (k0 + k) * ld + row0 + row) : u32x4{0u, 0u, 0u, 0u};
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) s[(row + i) * kStride + k] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    } else {
      const int row = tid >> 2, k = 8 * (tid & 3);
      const bool on = row0 + row < rows && k0 + k < K;   // K a multiple of 8
      *reinterpret_cast<u32x4*>(s + row * kStride + k) =
          on ? *reinterpret_cast<const u32x4*>(p + (row0 + row) * ld + k0 + k) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  f32x4 acc[2][2] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 32) {
    stage(std::bool_constant<AT>{}, a, lda, m0, M, k0, sa);
    stage(std::bool_constant<BT>{}, b, ldb, n0, N, k0, sb);
    __syncthreads();
    u32x4 fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = *reinterpret_cast<const u32x4*>(sa + (wm + 16 * i + r) * kStride + 8 * q);
      fb[i] = *reinterpret_cast<const u32x4*>(sb + (wn + 16 * i + r) * kStride + 8 * q);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (F16) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, fb[j]), __builtin_bit_cast(f16x8, fa[i]), acc[i][j], 0, 0, 0);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[j]), __builtin_bit_cast(bf16x8, fa[i]), acc[i][j], 0, 0, 0);
        }
      }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + wm + 16 * i + r, n = n0 + wn + 16 * j + 4 * q + e;
        if (m < M && n < N) store_as(c, cdt, m * N + n, acc[i][j][e]);
      }
}

template <bool F16, bool AT, bool BT>
hipError_t simple16(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t M, int64_t N, int64_t K, void* c, int cdt,
                    hipStream_t st) {
  const int64_t tiles = ((N + 63) / 64) * ((M + 63) / 64);
  if (tiles >= 1 << 24) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_simple16<F16, AT, BT>), dim3(static_cast<unsigned>(tiles)), dim3(256), 0, st, static_cast<const uint16_t*>(a), lda,
                     static_cast<const uint16_t*>(b), ldb, M, N, K, c, cdt);
  return hipGetLastError();
}

// h = act(g) * u from pre [M][2 I], four values a thread (I a multiple of 8).
__global__ __launch_bounds__(256) void k_ff_act(const float* __restrict__ pre, int64_t M, int64_t I, int gelu, void* __restrict__ h,
                                                int hdt) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, quads = M * (I >> 2);
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < quads; v += step) {
    const int64_t m = v / (I >> 2), i = 4 * (v - m * (I >> 2));
    const f32x4 g = *reinterpret_cast<const f32x4*>(pre + m * 2 * I + i), u = *reinterpret_cast<const f32x4*>(pre + m * 2 * I + I + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) store_as(h, hdt, m * I + i + e, act_of(g[e], gelu).value * u[e]);
  }
}

// [dg | du] from pre and dh, in the operands' type: the products that follow take 16-bit
// operands, and their results are 16-bit values of the same type.
template <bool F16>
__global__ __launch_bounds__(256) void k_ff_dpre(const float* __restrict__ pre, const uint16_t* __restrict__ dh, int64_t M,
                                                 int64_t I, int gelu, uint16_t* __restrict__ dpre) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, quads = M * (I >> 2);
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < quads; v += step) {
    const int64_t m = v / (I >> 2), i = 4 * (v - m * (I >> 2));
    const f32x4 g = *reinterpret_cast<const f32x4*>(pre + m * 2 * I + i), u = *reinterpret_cast<const f32x4*>(pre + m * 2 * I + I + i);
    const uint2 d = *reinterpret_cast<const uint2*>(dh + m * I + i);
    uint32_t dg[4], du[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t bits = (e < 2 ? d.x : d.y) >> (16 * (e & 1)) & 0xffffu;
      const float t = F16 ? static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits))) : __uint_as_float(bits << 16);
      const Act a = act_of(g[e], gelu);
      dg[e] = bits16<F16>(t * u[e] * a.slope);
      du[e] = bits16<F16>(t * a.value);
    }
    *reinterpret_cast<uint2*>(dpre + m * 2 * I + i) = make_uint2(dg[0] | dg[1] << 16, dg[2] | dg[3] << 16);
    *reinterpret_cast<uint2*>(dpre + m * 2 * I + I + i) = make_uint2(du[0] | du[1] << 16, du[2] | du[3] << 16);
  }
}

unsigned quad_grid(int64_t M, int64_t I) {
  const int64_t g = (M * (I >> 2) + 255) / 256;
  return static_cast<unsigned>(g < 65536 ? g : 65536);
}

}  // namespace

hipError_t launch_ff_act(const float* pre, int64_t M, int64_t I, int gelu, void* h, int hdt, hipStream_t st) {
  hipLaunchKernelGGL(k_ff_act, dim3(quad_grid(M, I)), dim3(256), 0, st, pre, M, I, gelu, h, hdt);
  return hipGetLastError();
}

hipError_t launch_gated_ff(const FfParams& p, hipStream_t st) {
  const hipError_t e = p.f16 ? simple16<true, false, false>(p.x, p.H, p.w, p.H, p.M, 2 * p.I, p.H, p.pre, 0, st)
                             : simple16<false, false, false>(p.x, p.H, p.w, p.H, p.M, 2 * p.I, p.H, p.pre, 0, st);
  return e != hipSuccess ? e : launch_ff_act(p.pre, p.M, p.I, p.gelu, p.h, p.f16 ? 2 : 1, st);
}

hipError_t launch_gated_ff_backward(const FfParams& p, hipStream_t st) {
  const unsigned grid = quad_grid(p.M, p.I);
  if (p.f16) {
    hipLaunchKernelGGL(k_ff_dpre<true>, dim3(grid), dim3(256), 0, st, p.pre, p.dh, p.M, p.I, p.gelu, p.dpre);
  } else {
    hipLaunchKernelGGL(k_ff_dpre<false>, dim3(grid), dim3(256), 0, st, p.pre, p.dh, p.M, p.I, p.gelu, p.dpre);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int dt = p.f16 ? 2 : 1;
  if (p.dx) {
    e = p.f16 ? simple16<true, false, true>(p.dpre, 2 * p.I, p.w, p.H, p.M, p.H, 2 * p.I, p.dx, dt, st)
              : simple16<false, false, true>(p.dpre, 2 * p.I, p.w, p.H, p.M, p.H, 2 * p.I, p.dx, dt, st);
    if (e != hipSuccess) return e;
  }
  if (p.dw) {
    e = p.f16 ? simple16<true, true, true>(p.dpre, 2 * p.I, p.x, p.H, 2 * p.I, p.H, p.M, p.dw, dt, st)
              : simple16<false, true, true>(p.dpre, 2 * p.I, p.x, p.H, 2 * p.I, p.H, p.M, p.dw, dt, st);
  }
  return e;
}

}  // namespace cubic
