// fp8.hip -- the block quantiser to e4m3 and the product of e4m3 activations and weights
// with fp32 scales per block of 128.
//
//   y[m][n] = sum_kb xs[m][kb] * ws[n / 128][kb] * (sum_{k in block kb} xq[m][k] wq[n][k]) (+ bias[n])
//
// An e4m3 value is exact in bf16 (three fraction bits, exponents -9 to 8), so a block's dot
// product on the bf16 MFMA has exact products and fp32 sums.
#include <algorithm>

#include "act_quant.h"
#include "common.h"
#include "dense.h"
#include "launch.h"

namespace cubic {
namespace {

// The larger of the magnitudes of 16 neighbouring lanes, NaN as the largest.
__device__ __forceinline__ float larger16(float v) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v = larger<true>(v, __shfl_xor(v, o, 64));
  return v;
}

// A launch takes fewer than 2^32 threads; what is more goes round again.
constexpr int64_t kMaxGrid = (1 << 24) - 1;

// One group per 16 lanes, eight values a lane.
template <bool XF16>
__global__ __launch_bounds__(256) void k_quant_fp8_rows(const uint16_t* __restrict__ x, int64_t groups, int64_t K, int64_t kb,
                                                        uint8_t* __restrict__ xq, float* __restrict__ xs) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 16;
  // whole groups of 16 lanes take part or leave
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4); g < groups; g += step) {
    const int64_t m = g / kb, b = g - m * kb;
    const int64_t k = b * 128 + 8 * (threadIdx.x & 15);
    const bool on = k < K;
    const u32x4 v = on ? *reinterpret_cast<const u32x4*>(x + m * K + k) : u32x4{0u, 0u, 0u, 0u};
    const float s = fp8_scale(larger16(absmax8<XF16, true>(v, 0.0f)));
    if (on) *reinterpret_cast<uint2*>(xq + m * K + k) = fp8_quant8<XF16>(v, s);
    if ((threadIdx.x & 15) == 0) xs[g] = s;
  }
}

// One block of 128 x 128 per workgroup, held in registers between the two passes.
template <bool XF16>
__global__ __launch_bounds__(256) void k_quant_fp8_blocks(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t kb,
                                                          uint8_t* __restrict__ xq, float* __restrict__ xs) {
  __shared__ float s_max[4];
  const int64_t blocks = (M + 127) / 128 * kb;
  for (int64_t at = blockIdx.x; at < blocks; at += gridDim.x) {
    const int64_t mb = at / kb, b = at - mb * kb;
    const int64_t k = b * 128 + 8 * (threadIdx.x & 15);
    u32x4 v[8];
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t m = mb * 128 + 16 * i + (threadIdx.x >> 4);
      v[i] = m < M && k < K ? *reinterpret_cast<const u32x4*>(x + m * K + k) : u32x4{0u, 0u, 0u, 0u};
      a = absmax8<XF16, true>(v[i], a);
    }
    a = wave_larger<true>(a);
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = a;
    __syncthreads();
    const float s = fp8_scale(larger<true>(larger<true>(s_max[0], s_max[1]), larger<true>(s_max[2], s_max[3])));
    __syncthreads();                           // read before the next block's are written
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t m = mb * 128 + 16 * i + (threadIdx.x >> 4);
      if (m < M && k < K) *reinterpret_cast<uint2*>(xq + m * K + k) = fp8_quant8<XF16>(v[i], s);
    }
    if (threadIdx.x == 0) xs[at] = s;
  }
}

// 64 x 64 outputs a workgroup, one block of 128 codes a step.
__global__ __launch_bounds__(256) void k_fp8_simple(Fp8Params p) {
  constexpr int kStride = 128 + 16;
  __shared__ __align__(16) unsigned char sa[64 * kStride], sb[64 * kStride];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t tn = (p.N + 63) / 64, tile = blockIdx.x;
  const int64_t m0 = tile / tn * 64, n0 = tile % tn * 64;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int64_t kb = (p.K + 127) / 128;
  f32x4 acc[2][2] = {};
  for (int64_t b = 0; b < kb; ++b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int idx = tid + 256 * i, row = idx >> 3, piece = idx & 7;
      const int64_t k = b * 128 + 16 * piece;
      const u32x4 zero{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(sa + row * kStride + 16 * piece) =
          m0 + row < p.M && k < p.K ? *reinterpret_cast<const u32x4*>(p.xq + (m0 + row) * p.K + k) : zero;
      *reinterpret_cast<u32x4*>(sb + row * kStride + 16 * piece) =
          n0 + row < p.N && k < p.K ? *reinterpret_cast<const u32x4*>(p.w + (n0 + row) * p.K + k) : zero;
    }
    __syncthreads();
    f32x4 part[2][2] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = e4m3x8_to_bf16(*reinterpret_cast<const u32x2*>(sa + (wm + 16 * i + r) * kStride + 32 * s + 8 * q));
        fb[i] = e4m3x8_to_bf16(*reinterpret_cast<const u32x2*>(sb + (wn + 16 * i + r) * kStride + 32 * s + 8 * q));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) part[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], part[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = m0 + wm + 16 * i + r;
      const float xs = m < p.M ? p.xs[m * kb + b] : 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = n0 + wn + 16 * j;
        const float s = xs * (n < p.N ? p.ws[(n >> 7) * kb + b] : 0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(part[i][j][e], s, acc[i][j][e]);
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
        if (m < p.M && n < p.N) store_as(p.y, p.ydt, m * p.N + n, acc[i][j][e] + (p.bias ? p.bias[n] : 0.0f));
      }
}

}  // namespace

hipError_t launch_quant_fp8(const uint16_t* x, bool xf16, int64_t M, int64_t K, bool blocks, uint8_t* xq, float* xs,
                            hipStream_t st) {
  const int64_t kb = (K + 127) / 128;
  if (blocks) {
    const unsigned grid = static_cast<unsigned>(std::min((M + 127) / 128 * kb, kMaxGrid));
    auto kern = xf16 ? k_quant_fp8_blocks<true> : k_quant_fp8_blocks<false>;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(256), 0, st, x, M, K, kb, xq, xs);
  } else {
    const unsigned grid = static_cast<unsigned>(std::min((M * kb + 15) / 16, kMaxGrid));
    auto kern = xf16 ? k_quant_fp8_rows<true> : k_quant_fp8_rows<false>;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(256), 0, st, x, M * kb, K, kb, xq, xs);
  }
  return hipGetLastError();
}

hipError_t launch_fp8(const Fp8Params& p, hipStream_t st) {
  const int64_t tiles = ((p.N + 63) / 64) * ((p.M + 63) / 64);
  if (tiles > kMaxGrid) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_fp8_simple, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace cubic
