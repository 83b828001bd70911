// tile.h -- what the dense tile kernels (gated_ff.hip, fp8.hip) share: buffer loads, the
// order of tiles over the compute units, and the way of a tile's results through LDS.
#pragma once
#include <algorithm>
#include <type_traits>
#include <utility>

#include "common.h"
#include "dense.h"
#include "launch.h"

namespace cubic {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kPast = 0xffffffffu;        // an offset behind every buffer: the load gives zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes),
                                           static_cast<int>(0x00020000u));
}
__device__ __forceinline__ u32x4 tile_load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(off), 0, 0));
}
// 16 bytes a lane straight into LDS, lane l's at lds + 16 l (lds the same in the whole wave).
// In assembly, since the compiler lets every transposed read of LDS wait for all such loads
// that it knows of (a product of 229 us took 314): the caller waits, by tile_wait and a barrier
// before what is loaded is read.
__device__ __forceinline__ u32x4 tile_lds_rsrc(const void* p, uint32_t bytes) {
  const uint64_t base = reinterpret_cast<uint64_t>(p);
  return u32x4{static_cast<uint32_t>(base), static_cast<uint32_t>(base >> 32) & 0xffffu, bytes, 0x00020000u};
}
__device__ __forceinline__ uint32_t tile_lds_at(unsigned char* lds) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)(lds)));
}
// AT: added to lds; voff the lane's offset, checked against the resource's size, and soff the
// wave's on top of it.
template <int AT>
__device__ __forceinline__ void tile_load_lds(const u32x4& rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds" ::"s"(lds), "n"(AT), "v"(voff),
               "s"(rsrc), "s"(soff)
               : "m0", "scc", "memory");
}
// The same with four bytes a lane, at lds + AT + 4 l.
template <int AT>
__device__ __forceinline__ void tile_load_lds4(const u32x4& rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dword %2, %3, %4 offen lds" ::"s"(lds), "n"(AT), "v"(voff),
               "s"(rsrc), "s"(soff)
               : "m0", "scc", "memory");
}
// stage(s, I) for s = 0 .. S - 1 with I = s % U known to the compiler.
template <int U, class Stage>
__device__ __forceinline__ void tile_stages(int S, Stage stage) {
  int s = 0;
  auto all = [&]<int... I>(std::integer_sequence<int, I...>) {
    for (; s + U <= S; s += U) (stage(s + I, std::integral_constant<int, I>{}), ...);
    const int left = S - s;
    ((I < left ? stage(s + I, std::integral_constant<int, I>{}) : void()), ...);
  };
  all(std::make_integer_sequence<int, U>{});
}
// Waits until at most N of this wave's global loads are on their way.
template <int N>
__device__ __forceinline__ void tile_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// A barrier that leaves global loads in flight.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Tile `t` of tm x tn to (row, column): neighbouring workgroup ids go to different XCDs, so
// each XCD takes a run of tiles, in groups of four tile rows (a run's tiles share operand
// rows in its L2).
__device__ __forceinline__ void tile_place(int t, int tm, int tn, int* im, int* in) {
  const int nt = tm * tn, base = nt >> 3, rem = nt & 7, x = t & 7;
  t = x * base + min(x, rem) + (t >> 3);
  const int per = 4 * tn, grp = t / per, r = t - grp * per;
  const int gm = min(4, tm - 4 * grp);
  *im = 4 * grp + r % gm;
  *in = r / gm;
}

// Writes a tile's results to y[m][n] (row stride ld) through LDS, so that rows leave in whole
// 16-byte pieces. The tile has WM x WN waves with MB x CB blocks of BLK x BLK (32 or 16) each, a
// lane holding row c and four neighbouring columns, 8 g + 4 h on in the block: value(i, j, g)
// gives them as four floats. Rows go in NP passes of what fits in kSpace bytes. Starts and
// ends with a barrier.
template <int BLK, int MB, int CB, int WM, int WN, int kBytes, int kSpace, class Value>
__device__ __forceinline__ void tile_write(unsigned char* smem, void* y, int ydt, int64_t ld, int64_t m0, int64_t M, int64_t n0,
                                           int64_t N, Value value) {
  constexpr int TC = BLK * CB * WN, kThreads = 64 * WM * WN, kStride = TC * kBytes + 16, kPer = 16 / kBytes;
  constexpr auto passes = [] {
    int np = 1;
    while (np < MB && BLK * MB * WM / np * kStride > kSpace) np *= 2;
    return np;
  };
  constexpr int NP = passes(), BP = MB / NP, kRows = BLK * BP * WM;
  static_assert(kRows * kStride <= 160 * 1024 && BP * NP == MB, "passes of whole blocks that fit");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & (BLK - 1), h = lane / BLK, wm = wave / WN, wn = wave % WN;
  const int cols = static_cast<int>(min(static_cast<int64_t>(TC), N - n0));
  const bool whole = ld % kPer == 0 && cols % kPer == 0;       // rows start on 16 bytes
#pragma unroll
  for (int ip = 0; ip < NP; ++ip) {
    __syncthreads();
#pragma unroll
    for (int ib = 0; ib < BP; ++ib) {
      const int i = ip * BP + ib;
      unsigned char* row = smem + (wm * BLK * BP + BLK * ib + c) * kStride;
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int g = 0; g < BLK / 8 * BLK / 32; ++g) {
          const int n = wn * BLK * CB + BLK * j + 8 * g + 4 * h;
          const f32x4 v = value(i, j, g);
          if constexpr (kBytes == 4) {
            *reinterpret_cast<f32x4*>(row + 4 * n) = v;
          } else {
            uint2 w;
            if (ydt == 2) {
              w = make_uint2(bits16<true>(v[0]) | bits16<true>(v[1]) << 16, bits16<true>(v[2]) | bits16<true>(v[3]) << 16);
            } else {
              w = make_uint2(bits16<false>(v[0]) | bits16<false>(v[1]) << 16, bits16<false>(v[2]) | bits16<false>(v[3]) << 16);
            }
            *reinterpret_cast<uint2*>(row + 2 * n) = w;
          }
        }
    }
    __syncthreads();
    auto global_row = [&](int r) {
      const int w = r / (BLK * BP);
      return m0 + w * BLK * MB + ip * BLK * BP + (r - w * BLK * BP);
    };
    unsigned char* out = static_cast<unsigned char*>(y);
    if (whole) {
      constexpr int kPieces = TC / kPer;
      for (int idx = tid; idx < kRows * kPieces; idx += kThreads) {
        const int r = idx / kPieces, q = idx - r * kPieces;
        const int64_t m = global_row(r);
        if (m < M && q * kPer < cols)
          *reinterpret_cast<u32x4*>(out + (m * ld + n0 + q * kPer) * kBytes) = *reinterpret_cast<const u32x4*>(smem + r * kStride + 16 * q);
      }
    } else {
      for (int idx = tid; idx < kRows * TC; idx += kThreads) {
        const int r = idx / TC, q = idx - r * TC;
        const int64_t m = global_row(r);
        if (m < M && q < cols) {
          if constexpr (kBytes == 2) {
            reinterpret_cast<uint16_t*>(out)[m * ld + n0 + q] = reinterpret_cast<const uint16_t*>(smem + r * kStride)[q];
          } else {
            reinterpret_cast<float*>(out)[m * ld + n0 + q] = reinterpret_cast<const float*>(smem + r * kStride)[q];
          }
        }
      }
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Tiles and slices. A product with few tiles splits its contraction into slices, whose fp32
// sums pass through the workspace ([slice][M][width]) and are added up in their order.
struct TilePlan {
  int shape, slices;       // of kTileShapes
};
constexpr int kTileShapes[][2] = {{256, 256}, {256, 128}, {128, 128}, {64, 128}, {64, 64}};
constexpr int kTileShapeCount = 5, kMaxSlices = 32;

// What the plans go by: cycles of a workgroup in each shape over a step of 128 bytes of the rows
// (64 values of 16 bits or 128 codes), as measured with every compute unit at work, and those of the
// last shape, two of which share a compute unit, where it has one to itself; a workgroup's start
// and end (17000 and 8000 measured for the first two shapes) come on top.
struct TileCosts {
  int64_t step[kTileShapeCount], last_alone;
};
inline int64_t plan_workgroup(int k, int64_t len, const TileCosts& c, bool alone) {
  return len * (alone && k == kTileShapeCount - 1 ? c.last_alone : c.step[k]) + 5000 + kTileShapes[k][0] * kTileShapes[k][1] / 6;
}
inline int64_t plan_tile_count(int k, int64_t M, int64_t width) {
  return ((M + kTileShapes[k][0] - 1) / kTileShapes[k][0]) * ((width + kTileShapes[k][1] - 1) / kTileShapes[k][1]);
}
inline int64_t plan_cus() { return device_cu_count() > 0 ? device_cu_count() : 256; }
// The join's launch and the slices' bytes.
inline int64_t plan_join(int slices, int64_t M, int64_t width) { return slices > 1 ? 5000 + M * width * 8 * slices / 1700 : 0; }

// The slices of least time for shape k, M rows, `width` columns of operand B and `stages` steps:
// rounds of workgroups over the compute units, and the join. No slice is empty.
inline TilePlan plan_shape(int k, int64_t cu, int64_t M, int64_t width, int64_t stages, const TileCosts& costs, int64_t* cost) {
  const int64_t tiles = plan_tile_count(k, M, width);
  TilePlan best{k, 1};
  *cost = INT64_MAX;
  for (int s = 1; s <= kMaxSlices; ++s) {
    if (s > 1 && (stages < 2 * s || tiles * s > 2 * cu)) break;
    const int64_t len = (stages + s - 1) / s;
    if (len * (s - 1) >= stages) continue;
    const int64_t c = (tiles * s + cu - 1) / cu * plan_workgroup(k, len, costs, tiles * s <= cu) + plan_join(s, M, width);
    if (c < *cost) {
      *cost = c;
      best.slices = s;
    }
  }
  return best;
}
inline TilePlan plan_tiles(int64_t M, int64_t width, int64_t stages, const TileCosts& costs) {
  const int64_t cu = plan_cus();
  TilePlan best{};
  int64_t cost = INT64_MAX;
  for (int k = 0; k < kTileShapeCount; ++k) {
    int64_t c;
    const TilePlan t = plan_shape(k, cu, M, width, stages, costs, &c);
    if (c < cost) {
      cost = c;
      best = t;
    }
  }
  return best;
}
inline size_t plan_bytes(const TilePlan& t, int64_t M, int64_t width) {
  return t.slices > 1 ? (static_cast<size_t>(t.slices) * M * width * 4 + 255) / 256 * 256 : 0;
}

// What follows the slices: y = their sum (+ bias) in its type, or gated y = act(gate) * up of
// the sum's halves, which pre receives where it is given.
struct JoinParams {
  const float* part;       // [slices][M][width]
  int slices;
  int64_t M, N, width;     // width N, gated 2 N
  const float* bias;
  void* y;
  int ydt, gelu;
  float* pre;
};
template <bool GATED, int V>                   // V neighbouring columns a thread
__global__ __launch_bounds__(256) void k_tile_join(JoinParams p) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, per = p.N / V, all = p.M * per, slice = p.M * p.width;
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < all; at += step) {
    const int64_t m = at / per, n = V * (at - m * per);
    auto sum = [&](int64_t col, float* v) {
      const float* q = p.part + m * p.width + col;
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 0.0f;
      for (int s = 0; s < p.slices; ++s, q += slice) {
        if constexpr (V == 4) {
          const f32x4 t = *reinterpret_cast<const f32x4*>(q);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += t[e];
        } else {
          v[0] += *q;
        }
      }
    };
    float v[V];
    sum(n, v);
    if constexpr (GATED) {
      float u[V];
      sum(p.N + n, u);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (p.pre) {
          p.pre[m * p.width + n + e] = v[e];
          p.pre[m * p.width + p.N + n + e] = u[e];
        }
        v[e] = act_of(v[e], p.gelu).value * u[e];
      }
    } else if (p.bias) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] += p.bias[n + e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) store_as(p.y, p.ydt, m * p.N + n + e, v[e]);
  }
}
template <bool GATED>
hipError_t launch_tile_join(const JoinParams& p, hipStream_t st) {
  const bool quads = p.N % 4 == 0;
  const int64_t items = p.M * (quads ? p.N / 4 : p.N);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((items + 255) / 256, 4096));
  if (quads) {
    hipLaunchKernelGGL((k_tile_join<GATED, 4>), dim3(grid), dim3(256), 0, st, p);
  } else {
    hipLaunchKernelGGL((k_tile_join<GATED, 1>), dim3(grid), dim3(256), 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace cubic
