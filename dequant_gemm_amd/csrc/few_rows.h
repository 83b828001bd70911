// few_rows.h -- the dense products of up to 64 activation rows (gated_ff.hip, fp8.hip): bound
// by the weight's bytes.
//
// Every workgroup takes an equal share of the weight rows (gated: of the columns of h, their
// gate and up rows), its sixteen waves a step of 64 bytes of each row in turn. Weights go
// from HBM to registers: a lane quad loads 64 contiguous bytes of a row, and the lanes
// exchange the pieces through the LDS crossbar into the MFMA's operand order when they are
// used. The activations pass through LDS in chunks of 64 KB, two buffers, one barrier a chunk
// that leaves the weight loads in flight; up to four rows that fit are staged whole. In fp8
// every workgroup can quantise the rows itself on their way into LDS: whole rows beside its first
// weight loads, or a chunk at a time. The waves' sums meet in LDS and are added up in their order.
//
// Measured: 44 MB of e4m3 weights (6144 x 7168) in 10.4 us of the kernel with one row, 13.2 us with 16;
// 58.7 MB of bf16 gate and up weights in 10.9 us (5.4 TB/s, partly from the last cache), 17 us of I 1024, H 8192
// with 48 rows. From 17 rows on the staging of the activations and the join of sixteen sums count.
#pragma once
#include <algorithm>
#include <type_traits>
#include <utility>

#include "launch.h"
#include "tile.h"

namespace cubic {

enum FewKind { kFewBf16, kFewF16, kFewFp8 };

struct FewParams {
  const void* x;           // 16 bits [M][K]; fp8: codes, or with WHOLE or QUANT 16-bit values to quantise
  const float* xs;         // fp8: [M][kb]
  const void* w;           // [N][K], gated: N gate rows and N up rows
  const float* ws;         // fp8: [ceil(rows / 128)][kb]
  const float* bias;       // [N] or NULL
  int64_t N, K;
  int M;
  void* y;                 // [M][N]
  int ydt, gelu;
  float* pre;              // gated: [M][2 N] or NULL
  int cols;                // of results per workgroup
  int rt;                  // of them per tile of 16
};

constexpr int kFewWaves = 16;
constexpr int64_t kFewMaxM = 64, kFewWholeM = 4, kFewQuantM = 8;
constexpr int64_t kFewWholeBytes = 32768;      // of a row held whole in LDS (four rows: 128 KB)

template <int KIND>
__device__ __forceinline__ f32x4 few_dot(const i32x4& a, const i32x4& b, f32x4 c) {
  if constexpr (KIND == kFewBf16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else if constexpr (KIND == kFewF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const u32x2 u{static_cast<uint32_t>(a[2 * s]), static_cast<uint32_t>(a[2 * s + 1])};
      const u32x2 v{static_cast<uint32_t>(b[2 * s]), static_cast<uint32_t>(b[2 * s + 1])};
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3x8_to_bf16(u), e4m3x8_to_bf16(v), c, 0, 0, 0);   // exact products
    }
    return c;
  }
}

// MT: tiles of 16 activation rows; SPC = 4 / MT steps per wave and chunk; NT: tiles of 16
// weight rows. Gated with NT 1: gate rows in the tile's first half, up rows in its second.
// QUANT: fp8, x in 16 bits, which every workgroup quantises a chunk at a time.
template <int KIND, int MT, int NT, bool WHOLE, bool GATED, bool XF16, bool QUANT>
__global__ __launch_bounds__(1024) void k_few_rows(FewParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr bool F8 = KIND == kFewFp8;
  constexpr int SPC = 4 / MT, PM = 4, kCode = F8 ? 1 : 2;
  constexpr int RM = WHOLE ? 4 : 16 * MT;      // activation rows held in LDS
  constexpr int kChunk = 65536, kScales = F8 && !WHOLE ? 2048 : 0;   // of a chunk: bytes, and of their scales
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const int M = p.M;
  const uint32_t KB = static_cast<uint32_t>(p.K) * kCode;        // bytes of a row, a multiple of 16
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * p.cols;
  const int cols = static_cast<int>(min(static_cast<int64_t>(p.cols), p.N - n0));
  const int nsteps = static_cast<int>((KB + 63) >> 6);
  const int iters = (nsteps + kFewWaves - 1) / kFewWaves;        // the longest wave's steps
  const int kb = static_cast<int>((p.K + 127) >> 7);

  // ---- weights: lane l loads piece l % 4 of row l / 4 of each tile ----
  __amdgpu_buffer_rsrc_t wrs[NT];
  uint32_t voff[NT], soff[NT];                 // the row's bytes and (in the MFMA's order) its scales
  float cs[PM][NT];
  u32x4 cb[PM][NT];
  const char* w = static_cast<const char*>(p.w);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if constexpr (!GATED) {
      wrs[t] = tile_rsrc(w + n0 * KB, static_cast<uint32_t>(cols) * KB);
      auto row = [&](int r) { return min(t * p.rt + min(r, p.rt - 1), cols - 1); };
      voff[t] = static_cast<uint32_t>(row(lane >> 2)) * KB + 16u * (lane & 3);
      if constexpr (F8) soff[t] = static_cast<uint32_t>((n0 + row(nl)) >> 7) * static_cast<uint32_t>(4 * kb);
    } else if constexpr (NT == 1) {
      // (the launcher sees to it that both parts lie within 32 bits)
      wrs[t] = tile_rsrc(w + n0 * KB, static_cast<uint32_t>((p.N + cols) * KB));
      auto col = [&](int r) { return min(r & 7, cols - 1); };
      voff[t] = static_cast<uint32_t>(((lane >> 5) ? p.N : 0) + col(lane >> 2)) * KB + 16u * (lane & 3);
      if constexpr (F8) soff[t] = static_cast<uint32_t>(((nl >> 3 ? p.N : 0) + n0 + col(nl)) >> 7) * static_cast<uint32_t>(4 * kb);
    } else {
      wrs[t] = tile_rsrc(w + (n0 + (t ? p.N : 0)) * KB, static_cast<uint32_t>(cols) * KB);
      voff[t] = static_cast<uint32_t>(min(lane >> 2, cols - 1)) * KB + 16u * (lane & 3);
      if constexpr (F8) soff[t] = static_cast<uint32_t>(((t ? p.N : 0) + n0 + min(nl, cols - 1)) >> 7) * static_cast<uint32_t>(4 * kb);
    }
  }
  // step i of this wave is K step 16 i + wave; past the last one and past K zeros (a
  // neighbouring row's values might be non-finite)
  auto issue = [&](auto u_c, int i) {
    constexpr int u = decltype(u_c)::value;
    const int s = i * kFewWaves + wave;
    const bool on = 64u * static_cast<uint32_t>(s) + 16u * (lane & 3) < KB;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      cb[u][t] = tile_load(wrs[t], on ? voff[t] + 64u * static_cast<uint32_t>(s) : kPast);
      if constexpr (F8) cs[u][t] = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(p.ws) + soff[t] + 4 * min(s >> 1, kb - 1));
    }
  };
  auto issue_first = [&] {
    __builtin_amdgcn_sched_barrier(0);
    [&]<int... U>(std::integer_sequence<int, U...>) {
      (issue(std::integral_constant<int, U>{}, U), ...);
    }(std::make_integer_sequence<int, PM>{});
    __builtin_amdgcn_sched_barrier(0);
  };

  // ---- activations: 16-byte piece j of row m at step st of a buffer: rows of 64 bytes, the
  // piece XORed with two row bits so that 16 rows read at one piece hit all banks ----
  auto place = [&](int st, int m, int j) { return ((st * RM + m) * 4 + (j ^ ((m >> 2) & 3))) * 16; };
  constexpr int XR = 4;                        // pieces per thread and chunk
  constexpr int kIn = QUANT ? 2 : 1;           // of them, of x
  u32x4 xv[XR * kIn];
  float xsv = 0.0f;
  const __amdgpu_buffer_rsrc_t xrs = tile_rsrc(p.x, kIn * static_cast<uint32_t>(M) * KB);
  constexpr int kPieces = 64 * SPC;            // pieces of a row in a chunk
  auto load_x = [&](int c) {
#pragma unroll
    for (int r = 0; r < XR; ++r) {
      const int idx = tid + 1024 * r;
      const int m = idx / kPieces;
      const uint32_t k = static_cast<uint32_t>(c) * (SPC * 1024) + 16u * (idx % kPieces);
#pragma unroll
      for (int h = 0; h < kIn; ++h)
        xv[kIn * r + h] = tile_load(xrs, m < M && k < KB ? kIn * (static_cast<uint32_t>(m) * KB + k) + 16u * h : kPast);
    }
    if constexpr (F8 && !QUANT) {                    // 8 SPC blocks of each row: thread to (block, row)
      const int m = tid % RM, b = c * (8 * SPC) + tid / RM;
      xsv = tid < 512 && m < M && b < kb ? p.xs[static_cast<int64_t>(m) * kb + b] : 0.0f;
    }
  };
  auto store_x = [&](int c) __attribute__((always_inline)) {   // (out of line its captures go to memory)
    unsigned char* buf = smem + (c & 1) * (kChunk + kScales);
    auto piece = [&](auto r_c) {
      constexpr int r = decltype(r_c)::value;
      const int idx = tid + 1024 * r;
      const int m = idx / kPieces, pk = idx % kPieces;
      if (m >= M) return;                      // (a wave's pieces are of one row)
      u32x4 codes = xv[kIn * r];
      if constexpr (QUANT) {                   // 16 values; eight neighbouring lanes hold a block
        const Fp8Scale s = fp8_scale_of(mag_value<XF16>(mag_lanes<8>(mag8(xv[kIn * r + 1], mag8(xv[kIn * r], 0u)))));
        const uint2 lo = fp8_quant8<XF16>(xv[kIn * r], s), hi = fp8_quant8<XF16>(xv[kIn * r + 1], s);
        codes = u32x4{lo.x, lo.y, hi.x, hi.y};
        if ((tid & 7) == 0) *reinterpret_cast<float*>(buf + kChunk + 4 * ((pk >> 3) * RM + m)) = s.s;
      }
      *reinterpret_cast<u32x4*>(buf + place(pk >> 2, m, pk & 3)) = codes;
    };
    [&]<int... R>(std::integer_sequence<int, R...>) {
      (piece(std::integral_constant<int, R>{}), ...);
    }(std::make_integer_sequence<int, XR>{});
    if constexpr (F8 && !QUANT) {
      if (tid < 512) *reinterpret_cast<float*>(buf + kChunk + 4 * tid) = xsv;
    }
  };

  const float* whole_scales = reinterpret_cast<const float*>(smem + nsteps * 256);   // WHOLE fp8: [block][4]
  if constexpr (WHOLE && F8) {
    // one vector of eight values per thread, row and round of 8192 values (K <= 32768)
    const int nvec = static_cast<int>(p.K >> 3);
    u32x4 v[4];
    const uint16_t* x = static_cast<const uint16_t*>(p.x);
    auto fetch = [&](int o) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
        v[m] = m < M && o + tid < nvec ? reinterpret_cast<const u32x4*>(x + static_cast<int64_t>(m) * p.K)[o + tid] : u32x4{0u, 0u, 0u, 0u};
    };
    fetch(0);
    issue_first();
    for (int o = 0; o < nsteps * 8; o += 1024) {
      if (o) fetch(o);
      const int vec = o + tid;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m < M) {
          const Fp8Scale s = fp8_scale_of(mag_value<XF16>(mag_lanes<16>(mag8(v[m], 0u))));
          // eight codes: half a piece; past K up to the last step's end zeros
          if (vec < nsteps * 8)
            *reinterpret_cast<uint2*>(smem + place(vec >> 3, m, (vec >> 1) & 3) + 8 * (vec & 1)) = fp8_quant8<XF16>(v[m], s);
          if ((tid & 15) == 0 && (vec >> 4) < kb) const_cast<float*>(whole_scales)[4 * (vec >> 4) + m] = s.s;
        }
      }
    }
    tile_barrier();
  } else if constexpr (WHOLE) {
    u32x4 v[4];
    const uint32_t pieces = static_cast<uint32_t>(nsteps) * 4;   // of a row, at most 2048
    auto fetch = [&](uint32_t o) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t k = 16u * (o + tid);
        v[m] = tile_load(xrs, m < M && k < KB ? static_cast<uint32_t>(m) * KB + k : kPast);
      }
    };
    fetch(0);
    issue_first();
    for (uint32_t o = 0; o < pieces; o += 1024) {
      if (o) fetch(o);
      const uint32_t pc = o + tid;
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (m < M && pc < pieces) *reinterpret_cast<u32x4*>(smem + place(pc >> 2, m, pc & 3)) = v[m];
    }
    tile_barrier();
  } else {
    load_x(0);
    issue_first();                             // activations ahead of the weights
  }

  f32x4 acc[MT][NT] = {};
  const int xaddr = 4 * (4 * nl + kq);
  const int ml = WHOLE ? (nl & 3) : nl;        // rows past M: their sums are not used
  for (int i0 = 0; i0 < iters; i0 += PM) {
    [&]<int... U>(std::integer_sequence<int, U...>) {
      (([&] {
         constexpr int u = U;
         const int i = i0 + u;
         if constexpr (!WHOLE && u % SPC == 0) {
           // chunk c in, chunk c + 1 on its way (the chunk before the last one read
           // the buffer that c overwrites; every wave is past it)
           const int c = i / SPC;
           if (i < iters) {
             store_x(c);
             load_x(c + 1);
             tile_barrier();
           }
         }
         const int s = i * kFewWaves + wave;
         if (s < nsteps) {
           const int st = WHOLE ? s : (i % SPC) * kFewWaves + wave;
           const unsigned char* buf = WHOLE ? smem : smem + ((i / SPC) & 1) * (kChunk + kScales);
           i32x4 b[NT];
#pragma unroll
           for (int t = 0; t < NT; ++t)
#pragma unroll
             for (int d = 0; d < 4; ++d) b[t][d] = __builtin_amdgcn_ds_bpermute(xaddr, static_cast<int>(cb[u][t][d]));
#pragma unroll
           for (int a = 0; a < MT; ++a) {
             const i32x4 av = *reinterpret_cast<const i32x4*>(buf + place(st, 16 * a + ml, kq));
             if constexpr (F8) {
               // the four rows' scales of the step's block (WHOLE: rows 0 .. 3, held by kq 0)
               const f32x4 sx = WHOLE ? *reinterpret_cast<const f32x4*>(whole_scales + 4 * (s >> 1))
                                      : *reinterpret_cast<const f32x4*>(buf + kChunk + 4 * ((st >> 1) * RM + 16 * a + 4 * kq));
#pragma unroll
               for (int t = 0; t < NT; ++t) {
                 const f32x4 part = few_dot<KIND>(av, b[t], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                 for (int r = 0; r < 4; ++r) acc[a][t][r] = fmaf(part[r], sx[r] * cs[u][t], acc[a][t][r]);
               }
             } else {
#pragma unroll
               for (int t = 0; t < NT; ++t) acc[a][t] = few_dot<KIND>(av, b[t], acc[a][t]);
             }
           }
         }
         issue(std::integral_constant<int, u>{}, i + PM);
         __builtin_amdgcn_sched_barrier(0);
       }()),
       ...);
    }(std::make_integer_sequence<int, PM>{});
  }

  // ---- the waves' sums meet in LDS: [wave][tile][MT][register][lane], the order in
  // which a wave writes 64 neighbouring words ----
  tile_barrier();                              // the activations are read
  float* red = reinterpret_cast<float*>(smem);
  constexpr int kTile = 16 * MT * 16;
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = 16 * a + 4 * kq + r;
        if (m < M) red[(wave * NT + t) * kTile + 256 * a + 64 * r + lane] = acc[a][t][r];
      }
  tile_barrier();
  auto sum = [&](int m, int t, int col) {
    const int at = 256 * (m >> 4) + 64 * (m & 3) + 16 * ((m >> 2) & 3) + col;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) v += red[(k * NT + t) * kTile + at];
    return v;
  };
  if constexpr (GATED) {
    for (int idx = tid; idx < M * 16; idx += 1024) {
      const int m = idx >> 4, j = idx & 15;
      if (j >= cols) continue;
      const float g = sum(m, 0, j), u = NT == 1 ? sum(m, 0, 8 + j) : sum(m, NT - 1, j);
      const int64_t n = n0 + j;
      if (p.pre) {
        p.pre[static_cast<int64_t>(m) * 2 * p.N + n] = g;
        p.pre[static_cast<int64_t>(m) * 2 * p.N + p.N + n] = u;
      }
      store_as(p.y, p.ydt, static_cast<int64_t>(m) * p.N + n, act_of(g, p.gelu).value * u);
    }
  } else {
    for (int idx = tid; idx < M * 32; idx += 1024) {
      const int m = idx >> 5, j = idx & 31;
      const int t = NT == 1 ? 0 : (j >= p.rt ? 1 : 0), col = j - t * p.rt;
      if (j >= cols || col >= p.rt) continue;
      const int64_t n = n0 + j;
      store_as(p.y, p.ydt, static_cast<int64_t>(m) * p.N + n, sum(m, t, col) + (p.bias ? p.bias[n] : 0.0f));
    }
  }
}

template <int KIND, int MT, int NT, bool WHOLE, bool GATED, bool XF16, bool QUANT>
hipError_t launch_few_k(const FewParams& p, hipStream_t st) {
  auto kern = k_few_rows<KIND, MT, NT, WHOLE, GATED, XF16, QUANT>;
  constexpr bool F8 = KIND == kFewFp8;
  const int nsteps = static_cast<int>((p.K * (F8 ? 1 : 2) + 63) / 64);
  const int red = kFewWaves * NT * 16 * MT * 16 * 4;
  const int x = WHOLE ? nsteps * 256 + (F8 ? static_cast<int>((p.K + 127) / 128) * 16 : 0) : 2 * (65536 + (F8 ? 2048 : 0));
  const int lds = std::max(red, x);
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), lds);
  if (e != hipSuccess) return e;
  const int64_t grid = (p.N + p.cols - 1) / p.cols;
  if (grid >= 1 << 22) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(1024), lds, st, p);
  return hipGetLastError();
}

// whole: p.x holds up to kFewWholeM rows to stage whole (fp8: 16-bit rows to quantise). quant: fp8,
// p.x holds up to kFewQuantM 16-bit rows to quantise a chunk at a time, beside one tile of weight rows.
template <int KIND, bool GATED>
hipError_t launch_few(FewParams p, bool whole, bool quant, bool xf16, hipStream_t st) {
  constexpr bool F8 = KIND == kFewFp8;
  const int64_t cu = device_cu_count() > 0 ? device_cu_count() : 256;
  // equal shares of the columns, at most two tiles of 16 rows a workgroup
  const int64_t most = GATED ? 16 : 32;
  const int64_t passes = (p.N + most * cu - 1) / (most * cu);
  const int64_t c = std::max<int64_t>(4, (p.N + cu * passes - 1) / (cu * passes));
  int nt;
  if (GATED) {
    nt = c > 8 || (p.N + 8) * p.K * (F8 ? 1 : 2) >= int64_t{1} << 32 ? 2 : 1;
    p.rt = static_cast<int>(c);
    p.cols = static_cast<int>(c);
  } else {
    nt = c > 16 ? 2 : 1;
    p.rt = static_cast<int>((c + nt - 1) / nt);
    p.cols = p.rt * nt;
  }
  auto go = [&](auto mt_c, auto whole_c, auto xf16_c, auto quant_c) {
    constexpr int MT = decltype(mt_c)::value;
    constexpr bool WHOLE = decltype(whole_c)::value, XF16 = decltype(xf16_c)::value, QUANT = decltype(quant_c)::value;
    // (e4m3 operands of two tiles by more rows than this go to the tile kernel: registers)
    constexpr bool kTwo = !QUANT && (!F8 || MT == 1);
    if constexpr (kTwo) {
      if (nt == 2) return launch_few_k<KIND, MT, 2, WHOLE, GATED, XF16, QUANT>(p, st);
    }
    return nt == 1 ? launch_few_k<KIND, MT, 1, WHOLE, GATED, XF16, QUANT>(p, st) : hipErrorInvalidValue;
  };
  using One = std::integral_constant<int, 1>;
  if (whole) {
    if constexpr (F8) {
      if (xf16) return go(One{}, std::true_type{}, std::true_type{}, std::false_type{});
    }
    return go(One{}, std::true_type{}, std::false_type{}, std::false_type{});
  }
  const std::false_type no;
  if constexpr (F8) {
    if (quant) return xf16 ? go(One{}, no, std::true_type{}, std::true_type{}) : go(One{}, no, no, std::true_type{});
  }
  if (p.M <= 16) return go(One{}, no, no, no);
  if (p.M <= 32) return go(std::integral_constant<int, 2>{}, no, no, no);
  return go(std::integral_constant<int, 4>{}, no, no, no);
}

}  // namespace cubic
