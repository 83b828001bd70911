// fp8.hip -- the block quantiser to e4m3 and the product of e4m3 activations and weights
// with fp32 scales per block of 128.
//
//   y[m][n] = sum_kb xs[m][kb] * ws[n / 128][kb] * (sum_{k in block kb} xq[m][k] wq[n][k]) (+ bias[n])
//
// (Block-scaled 8-bit weights of the dense parts beside the routed experts.) An e4m3 value is
// exact in bf16 (three fraction bits, exponents -9 to 8), so a block's dot product on the bf16
// MFMA has exact products and fp32 sums. The 8-bit MFMA, twice as fast, drops what lies below
// about 2^-14 of the largest of the products that it adds: its sums are off by 1.3e-5 to 2.2e-5
// in the 2-norm, and where large products cancel what is left may be lost whole.
//
// k_quant_fp8_rows, k_quant_fp8_blocks: bound by HBM. 4096 x 7168 rows: 19 us cold, 12 us beside a
// product (88 MB; 17 us at the 5.1 TB/s of a large copy).
//
// k_quant_fp8_blocks: 6144 x 7168 in 23.4 us (132 MB). Few rows (few_rows.h): 1 x 6144 x 7168 from
// bf16 10.5-11.2 us a call (44 MB: 8.6 us), 16 rows 13.2 us.
//
// k_fp8_tile (more rows; bound by the MFMA and the power it takes): 256 x 256 tiles of eight
// waves, 64 x 128 each, both operands straight into two LDS stages of 128 codes, one block of
// scales; A's fragments stay in registers through a stage, B's come one by one, both are
// converted there, and each 16 x 16 x 128 result goes into the sums by four fmas with the row's
// scale times the block's. Measured: 4096 x 4096 x 7168 in 171-180 us (1.34-1.4 PFLOP/s; the
// library's product in bf16 160 us), MFMA busy 57 % of the cycles, vector instructions
// (conversions) 56 %. 4096 x 6144 x 7168, a round and a half of these, takes 256 x 128 tiles:
// 305-316 us. Smaller tiles of 4096 x 4096 x 7168: 256 x 128 202-215 us, 128 x 128 226, 64 x 128
// 283, 64 x 64 275; those of 128 x 128 and less hold a stage's fragments ahead, with the ring's slots
// known to the compiler. Not faster: 128 x 128 by four waves (215 us, but 512 x 6144 x 7168 66
// against 52), 256 x 128 by waves of 128 x 32 (278, spills), with a ring of two or as 128 x 256 (202).
#include <algorithm>

#include "common.h"
#include "dense.h"
#include "few_rows.h"
#include "launch.h"
#include "tile.h"

namespace cubic {
namespace {

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
    const Fp8Scale s = fp8_scale_of(mag_value<XF16>(mag_lanes<16>(mag8(v, 0u))));
    if (on) *reinterpret_cast<uint2*>(xq + m * K + k) = fp8_quant8<XF16>(v, s);
    if ((threadIdx.x & 15) == 0) xs[g] = s.s;
  }
}

// One block of 128 x 128 per workgroup, held in registers between the two passes.
template <bool XF16>
__global__ __launch_bounds__(256) void k_quant_fp8_blocks(const uint16_t* __restrict__ x, int64_t M, int64_t K, int64_t kb,
                                                          uint8_t* __restrict__ xq, float* __restrict__ xs) {
  __shared__ uint32_t s_max[4];
  const int64_t blocks = (M + 127) / 128 * kb;
  for (int64_t at = blockIdx.x; at < blocks; at += gridDim.x) {
    const int64_t mb = at / kb, b = at - mb * kb;
    const int64_t k = b * 128 + 8 * (threadIdx.x & 15);
    u32x4 v[8];
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t m = mb * 128 + 16 * i + (threadIdx.x >> 4);
      v[i] = m < M && k < K ? *reinterpret_cast<const u32x4*>(x + m * K + k) : u32x4{0u, 0u, 0u, 0u};
      a = mag8(v[i], a);
    }
    a = mag_lanes<64>(a);
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = a;
    __syncthreads();
    const Fp8Scale s = fp8_scale_of(mag_value<XF16>(mag_max(mag_max(s_max[0], s_max[1]), mag_max(s_max[2], s_max[3]))));
    __syncthreads();                           // read before the next block's are written
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t m = mb * 128 + 16 * i + (threadIdx.x >> 4);
      if (m < M && k < K) *reinterpret_cast<uint2*>(xq + m * K + k) = fp8_quant8<XF16>(v[i], s);
    }
    if (threadIdx.x == 0) xs[at] = s.s;
  }
}

// ---------------------------------------------------------------------------
// A tile's shape: WM x WN waves with MB x NB blocks of 16 x 16 each, RING stages in LDS. AHEAD: a
// wave holds the fragments of a whole stage and reads the next one's meanwhile, for tiles whose
// MFMAs between a read and its use take less than the read.
template <int MB_, int NB_, int WM_, int WN_, int RING_, bool AHEAD_>
struct Tile8 {
  static constexpr bool kAhead = AHEAD_;
  static constexpr int MB = MB_, NB = NB_, WM = WM_, WN = WN_, W = WM * WN;
  static constexpr int TM = 16 * MB * WM, TN = 16 * NB * WN;
  // 128 codes of every row, the scales of the rows of A, those of B's blocks (a wave's load)
  static constexpr int kStage = 128 * (TM + TN) + 4 * TM + 256;
  // 1024-byte pieces of a stage per wave (eight rows each)
  static constexpr int LA = TM / 8 / W, LB = TN / 8 / W, NL = LA + LB;
  static_assert(LA * 8 * W == TM && LB * 8 * W == TN && TM < 64 * W && TM % 64 == 0 && 128 % (16 * NB) == 0, "whole pieces; a wave's rows in one block");
  static constexpr int kRing = RING_;
  static constexpr int kLds = kRing * kStage;
  static_assert(kRing >= 2 && kLds <= 160 * 1024, "one compute unit's LDS");
};

// One 16 x 16 block of results over the 128 codes of a stage. Codes that several blocks share are
// converted once, as far as registers allow.
__device__ __forceinline__ f32x4 fp8_dot(const i32x8& a, const i32x8& b) {
  f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s)
    part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        e4m3x8_to_bf16(u32x2{static_cast<uint32_t>(a[2 * s]), static_cast<uint32_t>(a[2 * s + 1])}),
        e4m3x8_to_bf16(u32x2{static_cast<uint32_t>(b[2 * s]), static_cast<uint32_t>(b[2 * s + 1])}), part, 0, 0, 0);
  return part;
}

// (AHEAD: two waves a SIMD, without which the compiler takes 330 registers, one workgroup to a
// compute unit, and up to 10 % more time)
template <class Shape, bool GATED>
__global__ __launch_bounds__(64 * Shape::W, Shape::kAhead ? 2 : 1) void k_fp8_tile(Fp8Params p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int MB = Shape::MB, NB = Shape::NB, WM = Shape::WM, WN = Shape::WN, W = Shape::W;
  constexpr int TM = Shape::TM, TN = Shape::TN, TC = GATED ? TN / 2 : TN, LA = Shape::LA, LB = Shape::LB, NL = Shape::NL;
  constexpr int kStage = Shape::kStage, kBOff = TM * 128, kSOff = kBOff + TN * 128;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t N = GATED ? p.N / 2 : p.N;     // columns of results
  int im, in;
  const int tm = static_cast<int>((p.M + TM - 1) / TM), tn = static_cast<int>((N + TC - 1) / TC);
  const int slice = static_cast<int>(blockIdx.x) / (tm * tn);
  tile_place(static_cast<int>(blockIdx.x) - slice * tm * tn, tm, tn, &im, &in);
  const int64_t m0 = static_cast<int64_t>(im) * TM, n0 = static_cast<int64_t>(in) * TC;
  const uint32_t K = static_cast<uint32_t>(p.K);
  const int64_t kb = (p.K + 127) >> 7;
  const int len = (static_cast<int>(kb) + p.slices - 1) / p.slices;
  const int s0 = slice * len, S = min(static_cast<int>(kb) - s0, len);   // stages s0 .. s0 + S - 1

  // ---- stage loads, straight into LDS: wave w takes rows 8 (W i + w) .. + 7 of A, then of B;
  // slot l % 8 of row l / 8 is lane l's and holds the row's piece l % 8 ^ (row / 2 % 8) (any
  // 16 rows read at one piece hit all banks) ----
  const uint32_t lane_k = 16u * ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
  const uint32_t base = static_cast<uint32_t>(8 * wave + (lane >> 3)) * K + lane_k;
  const uint32_t arows = static_cast<uint32_t>(min(static_cast<int64_t>(TM), p.M - m0));
  const uint32_t brows = static_cast<uint32_t>(min(static_cast<int64_t>(TC), N - n0));
  const uint8_t* bp[LB];
  uint32_t boff[LB];
#pragma unroll
  for (int g = 0; g < LB; ++g) {
    if constexpr (GATED) {                     // blocks of 16 rows are gate and up in turn
      const int row = 8 * (W * g + wave), blk = row >> 4;
      bp[g] = p.w + ((blk & 1) * N + n0) * p.K;
      boff[g] = static_cast<uint32_t>(16 * (blk >> 1) + (row & 15) + (lane >> 3)) * K + lane_k;
    } else {
      bp[g] = p.w + n0 * p.K;
      boff[g] = base + 8u * W * g * K;
    }
  }
  // scales: the first waves take the rows' of A, the next one those of B's two blocks (gated:
  // the block of the gate rows, of the up rows)
  const uint32_t kb4 = static_cast<uint32_t>(4 * kb);
  const bool of_a = wave < TM / 64;
  const int64_t b0 = n0 >> 7, b1 = GATED ? (N + n0) >> 7 : min(b0 + 1, (N - 1) >> 7);
  const void* sp = of_a ? static_cast<const void*>(p.xs + m0 * kb) : p.ws + b0 * kb;
  const uint32_t sbytes = of_a ? arows * kb4 : static_cast<uint32_t>((b1 - b0 + 1) * kb4);
  const uint32_t soff = of_a ? static_cast<uint32_t>(tid) * kb4 : lane == 0 ? 0u : lane == 1 ? sbytes - kb4 : kPast;
  constexpr int kRing = Shape::kRing;
  auto stage_at = [&](int s) { return smem + ((kRing & (kRing - 1)) ? s % kRing : s & (kRing - 1)) * kStage; };
  auto load = [&](int s, int i) {              // piece i of stage s; past K and past the rows zeros
    unsigned char* st = stage_at(s) + 1024 * wave;
    const uint32_t k = 128u * static_cast<uint32_t>(s0 + s);
    const bool on = k + lane_k < K;
    if (i < LA) {
      tile_load_lds<0>(tile_lds_rsrc(p.xq + m0 * p.K, arows * K), tile_lds_at(st + 1024 * W * i), on ? base + k + 8u * W * i * K : kPast, 0);
    } else {
      tile_load_lds<0>(tile_lds_rsrc(bp[i - LA], brows * K), tile_lds_at(st + kBOff + 1024 * W * (i - LA)), on ? boff[i - LA] + k : kPast, 0);
    }
  };
  auto load_scale = [&](int s) {
    if (wave <= TM / 64)
      tile_load_lds4<0>(tile_lds_rsrc(sp, sbytes), tile_lds_at(stage_at(s) + kSOff + 256 * wave), s < S ? soff + 4u * static_cast<uint32_t>(s0 + s) : kPast, 0);
  };

  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, q = lane >> 4;
  const uint32_t f0 = 128u * c + 16u * (q ^ (c >> 1)), f1 = 128u * c + 16u * ((q + 4) ^ (c >> 1));
  auto frag = [&](const unsigned char* at) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(at + f0), hi = *reinterpret_cast<const i32x4*>(at + f1);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto read_a = [&](int s, int i) { return frag(stage_at(s) + (wm * MB + i) * 2048); };
  auto read_b = [&](int s, int j) { return frag(stage_at(s) + kBOff + (wn * NB + j) * 2048); };
  auto read_scale = [&](int s, int i) { return *reinterpret_cast<const float*>(stage_at(s) + kSOff + 4 * ((wm * MB + i) * 16 + c)); };
  // the wave's weight rows lie in one block of scales (gated: gate and up in one each)
  const int wb = GATED ? 0 : static_cast<int>(((n0 + 16 * NB * wn) >> 7) - b0);
  auto read_wscale = [&](int s, int b) { return *reinterpret_cast<const float*>(stage_at(s) + kSOff + 4 * (TM + b)); };

  f32x4 acc[MB][NB] = {};
  // results are added this many blocks later (gated 256 x 256 with three spills 8 registers: 208 us of
  // 4096 x 7168 x 2048 against 194)
  constexpr int Q = MB * NB, kLag = GATED ? 2 : 3;
  static_assert(NB % 2 == 0, "fb[0] holds a stage's first block again");
  if constexpr (Shape::kAhead) {
    // Stage s: at its start the loads of the next stage are in LDS, and every wave has read this
    // one: the loads of the stage kRing behind it take its place.
    // Slots of the ring are known to the compiler and offsets made once: what counts beside the
    // MFMAs of such a tile is the number of other instructions.
    static_assert(kRing % 2 == 0);
    const u32x4 ra = tile_lds_rsrc(p.xq + m0 * p.K, arows * K);
    u32x4 rb[LB];
    uint32_t va[LA];
#pragma unroll
    for (int i = 0; i < LA; ++i) va[i] = base + 8u * W * i * K;
#pragma unroll
    for (int i = 0; i < LB; ++i) rb[i] = tile_lds_rsrc(bp[i], brows * K);
    const uint32_t lds = tile_lds_at(smem) + 1024u * wave;
    const int whole = static_cast<int>(K >> 7) - s0;           // of this slice's stages, those that are whole
    // Piece i of stage s into slot SLOT; stages and pieces come in their order.
    auto put = [&]<int SLOT, int I>(std::integral_constant<int, SLOT>, int s, std::integral_constant<int, I>) {
      const uint32_t k = 128u * static_cast<uint32_t>(s0 + s);
      if (I == 0 && s >= whole) {              // past K nothing is read, nor of the stages that follow
        asm volatile("" ::: "memory");
        const bool past = k + lane_k >= K;
#pragma unroll
        for (int i = 0; i < LA; ++i) va[i] = past ? kPast : va[i];
#pragma unroll
        for (int i = 0; i < LB; ++i) boff[i] = past ? kPast : boff[i];
      }
      if constexpr (I < LA) {
        tile_load_lds<SLOT * kStage + 1024 * W * I>(ra, lds, va[I], k);
      } else {
        tile_load_lds<SLOT * kStage + kBOff + 1024 * W * (I - LA)>(rb[I - LA], lds, boff[I - LA], k);
      }
    };
    auto times = [&]<int N0, int N1>(std::integral_constant<int, N0>, std::integral_constant<int, N1>, auto f) {
      [&]<int... T>(std::integer_sequence<int, T...>) {
        (f(std::integral_constant<int, N0 + T>{}), ...);
      }(std::make_integer_sequence<int, N1 - N0>{});
    };
    using I0 = std::integral_constant<int, 0>;
    i32x8 fa[2][MB], fb[2][NB];
    float sx[2][MB], w[2][2];
    constexpr int kReads = 1 + 2 * MB + NB, kOver = std::max(1, Q * 3 / 4);
    auto read = [&]<int TO, int SLOT>(std::integral_constant<int, TO>, std::integral_constant<int, SLOT>, int r) {
      if (r == 0) {
        w[TO][0] = read_wscale(SLOT, wb);
        w[TO][1] = GATED ? read_wscale(SLOT, 1) : 0.0f;
      } else if (r <= MB) {
        sx[TO][r - 1] = read_scale(SLOT, r - 1);
      } else if (r <= 2 * MB) {
        fa[TO][r - 1 - MB] = read_a(SLOT, r - 1 - MB);
      } else {
        fb[TO][r - 1 - 2 * MB] = read_b(SLOT, r - 1 - 2 * MB);
      }
    };
    times(I0{}, std::integral_constant<int, kRing>{}, [&](auto slot) {
      load_scale(slot);
      times(I0{}, std::integral_constant<int, NL>{}, [&](auto i) { put(slot, slot, i); });
    });
    tile_wait<(kRing - 1) * NL>();
    tile_barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(I0{}, I0{}, r);
    tile_stages<kRing>(S, [&](int s, auto slot) {
      constexpr int kSlot = decltype(slot)::value, u = kSlot % 2;
      tile_wait<(kRing - 2) * NL>();
      tile_barrier();
      f32x4 part[kLag + 1];
      auto add = [&](int t) {
        const int i = t % MB, j = t / MB;
        const float f = sx[u][i] * w[u][GATED ? j & 1 : 0];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(part[t % (kLag + 1)][e], f, acc[i][j][e]);
      };
      times(I0{}, std::integral_constant<int, Q>{}, [&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        part[t % (kLag + 1)] = fp8_dot(fb[u][t / MB], fa[u][t % MB]);
        // in the first three quarters, so that they have arrived at the barrier
#pragma unroll
        for (int r = t * kReads / kOver; r < (t + 1) * kReads / kOver && r < kReads; ++r)
          read(std::integral_constant<int, 1 - u>{}, std::integral_constant<int, (kSlot + 1) % kRing>{}, r);
        if (t == 0) load_scale(s + kRing);
        times(std::integral_constant<int, t * NL / Q>{}, std::integral_constant<int, (t + 1) * NL / Q>{}, [&](auto i) { put(slot, s + kRing, i); });
        if (t >= kLag) add(t - kLag);
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int t = Q - kLag; t < Q; ++t) add(t);
    });
  } else {
    // a stage's loads are issued beside a last and a first part of the MFMAs
    constexpr int kLast = MB, kFirst = MB * (NB / 2), kN1 = NL * kLast / (kLast + kFirst);
#pragma unroll
    for (int r = 0; r + 1 < kRing; ++r) {
      load_scale(r);
#pragma unroll
      for (int i = 0; i < NL; ++i) load(r, i);
    }
#pragma unroll
    for (int i = 0; i < kN1; ++i) load(kRing - 1, i);
    // (the scales' loads, which not every wave has, are not counted: the waits are a little long)
    tile_wait<(kRing - 2) * NL + kN1>();
    tile_barrier();
    i32x8 fa[MB], fb[2];
    float sx[MB], w0, w1 = 0.0f;
    fb[0] = read_b(0, 0);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      fa[i] = read_a(0, i);
      sx[i] = read_scale(0, i);
    }
    w0 = read_wscale(0, wb);
    if constexpr (GATED) w1 = read_wscale(0, 1);
    for (int s = 0; s < S; ++s) {
      float sc0[MB], sc1[GATED ? MB : 1];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        sc0[i] = sx[i] * w0;
        if constexpr (GATED) sc1[i] = sx[i] * w1;
      }
      f32x4 part[kLag + 1];
      auto add = [&](int t) {
        const int i = t % MB, j = t / MB;
        const float f = GATED && (j & 1) ? sc1[GATED ? i : 0] : sc0[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(part[t % (kLag + 1)][e], f, acc[i][j][e]);
      };
#pragma unroll
      for (int t = 0; t < Q; ++t) {
        const int i = t % MB, j = t / MB;
        if (t == Q - kLast) {
          // every wave has this stage's last fragments in registers, and its loads of the
          // next stage are in LDS: that one is read from here on, and the stage after it
          // kRing behind it takes this one's place
          tile_wait<(kRing - 2) * NL>();
          tile_barrier();
          fb[(j + 1) & 1] = read_b(s + 1, 0);
        } else if (i == 0) {
          fb[(j + 1) & 1] = read_b(s, j + 1);
        }
        part[t % (kLag + 1)] = fp8_dot(fb[j & 1], fa[i]);
        if (j == NB - 1) {
          fa[i] = read_a(s + 1, i);
          sx[i] = read_scale(s + 1, i);
          if (i == 0) {
            w0 = read_wscale(s + 1, wb);
            if constexpr (GATED) w1 = read_wscale(s + 1, 1);
          }
        }
        if (t >= kLag) add(t - kLag);
        if (t >= Q - kLast) {
          constexpr int l1 = kN1;
          const int u = t - (Q - kLast);
#pragma unroll
          for (int r = u * l1 / kLast; r < (u + 1) * l1 / kLast; ++r) load(s + kRing, r);
        } else if (t < kFirst) {
#pragma unroll
          for (int r = kN1 + t * (NL - kN1) / kFirst; r < kN1 + (t + 1) * (NL - kN1) / kFirst; ++r) load(s - 1 + kRing, r);
          if (t == 0) load_scale(s - 1 + kRing);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int t = Q - kLag; t < Q; ++t) add(t);
    }
  }
  tile_wait<0>();                              // loads behind the last stage

  if constexpr (GATED) {
    if (p.slices > 1) {
      float* part = p.part + static_cast<int64_t>(slice) * p.M * p.N;
      tile_write<16, MB, NB / 2, WM, WN, 4, Shape::kLds>(smem, part, 0, p.N, m0, p.M, n0, N, [&](int i, int j, int) { return acc[i][2 * j]; });
      tile_write<16, MB, NB / 2, WM, WN, 4, Shape::kLds>(smem, part + N, 0, p.N, m0, p.M, n0, N, [&](int i, int j, int) { return acc[i][2 * j + 1]; });
      return;
    }
    tile_write<16, MB, NB / 2, WM, WN, 2, Shape::kLds>(smem, p.y, p.ydt, N, m0, p.M, n0, N, [&](int i, int j, int) {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_of(acc[i][2 * j][e], p.gelu).value * acc[i][2 * j + 1][e];
      return v;
    });
  } else {
    if (p.slices > 1) {
      tile_write<16, MB, NB, WM, WN, 4, Shape::kLds>(smem, p.part + static_cast<int64_t>(slice) * p.M * N, 0, N, m0, p.M, n0, N,
                                                     [&](int i, int j, int) { return acc[i][j]; });
      return;
    }
    auto value = [&](int i, int j, int) {
      f32x4 v = acc[i][j];
      if (p.bias) {
        const int64_t n = n0 + 16 * (wn * NB + j) + 4 * q;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += n + e < N ? p.bias[n + e] : 0.0f;
      }
      return v;
    };
    if (p.ydt == 0) {
      tile_write<16, MB, NB, WM, WN, 4, Shape::kLds>(smem, p.y, 0, N, m0, p.M, n0, N, value);
    } else {
      tile_write<16, MB, NB, WM, WN, 2, Shape::kLds>(smem, p.y, p.ydt, N, m0, p.M, n0, N, value);
    }
  }
}

template <class Shape, bool GATED>
hipError_t launch_tile8(const Fp8Params& p, hipStream_t st) {
  auto kern = k_fp8_tile<Shape, GATED>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), Shape::kLds);
  if (e != hipSuccess) return e;
  const int64_t N = GATED ? p.N / 2 : p.N, TC = GATED ? Shape::TN / 2 : Shape::TN;
  const int64_t tiles = ((p.M + Shape::TM - 1) / Shape::TM) * ((N + TC - 1) / TC) * p.slices;
  if (tiles * 64 * Shape::W >= int64_t{1} << 32) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles)), dim3(64 * Shape::W), Shape::kLds, st, p);
  return hipGetLastError();
}

// Slices are whole blocks of 128 codes. The costs at 2 GHz, from 4096 x 4096 x 7168 in 173, 205, 226, 283
// and 275 us, and 100 x 6144 x 7168 in 26.
constexpr TileCosts kCosts8 = {{5890, 3470, 1880, 1180, 580}, 830};
TilePlan plan8(int64_t M, int64_t N, int64_t K) { return plan_tiles(M, N, (K + 127) / 128, kCosts8); }

template <bool GATED>
hipError_t launch_fp8_tiles(Fp8Params p, hipStream_t st) {
  const TilePlan plan = plan8(p.M, p.N, p.K);
  p.slices = plan.slices;
  hipError_t e;
  switch (plan.shape) {
    case 0: e = launch_tile8<Tile8<4, 8, 4, 2, 2, false>, GATED>(p, st); break;
    case 1: e = launch_tile8<Tile8<4, 4, 4, 2, 3, false>, GATED>(p, st); break;
    case 2: e = launch_tile8<Tile8<2, 4, 4, 2, 4, true>, GATED>(p, st); break;
    case 3: e = launch_tile8<Tile8<2, 4, 2, 2, 4, true>, GATED>(p, st); break;
    default: e = launch_tile8<Tile8<2, 2, 2, 2, 4, true>, GATED>(p, st); break;
  }
  if (e != hipSuccess || plan.slices == 1) return e;
  return launch_tile_join<GATED>({p.part, plan.slices, p.M, GATED ? p.N / 2 : p.N, p.N, p.bias, p.y, p.ydt, p.gelu, nullptr}, st);
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

namespace {
FewParams few_params(const Fp8Params& p, bool gated) {
  FewParams f{};
  f.x = p.x ? static_cast<const void*>(p.x) : p.xq;
  f.xs = p.xs;
  f.w = p.w;
  f.ws = p.ws;
  f.bias = p.bias;
  f.N = gated ? p.N / 2 : p.N;
  f.K = p.K;
  f.M = static_cast<int>(p.M);
  f.y = p.y;
  f.ydt = p.ydt;
  f.gelu = p.gelu;
  return f;
}
}  // namespace

// Rows that the streaming kernel takes: up to 32 weight rows a compute unit, one pass of its workgroups. Measured against
// the tiles (N x K, us of a replay): one row 8192 x 4096 7.9 against 12.5, 10240 x 4096 15.7 against 14.0, 28672 x 4096 31
// against 25; 16 rows 6144 x 7168 13.2 against 15.6, 8192 x 7168 14.8 against 16.6, 10240 x 7168 22.9 against 18.8. Beyond 16 rows
// (wide: two tiles of weight rows a workgroup, not for them): 32 rows 2048 x 7168 11.3 against 11.8, 4096 x 7168 11.6
// against 13.9; 64 rows 1003 x 1936 8.9 against 10.5, 4096 x 4096 12.1 against 12.0, 2048 x 7168 16.3 against 12.5.
static bool fp8_wide(int64_t N) { return N > 16 * plan_cus(); }
static bool fp8_few(int64_t M, int64_t N, int64_t K) {
  if (N > 32 * plan_cus()) return false;
  return M <= 16 || (!fp8_wide(N) && (M <= 32 || (M <= kFewMaxM && K <= 4096)));
}

size_t fp8_part_bytes(int64_t M, int64_t N, int64_t K) { return fp8_few(M, N, K) ? 0 : plan_bytes(plan8(M, N, K), M, N); }

// Of those, the ones that are staged whole.
static bool fp8_whole(int64_t M, int64_t K) { return M <= kFewWholeM && K <= kFewWholeBytes; }
// Every workgroup quantises the rows itself, instead of a launch before the product's, where a graph replay does not
// lose by it (every workgroup repeats the work). Measured from bf16, in us (rows x K, N; replays, then calls; in the
// product against a launch of its own): 8 x 1024, N 1003, 7.0 and 8.8 against 7.0 and 11.9; 8 x 4096 7.7 and 8.5 against
// 7.8 and 11.1; N 4096 7.6 and 8.6 against 8.1 and 11.3. More rows: 16 x 1024 8.9 and 8.6 against 7.0 and 11.5; 37 x 1936
// 12.6 and 12.2 against 9.6 and 12.3. More values: 8 x 7168 10.7 and 10.4 against 9.3 and 11.3. Wide: 8 x 1936, N 7168, 9.9
// and 9.5 against 9.0 and 11.1; 8 x 7168 19.2 and 18.7 against 15.6 and 15.1.
bool fp8_quantises(int64_t M, int64_t N, int64_t K) {
  return fp8_few(M, N, K) && (fp8_whole(M, K) || (M <= kFewQuantM && !fp8_wide(N) && M * K <= 32 * 1024));
}

hipError_t launch_fp8(const Fp8Params& p, bool xf16, hipStream_t st) {
  if (!fp8_few(p.M, p.N, p.K)) return launch_fp8_tiles<false>(p, st);
  return launch_few<kFewFp8, false>(few_params(p, false), p.x && fp8_whole(p.M, p.K), p.x != nullptr, xf16, st);
}

hipError_t launch_fp8_gated(const Fp8Params& p, bool xf16, hipStream_t st) {
  if (!fp8_few(p.M, p.N, p.K)) return launch_fp8_tiles<true>(p, st);
  return launch_few<kFewFp8, true>(few_params(p, true), p.x && fp8_whole(p.M, p.K), p.x != nullptr, xf16, st);
}

}  // namespace cubic
