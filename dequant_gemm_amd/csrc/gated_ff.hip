// gated_ff.hip -- the gated feed-forward block over 16-bit weights and its backward pass.
//
//   [g | u] = x W^T,  h = act(g) * u;   dg = dh * u * act'(g),  du = dh * act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// (The gated block of the dense parts beside the routed experts, whose own form cubic_moe_mlp
// computes.) All three products take 16-bit operands and keep fp32 sums. dg and du are rounded to
// 16 bits on the way to the last two, as large an error as the results' own rounding (two 16-bit
// halves of them would take the backward products of 4096 x 7168 x 2048 from 420 to 750 us); the
// pre-activations between the passes are fp32, since theirs would come on top. In fp16 dg and du
// are scaled by powers of two, each row's for dx and each column's for dw, which the results get
// back: they may lie outside the type's range where dx and dw do not. That takes two more
// launches (4096 x 2048 in 22 us) and dg and du twice.
//
// Up to 64 rows (few_rows.h): 1 x 7168 x 2048 (58.7 MB of weights) 10.6-11 us, 5.4 TB/s.
//
// tile16 (more rows; bound by the MFMA and the power it takes): 256 x 256 tiles of eight waves, 64 x
// 128 each, operands straight into two LDS stages of 64 k with a barrier every 32 MFMAs a wave;
// gate and up rows alternate in blocks of 32, so that a wave holds both of a column and h
// leaves from the registers. Operands whose contraction runs down the rows (w for dx; dpre and x
// for dw) lie in LDS as they are and come out through the transposing reads, so nothing is
// transposed in memory. Measured, 4096 x 7168 x 2048 in bf16: forward 177-190 us (1.27-1.36
// PFLOP/s; the library's product of that size alone 153-160 us), both products of the backward
// pass 410-430 us (library 192 + 222), dpre 20 us (117 MB). MFMA busy 65 % of the cycles at 1.8 GHz;
// on zeros 128 us (library 110). Not faster: operands through registers (189 us; with a barrier
// every 16 MFMAs 207), four waves of 128 x 128 (180), two workgroups of four waves to a compute unit
// (245), rings of four stages of 32 k (213), the barrier later in the step, reads earlier, wave
// priorities (all within 2 us). Every load from the same lines: 4 % less.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "dense.h"
#include "few_rows.h"
#include "launch.h"
#include "tile.h"

namespace cubic {
namespace {

// The power of two that brings magnitudes up to the one with these bits (0: none) below 2^15: what is
// scaled by it keeps fp16's eleven bits down to 2^-29 of the largest one, and 2^-40 of it below.
__device__ __forceinline__ int range_exp(uint32_t bits) { return bits == 0u ? 0 : static_cast<int>(bits >> 23) - 141; }

// ---------------------------------------------------------------------------
// C[m][n] = sum_k A(m, k) B(n, k) in 16-bit operands and fp32 sums. A(m, k) is a[m * lda + k],
// or with AT a[k * lda + m] (the contraction runs down the rows); B likewise.
struct TileParams {
  const uint16_t *a, *b;
  int64_t lda, ldb;
  int64_t M, N, K;
  void* y;                 // [M][N] in bf16 (ydt 1) or fp16 (2)
  int ydt;
  // gated form: b holds N gate rows and N up rows behind them; y gets act(gate) * up and,
  // where it is given, pre [M][2 N] both
  float* pre;
  int gelu;
  // slices of the contraction, and where their sums go if there are several: fp32
  // [slices][M][N], gated [slices][M][2 N]
  int slices;
  float* part;
  const uint32_t* range;   // SCALED: [M] bits of the largest magnitudes by which A's rows are scaled (range_exp)
};

// A tile's shape: WM x WN waves with MB x NB blocks of 32 x 32 each; stages of KS steps of 16 k,
// RING of them in LDS (one is read, the others are on their way), the loads of a stage issued
// over SPREAD steps. AHEAD: a wave holds the fragments of a whole stage and reads the next
// one's meanwhile, for tiles whose steps are shorter than a read of LDS takes.
template <int MB_, int NB_, int WM_, int WN_, int KS_, int RING_, int SPREAD_, bool AHEAD_>
struct Tile16 {
  static constexpr int MB = MB_, NB = NB_, WM = WM_, WN = WN_, W = WM * WN, KS = KS_, kRing = RING_, kSpread = SPREAD_;
  static constexpr bool kAhead = AHEAD_;
  static constexpr int TM = 32 * MB * WM, TN = 32 * NB * WN;
  static constexpr int kRow = 32 * KS;                           // bytes of a stage's row
  static constexpr int kStage = kRow * (TM + TN);
  // 1024-byte pieces of a stage per wave
  static constexpr int LA = TM * kRow / 1024 / W, LB = TN * kRow / 1024 / W, NL = LA + LB;
  static_assert(LA * 1024 * W == TM * kRow && LB * 1024 * W == TN * kRow && kSpread <= KS, "whole pieces");
  // (results of the largest tile pass through LDS as a whole)
  static constexpr int kLds = std::max(kRing * kStage, TM * TN > 32768 ? 148 * 1024 : 36 * 1024);
  static_assert(kRing >= 2 && kLds <= 160 * 1024 && (kRing - 2) * NL + NL <= 63, "one compute unit's LDS, a wave's loads on their way");
};

// One operand's stages: rows of 32 KS bytes, or with T 16 KS rows (one k each) of 2 ROWS bytes.
// A piece of 1024 bytes is a wave's load: some rows; in LDS its 16-byte parts lie in the
// lanes' order, and lanes load the part that belongs there.
template <bool T, int ROWS, int W, int KS>
struct Operand {
  static constexpr int kParts = T ? ROWS / 8 : 2 * KS;           // 16-byte parts of a row
  static constexpr int kPer = 64 / kParts;                       // rows of a wave's load
  static constexpr int L = ROWS * 32 * KS / 1024 / W;            // pieces of a wave and stage
  u32x4 rsrc[L];                               // one, but for gate and up rows
  uint32_t voff[L], soff, inc;                 // a lane's offsets, the stage's on top
  uint32_t lane_k;
  int K;

  // from stage s0 on
  __device__ __forceinline__ void init(const uint16_t* base, int64_t ld, int64_t row0, int64_t rows, int64_t K_, int wave, int s0) {
    const int lane = threadIdx.x & 63;
    K = static_cast<int>(K_);
    const int row = kPer * wave + lane / kParts, at = lane % kParts;
    const uint32_t ld2 = static_cast<uint32_t>(2 * ld);
#pragma unroll
    for (int g = 0; g < L; ++g) {
      if constexpr (T) {
        const int part = ((at >> 2) ^ swizzle(row)) * 4 + (at & 3);
        lane_k = static_cast<uint32_t>(row);
        voff[g] = 8 * part < rows - row0 ? static_cast<uint32_t>(row + kPer * W * g) * ld2 + 16u * part : kPast;   // rows a multiple of 8
        rsrc[g] = tile_lds_rsrc(base + row0 + static_cast<int64_t>(s0) * (16 * KS) * ld, 16u * KS * ld2);
      } else {
        lane_k = 16u * (at ^ swizzle(row));
        voff[g] = static_cast<uint32_t>(row + kPer * W * g) * ld2 + lane_k;
        rsrc[g] = tile_lds_rsrc(base + row0 * ld, static_cast<uint32_t>(min(static_cast<int64_t>(ROWS), rows - row0)) * ld2);
      }
    }
    soff = T ? 0u : 32u * KS * static_cast<uint32_t>(s0);
    inc = T ? 16u * KS * ld2 : 32u * KS;
  }
  // Blocks of 32 rows are gate rows and up rows (`rows` further on) in turn, so that a wave
  // holds both of a column; row0 and rows count columns.
  __device__ __forceinline__ void init_gated(const uint16_t* base, int64_t ld, int64_t row0, int64_t rows, int64_t K_, int wave, int s0) {
    static_assert(!T);
    init(base, ld, row0, rows, K_, wave, s0);
    const int lane = threadIdx.x & 63;
    const uint32_t ld2 = static_cast<uint32_t>(2 * ld);
#pragma unroll
    for (int g = 0; g < L; ++g) {
      const int row = kPer * (W * g + wave), blk = row >> 5;
      rsrc[g] = tile_lds_rsrc(base + ((blk & 1) * rows + row0) * ld, static_cast<uint32_t>(min(static_cast<int64_t>(ROWS / 2), rows - row0)) * ld2);
      voff[g] = static_cast<uint32_t>(32 * (blk >> 1) + (row & 31) + lane / kParts) * ld2 + lane_k;
    }
  }
  // The order of a row's parts: any 16 rows read at one part hit all banks. T: the order of
  // its 64-byte segments: four k rows read at one segment hit all banks.
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (T) {
      constexpr int nseg = ROWS / 32;          // segments of a row
      return nseg >= 4 ? (row & 3) : nseg == 2 ? ((row >> 1) & 1) : 0;
    } else {
      return KS == 4 ? (row >> 1) & 7 : (row >> 2) & 3;
    }
  }
  // Before the loads of stage s, which is not whole or behind the last one: what lies past K is
  // not read (and nothing of the stages that follow, in which it lies past K too).
  __device__ __forceinline__ void cut(int s) {
#pragma unroll
    for (int g = 0; g < L; ++g) {
      const bool past = T ? 16 * KS * s + static_cast<int>(lane_k) + kPer * W * g >= K : 32u * KS * s + lane_k >= 2u * static_cast<uint32_t>(K);
      voff[g] = past ? kPast : voff[g];
    }
  }
  // after a stage's loads
  __device__ __forceinline__ void next() {
    if constexpr (T) {
#pragma unroll
      for (int g = 0; g < L; ++g) {
        const uint64_t at = (static_cast<uint64_t>(rsrc[g][1]) << 32 | rsrc[g][0]) + inc;
        rsrc[g][0] = static_cast<uint32_t>(at);
        rsrc[g][1] = static_cast<uint32_t>(at >> 32);
      }
    } else {
      soff += inc;
    }
  }
};

// Fragments of a wave's blocks of 32 rows, for k 16 ks .. + 15 of a stage: lane l has row l % 32
// and eight k from 8 (l / 32) on. Their addresses in LDS are made once for every slot of the
// ring: one for each step, or with T for each block.
template <bool T, int ROWS, int KS, int BLOCKS, int SLOTS>
struct Fragments {
  static constexpr int kAddr = T ? BLOCKS : KS;
  uint32_t at[SLOTS][kAddr];

  __device__ __forceinline__ void init(uint32_t lds, int stage, int first) {   // the wave's first block
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
#pragma unroll
      for (int n = 0; n < kAddr; ++n) {
        uint32_t v = lds + static_cast<uint32_t>(s * stage);
        if constexpr (T) {
          // four k rows of 16 columns at a time come transposed out of LDS
          const int grp = lane >> 4, kr = (lane & 15) >> 2;
          v += (8 * (grp >> 1) + kr) * (2 * ROWS) + (((first + n) ^ Operand<true, ROWS, 1, KS>::swizzle(kr)) << 6) + 32 * (grp & 1) + 8 * (lane & 3);
        } else {
          const int c = lane & 31, h = lane >> 5;
          v += (32 * first + c) * (32 * KS) + (((2 * n + h) ^ Operand<false, ROWS, 1, KS>::swizzle(c)) << 4);
        }
        asm("" : "+v"(v));                     // kept, instead of an addition beside every read
        at[s][n] = v;
      }
  }
  __device__ __forceinline__ s16x8 read(int slot, int ks, int i) const {
    if constexpr (T) {
      typedef __attribute__((address_space(3))) s16x4* LdsPtr;
      const uint32_t a = at[slot][i] + 16 * ks * (2 * ROWS);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(a));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(a + 4 * (2 * ROWS)));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      typedef __attribute__((address_space(3))) s16x8* LdsPtr;
      return *(LdsPtr)(at[slot][ks] + 32 * i * (32 * KS));
    }
  }
};

template <bool F16>
__device__ __forceinline__ f32x16 mma(const s16x8& a, const s16x8& b, const f32x16& c) {
  if constexpr (F16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
}

// One workgroup's share: tile and slice `block`.
template <class Shape, bool F16, bool AT, bool BT, bool GATED, bool SCALED>
__device__ __forceinline__ void tile16(const TileParams& p, int block, unsigned char* smem) {
  constexpr int MB = Shape::MB, NB = Shape::NB, WM = Shape::WM, WN = Shape::WN, W = Shape::W;
  constexpr int TM = Shape::TM, TN = Shape::TN, TC = GATED ? TN / 2 : TN, LA = Shape::LA, LB = Shape::LB, NL = Shape::NL, KS = Shape::KS;
  constexpr int kStage = Shape::kStage, kBOff = TM * Shape::kRow;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  int im, in;
  const int tm = static_cast<int>((p.M + TM - 1) / TM), tn = static_cast<int>((p.N + TC - 1) / TC);
  const int slice = block / (tm * tn);
  tile_place(block - slice * tm * tn, tm, tn, &im, &in);
  const int64_t m0 = static_cast<int64_t>(im) * TM, n0 = static_cast<int64_t>(in) * TC;

  const int all = static_cast<int>((p.K + 16 * KS - 1) / (16 * KS)), len = (all + p.slices - 1) / p.slices;
  const int s0 = slice * len, S = min(all - s0, len);   // stages s0 .. s0 + S - 1
  const int whole = static_cast<int>(p.K / (16 * KS)) - s0;   // of this slice's, those that are whole
  Operand<AT, TM, W, KS> A;
  A.init(p.a, p.lda, m0, p.M, p.K, wave, s0);
  Operand<BT, TN, W, KS> B;
  if constexpr (GATED) {
    B.init_gated(p.b, p.ldb, n0, p.N, p.K, wave, s0);
  } else {
    B.init(p.b, p.ldb, n0, p.N, p.K, wave, s0);
  }
  constexpr int kRing = Shape::kRing;
  const uint32_t lds = tile_lds_at(smem) + 1024u * wave;
  // Piece i of stage s, straight into LDS at slot SLOT of the ring. Stages and pieces come in
  // their order.
  auto load = [&]<int SLOT>(std::integral_constant<int, SLOT>, int s, auto i_c) {
    constexpr int i = decltype(i_c)::value;
    if (i == 0 && s >= whole) {
      asm volatile("" ::: "memory");           // a branch, rarely taken, and no selects in every stage
      A.cut(s0 + s);
      B.cut(s0 + s);
    }
    if constexpr (i < LA) {
      tile_load_lds<SLOT * kStage + 1024 * W * i>(A.rsrc[0], lds, A.voff[i], A.soff);
    } else {
      tile_load_lds<SLOT * kStage + kBOff + 1024 * W * (i - LA)>(B.rsrc[GATED ? i - LA : 0], lds, B.voff[i - LA], B.soff);
    }
    if constexpr (i == NL - 1) {
      A.next();
      B.next();
    }
  };
  // pieces L0 .. L1 - 1
  auto loads = [&]<int SLOT, int L0, int L1>(std::integral_constant<int, SLOT> slot, int s, std::integral_constant<int, L0>, std::integral_constant<int, L1>) {
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (load(slot, s, std::integral_constant<int, L0 + I>{}), ...);
    }(std::make_integer_sequence<int, L1 - L0>{});
  };
  const int wm = wave / WN, wn = wave % WN;
  Fragments<AT, TM, KS, MB, kRing> FA;
  Fragments<BT, TN, KS, NB, kRing> FB;
  FA.init(tile_lds_at(smem), kStage, wm * MB);
  FB.init(tile_lds_at(smem) + kBOff, kStage, wn * NB);
  auto read_a = [&](int slot, int ks, int i) { return FA.read(slot, ks, i); };
  auto read_b = [&](int slot, int ks, int j) { return FB.read(slot, ks, j); };

  f32x16 acc[MB][NB] = {};
  constexpr int Q = MB * NB;
  // f(t) for t = 0 .. N - 1, known to the compiler
  auto times = [&]<int N>(std::integral_constant<int, N>, auto f) {
    [&]<int... T>(std::integer_sequence<int, T...>) {
      (f(std::integral_constant<int, T>{}), ...);
    }(std::make_integer_sequence<int, N>{});
  };
  using I0 = std::integral_constant<int, 0>;
  using INL = std::integral_constant<int, NL>;
  if constexpr (Shape::kAhead) {
    // Stage s: its MFMAs (B times A, so that a lane's results are neighbouring columns of one
    // row) from fragments read before, spread between them the reads of the next stage's.
    // At its start the loads of the next stage are in LDS, and every wave has read this one:
    // the loads of the stage kRing behind it take its place.
    s16x8 fa[2][KS][MB], fb[2][KS][NB];
    constexpr int kReads = KS * (MB + NB), kTotal = KS * Q;
    auto read = [&](auto to_c, int slot, int r) {
      constexpr int to = decltype(to_c)::value;
      const int ks = r / (MB + NB), i = r % (MB + NB);
      if (i < MB) {
        fa[to][ks][i] = read_a(slot, ks, i);
      } else {
        fb[to][ks][i - MB] = read_b(slot, ks, i - MB);
      }
    };
    times(std::integral_constant<int, kRing>{}, [&](auto r) { loads(r, r, I0{}, INL{}); });
    tile_wait<(kRing - 1) * NL>();
    tile_barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(I0{}, 0, r);
    tile_stages<kRing % 2 ? 2 * kRing : kRing>(S, [&](int s, auto u_c) {
      constexpr int u = decltype(u_c)::value, at = u % 2, slot = u % kRing, to_slot = (u + 1) % kRing;
      tile_wait<(kRing - 2) * NL>();
      tile_barrier();
      times(std::integral_constant<int, kTotal>{}, [&](auto t_c) {
        constexpr int t = decltype(t_c)::value;
        constexpr int ks = t / Q, q = t % Q, i = q / NB, j = (i & 1) ? NB - 1 - q % NB : q % NB;
        acc[i][j] = mma<F16>(fb[at][ks][j], fa[at][ks][i], acc[i][j]);
        // in the first three quarters, so that they have arrived at the barrier
        constexpr int kOver = kTotal * 3 / 4;
#pragma unroll
        for (int r = t * kReads / kOver; r < (t + 1) * kReads / kOver && r < kReads; ++r) read(std::integral_constant<int, 1 - at>{}, to_slot, r);
        loads(std::integral_constant<int, slot>{}, s + kRing, std::integral_constant<int, t * NL / kTotal>{}, std::integral_constant<int, (t + 1) * NL / kTotal>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  } else {
    constexpr int SP = Shape::kSpread;         // steps over which a stage's loads are issued
    times(std::integral_constant<int, kRing - 1>{}, [&](auto r) { loads(r, r, I0{}, INL{}); });
    loads(std::integral_constant<int, kRing - 1>{}, kRing - 1, I0{}, std::integral_constant<int, NL / SP>{});
    tile_wait<(kRing - 2) * NL + NL / SP>();
    tile_barrier();
    s16x8 fa[2][MB], fb[2][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) fa[0][i] = read_a(0, 0, i);
#pragma unroll
    for (int j = 0; j < NB; ++j) fb[0][j] = read_b(0, 0, j);

    // A step of 16 k: the MFMAs of its fragments, spread between them the reads of the next
    // step's. Before a stage's last step every wave has read that stage and its loads of the
    // next one are in LDS: after the barrier that one is read, and the loads of the stage
    // kRing behind this one take its place, from the last step on over SP steps. While an MFMA
    // runs its wave issues nothing else, so what counts beside them is the number of other
    // instructions: addresses are made once, slots of the ring known to the compiler.
    tile_stages<kRing>(S, [&](int s, auto u_c) {
      constexpr int slot = decltype(u_c)::value, next_slot = (slot + 1) % kRing, last_slot = (slot + kRing - 1) % kRing;
      times(std::integral_constant<int, KS * Q>{}, [&](auto t_c) {
        constexpr int t = decltype(t_c)::value, ks = t / Q, q = t % Q, f = ks & 1;
        constexpr int i = q / NB, j = (i & 1) ? NB - 1 - q % NB : q % NB;
        if constexpr (ks == KS - 1 && q == 0) {
          tile_wait<(kRing - 2) * NL>();
          tile_barrier();
        }
        acc[i][j] = mma<F16>(fb[f][j], fa[f][i], acc[i][j]);
#pragma unroll
        for (int r = q * (MB + NB) / Q; r < (q + 1) * (MB + NB) / Q; ++r) {
          const int from = ks == KS - 1 ? next_slot : slot, kr = (ks + 1) % KS;
          if (r < MB) {
            fa[1 - f][r] = read_a(from, kr, r);
          } else {
            fb[1 - f][r - MB] = read_b(from, kr, r - MB);
          }
        }
        constexpr int part = ks == KS - 1 ? 0 : ks + 1;
        if constexpr (part < SP) {
          constexpr int l0 = part * NL / SP, l1 = (part + 1) * NL / SP;
          loads(std::integral_constant<int, ks == KS - 1 ? slot : last_slot>{}, (ks == KS - 1 ? s : s - 1) + kRing,
                std::integral_constant<int, l0 + q * (l1 - l0) / Q>{}, std::integral_constant<int, l0 + (q + 1) * (l1 - l0) / Q>{});
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  }
  tile_wait<0>();                              // loads behind the last stage

  auto quad = [&](int i, int j, int g) { return f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]}; };
  if constexpr (GATED) {
    float* pre = p.slices > 1 ? p.part + static_cast<int64_t>(slice) * p.M * 2 * p.N : p.pre;
    if (pre) {
      tile_write<32, MB, NB / 2, WM, WN, 4, Shape::kLds>(smem, pre, 0, 2 * p.N, m0, p.M, n0, p.N, [&](int i, int j, int g) { return quad(i, 2 * j, g); });
      tile_write<32, MB, NB / 2, WM, WN, 4, Shape::kLds>(smem, pre + p.N, 0, 2 * p.N, m0, p.M, n0, p.N, [&](int i, int j, int g) { return quad(i, 2 * j + 1, g); });
    }
    if (p.slices > 1) return;
    tile_write<32, MB, NB / 2, WM, WN, 2, Shape::kLds>(smem, p.y, p.ydt, p.N, m0, p.M, n0, p.N, [&](int i, int j, int g) {
      const f32x4 a = quad(i, 2 * j, g), u = quad(i, 2 * j + 1, g);
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_of(a[e], p.gelu).value * u[e];
      return v;
    });
  } else {
    int back[MB];                              // A's rows as they were: powers of two, exact
#pragma unroll
    for (int i = 0; i < MB; ++i)
      back[i] = SCALED ? range_exp(p.range[min(m0 + 32 * (wm * MB + i) + (static_cast<int>(threadIdx.x) & 31), p.M - 1)]) : 0;
    auto value = [&](int i, int j, int g) {
      f32x4 v = quad(i, j, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = SCALED ? ldexpf(v[e], back[i]) : v[e];
      return v;
    };
    if (p.slices > 1) {
      tile_write<32, MB, NB, WM, WN, 4, Shape::kLds>(smem, p.part + static_cast<int64_t>(slice) * p.M * p.N, 0, p.N, m0, p.M, n0, p.N, value);
    } else {
      tile_write<32, MB, NB, WM, WN, 2, Shape::kLds>(smem, p.y, p.ydt, p.N, m0, p.M, n0, p.N, value);
    }
  }
}

template <class Shape, bool F16>
__global__ __launch_bounds__(64 * Shape::W) void k_ff_forward(TileParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  tile16<Shape, F16, false, false, true, false>(p, static_cast<int>(blockIdx.x), smem);
}

// The backward pass's two products in one launch, so that the compute units that the first one
// leaves idle take up the second: dx = dpre w (its first workgroups), dw = dpre^T x.
template <class Shape, bool F16>
__global__ __launch_bounds__(64 * Shape::W) void k_ff_backward(TileParams dx, TileParams dw, int first) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int block = static_cast<int>(blockIdx.x);
  if (block < first) {
    tile16<Shape, F16, false, true, false, F16>(dx, block, smem);
  } else {
    tile16<Shape, F16, true, true, false, F16>(dw, block - first, smem);
  }
}

constexpr int kKS = 4;                         // a stage's steps, in every shape
// For the plans. A 64 x 64 tile of the forward product that has a compute unit to itself: 256 x 7168 x 2048 in
// 26.5 us.
constexpr TileCosts kCosts16 = {{3232, 1752, 1190, 908, 626}, 430}, kCostsBack = {{3232, 1752, 1190, 908, 626}, 626};
// f(shape) with shape k of kTileShapes
template <class F>
hipError_t with_shape(int k, F f) {
  switch (k) {
    case 0: return f(Tile16<2, 4, 4, 2, kKS, 2, 2, false>{});
    case 1: return f(Tile16<2, 2, 4, 2, kKS, 3, 1, false>{});
    case 2: return f(Tile16<1, 2, 4, 2, kKS, 4, 1, true>{});
    case 3: return f(Tile16<1, 2, 2, 2, kKS, 3, 1, true>{});
    default: return f(Tile16<1, 2, 2, 1, kKS, 4, 1, true>{});
  }
}

int64_t stages16(int64_t K) { return (K + 16 * kKS - 1) / (16 * kKS); }
TilePlan plan_forward(int64_t M, int64_t H, int64_t I) { return plan_tiles(M, 2 * I, stages16(H), kCosts16); }

// Both products in one launch, where they share a shape and fill each other's rounds, or each
// in its own. Does not depend on which of them is asked for, and so neither do the results.
struct BackwardPlan {
  TilePlan dx, dw;
  bool together;
};
BackwardPlan plan_backward(int64_t M, int64_t H, int64_t I) {
  const int64_t cu = plan_cus(), sx = stages16(2 * I), sw = stages16(M);
  BackwardPlan one{}, two{};
  int64_t cost1 = INT64_MAX, costx = INT64_MAX, costw = INT64_MAX;
  for (int k = 0; k < kTileShapeCount; ++k) {
    int64_t cx, cw;
    const TilePlan x = plan_shape(k, cu, M, H, sx, kCostsBack, &cx), w = plan_shape(k, cu, 2 * I, H, sw, kCostsBack, &cw);
    if (cx < costx) {
      costx = cx;
      two.dx = x;
    }
    if (cw < costw) {
      costw = cw;
      two.dw = w;
    }
    const int64_t nx = plan_tile_count(k, M, H) * x.slices, nw = plan_tile_count(k, 2 * I, H) * w.slices;
    const int64_t tx = plan_workgroup(k, (sx + x.slices - 1) / x.slices, kCostsBack, false), tw = plan_workgroup(k, (sw + w.slices - 1) / w.slices, kCostsBack, false);
    // workgroups follow each other without waiting for a round; the last ones run half alone
    const int64_t longest = std::max(tx, tw);
    const int64_t c = std::max(longest, (nx * tx + nw * tw) / cu + longest / 2) + plan_join(x.slices, M, H) + plan_join(w.slices, 2 * I, H);
    if (c < cost1) {
      cost1 = c;
      one = {x, w, true};
    }
  }
  return cost1 <= costx + costw + 4000 ? one : two;    // 4000: a launch
}

template <class Shape>
int64_t tile_count(const TileParams& p, int64_t columns) {
  return ((p.M + Shape::TM - 1) / Shape::TM) * ((p.N + columns - 1) / columns) * p.slices;
}

// dg and du of four neighbouring columns i of row m, in fp32.
struct Dpre {
  f32x4 dg, du;
};
template <bool F16>
__device__ __forceinline__ Dpre dpre_of(const float* __restrict__ pre, const uint16_t* __restrict__ dh, int64_t m, int64_t i, int64_t I, int gelu) {
  const f32x4 g = *reinterpret_cast<const f32x4*>(pre + m * 2 * I + i), u = *reinterpret_cast<const f32x4*>(pre + m * 2 * I + I + i);
  const uint2 d = *reinterpret_cast<const uint2*>(dh + m * I + i);
  Dpre r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t bits = (e < 2 ? d.x : d.y) >> (16 * (e & 1)) & 0xffffu;
    const float t = F16 ? static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits))) : __uint_as_float(bits << 16);
    const Act a = act_of(g[e], gelu);
    r.dg[e] = t * u[e] * a.slope;
    r.du[e] = t * a.value;
  }
  return r;
}

// The largest finite magnitudes of every row and every column of [dg | du], as bits, into `rows`
// [M] and `cols` [2 I], which hold zeros (the atomic maxima do not depend on their order). A lane has
// four columns, a workgroup a run of `run` rows, a multiple of 16, its waves four of them at a time;
// what the waves found in a column meets in LDS, since atomics are what takes time: 4096 x 2048 in
// runs of 4, 16 and 64 rows: 89, 34 and 19 us (84 MB).
__global__ __launch_bounds__(256) void k_ff_range(const float* __restrict__ pre, const uint16_t* __restrict__ dh, int64_t M, int64_t I,
                                                  int gelu, int run, uint32_t* __restrict__ rows, uint32_t* __restrict__ cols) {
  __shared__ uint32_t s_cols[2][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t qs = I >> 2, qb = (qs + 63) / 64, jobs = (M + run - 1) / run * qb;
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int64_t mb = job / qb, q0 = (job - mb * qb) * 64;
    const int64_t i = 4 * min(q0 + lane, qs - 1), end = min((mb + 1) * run, M);   // (lanes behind the last column take it too)
    uint32_t cg[4] = {}, cu[4] = {};
    for (int64_t m0 = mb * run + 4 * wave; m0 < end; m0 += 16) {
      uint32_t top[4] = {};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const Dpre d = dpre_of<true>(pre, dh, min(m0 + r, M - 1), i, I, gelu);    // (the last row again)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          auto take = [&](float v, uint32_t& c) {
            const uint32_t b = __float_as_uint(v) & 0x7fffffffu, f = b < 0x7f800000u ? b : 0u;
            c = max(c, f);
            top[r] = max(top[r], f);
          };
          take(d.dg[e], cg[e]);
          take(d.du[e], cu[e]);
        }
      }
#pragma unroll
      for (int l = 32; l > 0; l >>= 1)
#pragma unroll
        for (int r = 0; r < 4; ++r) top[r] = max(top[r], static_cast<uint32_t>(__shfl_xor(static_cast<int>(top[r]), l, 64)));
      if (lane < 4 && m0 + lane < M) {
        const uint32_t t = lane == 0 ? top[0] : lane == 1 ? top[1] : lane == 2 ? top[2] : top[3];
        if (t != 0u) atomicMax(rows + m0 + lane, t);
      }
    }
    s_cols[0][threadIdx.x] = 0u;
    s_cols[1][threadIdx.x] = 0u;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      atomicMax(&s_cols[0][4 * lane + e], cg[e]);
      atomicMax(&s_cols[1][4 * lane + e], cu[e]);
    }
    __syncthreads();
    const int64_t col = 4 * q0 + threadIdx.x;
    if (col < I) {
      if (s_cols[0][threadIdx.x] != 0u) atomicMax(cols + col, s_cols[0][threadIdx.x]);
      if (s_cols[1][threadIdx.x] != 0u) atomicMax(cols + I + col, s_cols[1][threadIdx.x]);
    }
    __syncthreads();                           // read before the next job's are written
  }
}

template <bool F16>
__device__ __forceinline__ void store_dpre(const f32x4& v, uint16_t* at) {
  *reinterpret_cast<uint2*>(at) = make_uint2(bits16<F16>(v[0]) | bits16<F16>(v[1]) << 16, bits16<F16>(v[2]) | bits16<F16>(v[3]) << 16);
}

// [dg | du] from pre and dh, in the operands' type: the products that follow take 16-bit
// operands, and their results are 16-bit values of the same type. In fp16 dg and du need not lie in the type's range
// where dx and dw do, so there are two of them: with rows scaled by powers of two for dx, with
// columns scaled for dw; either may be NULL.
__global__ __launch_bounds__(256) void k_ff_dpre_bf16(const float* __restrict__ pre, const uint16_t* __restrict__ dh, int64_t M, int64_t I, int gelu,
                                                      uint16_t* __restrict__ dpre) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, quads = M * (I >> 2);
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < quads; v += step) {
    const int64_t m = v / (I >> 2), i = 4 * (v - m * (I >> 2));
    const Dpre d = dpre_of<false>(pre, dh, m, i, I, gelu);
    store_dpre<false>(d.dg, dpre + m * 2 * I + i);
    store_dpre<false>(d.du, dpre + m * 2 * I + I + i);
  }
}
__global__ __launch_bounds__(256) void k_ff_dpre_f16(const float* __restrict__ pre, const uint16_t* __restrict__ dh, int64_t M, int64_t I, int gelu,
                                                     const uint32_t* __restrict__ rows, const uint32_t* __restrict__ cols, uint16_t* __restrict__ for_x,
                                                     uint16_t* __restrict__ for_w) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, quads = M * (I >> 2);
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; v < quads; v += step) {
    const int64_t m = v / (I >> 2), i = 4 * (v - m * (I >> 2));
    const Dpre d = dpre_of<true>(pre, dh, m, i, I, gelu);
    auto store = [&](const f32x4& t, int64_t col) {
      f32x4 s;
      if (for_x) {
        const int e0 = range_exp(rows[m]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = ldexpf(t[e], -e0);
        store_dpre<true>(s, for_x + m * 2 * I + col);
      }
      if (for_w) {
        const u32x4 c = *reinterpret_cast<const u32x4*>(cols + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = ldexpf(t[e], -range_exp(c[e]));
        store_dpre<true>(s, for_w + m * 2 * I + col);
      }
    };
    store(d.dg, i);
    store(d.du, I + i);
  }
}

unsigned quad_grid(int64_t M, int64_t I) {
  const int64_t g = (M * (I >> 2) + 255) / 256;
  return static_cast<unsigned>(g < 65536 ? g : 65536);
}

}  // namespace

// Rows that the streaming kernel takes: every workgroup stages all of them, in each of its passes of 16 columns a
// compute unit. Measured against the tiles (H / I, us of a replay): 4 rows 4096 / 8192 22.6 against 25.6, 4096 / 14336 35.0
// against 35.1; 16 rows 7168 / 2048 13.3 against 19.3, 4096 / 6144 22.4 against 21.7, 4096 / 14336 44 against 35; 32 rows
// 7168 / 2048 15.8 against 20.0, 2048 / 4352 16.6 against 14.8; 64 rows 2048 / 1024 10.1 against 13.0, 4096 / 4096 19.7
// against 18.4, 7168 / 2048 21.6 against 18.7.
static bool ff_few(int64_t M, int64_t H, int64_t I) {
  const int64_t pass = 16 * plan_cus();
  return M <= 4 || (M <= 16 && 2 * I <= 3 * pass) || (I <= pass && (M <= 32 || (M <= kFewMaxM && H <= 4096)));
}

size_t gated_ff_part_bytes(int64_t M, int64_t H, int64_t I) {
  return ff_few(M, H, I) ? 0 : plan_bytes(plan_forward(M, H, I), M, 2 * I);
}

size_t gated_ff_backward_part_bytes(int64_t M, int64_t H, int64_t I) {
  const BackwardPlan plan = plan_backward(M, H, I);
  return plan_bytes(plan.dx, M, H) + plan_bytes(plan.dw, 2 * I, H);
}

hipError_t launch_gated_ff(const FfParams& p, hipStream_t st) {
  const int dt = p.f16 ? 2 : 1;
  if (ff_few(p.M, p.H, p.I)) {
    FewParams f{};
    f.x = p.x;
    f.w = p.w;
    f.N = p.I;
    f.K = p.H;
    f.M = static_cast<int>(p.M);
    f.y = p.h;
    f.ydt = dt;
    f.gelu = p.gelu;
    f.pre = p.pre;
    const bool whole = p.M <= kFewWholeM && 2 * p.H <= kFewWholeBytes;
    return p.f16 ? launch_few<kFewF16, true>(f, whole, false, false, st) : launch_few<kFewBf16, true>(f, whole, false, false, st);
  }
  const TilePlan plan = plan_forward(p.M, p.H, p.I);
  const TileParams t{p.x, p.w, p.H, p.H, p.M, p.I, p.H, p.h, dt, p.pre, p.gelu, plan.slices, p.part, nullptr};
  const hipError_t e = with_shape(plan.shape, [&](auto shape) {
    using Shape = decltype(shape);
    auto kern = p.f16 ? k_ff_forward<Shape, true> : k_ff_forward<Shape, false>;
    const int64_t grid = tile_count<Shape>(t, Shape::TN / 2);
    if (grid * 64 * Shape::W >= int64_t{1} << 32) return hipErrorInvalidValue;
    const hipError_t l = allow_lds(reinterpret_cast<const void*>(kern), Shape::kLds);
    if (l != hipSuccess) return l;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(64 * Shape::W), Shape::kLds, st, t);
    return hipGetLastError();
  });
  if (e != hipSuccess || plan.slices == 1) return e;
  return launch_tile_join<true>({p.part, plan.slices, p.M, p.I, 2 * p.I, nullptr, p.h, dt, p.gelu, p.pre}, st);
}

hipError_t launch_gated_ff_backward(const FfParams& p, hipStream_t st) {
  const unsigned quads = quad_grid(p.M, p.I);
  const int dt = p.f16 ? 2 : 1;
  const BackwardPlan plan = plan_backward(p.M, p.H, p.I);
  float* part = p.part;
  float* part_w = reinterpret_cast<float*>(reinterpret_cast<char*>(part) + plan_bytes(plan.dx, p.M, p.H));
  // the largest magnitudes of the columns, on 16 bytes, then of the rows
  uint32_t *cols = p.range, *rows = p.range + 2 * p.I;
  const TileParams x{p.dpre, p.w, 2 * p.I, p.H, p.M, p.H, 2 * p.I, p.dx, dt, nullptr, 0, plan.dx.slices, part, rows};
  const TileParams w{p.f16 ? p.dpre_w : p.dpre, p.x, 2 * p.I, p.H, 2 * p.I, p.H, p.M, p.dw, dt, nullptr, 0, plan.dw.slices, part_w, cols};
  auto launch = [&](int shape_index, bool with_x, bool with_w) {
    if (!with_x && !with_w) return hipSuccess;
    return with_shape(shape_index, [&](auto shape) {
      using Shape = decltype(shape);
      auto kern = p.f16 ? k_ff_backward<Shape, true> : k_ff_backward<Shape, false>;
      const int64_t first = with_x ? tile_count<Shape>(x, Shape::TN) : 0, grid = first + (with_w ? tile_count<Shape>(w, Shape::TN) : 0);
      if (grid * 64 * Shape::W >= int64_t{1} << 32) return hipErrorInvalidValue;
      const hipError_t l = allow_lds(reinterpret_cast<const void*>(kern), Shape::kLds);
      if (l != hipSuccess) return l;
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(64 * Shape::W), Shape::kLds, st, x, w, static_cast<int>(first));
      return hipGetLastError();
    });
  };
  auto products = [&](bool with_x, bool with_w) {
    if (plan.together) return launch(plan.dx.shape, with_x, with_w);
    const hipError_t l = launch(plan.dx.shape, with_x, false);
    return l != hipSuccess ? l : launch(plan.dw.shape, false, with_w);
  };
  hipError_t e;
  if (p.f16) {
    e = launch_fill_zero(reinterpret_cast<float*>(p.range), p.M + 2 * p.I, false, st);
    if (e != hipSuccess) return e;
    // runs that give each compute unit two workgroups, of 16 rows at least
    const int64_t wide = (p.I / 4 + 63) / 64, run = std::clamp<int64_t>(p.M * wide / (2 * plan_cus()) / 16 * 16, 16, 128);
    const int64_t jobs = (p.M + run - 1) / run * wide;
    hipLaunchKernelGGL(k_ff_range, dim3(static_cast<unsigned>(std::min<int64_t>(jobs, 65536))), dim3(256), 0, st, p.pre, p.dh, p.M, p.I, p.gelu,
                       static_cast<int>(run), rows, cols);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto dpre = [&](bool for_x, bool for_w) {
      hipLaunchKernelGGL(k_ff_dpre_f16, dim3(quads), dim3(256), 0, st, p.pre, p.dh, p.M, p.I, p.gelu, rows, cols, for_x ? p.dpre : nullptr,
                         for_w ? p.dpre_w : nullptr);
      return hipGetLastError();
    };
    if (p.dpre_w != p.dpre || !p.dx || !p.dw) {
      e = dpre(p.dx != nullptr, p.dw != nullptr);
      if (e == hipSuccess) e = products(p.dx != nullptr, p.dw != nullptr);
    } else {                                   // one after the other in one place
      e = dpre(true, false);
      if (e == hipSuccess) e = products(true, false);
      if (e == hipSuccess) e = dpre(false, true);
      if (e == hipSuccess) e = products(false, true);
    }
  } else {
    hipLaunchKernelGGL(k_ff_dpre_bf16, dim3(quads), dim3(256), 0, st, p.pre, p.dh, p.M, p.I, p.gelu, p.dpre);
    e = hipGetLastError();
    if (e == hipSuccess) e = products(p.dx != nullptr, p.dw != nullptr);
  }
  if (e == hipSuccess && p.dx && plan.dx.slices > 1)
    e = launch_tile_join<false>({part, plan.dx.slices, p.M, p.H, p.H, nullptr, p.dx, dt, 0, nullptr}, st);
  if (e == hipSuccess && p.dw && plan.dw.slices > 1)
    e = launch_tile_join<false>({part_w, plan.dw.slices, 2 * p.I, p.H, p.H, nullptr, p.dw, dt, 0, nullptr}, st);
  return e;
}

}  // namespace cubic
