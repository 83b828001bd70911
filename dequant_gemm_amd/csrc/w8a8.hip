// w8a8.hip -- the int8 product of per-token activations and per-channel weights.
//
//   y[m][n] = fp32(sum_k xq[m][k] * wq[n][k]) * w_scale[n] * x_scale[m] (+ bias[n])
//
// (The msModelSlim article's W8A8 scheme, which it gives the projections and shared
// experts that stay beside the routed experts.) The dot product is exact in int32, so
// the split of K between waves does not change results.
//
// k_w8a8_rows (up to 64 rows; bound by the weight's bytes): every workgroup takes an
// equal share of the weight rows, its sixteen waves a step of 64 codes each in turn.
// Weights go from HBM to registers: a lane quad loads 64 contiguous bytes of a row
// (loads in MFMA operand order would touch a row a lane and take the address unit four
// times as long), and the lanes exchange the words through the LDS crossbar when they
// are used. The activations pass through LDS in chunks of 64 KB, two buffers, one
// barrier a chunk that leaves the weight loads in flight. Up to four bf16 or fp16 rows
// are quantised by every workgroup itself, beside its first weight loads, which saves a
// launch; with more rows the quantiser is a launch of its own (every workgroup quantising
// 37 rows of 1928, chunk by chunk: 43 us instead of 10).
//
// Measured: 6144 x 7168, one bf16 row: 44.1 MB in 9.8-10.2 us (4.4 TB/s; a large copy
// runs at 5.1); 7168 x 2048, 64 rows: 9.7 us, where the launch, the chunks' round trips
// and the join of sixteen waves' sums count, not the 3 us of the weight's bytes.
//
// k_w8a8_tile (more rows; bound by the int8 MFMA, at the clock that its power allows):
// eight waves a tile of 256 rows (four a smaller one), both operands in two LDS stages of
// 64 codes, filled through registers two stages ahead, so that a stage costs one barrier;
// the result leaves through LDS in 16-byte pieces. Measured: 4096 x 6144 x 7168 in
// 181-220 us by box and clock (1.64-2.0 POP/s; the library's int8 product 168-184 us on
// the same boxes), 151 us on zeros (less power, a higher clock; library 141). MFMA busy
// 54 % of the cycles. Not faster: four waves with direct global-to-LDS stages (192-225)
// or through registers (196-230), 256 x 256 tiles (209; a second, half-empty round of
// tiles), 128 x 192 tiles two to a compute unit (227), fragment reads moved ahead, wave
// priorities and workgroups at rotated K offsets (all within 2 us). Faster than 2-byte
// stores from the MFMA layout: 30 us.
#include <algorithm>
#include <utility>

#include "act_quant.h"
#include "common.h"
#include "launch.h"

namespace cubic {
namespace {

constexpr uint32_t kW8Rsrc3 = 0x00020000u;     // raw buffer, 32-bit data format
constexpr int kRowsWaves = 16;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t w8_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes),
                                           static_cast<int>(kW8Rsrc3));
}
__device__ __forceinline__ void w8_lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One result: the product's rounding steps, in this order everywhere.
__device__ __forceinline__ float w8_result(int acc, float ws, float xs, bool has_bias, float bias) {
  const float v = static_cast<float>(acc) * ws;
  return has_bias ? fmaf(v, xs, bias) : v * xs;
}

struct RowsParams {
  W8Params q;
  int rows, rt;            // weight rows per workgroup, and per tile of 16
};

// MT: tiles of 16 activation rows; SPC = 4 / MT steps per wave and chunk. QUANT: up
// to four rows of bf16 (or, XF16, fp16) values are quantised into LDS as a whole.
template <int MT, int NT, bool QUANT, bool XF16>
__global__ __launch_bounds__(1024) void k_w8a8_rows(RowsParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int SPC = 4 / MT, PM = 4;
  constexpr int RM = QUANT ? 4 : 16 * MT;      // activation rows held in LDS
  const W8Params& w = p.q;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const int M = static_cast<int>(w.M), K = static_cast<int>(w.K);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * p.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), w.N - n0));
  const int nsteps = (K + 63) >> 6;
  const int iters = (nsteps + kRowsWaves - 1) / kRowsWaves;      // the longest wave's steps

  // ---- weights: lane l loads piece l % 4 of row l / 4 of each tile ----
  const uint32_t wbytes = static_cast<uint32_t>(rows) * static_cast<uint32_t>(K);
  const __amdgpu_buffer_rsrc_t wrs = w8_rsrc(w.w + n0 * K, wbytes);
  uint32_t voff[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    voff[i] = static_cast<uint32_t>(min(i * p.rt + min(lane >> 2, p.rt - 1), rows - 1)) * static_cast<uint32_t>(K) +
              16u * (lane & 3);
  u32x4 cb[PM][NT];
  // step i of this wave is K step 16 i + wave; past the last one nothing is read
  auto issue = [&](auto u_c, int i) {
    constexpr int u = decltype(u_c)::value;
    const int s = i * kRowsWaves + wave;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t off = s < nsteps ? voff[t] + 64u * static_cast<uint32_t>(s) : wbytes;
      cb[u][t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wrs, off, 0, 0));
    }
  };

  // ---- activations ----
  // 16-byte piece j of row m at step st of a buffer: rows of 64 bytes, the piece
  // XORed with two row bits so that 16 rows read at one piece hit all banks
  auto place = [&](int st, int m, int j) { return ((st * RM + m) * 4 + (j ^ ((m >> 2) & 3))) * 16; };
  constexpr int XR = 4;                        // pieces per thread and chunk
  u32x4 xv[XR];
  const __amdgpu_buffer_rsrc_t xrs = w8_rsrc(w.xq, static_cast<uint32_t>(M) * static_cast<uint32_t>(K));
  constexpr int kPieces = 64 * SPC;            // pieces of a row in a chunk
  auto load_x = [&](int c) {
#pragma unroll
    for (int r = 0; r < XR; ++r) {
      const int idx = tid + 1024 * r;
      const int m = idx / kPieces;
      const int k = c * (SPC * 1024) + 16 * (idx % kPieces);
      const uint32_t off = m < M && k < K ? static_cast<uint32_t>(m) * static_cast<uint32_t>(K) + k
                                          : static_cast<uint32_t>(M) * static_cast<uint32_t>(K);
      u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xrs, off, 0, 0));
      if (k + 8 >= K) { v.z = 0u; v.w = 0u; }  // K is a multiple of 8: the piece may end in the next row
      xv[r] = v;
    }
  };
  auto store_x = [&](int c) {
    unsigned char* buf = smem + (c & 1) * 65536;
#pragma unroll
    for (int r = 0; r < XR; ++r) {
      const int idx = tid + 1024 * r;
      const int m = idx / kPieces, pk = idx % kPieces;
      if (m < M) *reinterpret_cast<u32x4*>(buf + place(pk >> 2, m, pk & 3)) = xv[r];
    }
  };

  __shared__ float s_red[QUANT ? 4 * kRowsWaves : 1];
  float qscale[QUANT ? 4 : 1];
  if constexpr (QUANT) {
    // K <= 8192: one vector of eight values per thread and row
    const int nvec = K >> 3;
    u32x4 v[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
      v[m] = m < M && tid < nvec ? reinterpret_cast<const u32x4*>(w.x + static_cast<int64_t>(m) * K)[tid]
                                 : u32x4{0u, 0u, 0u, 0u};
    __builtin_amdgcn_sched_barrier(0);
    [&]<int... U>(std::integer_sequence<int, U...>) {
      (issue(std::integral_constant<int, U>{}, U), ...);
    }(std::make_integer_sequence<int, PM>{});
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (m < M) {
        const float a = wave_larger<true>(absmax8<XF16, true>(v[m], 0.0f));
        if (lane == 0) s_red[m * kRowsWaves + wave] = a;
      }
    }
    w8_lds_barrier();
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      qscale[m] = 0.0f;
      if (m < M) {
        float a = 0.0f;
#pragma unroll
        for (int k = 0; k < kRowsWaves; ++k) a = larger<true>(a, s_red[m * kRowsWaves + k]);
        const float sx = scale_of<true>(a);
        qscale[m] = sx;
        const bool fast = sx >= 0x1p-100f && sx <= 0x1p100f;
        const uint2 c = quant8<XF16>(v[m], sx, __builtin_amdgcn_rcpf(sx), fast);
        // eight codes: half a piece; past K up to the last step's end zeros
        if (tid < nsteps * 8)
          *reinterpret_cast<uint2*>(smem + place(tid >> 3, m, (tid >> 1) & 3) + 8 * (tid & 1)) =
              tid < nvec ? c : make_uint2(0u, 0u);
      }
    }
    w8_lds_barrier();
  } else {
    load_x(0);
    __builtin_amdgcn_sched_barrier(0);         // activations ahead of the weights
    [&]<int... U>(std::integer_sequence<int, U...>) {
      (issue(std::integral_constant<int, U>{}, U), ...);
    }(std::make_integer_sequence<int, PM>{});
    __builtin_amdgcn_sched_barrier(0);
  }

  i32x4 acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[a][t] = i32x4{0, 0, 0, 0};
  const int xaddr = 4 * (4 * nl + kq);
  const int ml = QUANT ? (nl & 3) : nl;        // rows past M: their sums are not used
  for (int i0 = 0; i0 < iters; i0 += PM) {
    [&]<int... U>(std::integer_sequence<int, U...>) {
      (([&] {
         constexpr int u = U;
         const int i = i0 + u;
         if constexpr (!QUANT && u % SPC == 0) {
           // chunk c in, chunk c + 1 on its way (the chunk before the last one read
           // the buffer that c overwrites; every wave is past it)
           const int c = i / SPC;
           if (i < iters) {
             store_x(c);
             load_x(c + 1);
             w8_lds_barrier();
           }
         }
         if (i * kRowsWaves + wave < nsteps) {
           const int st = QUANT ? i * kRowsWaves + wave : (i % SPC) * kRowsWaves + wave;
           const unsigned char* buf = QUANT ? smem : smem + ((i / SPC) & 1) * 65536;
           i32x4 b[NT];
#pragma unroll
           for (int t = 0; t < NT; ++t)
#pragma unroll
             for (int d = 0; d < 4; ++d) b[t][d] = __builtin_amdgcn_ds_bpermute(xaddr, static_cast<int>(cb[u][t][d]));
#pragma unroll
           for (int a = 0; a < MT; ++a) {
             const i32x4 av = *reinterpret_cast<const i32x4*>(buf + place(st, 16 * a + ml, kq));
#pragma unroll
             for (int t = 0; t < NT; ++t)
               acc[a][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, b[t], acc[a][t], 0, 0, 0);
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
  w8_lds_barrier();                            // the activations are read
  int* red = reinterpret_cast<int*>(smem);
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
  w8_lds_barrier();
  for (int idx = tid; idx < M * 32; idx += 1024) {
    const int m = idx >> 5, j = idx & 31;
    const int t = NT == 1 ? 0 : (j >= p.rt ? 1 : 0), col = j - t * p.rt;
    if (j >= rows || col >= p.rt) continue;
    const int at = 256 * (m >> 4) + 64 * (m & 3) + 16 * ((m >> 2) & 3) + col;
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kRowsWaves; ++k) sum += red[(k * NT + t) * kTile + at];
    const int64_t n = n0 + j;
    float xs;
    if constexpr (QUANT) {
      xs = m == 0 ? qscale[0] : m == 1 ? qscale[1] : m == 2 ? qscale[2] : qscale[3];
    } else {
      xs = w.xs[m];
    }
    store_out(static_cast<float*>(w.y), w.ybf16 != 0, static_cast<int64_t>(m) * w.N + n,
              w8_result(sum, w.ws[n], xs, w.bias != nullptr, w.bias ? w.bias[n] : 0.0f));
  }
}

// ---------------------------------------------------------------------------
// A tile's shape: WM x WN waves with MB x NB blocks of 32 x 32 each.
template <int MB_, int NB_, int WM_, int WN_>
struct Tile {
  static constexpr int MB = MB_, NB = NB_, WM = WM_, WN = WN_, W = WM * WN;
  static constexpr int TM = 32 * MB * WM, TN = 32 * NB * WN;
  static constexpr int kStage = 64 * (TM + TN);                  // 64 codes of every row
  // 16-row pieces of a stage per wave (the last ones may be past the tile)
  static constexpr int LA = (TM / 16 + W - 1) / W, LB = (TN / 16 + W - 1) / W, NL = LA + LB;
  // The epilogue takes the tile's rows in NP passes of what fits its share of LDS.
  static constexpr int kLdsTarget = W == 8 ? 144 * 1024 : 40 * 1024;
  static constexpr int out_bytes(int np, int bytes) { return TM / np * (TN * bytes + 16) + 8 * TN; }
  static constexpr int passes(int bytes) {
    int np = 1;
    while (np < MB && out_bytes(np, bytes) > kLdsTarget) np *= 2;
    return np;
  }
  static constexpr int max3(int x, int y, int z) { return x > y ? (x > z ? x : z) : (y > z ? y : z); }
  static constexpr int kLds = max3(2 * kStage, out_bytes(passes(2), 2), out_bytes(passes(4), 4));
  static_assert(kLds <= 160 * 1024, "one compute unit's LDS");
};

template <class Shape>
__global__ __launch_bounds__(64 * Shape::W) void k_w8a8_tile(W8Params p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int MB = Shape::MB, NB = Shape::NB, WN = Shape::WN, W = Shape::W, kThreads = 64 * W;
  constexpr int TM = Shape::TM, TN = Shape::TN, LA = Shape::LA, NL = Shape::NL;
  constexpr int kLoads1 = (NL + 1) / 2;        // pieces of a stage that move in the half step after the barrier
  constexpr int kStage = Shape::kStage, kBOff = TM * 64;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int K = static_cast<int>(p.K);

  // Tiles to workgroups: neighbouring workgroup ids go to different XCDs, so each XCD
  // takes a run of tiles, in groups of four tile rows (a run's tiles share operand rows
  // in its L2).
  const int tm = static_cast<int>((p.M + TM - 1) / TM), tn = static_cast<int>((p.N + TN - 1) / TN);
  int t = static_cast<int>(blockIdx.x);
  {
    const int nt = tm * tn, base = nt >> 3, rem = nt & 7, x = t & 7;
    t = x * base + min(x, rem) + (t >> 3);
  }
  const int per = 4 * tn, grp = t / per, in = t - grp * per;
  const int gm = min(4, tm - 4 * grp);
  const int64_t m0 = static_cast<int64_t>(4 * grp + in % gm) * TM;
  const int64_t n0 = static_cast<int64_t>(in / gm) * TN;

  // ---- stage loads: wave w takes rows 16 (W i + w) .. + 15 of A, then of B; lane l
  // loads the 16-byte piece l % 4 of row l / 4 (64 contiguous bytes a lane quad) into
  // registers and writes it to slot piece ^ (row / 4 % 4) of the row (any 16 rows read
  // at one piece hit all banks) ----
  const uint32_t abytes = static_cast<uint32_t>(min(static_cast<int64_t>(TM), p.M - m0)) * static_cast<uint32_t>(K);
  const uint32_t bbytes = static_cast<uint32_t>(min(static_cast<int64_t>(TN), p.N - n0)) * static_cast<uint32_t>(K);
  const __amdgpu_buffer_rsrc_t ars = w8_rsrc(p.xq + m0 * K, abytes);
  const __amdgpu_buffer_rsrc_t brs = w8_rsrc(p.w + n0 * K, bbytes);
  const uint32_t lane_k = 16u * (lane & 3);
  const uint32_t abase = static_cast<uint32_t>(16 * wave + (lane >> 2)) * static_cast<uint32_t>(K) + lane_k;
  const uint32_t bbase = static_cast<uint32_t>(16 * wave + (lane >> 2)) * static_cast<uint32_t>(K) + lane_k;
  const uint32_t slot = 64u * (lane >> 2) + 16u * ((lane & 3) ^ ((lane >> 4) & 3));
  const int S = (K + 63) >> 6;
  u32x4 gr[2][NL];                             // pieces on their way: stages of either parity
  auto load = [&](auto set_c, int s, int i) {  // piece i of stage s; past K nothing is read: zeros
    constexpr int set = decltype(set_c)::value;
    const uint32_t k = 64u * static_cast<uint32_t>(s);
    const bool on = k + lane_k < static_cast<uint32_t>(K);
    const int g = i < LA ? i : i - LA;         // pieces past the tile read nothing
    if (i < LA) {
      const uint32_t off = on && 16 * (W * g + wave) < TM ? abase + k + 16u * W * g * static_cast<uint32_t>(K) : abytes;
      gr[set][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ars, off, 0, 0));
    } else {
      const uint32_t off = on && 16 * (W * g + wave) < TN ? bbase + k + 16u * W * g * static_cast<uint32_t>(K) : bbytes;
      gr[set][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(brs, off, 0, 0));
    }
  };
  auto store = [&](auto set_c, int s, int i) { // piece i of stage s into LDS
    constexpr int set = decltype(set_c)::value;
    unsigned char* st = smem + (s & 1) * kStage;
    u32x4 v = gr[set][i];
    const int g = i < LA ? i : i - LA;
    if (i < LA) {
      // K a multiple of 8, not of 16: the last piece's upper half belongs to the next
      // row (zeros in A make it count nothing)
      if (64u * static_cast<uint32_t>(s) + lane_k + 8u >= static_cast<uint32_t>(K)) { v.z = 0u; v.w = 0u; }
      if (16 * (W * g + wave) < TM) *reinterpret_cast<u32x4*>(st + (W * g + wave) * 1024 + slot) = v;
    } else {
      if (16 * (W * g + wave) < TN) *reinterpret_cast<u32x4*>(st + kBOff + (W * g + wave) * 1024 + slot) = v;
    }
  };

  const int wm = wave / WN, wn = wave % WN;
  const uint32_t swz = (c >> 2) & 3;
  auto frag = [&](const unsigned char* st, int row, int ks) {
    return *reinterpret_cast<const i32x4*>(st + row * 64 + (((2 * ks + h) ^ swz) << 4));
  };
  auto read_a = [&](int s, int ks, int i) {
    return frag(smem + (s & 1) * kStage, wm * 32 * MB + 32 * i + c, ks);
  };
  auto read_b = [&](int s, int ks, int j) {
    return frag(smem + (s & 1) * kStage + kBOff, wn * 32 * NB + 32 * j + c, ks);
  };

  i32x16 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using IL = std::integral_constant<int, kLoads1>;
  using IN = std::integral_constant<int, NL>;
#pragma unroll
  for (int i = 0; i < NL; ++i) load(I0{}, 0, i);
#pragma unroll
  for (int i = 0; i < NL; ++i) load(I1{}, 1, i);
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    store(I0{}, 0, i);
    load(I0{}, 2, i);
  }
  w8_lds_barrier();
#pragma unroll
  for (int i = 0; i < kLoads1; ++i) {
    store(I1{}, 1, i);
    load(I1{}, 3, i);
  }
  i32x4 fa[2][MB], fb[2][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i) fa[0][i] = read_a(0, 0, i);
#pragma unroll
  for (int j = 0; j < NB; ++j) fb[0][j] = read_b(0, 0, j);

  // One half step: the MFMAs of fragments f (weights times activations, so that a
  // lane's results are consecutive channels of one row). Spread between them: the
  // reads of the other half's fragments, and for pieces l0 .. l1 - 1 of stage s_st the
  // write to LDS and the load of the piece two stages later into its registers.
  auto half = [&](auto f_c, int s_read, int ks, auto set_c, int s_st, auto l0_c, auto l1_c) {
    constexpr int f = decltype(f_c)::value, l0 = decltype(l0_c)::value, l1 = decltype(l1_c)::value;
    constexpr int Q = MB * NB;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = q / NB, j = (i & 1) ? NB - 1 - q % NB : q % NB;
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[f][j], fa[f][i], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int r = q * (MB + NB) / Q; r < (q + 1) * (MB + NB) / Q; ++r) {
        if (r < MB) {
          fa[1 - f][r] = read_a(s_read, ks, r);
        } else {
          fb[1 - f][r - MB] = read_b(s_read, ks, r - MB);
        }
      }
#pragma unroll
      for (int r = l0 + q * (l1 - l0) / Q; r < l0 + (q + 1) * (l1 - l0) / Q; ++r) {
        store(set_c, s_st, r);
        load(set_c, s_st + 2, r);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Stage s: its second half's fragments are read beside the first half's MFMAs; then
  // stage s + 1 is whole in LDS (its last pieces were written there) and every wave is
  // done with stage s, so that after the barrier stage s + 1 is read and stage s + 2
  // takes the place of s.
  auto stage = [&](int s, auto next_c, auto after_c) {
    half(I0{}, s, 1, next_c, s + 1, IL{}, IN{});
    w8_lds_barrier();
    half(I1{}, s + 1, 0, after_c, s + 2, I0{}, IL{});
  };
  int s = 0;
  for (; s + 1 < S; s += 2) {
    stage(s, I1{}, I0{});
    stage(s + 1, I0{}, I1{});
  }
  if (s < S) stage(s, I1{}, I0{});
  __syncthreads();

  // ---- epilogue: D row n = 8 (e / 4) + 4 h + e % 4 of block (i, j), column m = c;
  // through LDS, so that rows leave in whole 16-byte pieces ----
  float* s_ws = reinterpret_cast<float*>(smem);
  float* s_bias = s_ws + TN;
  unsigned char* tile = smem + 8 * TN;
  for (int i = tid; i < TN; i += kThreads) {
    const bool on = n0 + i < p.N;
    s_ws[i] = on ? p.ws[n0 + i] : 0.0f;
    s_bias[i] = on && p.bias ? p.bias[n0 + i] : 0.0f;
  }
  float xs[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int64_t m = m0 + wm * 32 * MB + 32 * i + c;
    xs[i] = p.xs[m < p.M ? m : p.M - 1];
  }
  __syncthreads();
  auto write_out = [&](auto bytes_c) {
    constexpr int kBytes = decltype(bytes_c)::value;             // of a result
    constexpr int NP = Shape::passes(kBytes);
    constexpr int BP = MB / NP, kRows = TM / NP, kStride = TN * kBytes + 16;
    constexpr int kPer = 16 / kBytes;                            // results of a piece
    const bool whole = p.N % kPer == 0;                          // rows start on 16 bytes
#pragma unroll
    for (int ip = 0; ip < NP; ++ip) {
      if (ip) __syncthreads();
#pragma unroll
      for (int ib = 0; ib < BP; ++ib) {
        const int i = ip * BP + ib;
        unsigned char* row = tile + (wm * 32 * BP + 32 * ib + c) * kStride;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int nl = wn * 32 * NB + 32 * j + 8 * g + 4 * h;
            const f32x4 ws = *reinterpret_cast<const f32x4*>(s_ws + nl);
            const f32x4 bs = *reinterpret_cast<const f32x4*>(s_bias + nl);
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = w8_result(acc[i][j][4 * g + r], ws[r], xs[i], p.bias != nullptr, bs[r]);
            store_out4(reinterpret_cast<float*>(row), kBytes == 2, nl, v);
          }
      }
      __syncthreads();
      const int cols = static_cast<int>(min(static_cast<int64_t>(TN), p.N - n0));
      auto global_row = [&](int r) {
        const int w = r / (32 * BP);
        return m0 + w * 32 * MB + ip * 32 * BP + (r - w * 32 * BP);
      };
      unsigned char* y = static_cast<unsigned char*>(p.y);
      if (whole) {
        constexpr int kPieces = TN / kPer;
        for (int idx = tid; idx < kRows * kPieces; idx += kThreads) {
          const int r = idx / kPieces, q = idx - r * kPieces;
          const int64_t m = global_row(r);
          if (m < p.M && q * kPer < cols)
            *reinterpret_cast<u32x4*>(y + (m * p.N + n0 + q * kPer) * kBytes) =
                *reinterpret_cast<const u32x4*>(tile + r * kStride + 16 * q);
        }
      } else {
        for (int idx = tid; idx < kRows * TN; idx += kThreads) {
          const int r = idx / TN, q = idx - r * TN;
          const int64_t m = global_row(r);
          if (m < p.M && q < cols) {
            if constexpr (kBytes == 2) {
              reinterpret_cast<uint16_t*>(y)[m * p.N + n0 + q] = reinterpret_cast<const uint16_t*>(tile + r * kStride)[q];
            } else {
              reinterpret_cast<float*>(y)[m * p.N + n0 + q] = reinterpret_cast<const float*>(tile + r * kStride)[q];
            }
          }
        }
      }
    }
  };
  if (p.ybf16) {
    write_out(std::integral_constant<int, 2>{});
  } else {
    write_out(std::integral_constant<int, 4>{});
  }
}

template <int MT, int NT, bool QUANT, bool XF16>
hipError_t launch_rows_k(const RowsParams& p, unsigned grid, hipStream_t st) {
  auto kern = k_w8a8_rows<MT, NT, QUANT, XF16>;
  const int nsteps = static_cast<int>((p.q.K + 63) / 64);
  const int red = kRowsWaves * NT * 16 * MT * 16 * 4;
  const int x = QUANT ? nsteps * 256 : 131072;
  const int lds = std::max(red, x);
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(1024), lds, st, p);
  return hipGetLastError();
}

template <bool QUANT, bool XF16>
hipError_t launch_rows(const W8Params& q, hipStream_t st) {
  const int64_t cu = device_cu_count() > 0 ? device_cu_count() : 256;
  RowsParams p{q, 0, 0};
  // equal shares of the rows, at most two tiles of 16 a workgroup
  const int64_t passes = (q.N + 32 * cu - 1) / (32 * cu);
  const int64_t r = std::max<int64_t>(4, (q.N + cu * passes - 1) / (cu * passes));
  const int nt = r > 16 ? 2 : 1;
  p.rt = static_cast<int>((r + nt - 1) / nt);
  p.rows = p.rt * nt;
  const unsigned grid = static_cast<unsigned>((q.N + p.rows - 1) / p.rows);
  if constexpr (QUANT) {
    return nt == 1 ? launch_rows_k<1, 1, true, XF16>(p, grid, st) : launch_rows_k<1, 2, true, XF16>(p, grid, st);
  } else {
    if (q.M <= 16)
      return nt == 1 ? launch_rows_k<1, 1, false, false>(p, grid, st) : launch_rows_k<1, 2, false, false>(p, grid, st);
    if (q.M <= 32)
      return nt == 1 ? launch_rows_k<2, 1, false, false>(p, grid, st) : launch_rows_k<2, 2, false, false>(p, grid, st);
    return nt == 1 ? launch_rows_k<4, 1, false, false>(p, grid, st) : launch_rows_k<4, 2, false, false>(p, grid, st);
  }
}

template <class Shape>
hipError_t launch_tile(const W8Params& p, hipStream_t st) {
  auto kern = k_w8a8_tile<Shape>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), Shape::kLds);
  if (e != hipSuccess) return e;
  const int64_t tiles = ((p.M + Shape::TM - 1) / Shape::TM) * ((p.N + Shape::TN - 1) / Shape::TN);
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles)), dim3(64 * Shape::W), Shape::kLds, st, p);
  return hipGetLastError();
}

constexpr int64_t kRowsMaxM = 64;
constexpr int64_t kQuantMaxM = 4, kQuantMaxK = 8192;

}  // namespace

bool w8a8_quantises(int64_t M, int64_t K) { return M <= kQuantMaxM && K <= kQuantMaxK; }

hipError_t launch_w8a8_linear(const W8Params& p, bool xf16, hipStream_t st) {
  return xf16 ? launch_rows<true, true>(p, st) : launch_rows<true, false>(p, st);
}

hipError_t launch_w8a8(const W8Params& p, hipStream_t st) {
  if (p.M <= kRowsMaxM) return launch_rows<false, false>(p, st);
  // The tile with the least time by a simple model: waves of workgroups over the
  // compute units times the larger of a stage's MFMA and LDS-fill cycles.
  const int64_t cu = device_cu_count() > 0 ? device_cu_count() : 256;
  static constexpr int kTiles[][2] = {{256, 256}, {256, 192}, {256, 128}, {128, 256}, {128, 128}, {128, 64}, {64, 128}, {64, 64}};
  int best = 0;
  int64_t cost = INT64_MAX;
  for (int k = 0; k < 8; ++k) {
    const int tm = kTiles[k][0], tn = kTiles[k][1];
    const int64_t tiles = ((p.M + tm - 1) / tm) * ((p.N + tn - 1) / tn);
    const int64_t per = std::max(tm * tn / 64, tm + tn) + 64;   // a stage of 64 codes, and its barrier
    const int64_t c = (tiles + cu - 1) / cu * per;
    if (c < cost) { cost = c; best = k; }
  }
  switch (best) {
    case 0: return launch_tile<Tile<2, 4, 4, 2>>(p, st);
    case 1: return launch_tile<Tile<2, 3, 4, 2>>(p, st);
    case 2: return launch_tile<Tile<2, 2, 4, 2>>(p, st);
    case 3: return launch_tile<Tile<2, 2, 2, 4>>(p, st);
    case 4: return launch_tile<Tile<2, 2, 2, 2>>(p, st);
    case 5: return launch_tile<Tile<2, 1, 2, 2>>(p, st);
    case 6: return launch_tile<Tile<1, 2, 2, 2>>(p, st);
    default: return launch_tile<Tile<1, 1, 2, 2>>(p, st);
  }
}

}  // namespace cubic
