// moe_layer.hip -- the router (cubic_moe_topk) and the whole routed-expert
// layer for a few tokens (cubic_moe_layer) in two kernels.
//
//   ids, w  = the router of each token's logits (router.h)
//   [g | u] = x_t * GU_e^T;  h = bf16(SiLU(g) * u);  y_t = sum_j w_tj * (h_tj * D_e^T)
//
// The layer is bound by HBM as long as decoding a code costs little and codes are read once
// for all rows that share them. Both products run on the int8 MFMA, whose sums are exact: the
// activations are fixed-point numbers of 30 bits under a power of two for each block of 128
// or 256 (a macro step), in four planes of signed base-256 digits, which are four rows of
// one 16 x 16 x 64 tile; four tokens fill its rows. A bf16 number has eight significant bits,
// so a value is exact down to 2^-22 of its block's largest and below that off by at most 2^-30
// of it; blocks whose largest value is below 2^-90 are multiples of 2^-120. A step's sum is
// rounded to fp32 where it leaves the integers, and steps are added up in fp32. (Two e4m3
// halves on the scaled 16 x 16 x 128 MFMA are as many rows for eight tokens, and 2-bit codes
// e2m1 nibbles, but that MFMA aligns 128 products to the largest and drops what lies about
// 2^-14 below it: sums off by 2^-16, and by 2^-11 of the largest product where large products
// cancel. Against it the layer takes 2 % longer with one and with four tokens of 7168 / 3 K,
// 20 % with eight.)
// 2-bit codes {00, 01, 11} = {0, +1, -1}: a field in the top bits of a byte is the signed byte
// 64 code, so sixteen codes take three shifts and four masks. The field 10 counts as -2 there;
// where a wave sees one, a slow pass adds what its level lacks.
//
// Kernel 1 (k_layer_up): every workgroup runs the router of all tokens (one wave
// each), splits x into LDS, and then walks its share of the units (touched
// expert, 16 gate rows and the 16 up rows beside them); a unit's codes serve all tokens. Rows
// of x that do not fit in LDS are taken in several launches, whose sums go through the
// workspace. Kernel 2 (k_layer_down): every workgroup takes an equal share of the output rows
// and all pairs, one (pair, K part) per wave at a time, so the router-weighted sum never
// leaves the workgroup: no atomics, and the order of the sums does not depend on timing. Pairs
// of one expert read its codes again, one soon after the other (from L2), and decode them again.
//
// Measured (hidden 7168, intermediate 3 K, G512, on one card whose large copy runs at
// 5.1 TB/s): one token through 16 of 64 experts, 281 MB: kernel 1 43 us (8 us until the
// first load is issued: router, splitting, lists; then 5.7 TB/s), kernel 2 24 us, 67-70 us
// together; four tokens through about 52 of 128 experts, 930 MB: 109 + 74 us; 4 bits, G128,
// 2048 x 1024, two tokens of top-4 of 32: 13.5 + 8.8 us. Against
// loads in operand order, a barrier a round and seven steps in flight, the first version,
// kernel 1 took 62 us and kernel 2 26.
//
// 3- and 4-bit codes run on the same two kernels as sums of fixed functions of the code
// (CodesWide); wider codes, more tokens and shapes beyond the kernels' limits run as the router kernel
// followed by the routed MLP step (moe.hip).
#include <algorithm>

#include "gemv_core.h"
#include "launch.h"
#include "router.h"

namespace cubic {
namespace {

constexpr uint32_t kRsrc3 = 0x00020000u;       // raw buffer, 32-bit data format
constexpr int kLayerWaves = 16;                // one workgroup of 1024 threads per compute unit
constexpr int kLayerMaxT = 8;                  // two tiles of four tokens' planes
constexpr int kLayerMaxE = 1024;               // experts of one router wave (4 or 16 per lane)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t layer_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes),
                                           static_cast<int>(kRsrc3));
}

// Barrier of the workgroup's LDS traffic alone: the code loads in flight stay
// in flight (__syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---- activations in fixed point --------------------------------------------
// A block of activations (the codes of a macro step) shares an exponent: with ef the
// (clamped) exponent field of its largest magnitude, X = rint(v 2^(156 - ef)) lies in
// -2^30 .. 2^30 and is four signed bytes in base 256. The block's factor 2^(ef - 162) takes
// the 64 of a code's unit with it; it has to be a normal number, so blocks whose largest
// magnitude is below 2^-90 are multiples of 2^-120.
constexpr int kPlanes = 4;
__device__ __forceinline__ float fixed_factor(uint32_t ef) { return __uint_as_float((283u - ef) << 23); }
__device__ __forceinline__ float block_factor(uint32_t ef) { return __uint_as_float((ef - 35u) << 23); }

// X as four signed base-256 digits, the lowest in byte 0. (The limits are for values that are
// not finite, whose block's factor is NaN.)
__device__ __forceinline__ uint32_t digits(float v, float f) {
  const int x = __float2int_rn(__builtin_amdgcn_fmed3f(v * f, -0x1p30f, 0x1p30f));
  return (static_cast<uint32_t>(x) + 0x00808080u) ^ 0x00808080u;
}
// The largest of G (8 or 16) neighbouring lanes' values, in each of them.
template <int G>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = max(v, dpp_move<0xB1>(v));               // quad_perm [1, 0, 3, 2]
  v = max(v, dpp_move<0x4E>(v));               // quad_perm [2, 3, 0, 1]
  v = max(v, dpp_move<0x141>(v));              // row_half_mirror
  if constexpr (G == 16) v = max(v, dpp_move<0x140>(v));   // row_mirror
  return v;
}

// One operand: sixteen consecutive bf16 values (raw, two 16-byte pieces) of a block of
// 16 G values, whose operands lie in G neighbouring lanes. Returns the block's factor; plane
// r (weight 256^r) gets sixteen digits in the order in which the codes are decoded: dword q
// of 2-bit codes holds codes q, q + 4, q + 8, q + 12; of wider codes the even (q even) or odd
// ones of codes 8 (q / 2) .. + 7.
template <bool WIDE, int G>
__device__ __forceinline__ float split16(const u32x4& r0, const u32x4& r1, u32x4* plane) {
  float v[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = j < 4 ? r0[j & 3] : r1[j & 3];
    v[2 * j] = __uint_as_float(w << 16);
    v[2 * j + 1] = __uint_as_float(w & 0xffff0000u);
  }
  uint32_t top = 0u;                           // magnitudes order as their bits, what is not finite last
#pragma unroll
  for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  top = block_max<G>(top);
  const bool finite = top < 0x7f800000u;
  const uint32_t ef = finite ? max(top >> 23, 36u) : 36u;
  const float f = fixed_factor(ef);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = digits(v[WIDE ? 8 * (q >> 1) + (q & 1) + 2 * i : q + 4 * i], f);
    const uint32_t a = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), b = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u), e = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
    plane[0][q] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    plane[1][q] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    plane[2][q] = __builtin_amdgcn_perm(e, c, 0x05040100u);
    plane[3][q] = __builtin_amdgcn_perm(e, c, 0x07060302u);
  }
  return finite ? block_factor(ef) : __builtin_nanf("");
}

// Place of operand o (codes 16 o .. + 15 of a row) in a plane's bytes. Lane group kq of a
// macro step owns 32 SPL consecutive codes, 2 SPL operands; the MFMA of operand d takes the
// d-th of each group.
template <int SPL>
__device__ __forceinline__ int operand_place(int o) {
  constexpr int kOps = 2 * SPL;
  return 128 * SPL * (o / (4 * kOps)) + 64 * (o % kOps) + 16 * (o / kOps % 4);
}

// The four planes' sums of one token (rows 4 t .. 4 t + 3 of the MFMA are registers of one
// lane) as one number: both halves are exact integers, rounded to fp32 once each.
__device__ __forceinline__ float plane_sum(const i32x4& s) {
  return fmaf(static_cast<float>(s[3] * 256 + s[2]), 65536.0f, static_cast<float>(s[1] * 256 + s[0]));
}

// ---- the two kinds of codes ---------------------------------------------------
// Both multiply the activations' planes (rows 4 t .. + 3 of the MFMA for token t).
template <int SPL_>
struct Codes2 {
  static constexpr bool kWide = false;
  static constexpr int kBits = 2, SPL = SPL_;
  static constexpr int DW = 2 * SPL_;          // dwords of a lane's loads: one an operand
};
// 3- and 4-bit codes j = -M .. K (M = 2^(B-1), K = M - 1): with n = |j| and c = 1 - a - b
// their level s (a t + b t |t| + c t^3), t = j / K, is a sum of three fixed odd functions
//   p1 = j,  p2 = +-n (M - n),  p3 = +-n (M - n) (n - M / 2):
//   level = s ((a / K + M b / K^2 + M^2 c / K^3) p1 - (b / K^2 + 1.5 M c / K^3) p2 - c / K^3 p3)
// whose values are small integers, looked up four at a time by byte permutes in registers and
// summed exactly against the planes; the coefficients of a group enter with its scale. A table
// of a group's levels costs its building and an LDS read a code (2048 x 1024, W4 G128, two
// tokens: 17.5 + 11.2 us with tables).
// 4 bits: a code is -8 sign + l. 16 p1 is the nibble in a byte's upper half; the low bits l of
// j and of -j add up to 8, where l (8 - l) is even and p3 odd, so p3 needs only l, and p2 the
// sign, spread over its byte by a permute.
// 3 bits: three look-ups in eight entries.
template <int B>
struct CodesWide {
  static constexpr bool kWide = true;
  static constexpr int kBits = B, SPL = 1;
  static constexpr int DW = B;
  static constexpr int M = 1 << (B - 1), K = M - 1;
  static constexpr int kP1 = B == 4 ? 16 : 1;  // p1's factor
};

// Four bytes of f(j0) .. f(j0 + 3).
template <class Fn>
constexpr uint32_t i8_bytes(Fn f, int j0) {
  uint32_t v = 0;
  for (int i = 0; i < 4; ++i) v |= (static_cast<uint32_t>(f(j0 + i)) & 0xffu) << (8 * i);
  return v;
}
// Operand d (16 codes) of the lane's 32: b[0] = kP1 p1, b[1] = p2, b[2] = p3.
template <int B>
__device__ __forceinline__ void poly_decode(const uint32_t* w, int d, i32x4* b) {
  if constexpr (B == 4) {
    constexpr auto p2 = [](int l) { return l * (8 - l); };
    constexpr auto m2 = [](int l) { return -l * (8 - l); };
    constexpr auto p3 = [](int l) { return l * (8 - l) * (l - 4); };
    constexpr uint32_t a0 = i8_bytes(p2, 0), a4 = i8_bytes(p2, 4), n0 = i8_bytes(m2, 0), n4 = i8_bytes(m2, 4);
    constexpr uint32_t c0 = i8_bytes(p3, 0), c4 = i8_bytes(p3, 4);
#pragma unroll
    for (int u = 0; u < 2; ++u) {              // eight codes: the even ones, then the odd ones
      const uint32_t v = w[2 * d + u], vl = v << 4;
      const uint32_t le = v & 0x07070707u, lo = (v >> 4) & 0x07070707u;
      // the sign bits of four bytes as byte masks (selectors 8 .. 11: bytes 1, 3 of either source)
      const uint32_t se = __builtin_amdgcn_perm(vl, vl << 8, 0x0b090a08u);
      const uint32_t so = __builtin_amdgcn_perm(v, v << 8, 0x0b090a08u);
      b[0][2 * u] = static_cast<int>(vl & 0xF0F0F0F0u);
      b[0][2 * u + 1] = static_cast<int>(v & 0xF0F0F0F0u);
      b[1][2 * u] = static_cast<int>((__builtin_amdgcn_perm(n4, n0, le) & se) | (__builtin_amdgcn_perm(a4, a0, le) & ~se));
      b[1][2 * u + 1] = static_cast<int>((__builtin_amdgcn_perm(n4, n0, lo) & so) | (__builtin_amdgcn_perm(a4, a0, lo) & ~so));
      b[2][2 * u] = static_cast<int>(__builtin_amdgcn_perm(c4, c0, le));
      b[2][2 * u + 1] = static_cast<int>(__builtin_amdgcn_perm(c4, c0, lo));
    }
  } else {
    // codes 0 .. 3 are their values, 4 .. 7 those less 8
    constexpr auto sign = [](int j) { return j < 0 ? -1 : 1; };
    constexpr auto p1 = [](int j) { return j; };
    constexpr auto p2 = [sign](int j) { return j * (4 - sign(j) * j); };
    constexpr auto p3 = [sign](int j) { return j * (4 - sign(j) * j) * (sign(j) * j - 2); };
    constexpr uint32_t t[3][2] = {{i8_bytes(p1, 0), i8_bytes(p1, -4)},
                                  {i8_bytes(p2, 0), i8_bytes(p2, -4)},
                                  {i8_bytes(p3, 0), i8_bytes(p3, -4)}};
#pragma unroll
    for (int u = 0; u < 2; ++u) {              // 24 bits: eight codes
      const int g = 2 * d + u;
      const uint32_t v = g == 0 ? w[0] : g == 1 ? __builtin_amdgcn_alignbit(w[1], w[0], 24)
                                     : g == 2 ? __builtin_amdgcn_alignbit(w[2], w[1], 16) : w[2] >> 8;
      // fields of three bits at 0, 3, 6, 9 and 16, 19, 22, 25; then those of even and odd codes in bytes
      const uint32_t y = (v & 0xFFFu) | ((v & 0xFFF000u) << 4);
      const uint32_t se = (y & 0x00070007u) | ((y & 0x01C001C0u) << 2);
      const uint32_t so = ((y >> 3) & 0x00070007u) | ((y & 0x0E000E00u) >> 1);
#pragma unroll
      for (int f = 0; f < 3; ++f) {
        b[f][2 * u] = static_cast<int>(__builtin_amdgcn_perm(t[f][1], t[f][0], se));
        b[f][2 * u + 1] = static_cast<int>(__builtin_amdgcn_perm(t[f][1], t[f][0], so));
      }
    }
  }
}

// ---- a wave's stream of code tiles ------------------------------------------
// NT tiles of 16 weight rows, macro steps of SPL * 128 codes, in blocks of PM
// steps that are in flight together. The MFMA wants row nl and K quarter kq in lane
// 16 kq + nl, but the address unit takes four neighbouring lanes at a time: loads in
// that order touch four rows a quad, and a load instruction takes four times as
// long. So lane l loads quarter l % 4 of row l / 4 (64 contiguous bytes a quad, the
// group scales of four steps likewise), and the lanes exchange the words through
// the LDS crossbar when they are used (ds_bpermute, no LDS memory).
struct CodeSrc {                               // a unit's code and scale buffers (wave-uniform)
  __amdgpu_buffer_rsrc_t code, scale, shape;   // (shape: of wide codes only)
};

struct Groups {                                // steps per group: as a shift, or (shift < 0) by a reciprocal
  int shift;
  uint32_t mul;
  __device__ __forceinline__ int of(int t) const {   // t < 2^16
    return shift >= 0 ? t >> shift : static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(t)) * mul) >> 32);
  }
};

template <class F, int PM, int NT>
struct CodeStream {
  static constexpr int DW = F::DW;             // code dwords per lane, tile and step
  static constexpr int SR = (PM + 3) / 4;      // scale registers per tile and block (four steps each)
  uint32_t cb[PM][NT][DW];
  float sc[NT][SR], scn[NT][SR];               // of the current block, and of the next
  uint32_t ab[NT][F::kWide ? SR : 1], abn[NT][F::kWide ? SR : 1];   // shape parameters likewise (wide codes)

  // step t into slot U; vcode: the lane's byte offset per tile
  template <int U>
  __device__ __forceinline__ void issue(const CodeSrc& src, const uint32_t* vcode, int t) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if constexpr (DW == 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(src.code, vcode[i], t * (4 * DW * 4), 0);
        cb[U][i][0] = v.x; cb[U][i][1] = v.y; cb[U][i][2] = v.z; cb[U][i][3] = v.w;
      } else if constexpr (DW == 3) {
        typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
        const u32x3 v = __builtin_amdgcn_raw_buffer_load_b96(src.code, vcode[i], t * (4 * DW * 4), 0);
        cb[U][i][0] = v.x; cb[U][i][1] = v.y; cb[U][i][2] = v.z;
      } else {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(src.code, vcode[i], t * (4 * DW * 4), 0);
        cb[U][i][0] = v.x; cb[U][i][1] = v.y;
      }
    }
  }
  // the group scales of a block into scn: lane l takes row l / 4 at the block's
  // steps 4 r + l % 4; step(i) is the i-th step of the block
  template <class Step>
  __device__ __forceinline__ void issue_scales(const CodeSrc& src, const uint32_t* vscale, const Groups& gr, int lane,
                                               Step step) {
#pragma unroll
    for (int r = 0; r < SR; ++r) {
      const uint32_t g = 4u * static_cast<uint32_t>(gr.of(step(4 * r + (lane & 3))));
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        scn[i][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(src.scale, vscale[i] + g, 0, 0));
        if constexpr (F::kWide) abn[i][r] = __builtin_amdgcn_raw_buffer_load_b32(src.shape, vscale[i] + g, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void take_scales() {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < SR; ++r) {
        sc[i][r] = scn[i][r];
        if constexpr (F::kWide) ab[i][r] = abn[i][r];
      }
  }
  // slot U in operand order: w[tile][dword], s[tile] and (wide codes) a | b in sh[tile]
  template <int U>
  __device__ __forceinline__ void take(int nl, int kq, uint32_t (*w)[DW], float* s, uint32_t* sh) {
    auto from = [](int lane, uint32_t v) {
      return static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(4 * lane, static_cast<int>(v)));
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int d = 0; d < DW; ++d) w[i][d] = from(4 * nl + kq, cb[U][i][d]);
      s[i] = __uint_as_float(from(4 * nl + (U & 3), __float_as_uint(sc[i][U / 4])));
      if constexpr (F::kWide) sh[i] = from(4 * nl + (U & 3), ab[i][U / 4]);
    }
  }
};

// The activations of a lane: its row (a token's plane) and its token's block factors in
// LDS, per tile of sixteen rows (four tokens).
template <int MT>
struct Acts {
  const uint8_t* row[MT];
  const float* factor[MT];
};

// One macro step of 2-bit codes: the step's sums, times block factor and group scale, go to
// acc[tile][tokens' tile]. A field in a byte's top bits is the signed byte 64 code.
// MODE 0: the field 10 counts as -2 and is collected in bad. MODE 1: the field 10 alone, as +1
// (the slow pass).
template <int SPL, int NT, int MT, int MODE>
__device__ __forceinline__ void layer_step(const uint32_t (*w)[2 * SPL], const float* sc, const Acts<MT>& x, int t, int kq,
                                           float (*acc)[MT], uint32_t& bad) {
  i32x4 part[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[i][m] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int d = 0; d < 2 * SPL; ++d) {
    i32x4 a[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) a[m] = *reinterpret_cast<const i32x4*>(x.row[m] + t * (128 * SPL) + 64 * d + 16 * kq);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t v = w[i][d];
      i32x4 b;
      if constexpr (MODE == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = static_cast<int>((v << (6 - 2 * q)) & 0xC0C0C0C0u);
        bad |= v & ~(v << 1);
      } else {
        const uint32_t f = (v & ~(v << 1) & 0xAAAAAAAAu) >> 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = static_cast<int>((f << (6 - 2 * q)) & 0x40404040u);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) part[i][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[m], b, part[i][m], 0, 0, 0);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const float f = x.factor[m][t];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][m] = fmaf(f, sc[i] * plane_sum(part[i][m]), acc[i][m]);
  }
}

// The same for wide codes, sh: the tiles' shapes a | b.
template <int B, int NT, int MT>
__device__ __forceinline__ void wide_step(const uint32_t (*w)[B], const float* sc, const uint32_t* sh, const Acts<MT>& x,
                                          int t, int kq, float (*acc)[MT]) {
  constexpr float K = CodesWide<B>::K, M = CodesWide<B>::M;
  i32x4 a[2][MT];
#pragma unroll
  for (int d = 0; d < 2; ++d)
#pragma unroll
    for (int m = 0; m < MT; ++m) a[d][m] = *reinterpret_cast<const i32x4*>(x.row[m] + t * 128 + 64 * d + 16 * kq);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    i32x4 part[3][MT];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      i32x4 b[3];
      poly_decode<B>(w[i], d, b);
#pragma unroll
      for (int f = 0; f < 3; ++f)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          constexpr i32x4 zero = {0, 0, 0, 0};
          part[f][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[d][m], b[f], d ? part[f][m] : zero, 0, 0, 0);
        }
    }
    // (64: a code's unit in the block factor)
    const float sa = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(sh[i] & 0xffffu)));
    const float sb = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(sh[i] >> 16)));
    const float c = (1.0f - sa - sb) * (64.0f / (K * K * K));
    constexpr float p1 = 1.0f / CodesWide<B>::kP1;
    const float k1 = sc[i] * fmaf(M * M * p1, c, fmaf(sb, 64.0f * M * p1 / (K * K), sa * (64.0f * p1 / K)));
    const float k2 = sc[i] * -fmaf(1.5f * M, c, sb * (64.0f / (K * K)));
    const float k3 = sc[i] * -c;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float v = fmaf(k3, plane_sum(part[2][m]), fmaf(k2, plane_sum(part[1][m]), k1 * plane_sum(part[0][m])));
      acc[i][m] = fmaf(x.factor[m][t], v, acc[i][m]);
    }
  }
}

// The slow pass: the level of the field 10 (code -2) is -q(2) s, q(2) = 2 a + 4 b +
// 8 (1 - a - b), of which the sums above hold -2 s; the rest is added step by step. Loads in
// operand order: vcode, vscale as in the stream, but of row nl and quarter kq.
template <int SPL, int NT, int MT>
__device__ __forceinline__ void layer_extra(const CodeSrc& src, const __amdgpu_buffer_rsrc_t& shp,
                                            const uint32_t* vcode, const uint32_t* vscale, int tb, int te, int by,
                                            const Groups& gr, const Acts<MT>& x, int t0, int kq, float (*acc)[MT]) {
#pragma unroll 1
  for (int t = tb; t < te; t += by) {
    CodeStream<Codes2<SPL>, 1, NT> st;
    st.template issue<0>(src, vcode, t);
    const int g = gr.of(t);
    float lev[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float s = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(src.scale, vscale[i], g * 4, 0));
      const uint32_t ab = __builtin_amdgcn_raw_buffer_load_b32(shp, vscale[i], g * 4, 0);
      const double a = f16_bits_to_f64(static_cast<uint16_t>(ab & 0xffffu));
      const double b = f16_bits_to_f64(static_cast<uint16_t>(ab >> 16));
      lev[i] = static_cast<float>(-static_cast<double>(s) * (level_numerator(a, b, 2, 1) - 2.0));
    }
    uint32_t none = 0u;
    layer_step<SPL, NT, MT, 1>(st.cb[0], lev, x, t - t0, kq, acc, none);
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// cubic_moe_topk: one wave per token.
// ---------------------------------------------------------------------------
template <int EPL>
__global__ __launch_bounds__(256) void k_moe_topk(RouterParams p, int64_t T, int32_t* __restrict__ ids,
                                                  float* __restrict__ weights) {
  __shared__ uint32_t cand[4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (t >= T) return;                          // no barrier in this kernel
  wave_topk<EPL>(p, t, lane, cand[wave], [&](int slot, int id, float w) {
    ids[t * p.topk + slot] = id;
    weights[t * p.topk + slot] = w;
  });
}

static RouterParams router_params(const MoeRouter& r) {
  return RouterParams{r.logits, r.bias, r.dtype, r.E, r.topk, r.sigmoid, r.renorm, r.scale};
}

hipError_t launch_moe_topk(const MoeRouter& r, int64_t T, int32_t* ids, float* weights, hipStream_t st) {
  const RouterParams p = router_params(r);
  const dim3 grid(static_cast<unsigned>((T + 3) / 4)), block(256);
  if (p.E <= 256) {
    hipLaunchKernelGGL(k_moe_topk<4>, grid, block, 0, st, p, T, ids, weights);
  } else if (p.E <= 1024) {
    hipLaunchKernelGGL(k_moe_topk<16>, grid, block, 0, st, p, T, ids, weights);
  } else {
    hipLaunchKernelGGL(k_moe_topk<32>, grid, block, 0, st, p, T, ids, weights);
  }
  return hipGetLastError();
}

namespace {

// Routing record that kernel 1 leaves for kernel 2: rec[0] = pairs with an
// expert, then (pair, expert) of each, grouped by expert.
struct LayerUpParams {
  RouterParams r;
  const uint16_t* x;       // bf16 [T][H]
  int T;
  int H, I;
  const uint8_t* codes;    // gate_up, expert 0
  const float* scales;
  const uint16_t* shapes;
  int64_t code_bytes;
  int gpr;                 // groups per row
  Groups groups;           // steps per group
  float share;             // 1 / (workgroups * waves)
  int batch;               // rounds between the joins of the waves' sums
  int k0, steps;           // macro steps of this launch: k0 .. k0 + steps - 1
  int add, last;           // the sums start from `partial`; they are whole (else they go there)
  float* partial;          // [T*topk][2I]
  float* weights;          // [T][topk] out, for kernel 2
  int32_t* ids_user;       // [T][topk] out for the caller, or NULL
  float* weights_user;
  int32_t* rec;
  uint16_t* h;             // bf16 [T*topk][I]
};

// K parts of kernel 1: the waves of a tile, so many that the slowest workgroup has the
// least to do (units: touched experts' tiles; kRoundCost: eighths of a step that a round
// costs beside its steps). At least two teams: h leaves in pieces of two tiles. The
// number of touched experts is known on the device alone: taken for the largest possible
// one (64 for 8 tokens of top-8, where 41 are usual), the last of two rounds was a third
// full, and 4 bits, 7168 x 2 K took 250 us.
constexpr int kRoundCost = 4;
__host__ __device__ inline int layer_up_max_parts(int nmacro) { return nmacro >= 8 ? 8 : nmacro >= 4 ? 4 : nmacro >= 2 ? 2 : 1; }
// share: 1 / (workgroups * waves). (Every workgroup computes the same; integer divisions
// take 0.5 us.)
__device__ __forceinline__ int layer_up_parts(int units, int nmacro, float share) {
  int best = 1;
  float cost = __builtin_inff();
  const int most = layer_up_max_parts(nmacro);
  const float whole = static_cast<float>(units) * share;
#pragma unroll
  for (int sh = 0; sh <= 3; ++sh) {
    const int ks = 1 << sh;
    const float rounds = ceilf(whole * static_cast<float>(ks) - 1e-3f);
    const float c = rounds * static_cast<float>(((nmacro + ks - 1) >> sh) * 8 + kRoundCost);
    if (ks <= most && c < cost) { cost = c; best = ks; }
  }
  return best;
}

struct LayerUpLds {
  int xq, xf, red, first, id, w, exp, slot, cand, misc, total;   // byte offsets
  int xq_stride, xf_stride;
};
// K: the activations of a token that a launch takes.
__host__ __device__ inline LayerUpLds layer_up_lds(int T, int topk, int K, int batch) {
  LayerUpLds L;
  const int P = T * topk;
  auto up16 = [](int v) { return (v + 15) & ~15; };
  // Rows of the MFMA: four planes a token; 16 bytes of padding each: the rows' reads hit
  // other banks. Block factors: at most one per 128 values.
  L.xq_stride = K + 16;
  L.xf_stride = K / 128;
  int o = 0;
  L.xq = o;    o += kPlanes * T * L.xq_stride;
  L.xf = o;    o += up16(T * L.xf_stride * 4);
  // partial sums, two batches of rounds: [2][batch][waves][2 tiles][T][16]; the
  // first-pair table of the experts uses the same bytes before the first round
  const int red = 2 * batch * kLayerWaves * 2 * T * 16 * 4;
  L.red = o;   o += red > kLayerMaxE * 4 ? red : kLayerMaxE * 4;
  L.first = L.red;
  L.id = o;    o += up16(P * 4);
  L.w = o;     o += up16(P * 4);
  L.exp = o;   o += up16(P * 4);
  L.slot = o;  o += up16(P * 8);
  L.cand = o;  o += kLayerMaxT * 64 * 4;
  L.misc = o;  o += 64;
  L.total = o;
  return L;
}

template <class F, int PM, int EPL, int MT>
__global__ __launch_bounds__(1024) void k_layer_up(LayerUpParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int SPL = F::SPL;
  using Stream = CodeStream<F, PM, 2>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const int T = p.T, topk = p.r.topk, P = T * topk;
  const int K = p.steps * SPL * 128;
  const LayerUpLds L = layer_up_lds(T, topk, K, p.batch);
  int32_t* s_first = reinterpret_cast<int32_t*>(smem + L.first);
  int32_t* s_id = reinterpret_cast<int32_t*>(smem + L.id);
  float* s_w = reinterpret_cast<float*>(smem + L.w);
  int32_t* s_exp = reinterpret_cast<int32_t*>(smem + L.exp);
  uint8_t* s_slot = smem + L.slot;             // [touched][8]: the token's slot, 0xff: not routed here
  int32_t* s_misc = reinterpret_cast<int32_t*>(smem + L.misc);

  // ---- the tokens' routers (one wave each), and x split into its halves ----
  if (wave < T) {
    // everything after waits for these waves
    __builtin_amdgcn_s_setprio(3);
    wave_topk<EPL>(p.r, wave, lane, reinterpret_cast<uint32_t*>(smem + L.cand) + 64 * wave,
                               [&](int slot, int id, float w) {
                                 s_id[wave * topk + slot] = id;
                                 s_w[wave * topk + slot] = w;
                               });
    __builtin_amdgcn_s_setprio(0);
  }
  for (int e = tid; e < p.r.E; e += 1024) s_first[e] = INT32_MAX;
  for (int i = tid; i < 2 * P; i += 1024) reinterpret_cast<uint32_t*>(s_slot)[i] = 0xffffffffu;
  {
    // one operand of sixteen values a thread; the operands of a block lie in neighbouring lanes
    constexpr int G = 8 * SPL;
    const int per_row = K / 16, all = T * per_row;
    for (int v0 = 0; v0 < all; v0 += 1024) {
      const int v = v0 + tid;
      const bool on = v < all;                 // whole blocks: all is a multiple of G
      const int t = on ? v / per_row : 0;
      const int o = on ? v - t * per_row : 0;
      const u32x4* src = reinterpret_cast<const u32x4*>(p.x + static_cast<int64_t>(t) * p.H + p.k0 * (SPL * 128) + 16 * o);
      u32x4 plane[kPlanes];
      const float f = split16<F::kWide, G>(src[0], src[1], plane);
      if (on) {
        unsigned char* dst = smem + L.xq + kPlanes * t * L.xq_stride + operand_place<SPL>(o);
#pragma unroll
        for (int r = 0; r < kPlanes; ++r) *reinterpret_cast<u32x4*>(dst + r * L.xq_stride) = plane[r];
        if (o % G == 0) reinterpret_cast<float*>(smem + L.xf)[t * L.xf_stride + o / G] = f;
      }
    }
  }
  __syncthreads();
  // ---- touched experts in the order of their first pair ----
  const int pe = tid < P ? s_id[tid] : -1;
  if (pe >= 0) atomicMin(&s_first[pe], tid);
  __syncthreads();
  const bool lead = pe >= 0 && s_first[pe] == tid;
  const uint64_t leads = __ballot(lead), routed = __ballot(pe >= 0);
  if (lane == 0 && wave < 8) {                 // P <= 512 threads
    s_misc[wave] = __popcll(leads);
    s_misc[8 + wave] = __popcll(routed);
  }
  __syncthreads();
  int n = 0, before = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = s_misc[k];
    before += k < wave ? c : 0;
    n += c;
  }
  n = __builtin_amdgcn_readfirstlane(n);
  if (lead) {
    const int a = before + __popcll(leads & ((uint64_t{1} << lane) - 1u));
    s_exp[a] = pe;
    s_first[pe] = -1 - a;                      // from here on the expert's place
  }
  __syncthreads();
  const int pa = pe >= 0 ? -1 - s_first[pe] : 0;
  const int pt = tid / topk;                   // the pair's token
  if (pe >= 0) s_slot[8 * pa + pt] = static_cast<uint8_t>(tid - pt * topk);
  __syncthreads();
  if (blockIdx.x == 0) {
    // for kernel 2 and the caller: weights, ids and the pairs grouped by expert
    if (tid < P) {
      const float w = s_w[tid];
      p.weights[tid] = w;
      if (p.ids_user) p.ids_user[tid] = pe;
      if (p.weights_user) p.weights_user[tid] = w;
    }
    if (pe >= 0) {
      // slots are below 64: the top bit of a byte is set where no token is
      int pos = 0;
      for (int a = 0; a < pa; ++a)
        pos += 8 - __popcll(*reinterpret_cast<const uint64_t*>(s_slot + 8 * a) & 0x8080808080808080ull);
      const uint64_t own = *reinterpret_cast<const uint64_t*>(s_slot + 8 * pa);
      pos += pt - __popcll(own & 0x8080808080808080ull & ((uint64_t{1} << (8 * pt)) - 1u));
      p.rec[2 + 2 * pos] = tid;
      p.rec[3 + 2 * pos] = pe;
    }
    if (tid == 0) {
      int all = 0;
      for (int k = 0; k < 8; ++k) all += s_misc[8 + k];
      p.rec[0] = all;
    }
  }

  // ---- units: round r, workgroup b, team m -> (r grid + b) teams + m ----
  const int tiles = p.I / 16;
  const int total = n * tiles;
  const int nmacro = p.steps, k0 = p.k0;
  const int ks = __builtin_amdgcn_readfirstlane(layer_up_parts(total, nmacro, p.share));
  const int teams = kLayerWaves / ks;
  const int team = wave / ks, part = wave - team * ks;
  // this wave's steps: part, part + ks, ... (the team's waves read neighbouring
  // pieces of a row at any time)
  const int steps = (nmacro - part + ks - 1) / ks;
  const uint32_t row_bytes = static_cast<uint32_t>(p.H * F::kBits / 8);
  // a gate row of the tile, and the up row I rows below it
  auto lane_offsets = [&](int row, int quarter, uint32_t* vc, uint32_t* vs) {
    vc[0] = row * row_bytes + quarter * (4 * F::DW);
    vc[1] = vc[0] + static_cast<uint32_t>(p.I) * row_bytes;
    vs[0] = static_cast<uint32_t>(row * p.gpr * 4);
    vs[1] = vs[0] + static_cast<uint32_t>(p.I * p.gpr * 4);
  };
  uint32_t vcode[2], vscale[2];
  lane_offsets(lane >> 2, lane & 3, vcode, vscale);
  Acts<MT> acts;
#pragma unroll
  for (int m = 0; m < MT; ++m) {               // rows past the tokens are not used
    const int t = 4 * m + (nl >> 2), u = 4 * m + kq;
    acts.row[m] = smem + L.xq + (t < T ? 4 * t + (nl & 3) : 0) * L.xq_stride;
    acts.factor[m] = reinterpret_cast<const float*>(smem + L.xf) + (u < T ? u : 0) * L.xf_stride;
  }

  auto unit_row = [&](int u, int64_t& e, int& j) {
    const int uu = u < total ? u : 0;
    const int a = uu / tiles;
    j = uu - a * tiles;
    e = __builtin_amdgcn_readfirstlane(s_exp[a]);
  };
  auto source = [&](int u) {
    CodeSrc s;
    int64_t e;
    int j;
    unit_row(u, e, j);
    const uint32_t rows = u < total ? static_cast<uint32_t>(p.I + 16) : 0u;   // no unit: every load is out of range
    s.code = layer_rsrc(p.codes + e * p.code_bytes + static_cast<int64_t>(16 * j) * row_bytes, rows * row_bytes);
    s.scale = layer_rsrc(p.scales + (e * 2 * p.I + 16 * j) * p.gpr, rows * 4u * static_cast<uint32_t>(p.gpr));
    s.shape = layer_rsrc(p.shapes + 2 * (e * 2 * p.I + 16 * j) * p.gpr, rows * 4u * static_cast<uint32_t>(p.gpr));
    return s;
  };
  if (n == 0) return;                          // no expert taken at all (block-uniform)
  const int stride = static_cast<int>(gridDim.x) * teams;
  int u = static_cast<int>(blockIdx.x) * teams + team;
  const int rounds = (total - static_cast<int>(blockIdx.x) * teams + stride - 1) / stride;   // block-uniform
  if (rounds <= 0) return;

  Stream st;
  CodeSrc cur = source(u);
  st.issue_scales(cur, vscale, p.groups, lane, [&](int i) { return k0 + part + min(i, steps - 1) * ks; });
  [&]<int... U>(std::integer_sequence<int, U...>) {
    (st.template issue<U>(cur, vcode, k0 + part + min(U, steps - 1) * ks), ...);
  }(std::make_integer_sequence<int, PM>{});

  float* red = reinterpret_cast<float*>(smem + L.red);
  const int red_wave = 2 * T * 16, red_round = kLayerWaves * red_wave;
  int slot_r = 0, half = 0, r0 = 0;            // round of the batch, its buffer, its first round
  for (int r = 0; r < rounds; ++r) {
    const CodeSrc nxt = source(u + stride);
    float acc[2][MT] = {};
    uint32_t bad = 0u;
    for (int t0 = 0; t0 < steps; t0 += PM) {
      // the next block: this unit's next PM steps, or the next unit's first
      st.take_scales();
      const bool more = t0 + PM < steps;
      CodeSrc src;
      src.code = more ? cur.code : nxt.code;
      src.scale = more ? cur.scale : nxt.scale;
      if constexpr (F::kWide) src.shape = more ? cur.shape : nxt.shape;
      const int tn = more ? t0 + PM : 0;
      st.issue_scales(src, vscale, p.groups, lane, [&](int i) { return k0 + part + min(tn + i, steps - 1) * ks; });
      [&]<int... U>(std::integer_sequence<int, U...>) {
        (([&] {
           if (t0 + U < steps) {
             uint32_t w[2][F::DW];
             float s[2];
#pragma unroll
             for (int i = 0; i < 2; ++i)
#pragma unroll
               for (int d = 0; d < Stream::DW; ++d) asm volatile("" : "+v"(st.cb[U][i][d]));
             uint32_t sh[2];
             st.template take<U>(nl, kq, w, s, sh);
             const int t = part + (t0 + U) * ks;
             if constexpr (F::kWide) {
               wide_step<F::kBits, 2, MT>(w, s, sh, acts, t, kq, acc);
             } else {
               layer_step<SPL, 2, MT, 0>(w, s, acts, t, kq, acc, bad);
             }
           }
           st.template issue<U>(src, vcode, k0 + part + min(tn + U, steps - 1) * ks);
           __builtin_amdgcn_sched_barrier(0);
         }()),
         ...);
      }(std::make_integer_sequence<int, PM>{});
    }
    if constexpr (!F::kWide) {
      if (u < total && __any((bad & 0xAAAAAAAAu) != 0u)) {
        int64_t e;
        int j;
        unit_row(u, e, j);
        const __amdgpu_buffer_rsrc_t shp = layer_rsrc(p.shapes + 2 * (e * 2 * p.I + 16 * j) * p.gpr,
                                                      static_cast<uint32_t>(p.I + 16) * 4u * static_cast<uint32_t>(p.gpr));
        uint32_t vc[2], vs[2];
        lane_offsets(nl, kq, vc, vs);
        layer_extra<SPL, 2, MT>(cur, shp, vc, vs, k0 + part, k0 + nmacro, ks, p.groups, acts, k0, kq, acc);
      }
    }
    // partial sums of the team's waves meet in LDS; lane group kq holds tokens kq and 4 + kq
    float* rb = red + (half * p.batch + slot_r) * red_round;
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (4 * m + kq < T)
#pragma unroll
        for (int i = 0; i < 2; ++i) rb[wave * red_wave + (i * T + 4 * m + kq) * 16 + nl] = acc[i][m];
    cur = nxt;
    u += stride;
    ++slot_r;
    if (slot_r < p.batch && r + 1 < rounds) continue;
    // A join of the waves every `batch` rounds: in between they run apart, so that a
    // wave whose loads come late holds nobody up. Two batches of sums: one barrier.
    lds_barrier();
    // h of two neighbouring tiles: 32 values per half wave
    const int pairs = teams / 2;
    const int nsub = slot_r * pairs * T;
    const float* hb = red + half * p.batch * red_round;
    for (int s0 = 0; s0 < nsub; s0 += 32) {
      const int sub = s0 + (tid >> 5);
      const int c = tid & 31;
      const int t = sub % T, rp = sub / T;
      const int rr = rp / pairs, pr = rp - rr * pairs;
      const int u0 = ((r0 + rr) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x)) * teams + 2 * pr;
      const bool in = sub < nsub && u0 < total;
      const int a = in ? u0 / tiles : 0;
      const int j = in ? u0 - a * tiles : 0;
      const int slot = in ? s_slot[8 * a + t] : 0xff;
      float g = 0.0f, uu = 0.0f;
      if (in) {
        const float* src = hb + rr * red_round + (2 * pr + (c >> 4)) * ks * red_wave + t * 16 + (c & 15);
        for (int k = 0; k < ks; ++k) {
          g += src[k * red_wave];
          uu += src[k * red_wave + T * 16];
        }
      }
      if (slot == 0xff) continue;
      const int64_t pair = t * topk + slot;
      float* sums = p.partial + pair * 2 * p.I + 16 * j + c;
      if (p.add) {
        g += sums[0];
        uu += sums[p.I];
      }
      if (p.last) {
        const float v = g / (1.0f + expf(-g)) * uu;
        // rounded to bf16, as the down product's activations are (NaN stays NaN)
        p.h[pair * p.I + 16 * j + c] = v != v ? uint16_t{0x7fc0u} : static_cast<uint16_t>(bf16_rne_bits(v));
      } else {
        sums[0] = g;
        sums[p.I] = uu;
      }
    }
    half ^= 1;
    slot_r = 0;
    r0 = r + 1;
  }
}

struct LayerDownParams {
  const int32_t* rec;
  const float* weights;    // [T][topk]
  int T, topk;
  const uint16_t* h;       // bf16 [pair][I]
  const uint8_t* codes;    // down, expert 0
  const float* scales;
  const uint16_t* shapes;
  int64_t code_bytes;
  int gpr;
  Groups groups;
  int H, I;
  int rows, rt;            // output rows per workgroup, and per tile
  int ks;                  // K parts per pair
  void* y;                 // [T][H]
  int ybf16;
};

struct LayerDownLds {
  int wave_bytes, hstride, factor, sum, total;
};
__host__ __device__ inline LayerDownLds layer_down_lds(int T, int I, int spl, int ks) {
  LayerDownLds L;
  const int nmacro = I / (spl * 128);
  const int steps = (nmacro + ks - 1) / ks;    // of a part
  L.hstride = steps * spl * 128 + 16;
  L.factor = kPlanes * L.hstride;
  L.wave_bytes = L.factor + ((steps * 4 + 15) & ~15);
  L.sum = kLayerWaves * L.wave_bytes;
  L.total = L.sum + kLayerWaves * T * 32 * 4;
  return L;
}

// One (pair, K part): the pair, its steps [tb, te), its expert; live 0: none.
struct DownItem {
  int pair, tb, te;
  int64_t e;
  uint32_t live;
};

// An item's h on its way into the planes of the wave's LDS, one operand a lane: it waits in
// registers, so that it is loaded before the codes of its item. (Split here and not by kernel
// 1: a block's values come from several of its workgroups.)
template <class F>
struct DownActs {
  static constexpr int G = 8 * F::SPL;
  u32x4 v[2];
  __device__ __forceinline__ void load(const LayerDownParams& p, const DownItem& q, int lane) {
    const int o = min(lane, (q.te - q.tb) * G - 1);
    const u32x4* src = reinterpret_cast<const u32x4*>(p.h + static_cast<int64_t>(q.pair) * p.I + q.tb * (16 * G) + 16 * o);
    v[0] = src[0];
    v[1] = src[1];
  }
  __device__ __forceinline__ void store(const DownItem& q, uint8_t* hreg, const LayerDownLds& L, int lane) const {
    u32x4 plane[kPlanes];
    const float f = split16<F::kWide, G>(v[0], v[1], plane);
    if (lane < (q.te - q.tb) * G) {            // whole blocks
      uint8_t* dst = hreg + operand_place<F::SPL>(lane);
#pragma unroll
      for (int r = 0; r < kPlanes; ++r) *reinterpret_cast<u32x4*>(dst + r * L.hstride) = plane[r];
      if (lane % G == 0) reinterpret_cast<float*>(hreg + L.factor)[lane / G] = f;
    }
  }
};

template <class F, int PM, int NT>
__global__ __launch_bounds__(1024) void k_layer_down(LayerDownParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int SPL = F::SPL;
  using Stream = CodeStream<F, PM, NT>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const LayerDownLds L = layer_down_lds(p.T, p.I, SPL, p.ks);
  uint8_t* hreg = smem + wave * L.wave_bytes;
  float* sums = reinterpret_cast<float*>(smem + L.sum) + wave * p.T * 32;
  for (int i = lane; i < p.T * 32; i += 64) sums[i] = 0.0f;
  wave_lds_order();
  const int n0 = static_cast<int>(blockIdx.x) * p.rows;
  const int rows = min(p.rows, p.H - n0);
  const int items = p.rec[0] * p.ks;
  const int nmacro = p.I / (SPL * 128);
  const uint32_t row_bytes = static_cast<uint32_t>(p.I * F::kBits / 8);
  // a row of each tile (past the workgroup's rows: its last one, whose sums are not used)
  auto lane_offsets = [&](int row, int quarter, uint32_t* vc, uint32_t* vs) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = min(i * p.rt + min(row, p.rt - 1), rows - 1);
      vc[i] = r * row_bytes + quarter * (4 * F::DW);
      vs[i] = static_cast<uint32_t>(r * p.gpr * 4);
    }
  };
  uint32_t vcode[NT], vscale[NT];
  lane_offsets(lane >> 2, lane & 3, vcode, vscale);
  using Item = DownItem;
  auto item_of = [&](int it) {
    Item q;
    q.live = it < items ? 1u : 0u;
    const int ii = it < items ? it : 0;
    const int job = ii / p.ks, part = ii - job * p.ks;
    q.pair = __builtin_amdgcn_readfirstlane(p.rec[2 + 2 * job]);
    q.e = __builtin_amdgcn_readfirstlane(p.rec[3 + 2 * job]);
    q.tb = part * nmacro / p.ks;
    q.te = (part + 1) * nmacro / p.ks;
    return q;
  };
  auto source = [&](const Item& q) {
    CodeSrc s;
    s.code = layer_rsrc(p.codes + q.e * p.code_bytes + static_cast<int64_t>(n0) * row_bytes,
                        q.live * static_cast<uint32_t>(rows) * row_bytes);
    s.scale = layer_rsrc(p.scales + (q.e * p.H + n0) * p.gpr,
                         q.live * static_cast<uint32_t>(rows) * 4u * static_cast<uint32_t>(p.gpr));
    s.shape = layer_rsrc(p.shapes + 2 * (q.e * p.H + n0) * p.gpr,
                         q.live * static_cast<uint32_t>(rows) * 4u * static_cast<uint32_t>(p.gpr));
    return s;
  };
  int it = wave;
  if (it < items) {                            // wave-uniform; the barrier comes after
    Stream st;
    DownActs<F> hst;
    Item q = item_of(it);
    CodeSrc cur = source(q);
    hst.load(p, q, lane);
    __builtin_amdgcn_sched_barrier(0);
    st.issue_scales(cur, vscale, p.groups, lane, [&](int i) { return min(q.tb + i, q.te - 1); });
    [&]<int... U>(std::integer_sequence<int, U...>) {
      (st.template issue<U>(cur, vcode, min(q.tb + U, q.te - 1)), ...);
    }(std::make_integer_sequence<int, PM>{});
    // rows 0 .. 3: the pair's planes (the others repeat them)
    const Acts<1> acts{{hreg + (nl & 3) * L.hstride}, {reinterpret_cast<const float*>(hreg + L.factor)}};
    for (; it < items; it += kLayerWaves) {
      hst.store(q, hreg, L, lane);             // the part's h into this wave's LDS
      wave_lds_order();
      const Item qn = item_of(it + kLayerWaves);
      const CodeSrc nxt = source(qn);
      const float w = p.weights[q.pair];
      hst.load(p, qn, lane);                   // ahead of the next item's codes
      float acc[NT][1] = {};
      uint32_t bad = 0u;
      for (int t0 = q.tb; t0 < q.te; t0 += PM) {
        st.take_scales();
        const bool more = t0 + PM < q.te;
        CodeSrc src;
        src.code = more ? cur.code : nxt.code;
        src.scale = more ? cur.scale : nxt.scale;
        if constexpr (F::kWide) src.shape = more ? cur.shape : nxt.shape;
        const int tn = more ? t0 + PM : qn.tb, last = (more ? q.te : qn.te) - 1;
        st.issue_scales(src, vscale, p.groups, lane, [&](int i) { return min(tn + i, last); });
        [&]<int... U>(std::integer_sequence<int, U...>) {
          (([&] {
             if (t0 + U < q.te) {
               uint32_t w4[NT][F::DW];
               float s[NT];
#pragma unroll
               for (int i = 0; i < NT; ++i)
#pragma unroll
                 for (int d = 0; d < Stream::DW; ++d) asm volatile("" : "+v"(st.cb[U][i][d]));
               uint32_t sh[NT];
               st.template take<U>(nl, kq, w4, s, sh);
               if constexpr (F::kWide) {
                 wide_step<F::kBits, NT, 1>(w4, s, sh, acts, t0 + U - q.tb, kq, acc);
               } else {
                 layer_step<SPL, NT, 1, 0>(w4, s, acts, t0 + U - q.tb, kq, acc, bad);
               }
             }
             st.template issue<U>(src, vcode, min(tn + U, last));
             __builtin_amdgcn_sched_barrier(0);
           }()),
           ...);
        }(std::make_integer_sequence<int, PM>{});
      }
      if constexpr (!F::kWide) {
        if (__any((bad & 0xAAAAAAAAu) != 0u)) {
          const __amdgpu_buffer_rsrc_t shp = layer_rsrc(p.shapes + 2 * (q.e * p.H + n0) * p.gpr,
                                                        static_cast<uint32_t>(rows) * 4u * static_cast<uint32_t>(p.gpr));
          uint32_t vc[NT], vs[NT];
          lane_offsets(nl, kq, vc, vs);
          layer_extra<SPL, NT, 1>(cur, shp, vc, vs, q.tb, q.te, 1, p.groups, acts, q.tb, kq, acc);
        }
      }
      if (kq == 0) {
        const int t = q.pair / p.topk;
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (nl < p.rt) sums[t * 32 + i * p.rt + nl] += w * acc[i][0];
      }
      wave_lds_order();
      q = qn;
      cur = nxt;
    }
  }
  __syncthreads();
  // the waves' sums in wave order
  const float* all = reinterpret_cast<const float*>(smem + L.sum);
  for (int i = tid; i < p.T * 32; i += 1024) {
    const int t = i >> 5, r = i & 31;
    if (r >= rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kLayerWaves; ++k) v += all[k * p.T * 32 + i];
    store_out(static_cast<float*>(p.y), p.ybf16 != 0, static_cast<int64_t>(t) * p.H + n0 + r, v);
  }
}

Groups group_steps(int group, int spl) {
  const int spg = group / (128 * spl);
  if ((spg & (spg - 1)) != 0) return Groups{-1, static_cast<uint32_t>((uint64_t{1} << 32) / static_cast<uint32_t>(spg) + 1)};
  int s = 0;
  while ((1 << s) < spg) ++s;
  return Groups{s, 0u};
}

int layer_spl(int bits, int group) { return bits == 2 && group % 256 == 0 ? 2 : 1; }

constexpr int kLayerLds = 160 * 1024;

// Launches of kernel 1: the fewest whose shares of the row fit in LDS (four bytes a value).
// Each routes again and passes its sums on through the workspace, some 8 us, where shorter
// runs of tokens would read the shared experts' codes again (7168 / 3 K, top-16 of 128, eight
// tokens: 100 + 106 us in two launches; two runs of four 218).
int layer_up_launches(int T, int topk, int H, int spl) {
  const int nmacro = H / (spl * 128);
  int n = 1;
  while (n < nmacro && layer_up_lds(T, topk, (nmacro + n - 1) / n * spl * 128, 1).total > kLayerLds) ++n;
  return n;
}

// K parts of kernel 2: of at most 1024 values, one operand a lane (7168 / 3 K, top-16 of 128,
// four tokens: 73 us against 81 with parts of 1536), and enough items for every wave.
constexpr int kDownPart = 1024;
int layer_down_parts(int T, int topk, int I, int spl) {
  const int nmacro = I / (spl * 128);
  const int jobs = T * topk;
  int ks = (I + kDownPart - 1) / kDownPart;
  while (ks < nmacro && jobs * ks < kLayerWaves) ks *= 2;
  return std::min(ks, nmacro);
}

}  // namespace

// One run of the two kernels: 2- to 4-bit codes, up to eight tokens.
static bool layer_fits(int64_t T, int topk, int E, int64_t H, int64_t I, int up_bits, int dn_bits) {
  if (up_bits < 2 || up_bits > 4 || dn_bits < 2 || dn_bits > 4) return false;
  if (T < 1 || T > kLayerMaxT || E > kLayerMaxE || topk > kRouterMaxTopk) return false;
  if (H > 65536 || I > 65536 || (I + 16) * (H * up_bits / 8) >= (int64_t{1} << 32)) return false;   // 32-bit tile offsets
  return true;
}

// Tokens of one run of the two kernels; 0: the composed path. Nine to 64 tokens take
// runs of up to eight: an expert that tokens of several runs share is read again, yet that is
// ahead of the composed path (us, runs against composed; 2048 x 1024, 2 bits, top-8 of 128: 16
// tokens 81 / 161, 64: 319 / 424; top-4 of 16, 64 tokens: 187 / 214; 4 bits, top-4 of 32: 16
// tokens 95 / 140, 64: 367 / 487; 7168 x 2 K, 4 bits, top-8 of 64: 64 tokens 2578 / 4644) but
// - where launches count, not rates: 2 bits, top-2 of 8, 512 x 256 (0.8 MB): 16 tokens 33 / 29;
//   top-4 of 16, 1024 x 512 (6 MB): 16 tokens 43 / 47, 32: 84 / 67. Wider codes are ahead with
//   a third of the bytes (4 bits, 1.6 MB: 16 tokens 37 / 47, 64: 144 / 114; 3 bits, 9 MB: 32
//   tokens 109 / 122, 64: 217 / 214);
// - with 2-bit codes and rows that take several launches of kernel 1 (7168 / 3 K, top-16 of
//   128: 16 tokens 719 / 832, 24: 1080 / 1104, 32: 1434 / 1399, 64: 2863 / 2686).
int64_t moe_layer_tokens(int64_t T, int topk, int E, int64_t H, int64_t I, int up_bits, int up_group, int dn_bits) {
  if (T < 1 || T > 8 * kLayerMaxT) return 0;
  const int64_t runs = (T + kLayerMaxT - 1) / kLayerMaxT, n = (T + runs - 1) / runs;
  if (!layer_fits(n, topk, E, H, I, up_bits, dn_bits)) return 0;
  if (runs == 1) return n;
  const bool two = up_bits == 2 && dn_bits == 2;
  const int64_t bytes = H * I * (2 * up_bits + dn_bits) / 8 * std::min<int64_t>(E, T * topk);
  if ((two ? 1 : 3) * bytes < runs * (int64_t{2} << 20)) return 0;
  const int launches = layer_up_launches(static_cast<int>(n), topk, static_cast<int>(H), layer_spl(up_bits, up_group));
  if (two && launches > 1 && runs > 3) return 0;
  return n;
}

namespace {

template <class Kern, class Par>
hipError_t launch_layer(Kern kern, unsigned grid, int lds, const Par& p, hipStream_t st) {
  if (lds > 64 * 1024) {
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kern), lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3(grid), dim3(1024), static_cast<size_t>(lds), st, p);
  return hipGetLastError();
}

}  // namespace

static hipError_t launch_layer_run(const MoeRouter& r, const uint16_t* x, int T, const MoeLayerWeight& up,
                                   const MoeLayerWeight& dn, int H, int I, const MoeLayerBuffers& b,
                                   int32_t* ids_user, float* weights_user, void* y, int ybf16, hipStream_t st) {
  const int cu = device_cu_count();
  const int cus = cu > 0 ? cu : 256;
  LayerUpParams p{};
  p.r = router_params(r);
  p.x = x;
  p.T = T;
  p.H = H;
  p.I = I;
  p.codes = up.codes;
  p.scales = up.scales;
  p.shapes = up.shapes;
  p.code_bytes = up.code_bytes;
  p.gpr = H / up.group;
  const int spl = layer_spl(up.bits, up.group), dspl = layer_spl(dn.bits, dn.group);
  p.groups = group_steps(up.group, spl);
  p.partial = b.partial;
  p.weights = b.weights;
  p.ids_user = ids_user;
  p.weights_user = weights_user;
  p.rec = b.rec;
  p.h = b.h;
  const int nmacro = H / (spl * 128), launches = layer_up_launches(T, r.topk, H, spl);
  const int64_t units = static_cast<int64_t>(std::min(r.E, T * r.topk)) * (I / 16);
  hipError_t e;
  const bool few = r.E <= 256;                 // a router wave with 4 experts a lane, or 16
  // steps in flight: up to four tokens, and more (whose second tile takes registers: more spill)
  auto up_kernel = [&](auto f_c, auto pm_c, auto pm2_c) {
    using F = decltype(f_c);
    constexpr int PM = decltype(pm_c)::value, PM2 = decltype(pm2_c)::value;
    hipError_t err = hipSuccess;
    for (int c = 0; c < launches && err == hipSuccess; ++c) {
      p.k0 = c * nmacro / launches;
      p.steps = (c + 1) * nmacro / launches - p.k0;
      p.add = c > 0;
      p.last = c == launches - 1;
      const int teams = kLayerWaves / layer_up_max_parts(p.steps);   // at least
      const unsigned grid = static_cast<unsigned>(std::min<int64_t>(cus, (units + teams - 1) / teams));
      p.share = 1.0f / (static_cast<float>(grid) * kLayerWaves);
      const int K = p.steps * spl * 128;
      p.batch = 4;
      while (p.batch > 1 && layer_up_lds(T, r.topk, K, p.batch).total > kLayerLds) --p.batch;
      const int lds = layer_up_lds(T, r.topk, K, p.batch).total;
      if (T > 4) {
        err = few ? launch_layer(k_layer_up<F, PM2, 4, 2>, grid, lds, p, st) : launch_layer(k_layer_up<F, PM2, 16, 2>, grid, lds, p, st);
      } else {
        err = few ? launch_layer(k_layer_up<F, PM, 4, 1>, grid, lds, p, st) : launch_layer(k_layer_up<F, PM, 16, 1>, grid, lds, p, st);
      }
    }
    return err;
  };
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  using I8 = std::integral_constant<int, 8>;
  if (up.bits == 2) {
    e = spl == 2 ? up_kernel(Codes2<2>{}, I4{}, I2{}) : up_kernel(Codes2<1>{}, I8{}, I4{});
  } else {
    e = up.bits == 3 ? up_kernel(CodesWide<3>{}, I2{}, I2{}) : up_kernel(CodesWide<4>{}, I2{}, I2{});
  }
  if (e != hipSuccess) return e;

  LayerDownParams d{};
  d.rec = b.rec;
  d.weights = b.weights;
  d.T = T;
  d.topk = r.topk;
  d.h = b.h;
  d.codes = dn.codes;
  d.scales = dn.scales;
  d.shapes = dn.shapes;
  d.code_bytes = dn.code_bytes;
  d.gpr = I / dn.group;
  d.groups = group_steps(dn.group, dspl);
  d.H = H;
  d.I = I;
  d.rows = std::min(32, std::max(4, (H + cus - 1) / cus));
  const int nt = d.rows > 16 ? 2 : 1;
  d.rt = (d.rows + nt - 1) / nt;
  d.rows = d.rt * nt;
  d.ks = layer_down_parts(T, r.topk, I, dspl);
  d.y = y;
  d.ybf16 = ybf16;
  const unsigned dgrid = static_cast<unsigned>((H + d.rows - 1) / d.rows);
  const int dlds = layer_down_lds(T, I, dspl, d.ks).total;
  auto down_kernel = [&](auto f_c, auto pm_c) {
    using F = decltype(f_c);
    constexpr int PM = decltype(pm_c)::value;
    return nt == 2 ? launch_layer(k_layer_down<F, PM, 2>, dgrid, dlds, d, st)
                   : launch_layer(k_layer_down<F, PM, 1>, dgrid, dlds, d, st);
  };
  if (dn.bits == 2) return dspl == 2 ? down_kernel(Codes2<2>{}, I4{}) : down_kernel(Codes2<1>{}, I8{});
  return dn.bits == 3 ? down_kernel(CodesWide<3>{}, I2{}) : down_kernel(CodesWide<4>{}, I2{});
}

hipError_t launch_moe_layer(const MoeRouter& r, const uint16_t* x, int T, int run, const MoeLayerWeight& up,
                            const MoeLayerWeight& dn, int H, int I, const MoeLayerBuffers& b, int32_t* ids_user,
                            float* weights_user, void* y, int ybf16, hipStream_t st) {
  for (int t0 = 0; t0 < T; t0 += run) {        // the runs follow each other on the stream and share the buffers
    MoeRouter rt = r;
    rt.logits = static_cast<const char*>(r.logits) + static_cast<int64_t>(t0) * r.E * (r.dtype == 0 ? 4 : 2);
    const int64_t at = static_cast<int64_t>(t0) * H;
    const hipError_t e = launch_layer_run(rt, x + at, std::min(run, T - t0), up, dn, H, I, b,
                                          ids_user ? ids_user + static_cast<int64_t>(t0) * r.topk : nullptr,
                                          weights_user ? weights_user + static_cast<int64_t>(t0) * r.topk : nullptr,
                                          static_cast<char*>(y) + at * (ybf16 ? 2 : 4), ybf16, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace cubic
