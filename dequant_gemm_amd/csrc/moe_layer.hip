// moe_layer.hip -- the router (cubic_moe_topk) and the whole routed-expert
// layer for a few tokens (cubic_moe_layer) in two kernels.
//
//   ids, w  = the router of each token's logits (router.h)
//   [g | u] = x_t * GU_e^T;  h = bf16(SiLU(g) * u);  y_t = sum_j w_tj * (h_tj * D_e^T)
//
// Every touched expert's codes are read once and each serves one to eight
// rows, so the layer is bound by HBM as long as decoding a code costs little.
// The 2-bit codes {00, 01, 11} = {0, +1, -1} are therefore turned into 4-bit
// floats: field b1 b0 in the top half of a nibble is the e2m1 number {0, +2, -2}
// (sign b1, exponent b0), so sixteen codes take one shift and two masks (the
// field 10 reads as -0 and contributes nothing; where a wave sees one, a slow
// pass adds its level's sum). The activations are split exactly into two
// e4m3 halves: a bf16 number has eight significant bits, hi takes the upper
// four rounded to nearest and lo the (signed) rest, with one power-of-two block
// scale for 32 consecutive values. hi and lo (and the tokens) are rows of the
// same 16 x 16 x 128 MFMA. Values below 2^-14 of their block's largest are off by up to
// 2^-22 of it, and blocks whose largest value is below 2^-116 by up to 2^-138. The MFMA
// aligns the products of its 128 codes to the largest and drops what lies about 2^-14
// below it: measured, its sums of normal values are off by 2^-18 to 2^-19 (rms; exact
// where the products span less), by 2^-16 where outliers of 40 times the rest are among
// them, and at worst by 2^-11 of the largest product. Steps are added up in fp32. The
// result is 2^-16 off where an fp32 sum would be 2^-24, which moves about one h in a
// hundred to the neighbouring bf16 number; exact sums would need a third row a token, and
// hold five tokens.
//
// Kernel 1 (k_layer_up): every workgroup runs the router of all tokens (one wave
// each), splits x into LDS, and then walks its share of the units (touched
// expert, 16 gate rows and the 16 up rows beside them). Kernel 2 (k_layer_down):
// every workgroup takes an equal share of the output rows and all pairs, one
// (pair, K part) per wave at a time, so the router-weighted sum never leaves the
// workgroup: no atomics, and the order of the sums does not depend on timing.
//
// Measured (hidden 7168, intermediate 3 K, G512, on one card whose large copy runs at
// 5.1 TB/s): one token through 16 of 64 experts, 281 MB: kernel 1 42 us (8 us until the
// first load is issued: router, splitting, lists; then 5.7 TB/s), kernel 2 21 us
// (5.9 TB/s while streaming), 56-64 us together; four tokens through about 52 of 128
// experts, 930 MB: 112 + 64 us; 4 bits, G128, 2048 x 1024, two tokens of top-4 of 32: 12.7
// + 8.6 us. HBM traffic is 1.00 of the codes and scales. Against
// loads in operand order, a barrier a round and seven steps in flight, the first version,
// kernel 1 took 62 us and kernel 2 26.
//
// 3- and 4-bit codes run on the same two kernels as sums of fixed functions of the code
// (CodesWide); wider codes, more tokens and shapes beyond the kernels' LDS run as the router kernel
// followed by the routed MLP step (moe.hip).
#include <algorithm>

#include "gemv_core.h"
#include "launch.h"
#include "router.h"

namespace cubic {
namespace {

constexpr uint32_t kRsrc3 = 0x00020000u;       // raw buffer, 32-bit data format
constexpr int kLayerWaves = 16;                // one workgroup of 1024 threads per compute unit
constexpr int kLayerMaxT = 8;                  // hi and lo rows of eight tokens fill the MFMA's 16 rows
constexpr int kLayerMaxE = 1024;               // experts of one router wave (4 or 16 per lane)
constexpr int kLayerMaxPairs = kLayerMaxT * kRouterMaxTopk;

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

// ---- the two e4m3 halves of bf16 values -----------------------------------
// Block scale of a largest magnitude (finite; its fp32 bits): with ef the
// (clamped) exponent field, v * 2^(134 - ef) lies below 256 and its largest
// in [128, 256). Scale bytes (E8M0): ef - 7 for hi, ef - 11 for lo.
__device__ __forceinline__ uint32_t block_exponent(float amax) {
  const uint32_t ef = __float_as_uint(amax) >> 23;
  return ef < 11u ? 11u : ef;
}
__device__ __forceinline__ float block_factor(uint32_t ef) { return __uint_as_float((261u - ef) << 23); }

// Halves of two values: bytes 0 and 1 of hi and lo. Non-finite values become
// NaN (0x7f) in hi, so their rows come out NaN.
__device__ __forceinline__ void split2(float a, float b, float f, uint32_t& hi, uint32_t& lo) {
  const bool fa = fabsf(a) < __builtin_inff(), fb = fabsf(b) < __builtin_inff();
  const float va = fa ? a * f : 0.0f, vb = fb ? b * f : 0.0f;
  hi = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(va, vb, 0, false)) & 0xffffu;
  const float ra = (va - __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(hi), 0)) * 16.0f;
  const float rb = (vb - __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(hi), 1)) * 16.0f;
  lo = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(ra, rb, 0, false)) & 0xffffu;
  hi = (fa ? hi : (hi & 0xff00u) | 0x7fu);
  hi = (fb ? hi : (hi & 0x00ffu) | 0x7f00u);
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a < __builtin_inff() ? a : 0.0f;
}

// Place of code c (0..31) of a 32-code chunk among the chunk's 32 operand bytes. 2-bit
// codes: dword d of the decoded chunk holds the even (d even) or odd codes of code word
// d / 2; wider codes: the even or odd ones of codes 8 (d / 2) .. + 7.
__device__ __forceinline__ int code_slot(int c, bool wide) {
  return 16 * (c >> 4) + (wide ? 8 * ((c & 15) >> 3) + 4 * (c & 1) + ((c & 7) >> 1) : 8 * (c & 1) + ((c & 15) >> 1));
}
// Place of 32-chunk b of a row: with SPL = 2 a lane's 16-byte load holds two
// chunks, which feed two MFMAs (a macro step of 256 codes, lane group kq takes
// chunks 2 kq and 2 kq + 1, MFMA h the h-th of each).
template <int SPL>
__device__ __forceinline__ int chunk_place(int b) {
  return SPL == 2 ? (b & ~7) + ((b & 1) << 2) + ((b & 7) >> 1) : b;
}

// ---- the two kinds of codes ---------------------------------------------------
// Both multiply the activations' e4m3 halves (rows 2 t and 2 t + 1 of the MFMA for token
// t). 2-bit codes are e2m1 nibbles; a lane's operand is one or two 32-code chunks.
template <int SPL_>
struct Codes2 {
  static constexpr bool kWide = false;
  static constexpr int kBits = 2, SPL = SPL_;
  static constexpr int DW = 2 * SPL_, W = DW;  // dwords of a lane's loads, and of its operand codes
  static constexpr int kPiece = 4 * DW;        // bytes between the loads of neighbouring lanes
};
// 3- and 4-bit codes j = -M .. K (M = 2^(B-1), K = M - 1): with n = |j| and c = 1 - a - b
// their level s (a t + b t |t| + c t^3), t = j / K, is a sum of three fixed odd functions
//   p1 = j,  p2 = +-n (M - n),  p3 = +-n (M - n) (n - M / 2):
//   level = s ((a / K + M b / K^2 + M^2 c / K^3) p1 - (b / K^2 + 1.5 M c / K^3) p2 - c / K^3 p3)
// whose products with the activations' halves MFMAs sum exactly: the values are e4m3
// numbers (four significant bits), looked up four at a time by byte permutes in registers,
// and the coefficients of a group enter with its scale. A table of a group's levels costs
// its building and an LDS read a code (2048 x 1024, W4 G128, two tokens: 17.5 + 11.2 us
// with tables).
// 4 bits: a code is -8 sign + l. The low bits l of j and of -j add up to 8, where p2 is
// even and p3 odd, so both need only l, and p2 the sign; p1 = (l - 4) +- 4, and p3 + l - 4
// has four significant bits (p3 has not): fourteen operations for eight codes and four
// MFMAs. Whole 16-entry look-ups of three functions took 26 and three (7168 x 2 K, 8
// tokens: 419 us against 291 to 310); l and the unsigned code as they stand (small e4m3
// numbers) take twelve, but their sums' cancellation costs two bits (2^-14.5). 3 bits:
// three look-ups in eight entries.
// The MFMA wants codes 16 kq .. + 15 and 64 + 16 kq .. + 15 of a step in lane group kq.
// 4 bits: loaded as 8-byte pieces of either half; 3 bits: as 12-byte chunks of 32 codes,
// of which two lane groups take a half each.
template <int B>
struct CodesWide {
  static constexpr bool kWide = true;
  static constexpr int kBits = B, SPL = 1;
  static constexpr int DW = B, W = 4;
  static constexpr int kPiece = B == 4 ? 8 : 12;
  static constexpr int M = 1 << (B - 1), K = M - 1;
  static constexpr int kSums = B == 4 ? 4 : 3; // MFMAs a step
};

// An integer of at most four significant bits as an e4m3 number.
constexpr uint32_t e4m3_int(int v) {
  uint32_t m = static_cast<uint32_t>(v < 0 ? -v : v), e = 0;
  if (m == 0) return 0u;
  while (m >= 16u) { m >>= 1; ++e; }           // (exact: the bits shifted out are zero)
  while (m < 8u) { m <<= 1; --e; }
  return ((e + 10u) << 3 | (m & 7u)) | (v < 0 ? 0x80u : 0u);   // m 2^e = m/8 2^(e+3), bias 7
}
// Four bytes of f(j0) .. f(j0 + 3).
template <class Fn>
constexpr uint32_t e4m3_bytes(Fn f, int j0) {
  uint32_t v = 0;
  for (int i = 0; i < 4; ++i) v |= e4m3_int(f(j0 + i)) << (8 * i);
  return v;
}
// The lane's 32 operand codes (w: 16 and 16; the even and odd ones of eight in turn) as
// bytes. 4 bits: b = l - 4, +-4, p2, p3 + l - 4; 3 bits: p1, p2, p3.
template <int B>
__device__ __forceinline__ void poly_decode(const uint32_t* w, i32x8* b) {
  if constexpr (B == 4) {
    constexpr auto p2 = [](int l) { return l * (8 - l); };
    constexpr auto p3l4 = [](int l) { return l * (8 - l) * (l - 4) + l - 4; };
    constexpr auto l4 = [](int l) { return l - 4; };
    constexpr uint32_t four = e4m3_int(4) * 0x01010101u, d0 = e4m3_bytes(l4, 0), d4 = e4m3_bytes(l4, 4);
    constexpr uint32_t a0 = e4m3_bytes(p2, 0), a4 = e4m3_bytes(p2, 4), c0 = e4m3_bytes(p3l4, 0), c4 = e4m3_bytes(p3l4, 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {              // eight codes
      const uint32_t v = w[u], vs = v >> 4;
      const uint32_t le = v & 0x07070707u, lo = vs & 0x07070707u;
      b[0][2 * u] = static_cast<int>(__builtin_amdgcn_perm(d4, d0, le));
      b[0][2 * u + 1] = static_cast<int>(__builtin_amdgcn_perm(d4, d0, lo));
      b[1][2 * u] = static_cast<int>(((v << 4) & 0x80808080u) | four);
      b[1][2 * u + 1] = static_cast<int>((v & 0x80808080u) | four);
      b[2][2 * u] = static_cast<int>(((v << 4) & 0x80808080u) | __builtin_amdgcn_perm(a4, a0, le));
      b[2][2 * u + 1] = static_cast<int>((v & 0x80808080u) | __builtin_amdgcn_perm(a4, a0, lo));
      b[3][2 * u] = static_cast<int>(__builtin_amdgcn_perm(c4, c0, le));
      b[3][2 * u + 1] = static_cast<int>(__builtin_amdgcn_perm(c4, c0, lo));
    }
  } else {
    // codes 0 .. 3 are their values, 4 .. 7 those less 8
    constexpr auto sign = [](int j) { return j < 0 ? -1 : 1; };
    constexpr auto p1 = [](int j) { return j; };
    constexpr auto p2 = [sign](int j) { return j * (4 - sign(j) * j); };
    constexpr auto p3 = [sign](int j) { return j * (4 - sign(j) * j) * (sign(j) * j - 2); };
    constexpr uint32_t t[3][2] = {{e4m3_bytes(p1, 0), e4m3_bytes(p1, -4)},
                                  {e4m3_bytes(p2, 0), e4m3_bytes(p2, -4)},
                                  {e4m3_bytes(p3, 0), e4m3_bytes(p3, -4)}};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t* q = w + 2 * (u >> 1);    // 48 bits
      const uint32_t v = (u & 1) ? __builtin_amdgcn_alignbit(q[1], q[0], 24) : q[0];
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
      if constexpr (F::kBits == 4) {
        const u32x2 v0 = __builtin_amdgcn_raw_buffer_load_b64(src.code, vcode[i], t * 64, 0);
        const u32x2 v1 = __builtin_amdgcn_raw_buffer_load_b64(src.code, vcode[i], t * 64 + 32, 0);
        cb[U][i][0] = v0.x; cb[U][i][1] = v0.y; cb[U][i][2] = v1.x; cb[U][i][3] = v1.y;
      } else if constexpr (DW == 4) {
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
  __device__ __forceinline__ void take(int nl, int kq, uint32_t (*w)[F::W], float* s, uint32_t* sh) {
    auto from = [](int lane, uint32_t v) {
      return static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(4 * lane, static_cast<int>(v)));
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if constexpr (F::kBits == 3) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {          // chunk 2 h + kq / 2; its upper half for odd kq
          const int l = 4 * nl + 2 * h + (kq >> 1);
          const uint32_t d0 = from(l, cb[U][i][0]), d1 = from(l, cb[U][i][1]), d2 = from(l, cb[U][i][2]);
          w[i][2 * h] = (kq & 1) ? __builtin_amdgcn_alignbit(d2, d1, 16) : d0;
          w[i][2 * h + 1] = (kq & 1) ? d2 >> 16 : d1;
        }
      } else {
#pragma unroll
        for (int d = 0; d < DW; ++d) w[i][d] = from(4 * nl + kq, cb[U][i][d]);
      }
      s[i] = __uint_as_float(from(4 * nl + (U & 3), __float_as_uint(sc[i][U / 4])));
      if constexpr (F::kWide) sh[i] = from(4 * nl + (U & 3), ab[i][U / 4]);
    }
  }
};

// One macro step: A rows from LDS (xr: this lane's row, its bytes in operand
// order; sr: its scale bytes), B from the code words of NT tiles. The step's sum
// of hi + lo, times the group scale, goes to acc[tile][token 0 / 1 of the lane].
// MODE 0: the codes 0, +1, -1; their unused field is collected in bad. MODE 1:
// the unused field alone, as +1 (the slow pass).
template <int SPL, int NT, int MODE>
__device__ __forceinline__ void layer_step(const uint32_t (*w)[2 * SPL], const float* sc, const uint8_t* xr,
                                           const uint8_t* sr, int t, int kq, float (*acc)[2], uint32_t& bad) {
  uint32_t sx;
  if constexpr (SPL == 2) {
    sx = *reinterpret_cast<const uint16_t*>(sr + t * 8 + kq * 2);
  } else {
    sx = sr[t * 4 + kq];
  }
  f32x4 part[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) part[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < SPL; ++h) {
    const u32x4 a0 = *reinterpret_cast<const u32x4*>(xr + (t * SPL + h) * 128 + 16 * kq);
    const u32x4 a1 = *reinterpret_cast<const u32x4*>(xr + (t * SPL + h) * 128 + 64 + 16 * kq);
    const i32x8 a = {static_cast<int>(a0.x), static_cast<int>(a0.y), static_cast<int>(a0.z), static_cast<int>(a0.w),
                     static_cast<int>(a1.x), static_cast<int>(a1.y), static_cast<int>(a1.z), static_cast<int>(a1.w)};
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      i32x8 b = {};
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const uint32_t v = w[i][2 * h + d];
        if constexpr (MODE == 0) {
          b[2 * d] = static_cast<int>((v << 2) & 0xCCCCCCCCu);
          b[2 * d + 1] = static_cast<int>(v & 0xCCCCCCCCu);
          bad |= v & ~(v << 1);
        } else {
          const uint32_t f = v & ~(v << 1) & 0xAAAAAAAAu;
          b[2 * d] = static_cast<int>((f << 1) & 0x44444444u);
          b[2 * d + 1] = static_cast<int>((f >> 1) & 0x44444444u);
        }
      }
      // scale 2^-1 on the codes: the nibbles are +-2
      if (h == 0) {
        part[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, part[i], 0, 4, 0, static_cast<int>(sx), 0, 126);
      } else {
        part[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, part[i], 0, 4, 1, static_cast<int>(sx), 0, 126);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    acc[i][0] = fmaf(sc[i], part[i][0] + part[i][1], acc[i][0]);
    acc[i][1] = fmaf(sc[i], part[i][2] + part[i][3], acc[i][1]);
  }
}

// The same for wide codes, sh: the tiles' shapes a | b.
template <int B, int NT>
__device__ __forceinline__ void wide_step(const uint32_t (*w)[4], const float* sc, const uint32_t* sh, const uint8_t* xr,
                                          const uint8_t* sr, int t, int kq, float (*acc)[2]) {
  constexpr float K = CodesWide<B>::K, M = CodesWide<B>::M;
  constexpr int NS = CodesWide<B>::kSums;
  const int sx = sr[t * 4 + kq];
  const u32x4 a0 = *reinterpret_cast<const u32x4*>(xr + t * 128 + 16 * kq);
  const u32x4 a1 = *reinterpret_cast<const u32x4*>(xr + t * 128 + 64 + 16 * kq);
  const i32x8 a = {static_cast<int>(a0.x), static_cast<int>(a0.y), static_cast<int>(a0.z), static_cast<int>(a0.w),
                   static_cast<int>(a1.x), static_cast<int>(a1.y), static_cast<int>(a1.z), static_cast<int>(a1.w)};
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    i32x8 b[NS];
    poly_decode<B>(w[i], b);
    f32x4 part[NS];
#pragma unroll
    for (int f = 0; f < NS; ++f) {
      constexpr f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      part[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[f], zero, 0, 0, 0, sx, 0, 127);
    }
    const float sa = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(sh[i] & 0xffffu)));
    const float sb = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(sh[i] >> 16)));
    const float c = (1.0f - sa - sb) * (1.0f / (K * K * K));
    const float k1 = sc[i] * fmaf(M * M, c, fmaf(sb, M / (K * K), sa * (1.0f / K)));
    const float k2 = sc[i] * -fmaf(1.5f * M, c, sb * (1.0f / (K * K)));
    const float k3 = sc[i] * -c;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float p[NS];
#pragma unroll
      for (int f = 0; f < NS; ++f) p[f] = part[f][2 * m] + part[f][2 * m + 1];
      if constexpr (B == 4) {
        acc[i][m] = fmaf(k1, p[0] + p[1], acc[i][m]);
        acc[i][m] = fmaf(k2, p[2], acc[i][m]);
        acc[i][m] = fmaf(k3, p[3] - p[0], acc[i][m]);
      } else {
        acc[i][m] = fmaf(k1, p[0], acc[i][m]);
        acc[i][m] = fmaf(k2, p[1], acc[i][m]);
        acc[i][m] = fmaf(k3, p[2], acc[i][m]);
      }
    }
  }
}

// The slow pass: the level of the field 10 (code -2) is -q(2) s, q(2) = 2 a + 4 b +
// 8 (1 - a - b); its codes' sums are added step by step. Loads in operand order:
// vcode, vscale as in the stream, but of row nl and quarter kq.
template <int SPL, int NT>
__device__ __forceinline__ void layer_extra(const CodeSrc& src, const __amdgpu_buffer_rsrc_t& shp,
                                            const uint32_t* vcode, const uint32_t* vscale, int tb, int te, int by,
                                            const Groups& gr, const uint8_t* xr, const uint8_t* sr, int kq,
                                            float (*acc)[2]) {
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
      lev[i] = static_cast<float>(-static_cast<double>(s) * level_numerator(a, b, 2, 1));
    }
    uint32_t none = 0u;
    layer_step<SPL, NT, 1>(st.cb[0], lev, xr, sr, t, kq, acc, none);
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
  int down_spl;            // operand order of h: chunks per lane and step of 2-bit down codes; 0: wider codes
  int32_t* ids;            // [T][topk] out
  float* weights;
  int32_t* ids_user;       // a second copy for the caller, or NULL
  float* weights_user;
  int32_t* rec;
  uint8_t* hq;             // [T*topk][2][I] e4m3 halves of h in operand order
  uint8_t* hs;             // [T*topk][2][I / 32] block scales
};

// K parts of kernel 1: the waves of a tile, so many that the slowest workgroup has the
// least to do (units: touched experts' tiles; kRoundCost: eighths of a step that a round
// costs beside its steps). At least two teams: a scale block of h spans two tiles. The
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
  int xq, xs, red, first, id, w, exp, slot, cand, misc, total;   // byte offsets
  int xq_stride, xs_stride;
};
__host__ __device__ inline LayerUpLds layer_up_lds(int T, int topk, int H, int batch) {
  LayerUpLds L;
  const int P = T * topk;
  auto up16 = [](int v) { return (v + 15) & ~15; };
  // Rows of the MFMA: two halves a token; 16 bytes of padding each: the rows' reads hit
  // other banks.
  L.xq_stride = H + 16;
  L.xs_stride = up16(H / 32) + 16;
  int o = 0;
  L.xq = o;    o += 2 * T * L.xq_stride;
  L.xs = o;    o += 2 * T * L.xs_stride;
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

template <class F, int PM, int EPL>
__global__ __launch_bounds__(1024) void k_layer_up(LayerUpParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int SPL = F::SPL;
  using Stream = CodeStream<F, PM, 2>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nl = lane & 15, kq = lane >> 4;
  const int T = p.T, topk = p.r.topk, P = T * topk;
  const LayerUpLds L = layer_up_lds(T, topk, p.H, p.batch);
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
    // eight values a thread; four neighbouring threads share a 32-value block
    const int per_row = p.H / 8, all = T * per_row;
    for (int v0 = 0; v0 < all; v0 += 1024) {
      const int v = v0 + tid;
      const bool on = v < all;                 // whole blocks: all is a multiple of 16
      const int t = on ? v / per_row : 0;
      const int q = on ? v - t * per_row : 0;
      const u32x4 raw = *reinterpret_cast<const u32x4*>(p.x + static_cast<int64_t>(t) * p.H + 8 * q);
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(raw[j] << 16);
        f[2 * j + 1] = __uint_as_float(raw[j] & 0xffff0000u);
      }
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(f[j]));
      amax = fmaxf(amax, __shfl_xor(amax, 1));
      amax = fmaxf(amax, __shfl_xor(amax, 2));
      const uint32_t ef = block_exponent(amax);
      const float fac = block_factor(ef);
      // even codes, then odd codes, of the eight
      uint32_t hi[4], lo[4];
      split2(f[0], f[2], fac, hi[0], lo[0]);
      split2(f[4], f[6], fac, hi[1], lo[1]);
      split2(f[1], f[3], fac, hi[2], lo[2]);
      split2(f[5], f[7], fac, hi[3], lo[3]);
      if (on) {
        const int b = q >> 2, qd = q & 3;      // block of the row, quarter of the block
        const int at = 32 * chunk_place<SPL>(b) + code_slot(8 * qd, F::kWide);
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
          unsigned char* dst = smem + L.xq + (2 * t + pc) * L.xq_stride + at;
          const uint32_t* s = pc ? lo : hi;
          *reinterpret_cast<uint32_t*>(dst) = s[0] | (s[1] << 16);
          *reinterpret_cast<uint32_t*>(dst + (F::kWide ? 4 : 8)) = s[2] | (s[3] << 16);
          if (qd == 0) smem[L.xs + (2 * t + pc) * L.xs_stride + b] = static_cast<uint8_t>(ef - (pc ? 11u : 7u));
        }
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
    // for kernel 2 and the caller: ids, weights and the pairs grouped by expert
    if (tid < P) {
      const float w = s_w[tid];
      p.ids[tid] = pe;
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
  const int nmacro = p.H / (SPL * 128);
  const int ks = __builtin_amdgcn_readfirstlane(layer_up_parts(total, nmacro, p.share));
  const int teams = kLayerWaves / ks;
  const int team = wave / ks, part = wave - team * ks;
  // this wave's steps: part, part + ks, ... (the team's waves read neighbouring
  // pieces of a row at any time)
  const int steps = (nmacro - part + ks - 1) / ks;
  const uint32_t row_bytes = static_cast<uint32_t>(p.H * F::kBits / 8);
  // a gate row of the tile, and the up row I rows below it
  auto lane_offsets = [&](int row, int quarter, int piece, uint32_t* vc, uint32_t* vs) {
    vc[0] = row * row_bytes + quarter * piece;
    vc[1] = vc[0] + static_cast<uint32_t>(p.I) * row_bytes;
    vs[0] = static_cast<uint32_t>(row * p.gpr * 4);
    vs[1] = vs[0] + static_cast<uint32_t>(p.I * p.gpr * 4);
  };
  uint32_t vcode[2], vscale[2];
  lane_offsets(lane >> 2, lane & 3, F::kPiece, vcode, vscale);
  const int ml = nl < 2 * T ? nl : 0;           // rows past the tokens are not used
  const uint8_t* xr = smem + L.xq + ml * L.xq_stride;
  const uint8_t* sr = smem + L.xs + ml * L.xs_stride;

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
  st.issue_scales(cur, vscale, p.groups, lane, [&](int i) { return part + min(i, steps - 1) * ks; });
  [&]<int... U>(std::integer_sequence<int, U...>) {
    (st.template issue<U>(cur, vcode, part + min(U, steps - 1) * ks), ...);
  }(std::make_integer_sequence<int, PM>{});

  float* red = reinterpret_cast<float*>(smem + L.red);
  const int red_wave = 2 * T * 16, red_round = kLayerWaves * red_wave;
  int slot_r = 0, half = 0, r0 = 0;            // round of the batch, its buffer, its first round
  for (int r = 0; r < rounds; ++r) {
    const CodeSrc nxt = source(u + stride);
    float acc[2][2] = {};
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
      st.issue_scales(src, vscale, p.groups, lane, [&](int i) { return part + min(tn + i, steps - 1) * ks; });
      [&]<int... U>(std::integer_sequence<int, U...>) {
        (([&] {
           if (t0 + U < steps) {
             uint32_t w[2][F::W];
             float s[2];
#pragma unroll
             for (int i = 0; i < 2; ++i)
#pragma unroll
               for (int d = 0; d < Stream::DW; ++d) asm volatile("" : "+v"(st.cb[U][i][d]));
             uint32_t sh[2];
             st.template take<U>(nl, kq, w, s, sh);
             const int t = part + (t0 + U) * ks;
             if constexpr (F::kWide) {
               wide_step<F::kBits, 2>(w, s, sh, xr, sr, t, kq, acc);
             } else {
               layer_step<SPL, 2, 0>(w, s, xr, sr, t, kq, acc, bad);
             }
           }
           st.template issue<U>(src, vcode, part + min(tn + U, steps - 1) * ks);
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
        lane_offsets(nl, kq, F::kPiece, vc, vs);
        layer_extra<SPL, 2>(cur, shp, vc, vs, part, nmacro, ks, p.groups, xr, sr, kq, acc);
      }
    }
    // partial sums of the team's waves meet in LDS; lane group kq holds tokens 2 kq
    // and 2 kq + 1
    float* rb = red + (half * p.batch + slot_r) * red_round;
#pragma unroll
    for (int m = 0; m < 2; ++m)
      if (2 * kq + m < T)
#pragma unroll
        for (int i = 0; i < 2; ++i) rb[wave * red_wave + (i * T + 2 * kq + m) * 16 + nl] = acc[i][m];
    cur = nxt;
    u += stride;
    ++slot_r;
    if (slot_r < p.batch && r + 1 < rounds) continue;
    // A join of the waves every `batch` rounds: in between they run apart, so that a
    // wave whose loads come late holds nobody up. Two batches of sums: one barrier.
    lds_barrier();
    // h of two neighbouring tiles: one scale block of 32 values per half wave
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
      const float v = g / (1.0f + expf(-g)) * uu;
      // rounded to bf16, as the down product's activations are (NaN stays NaN)
      const float h = v != v ? v : __uint_as_float(bf16_rne_bits(v) << 16);
      float amax = finite_abs(h);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
      const uint32_t ef = block_exponent(amax);
      uint32_t hi, lo;
      split2(h, h, block_factor(ef), hi, lo);
      if (slot != 0xff) {
        const int b = j / 2;
        const int place = 32 * (p.down_spl == 2 ? chunk_place<2>(b) : b) + code_slot(c, p.down_spl == 0);
        uint8_t* hq = p.hq + static_cast<int64_t>(t * topk + slot) * 2 * p.I + place;
        hq[0] = static_cast<uint8_t>(hi);
        hq[p.I] = static_cast<uint8_t>(lo);
        if (c < 2) p.hs[(static_cast<int64_t>(t * topk + slot) * 2 + c) * (p.I / 32) + b] =
            static_cast<uint8_t>(ef - (c ? 11u : 7u));
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
  const uint8_t* hq;       // [pair][2][I]
  const uint8_t* hs;       // [pair][2][I / 32]
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
  int wave_bytes, hstride, sstride, sum, total;
};
__host__ __device__ inline LayerDownLds layer_down_lds(int T, int I, int spl, int ks) {
  LayerDownLds L;
  const int nmacro = I / (spl * 128);
  const int kp = (nmacro + ks - 1) / ks * spl * 128;             // K values of a part
  L.hstride = kp + 16;
  L.sstride = ((kp / 32 + 15) & ~15) + 16;
  L.wave_bytes = 2 * L.hstride + 2 * L.sstride;
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

// An item's h halves and block scales on their way into the wave's LDS: the first
// 6 KB (a part of 3 K values) wait in registers, so that they are loaded before the
// codes of their item; longer parts load the rest at the store.
template <int SPL>
struct DownActs {
  static constexpr int R = 6;
  u32x4 v[R];
  uint32_t sv;
  // 16-byte chunk i of the part's two half rows (n chunks each)
  static __device__ __forceinline__ const uint8_t* chunk(const LayerDownParams& p, const DownItem& q, int i, int n) {
    const int pc = i < n ? 0 : 1;
    return p.hq + (static_cast<int64_t>(q.pair) * 2 + pc) * p.I + q.tb * SPL * 128 + 16 * (i - pc * n);
  }
  static __device__ __forceinline__ int place(const LayerDownLds& L, int i, int n) {
    return i < n ? 16 * i : L.hstride + 16 * (i - n);
  }
  // dword i of the part's scales (m a row)
  static __device__ __forceinline__ const uint8_t* scale(const LayerDownParams& p, const DownItem& q, int i, int m) {
    const int pc = i < m ? 0 : 1;
    return p.hs + (static_cast<int64_t>(q.pair) * 2 + pc) * (p.I / 32) + q.tb * SPL * 4 + 4 * (i - pc * m);
  }
  __device__ __forceinline__ void load(const LayerDownParams& p, const DownItem& q, int lane) {
    const int n = (q.te - q.tb) * SPL * 8;
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = *reinterpret_cast<const u32x4*>(chunk(p, q, min(64 * r + lane, 2 * n - 1), n));
    sv = *reinterpret_cast<const uint32_t*>(scale(p, q, min(lane, n / 4 - 1), n / 8));
  }
  __device__ __forceinline__ void store(const LayerDownParams& p, const DownItem& q, uint8_t* hreg, uint8_t* sreg,
                                        const LayerDownLds& L, int lane) const {
    const int n = (q.te - q.tb) * SPL * 8, m = n / 8;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (64 * r + lane < 2 * n) *reinterpret_cast<u32x4*>(hreg + place(L, 64 * r + lane, n)) = v[r];
    for (int i = 64 * R + lane; i < 2 * n; i += 64)
      *reinterpret_cast<u32x4*>(hreg + place(L, i, n)) = *reinterpret_cast<const u32x4*>(chunk(p, q, i, n));
    if (lane < 2 * m) *reinterpret_cast<uint32_t*>(sreg + (lane < m ? 4 * lane : L.sstride + 4 * (lane - m))) = sv;
    for (int i = 64 + lane; i < 2 * m; i += 64)
      *reinterpret_cast<uint32_t*>(sreg + (i < m ? 4 * i : L.sstride + 4 * (i - m))) =
          *reinterpret_cast<const uint32_t*>(scale(p, q, i, m));
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
  uint8_t* sreg = hreg + 2 * L.hstride;
  float* sums = reinterpret_cast<float*>(smem + L.sum) + wave * p.T * 32;
  for (int i = lane; i < p.T * 32; i += 64) sums[i] = 0.0f;
  wave_lds_order();
  const int n0 = static_cast<int>(blockIdx.x) * p.rows;
  const int rows = min(p.rows, p.H - n0);
  const int items = p.rec[0] * p.ks;
  const int nmacro = p.I / (SPL * 128);
  const uint32_t row_bytes = static_cast<uint32_t>(p.I * F::kBits / 8);
  // a row of each tile (past the workgroup's rows: its last one, whose sums are not used)
  auto lane_offsets = [&](int row, int quarter, int piece, uint32_t* vc, uint32_t* vs) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = min(i * p.rt + min(row, p.rt - 1), rows - 1);
      vc[i] = r * row_bytes + quarter * piece;
      vs[i] = static_cast<uint32_t>(r * p.gpr * 4);
    }
  };
  uint32_t vcode[NT], vscale[NT];
  lane_offsets(lane >> 2, lane & 3, F::kPiece, vcode, vscale);
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
    DownActs<SPL> hst;
    Item q = item_of(it);
    CodeSrc cur = source(q);
    hst.load(p, q, lane);
    __builtin_amdgcn_sched_barrier(0);
    st.issue_scales(cur, vscale, p.groups, lane, [&](int i) { return min(q.tb + i, q.te - 1); });
    [&]<int... U>(std::integer_sequence<int, U...>) {
      (st.template issue<U>(cur, vcode, min(q.tb + U, q.te - 1)), ...);
    }(std::make_integer_sequence<int, PM>{});
    const uint8_t* xr = hreg + (nl == 1 ? L.hstride : 0);   // row 0: hi, row 1: lo
    const uint8_t* sr = sreg + (nl == 1 ? L.sstride : 0);
    for (; it < items; it += kLayerWaves) {
      hst.store(p, q, hreg, sreg, L, lane);    // the part's h into this wave's LDS
      wave_lds_order();
      const Item qn = item_of(it + kLayerWaves);
      const CodeSrc nxt = source(qn);
      const float w = p.weights[q.pair];
      hst.load(p, qn, lane);                   // ahead of the next item's codes
      float acc[NT][2] = {};
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
               uint32_t w4[NT][F::W];
               float s[NT];
#pragma unroll
               for (int i = 0; i < NT; ++i)
#pragma unroll
                 for (int d = 0; d < Stream::DW; ++d) asm volatile("" : "+v"(st.cb[U][i][d]));
               uint32_t sh[NT];
               st.template take<U>(nl, kq, w4, s, sh);
               if constexpr (F::kWide) {
                 wide_step<F::kBits, NT>(w4, s, sh, xr, sr, t0 + U - q.tb, kq, acc);
               } else {
                 layer_step<SPL, NT, 0>(w4, s, xr, sr, t0 + U - q.tb, kq, acc, bad);
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
          lane_offsets(nl, kq, F::kPiece, vc, vs);
          const int back = q.tb * SPL * 128;     // (steps count from the part's first in LDS)
          layer_extra<SPL, NT>(cur, shp, vc, vs, q.tb, q.te, 1, p.groups, xr - back, sr - q.tb * SPL * 4, kq, acc);
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

// K parts of kernel 2: enough items for every wave, and a part's h in LDS.
int layer_down_parts(int T, int topk, int I, int spl) {
  const int nmacro = I / (spl * 128);
  const int jobs = T * topk;
  int ks = 1;
  while (ks < nmacro && (jobs * ks < kLayerWaves || layer_down_lds(T, I, spl, ks).total > kLayerLds)) ks *= 2;
  return std::min(ks, nmacro);
}

}  // namespace

// One run of the two kernels: 2- to 4-bit codes, up to eight tokens, and activations,
// lists and partial sums in one compute unit's LDS.
static bool layer_fits(int64_t T, int topk, int E, int64_t H, int64_t I, int up_bits, int up_group, int dn_bits,
                       int dn_group) {
  if (up_bits < 2 || up_bits > 4 || dn_bits < 2 || dn_bits > 4) return false;
  if (T < 1 || T > kLayerMaxT || E > kLayerMaxE || topk > kRouterMaxTopk) return false;
  if (H > 65536 || I > 65536 || (I + 16) * (H * up_bits / 8) >= (int64_t{1} << 32)) return false;   // 32-bit tile offsets
  if (layer_up_lds(static_cast<int>(T), topk, static_cast<int>(H), 1).total > kLayerLds) return false;
  const int spl = layer_spl(dn_bits, dn_group);
  const int ks = layer_down_parts(static_cast<int>(T), topk, static_cast<int>(I), spl);
  return layer_down_lds(static_cast<int>(T), static_cast<int>(I), spl, ks).total <= kLayerLds;
}

// Tokens of one run of the two kernels; 0: the composed path. Nine to 64 tokens take
// runs of up to eight: an expert that tokens of several runs share is read again, but at
// twice the composed path's rate or more (2-bit codes, 2048 x 1024, top-8 of 128, 16
// tokens: 80 against 158 us, 64: 302 against 433; 7168 x 3 K, top-16 of 128, 64 tokens:
// 2.28 against 2.61 ms; 4 bits, 2048 x 1024, top-4 of 32, 64 tokens: 347 against 506).
// The composed path is ahead where many pairs of 2-bit codes share an expert (2048 x 1024,
// top-4 of 16: 40 tokens 128 against 128 us, 64 tokens 200 against 191), and with weights
// below 4 MB, where the launches count, not the rate (16 tokens, 512 x 256, top-2 of 8: 40
// against 33 us).
int64_t moe_layer_tokens(int64_t T, int topk, int E, int64_t H, int64_t I, int up_bits, int up_group, int dn_bits,
                         int dn_group) {
  if (T < 1 || T > 8 * kLayerMaxT) return 0;
  const int64_t runs = (T + kLayerMaxT - 1) / kLayerMaxT, n = (T + runs - 1) / runs;
  if (!layer_fits(n, topk, E, H, I, up_bits, up_group, dn_bits, dn_group)) return 0;
  if (up_bits == 2 && runs > 4 && T * topk > 10 * static_cast<int64_t>(E)) return 0;
  if (runs > 1 && 3 * H * I * up_bits / 8 * std::min<int64_t>(E, T * topk) < (int64_t{4} << 20)) return 0;
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
  const int nmacro = H / (spl * 128);
  p.down_spl = dn.bits == 2 ? dspl : 0;
  p.ids = b.ids;
  p.weights = b.weights;
  p.ids_user = ids_user;
  p.weights_user = weights_user;
  p.rec = b.rec;
  p.hq = b.hq;
  p.hs = b.hs;
  const int teams = kLayerWaves / layer_up_max_parts(nmacro);    // at least
  const int64_t units = static_cast<int64_t>(std::min(r.E, T * r.topk)) * (I / 16);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(cus, (units + teams - 1) / teams));
  p.share = 1.0f / (static_cast<float>(grid) * kLayerWaves);
  p.batch = 4;
  while (p.batch > 1 && layer_up_lds(T, r.topk, H, p.batch).total > kLayerLds) --p.batch;
  const int lds = layer_up_lds(T, r.topk, H, p.batch).total;
  hipError_t e;
  const bool few = r.E <= 256;                 // a router wave with 4 experts a lane, or 16
  auto up_kernel = [&](auto f_c, auto pm_c) {
    using F = decltype(f_c);
    constexpr int PM = decltype(pm_c)::value;
    return few ? launch_layer(k_layer_up<F, PM, 4>, grid, lds, p, st) : launch_layer(k_layer_up<F, PM, 16>, grid, lds, p, st);
  };
  using I2 = std::integral_constant<int, 2>;   // (more spill)
  using I4 = std::integral_constant<int, 4>;
  using I8 = std::integral_constant<int, 8>;
  if (up.bits == 2) {
    e = spl == 2 ? up_kernel(Codes2<2>{}, I4{}) : up_kernel(Codes2<1>{}, I8{});
  } else {
    e = up.bits == 3 ? up_kernel(CodesWide<3>{}, I2{}) : up_kernel(CodesWide<4>{}, I2{});
  }
  if (e != hipSuccess) return e;

  LayerDownParams d{};
  d.rec = b.rec;
  d.weights = b.weights;
  d.T = T;
  d.topk = r.topk;
  d.hq = b.hq;
  d.hs = b.hs;
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
