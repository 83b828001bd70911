// router.h -- one token's router on one wave: scores of its logits, the top
// experts and their weights (cubic_moe_topk; the few-token layer runs the same
// code in its first kernel).
//
//   p_e = softmax(l)_e or 1 / (1 + exp(-l_e));  key_e = p_e + bias_e, or l_e
//   without a bias (both scores are increasing in l); the topk largest keys,
//   ties to the lowest index;  w = p [/ sum of the taken p] * scale.
//
// Whole numbers come out, so the order has to be the definition's, not that of
// rounded keys: logits compare exactly as fp32 numbers, and biased keys are
// only narrowed down in fp32 (candidates whose fp32 key lies within its error
// bound of the cut) and then compared in fp64. What bounds a single token is
// the chain of dependent steps, so the cut is found by counting (ballots and
// scalar population counts in a bisection over the ordered key bits), the
// candidates above it take one lane each, their fp64 keys are evaluated side by
// side, and each lane counts the candidates ahead of its own. All loads are issued
// before the first value is used.
//
// Measured: one token, 896 experts, biased sigmoids: 4.9 us as a kernel of its own (an
// empty launch takes 1.7; with the loads issued one after another it took 16); 4096
// tokens 11.5 us (15 MB: 3 us at the copy rate; the fp32 keys and counts of 16 experts a
// lane bound it, 32 us in the first version).
#pragma once
#include "common.h"

namespace cubic {

struct RouterParams {
  const void* logits;      // [T][E]: fp32 (dtype 0), bf16 (1) or fp16 (2)
  const float* bias;       // [E] or NULL
  int dtype;
  int E, topk;
  int sigmoid;             // 0: softmax
  int renorm;
  float scale;
};

constexpr int kRouterMaxTopk = 64;       // one lane per taken expert

// Ascending unsigned order of fp32 values (no NaN).
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o >> 31) ? (o ^ 0x80000000u) : ~o);
}

// Reductions over the 64 lanes that end in every lane, in a fixed order: within
// each row of 16 lanes by DPP (quad swaps, half-row mirror, row mirror), then the
// four rows' results by readlane.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, Op op) {
  auto each_dword = [](T x, auto f) {
    if constexpr (sizeof(T) == 4) {
      return __builtin_bit_cast(T, f(__builtin_bit_cast(uint32_t, x)));
    } else {
      const uint64_t b = __builtin_bit_cast(uint64_t, x);
      const uint64_t lo = f(static_cast<uint32_t>(b)), hi = f(static_cast<uint32_t>(b >> 32));
      return __builtin_bit_cast(T, lo | (hi << 32));
    }
  };
  v = op(v, each_dword(v, [](uint32_t x) { return dpp_move<0xB1>(x); }));    // quad_perm [1, 0, 3, 2]
  v = op(v, each_dword(v, [](uint32_t x) { return dpp_move<0x4E>(x); }));    // quad_perm [2, 3, 0, 1]
  v = op(v, each_dword(v, [](uint32_t x) { return dpp_move<0x141>(x); }));   // row_half_mirror
  v = op(v, each_dword(v, [](uint32_t x) { return dpp_move<0x140>(x); }));   // row_mirror
  T r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    r[k] = each_dword(v, [k](uint32_t x) {
      return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), 16 * k));
    });
  return op(op(r[0], r[1]), op(r[2], r[3]));
}

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// A logit or bias as the router reads it: experts that are never taken (NaN,
// -inf) as -inf, +inf as FLT_MAX, -0 as +0.
__device__ __forceinline__ float router_value(float v) {
  return v > -__builtin_inff() ? fminf(v, 3.4028234663852886e38f) + 0.0f : -__builtin_inff();
}
__device__ __forceinline__ float router_logit(const RouterParams& p, int64_t at) {
  float l;
  if (p.dtype == 0) {
    l = static_cast<const float*>(p.logits)[at];
  } else {
    const uint16_t h = static_cast<const uint16_t*>(p.logits)[at];
    l = p.dtype == 1 ? bf16_to_f32(h) : static_cast<float>(__builtin_bit_cast(_Float16, h));
  }
  return router_value(l);
}

// The router of token t on one wave, EPL experts per lane (E <= 64 EPL; lane l,
// register i: expert 64 i + l). cand: 64 dwords of LDS of this wave. out(slot, id,
// weight) is called once for every slot 0 .. topk - 1, each by some lane (id -1: no
// expert left). Every lane of the wave has to call it.
template <int EPL, class Out>
__device__ __forceinline__ void wave_topk(const RouterParams& p, int64_t t, int lane, uint32_t* cand, Out&& out) {
  const int k = p.topk, E = p.E;
  const int64_t row = t * E;
  float l[EPL], b[EPL];
  // every load first, indices clamped
  if (p.dtype == 0) {
    const float* src = static_cast<const float*>(p.logits) + row;
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = src[min(64 * i + lane, E - 1)];
  } else {
    const uint16_t* src = static_cast<const uint16_t*>(p.logits) + row;
    uint16_t h[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) h[i] = src[min(64 * i + lane, E - 1)];
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      l[i] = p.dtype == 1 ? bf16_to_f32(h[i]) : static_cast<float>(__builtin_bit_cast(_Float16, h[i]));
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) b[i] = p.bias[min(64 * i + lane, E - 1)];
  }
  float lmax = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    l[i] = 64 * i + lane < E ? router_value(l[i]) : -__builtin_inff();
    lmax = fmaxf(lmax, l[i]);
  }
  // The softmax's denominator, where a key or a weight needs it.
  double total = 1.0;
  if (!p.sigmoid) {
    lmax = wave_reduce(lmax, [](float x, float y) { return fmaxf(x, y); });
    if (lmax > -__builtin_inff() && (p.bias || !p.renorm)) {
      total = 0.0;
      // four exponentials side by side: one by one they follow each other (one token of 896
      // experts: 7.9 us; this way 5.8, and 5.3 with a sum in fp32)
#pragma unroll
      for (int i0 = 0; i0 < EPL; i0 += 4) {
        if (64 * i0 < E) {
          double e4[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) e4[u] = exp(static_cast<double>(l[i0 + u]) - static_cast<double>(lmax));
          total += (e4[0] + e4[1]) + (e4[2] + e4[3]);
        }
      }
      total = wave_reduce(total, [](double x, double y) { return x + y; });
    }
  }
  uint32_t key[EPL];                           // ordered key; 0: not there or never taken
  uint32_t kmax = 0u;
  if (p.bias) {
    const float rt = 1.0f / static_cast<float>(total);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float bi = router_value(b[i]);
      const float ex = __expf(p.sigmoid ? -l[i] : l[i] - lmax);
      const float f = (p.sigmoid ? __builtin_amdgcn_rcpf(1.0f + ex) : ex * rt) + bi;
      key[i] = l[i] > -__builtin_inff() && bi > -__builtin_inff() ? order_bits(f) : 0u;
      kmax = max(kmax, key[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = l[i] > -__builtin_inff() ? order_bits(l[i]) : 0u;
      kmax = max(kmax, key[i]);
    }
  }
  auto count_ge = [&](uint32_t thr) {          // wave-uniform
    int n = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) n += __popcll(__ballot(key[i] >= thr));
    return n;
  };
  // An fp32 biased key is off by less than 2^-20 (1 + |key|): the score (hardware
  // exponential and reciprocal, the argument's rounding: below 2^-20 of a score
  // that is at most 1) and half an ulp of the sum. Keys of the definition's top k
  // lie at most two such errors below a cut that k fp32 keys reach.
  auto lower = [&](uint32_t cut) {
    const float v = order_value(cut);
    const float m = v - 0x1p-18f * (1.0f + fabsf(v));
    return m > -__builtin_inff() ? order_bits(m) : 1u;
  };
  // The cut: first the k-th largest of the lanes' largest keys, found by bisection
  // on one register (k lanes reach it, so at least k keys do, and few more where
  // large keys are spread over the lanes); only where more than 64 keys reach it,
  // a bisection that counts all keys.
  uint32_t cut = 1u;                           // every live key
  int n = count_ge(1u);
  bool many = false;
  const int limit = k + 8 < 64 ? k + 8 : 64;
  if (n > limit) {
    uint32_t lo = 1u;
    const uint32_t top = wave_reduce(kmax, [](uint32_t x, uint32_t y) { return max(x, y); }) + 1u;
    uint32_t hi = top;
    if (__popcll(__ballot(kmax != 0u)) >= k) {
      lo = wave_reduce(kmax, [](uint32_t x, uint32_t y) { return min(x, y); });
      lo = lo ? lo : 1u;
      while (hi - lo > 1u) {
        const uint32_t mid = lo + ((hi - lo) >> 1);
        const int c = __popcll(__ballot(kmax >= mid));
        if (c >= k) {
          lo = mid;
          if (c == k) break;
        } else {
          hi = mid;
        }
      }
      n = count_ge(lo);
    }
    cut = p.bias ? lower(lo) : lo;
    if (p.bias) n = count_ge(cut);
    hi = top;
    // count(lo) >= k > count(hi) throughout
    while (n > 64 && hi - lo > 1u) {
      const uint32_t mid = lo + ((hi - lo) >> 1);
      const int c = count_ge(mid);
      if (c >= k) {
        lo = mid;
        cut = p.bias ? lower(lo) : lo;
        n = p.bias ? count_ge(cut) : c;
      } else {
        hi = mid;
      }
    }
    many = n > 64;                             // ties (or near ties of biased keys) at the cut
  }
  int ec = -1;                                 // this lane's candidate
  if (!many) {
    int base = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool in = key[i] >= cut;
      const uint64_t m = __ballot(in);
      const int at = base + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32),
                                                      __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0));
      if (in) cand[at] = static_cast<uint32_t>(64 * i + lane);
      base += __popcll(m);
    }
    wave_lds_order();
    if (lane < n) ec = static_cast<int>(cand[lane]);
  } else {
    // More than 64 keys tie at the cut (or lie within the fp32 error of it): k rounds
    // of a wave-wide maximum over exact keys (rare, and slow).
    uint32_t taken = 0u;
    n = k;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
      double best = -__builtin_inf();
      int be = INT32_MAX;
#pragma unroll 1
      for (int i = 0; 64 * i < E; ++i) {
        const int e = 64 * i + lane;
        if (e >= E || ((taken >> i) & 1u)) continue;
        const float f = router_logit(p, row + e);
        if (!(f > -__builtin_inff())) continue;
        double v = static_cast<double>(f);
        if (p.bias) {
          const float bi = router_value(p.bias[e]);
          if (!(bi > -__builtin_inff())) continue;
          v = (p.sigmoid ? sigmoid64(f) : exp(v - static_cast<double>(lmax)) / total) + static_cast<double>(bi);
        }
        if (v > best || be == INT32_MAX) { best = v; be = e; }
      }
      double wb = best;
      int we = be;
#pragma unroll 1
      for (int o = 32; o >= 1; o >>= 1) {
        const double v = __shfl_xor(wb, o, 64);
        const int e = __shfl_xor(we, o, 64);
        if (e != INT32_MAX && (we == INT32_MAX || v > wb || (v == wb && e < we))) { wb = v; we = e; }
      }
      if (we == be && be != INT32_MAX) taken |= 1u << (be >> 6);
      if (lane == j) ec = we;
    }
  }
  // one candidate per lane: its score and key in fp64
  double pc = 0.0, kc = -__builtin_inf();
  if (ec >= 0) {
    const float lc = router_logit(p, row + ec);
    if (p.sigmoid) {
      pc = sigmoid64(lc);
    } else {
      pc = exp(static_cast<double>(lc) - static_cast<double>(lmax)) / total;
    }
    kc = p.bias ? pc + static_cast<double>(router_value(p.bias[ec])) : static_cast<double>(lc);
  }
  // Rank: candidates with a larger key, or an equal one at a lower index. The
  // candidates lie in index order (the rare path has them in rank order already).
  // Keys are compared as ordered integers; lanes past n hold the smallest one.
  int rank = many ? lane : 0;
  if (!many) {
    const uint64_t kb = __builtin_bit_cast(uint64_t, kc + 0.0);
    const uint64_t ok = ec >= 0 ? kb ^ ((kb >> 63) ? ~uint64_t{0} : uint64_t{1} << 63) : 0u;
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += 8) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = j0 + u;                  // n <= 64: j stays below 64
        const uint32_t jlo = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(ok)), j);
        const uint32_t jhi = __builtin_amdgcn_readlane(static_cast<int>(ok >> 32), j);
        const uint64_t oj = (static_cast<uint64_t>(jhi) << 32) | jlo;
        rank += (oj > ok || (oj == ok && j < lane)) ? 1 : 0;
      }
    }
  }
  const bool win = ec >= 0 && rank < k;
  double sum = 1.0;
  if (p.renorm) {
    sum = wave_reduce(win ? pc : 0.0, [](double x, double y) { return x + y; });
    if (!(sum > 0.0)) sum = 1.0;               // every taken score is zero: weights zero
  }
  if (win) out(rank, ec, static_cast<float>(pc / sum * static_cast<double>(p.scale)));
  if (lane >= n && lane < k) out(lane, -1, 0.0f);
  wave_lds_order();
}

}  // namespace cubic
