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
// the chain of dependent steps, so the cut is found by counting: a bisection
// over the ordered key bits, one ballot and one scalar population count per
// register and probe, that stops as soon as at least topk and at most
// topk + 16 keys lie above the probe. The candidates then take one
// lane each: their fp64 keys are evaluated side by side, and each lane counts
// the candidates ahead of its own.
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

__device__ __forceinline__ float wave_max_f(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
template <class F>
__device__ __forceinline__ F wave_sum_f(F v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// Expert lane * per + i of token t, as fp32; experts that are never taken
// (NaN or -inf logits, NaN or -inf biases) come back as -inf, +inf as FLT_MAX.
__device__ __forceinline__ float router_logit(const RouterParams& p, int64_t t, int e) {
  const int64_t at = t * p.E + e;
  float l;
  if (p.dtype == 0) {
    l = static_cast<const float*>(p.logits)[at];
  } else {
    const uint16_t h = static_cast<const uint16_t*>(p.logits)[at];
    l = p.dtype == 1 ? bf16_to_f32(h) : static_cast<float>(__builtin_bit_cast(_Float16, h));
  }
  if (!(l > -__builtin_inff())) return -__builtin_inff();         // NaN, -inf
  return fminf(l, 3.4028234663852886e38f) + 0.0f;                 // -0 as +0
}
__device__ __forceinline__ float router_bias(const RouterParams& p, int e) {
  const float b = p.bias[e];
  return b > -__builtin_inff() ? fminf(b, 3.4028234663852886e38f) : -__builtin_inff();   // NaN as -inf
}

// The router of token t on one wave, EPL experts per lane (E <= 64 EPL; lane l
// holds the consecutive experts l per .. l per + per - 1, per = ceil(E / 64), so
// that lower lanes hold lower indices). cand: 64 dwords of LDS of this wave.
// Lane j < topk returns slot j: id (-1: no expert left) and weight. Every lane
// of the wave has to call it.
template <int EPL>
__device__ __forceinline__ void wave_topk(const RouterParams& p, int64_t t, int lane, uint32_t* cand, int* id_out,
                                          float* w_out) {
  const int per = (p.E + 63) >> 6;
  const int e0 = lane * per;
  const int k = p.topk;
  float l[EPL];
  uint32_t key[EPL];                           // ordered key; 0: not there or never taken
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = i < per && e0 + i < p.E ? router_logit(p, t, e0 + i) : -__builtin_inff();
  float lmax = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < EPL; ++i) lmax = fmaxf(lmax, l[i]);
  lmax = wave_max_f(lmax);
  // softmax denominators: in fp64 where biased keys are compared, else in fp32
  double total64 = 0.0;
  float total = 0.0f;
  if (!p.sigmoid && lmax > -__builtin_inff()) {
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i < per && l[i] > -__builtin_inff()) total64 += exp(static_cast<double>(l[i]) - static_cast<double>(lmax));
      total64 = wave_sum_f(total64);
      total = static_cast<float>(total64);
    } else if (!p.renorm) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) total += l[i] > -__builtin_inff() ? expf(l[i] - lmax) : 0.0f;
      total = wave_sum_f(total);
    }
  }
  uint32_t kmax = 0u;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float f = l[i];
    if (p.bias && i < per && f > -__builtin_inff()) {
      const float b = router_bias(p, e0 + i);
      const float pr = p.sigmoid ? 1.0f / (1.0f + expf(-f)) : expf(f - lmax) / total;
      if (b > -__builtin_inff()) {
        f = pr + b;
      } else {
        f = l[i] = -__builtin_inff();
      }
    }
    key[i] = f > -__builtin_inff() ? order_bits(f) : 0u;
    kmax = key[i] > kmax ? key[i] : kmax;
  }
  auto count_ge = [&](uint32_t thr) {          // wave-uniform
    int n = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) n += __popcll(__ballot(key[i] >= thr));
    return n;
  };
  // An fp32 biased key is off by less than 2^-20 (1 + |key|): the score by a few
  // of its ulps (<= 2^-21), the sum by half an ulp. Keys of the definition's top k
  // lie at most two such errors below a cut that k fp32 keys reach.
  auto lower = [&](uint32_t cut) {
    if (!p.bias) return cut;
    const float v = order_value(cut);
    const float m = v - 0x1p-18f * (1.0f + fabsf(v));
    return m > -__builtin_inff() ? order_bits(m) : 1u;
  };
  const int live = count_ge(1u);
  uint32_t cut = 1u;                           // every live key
  int n = live;
  bool many = false;
  const int limit = k + 16 < 64 ? k + 16 : 64;   // a probe costs about as much as ranking a few candidates
  if (live > limit) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const uint32_t u = __shfl_xor(kmax, o, 64);
      kmax = u > kmax ? u : kmax;
    }
    // count(lo) >= k > count(hi) throughout; stop once the candidates fit the lanes
    uint32_t lo = 1u, hi = kmax + 1u;
    while (n > limit && hi - lo > 1u) {
      const uint32_t mid = lo + ((hi - lo) >> 1);
      const int c = count_ge(mid);
      if (c >= k) {
        lo = mid;
        cut = lower(lo);
        n = p.bias ? count_ge(cut) : c;
      } else {
        hi = mid;
      }
    }
    many = n > 64;                             // ties (or near ties of biased keys) at the cut
    if (many && !p.bias) {
      // more than 64 keys reach lo, the k-th key itself: the fewer than k above it,
      // and the lowest indices at it up to 64
      cut = lo;
    }
  }
  int ec = -1;                                 // this lane's candidate
  if (!many || !p.bias) {
    // candidates by ascending index; of more than 64 (unbiased ties) those above
    // the cut first
    int base = 0;
    const int above = many ? count_ge(cut + 1u) : 0;
    int tie_base = above;
    // positions count lane by lane, register by register: a candidate's place is
    // the number of candidates in lower lanes, then in lower registers of its own
    int mine = 0, mine_tie = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool in = many ? key[i] > cut : key[i] >= cut;
      mine += in;
      mine_tie += many && key[i] == cut;
    }
    // exclusive prefix over lanes
    int pre = mine, pre_tie = mine_tie;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(pre, o), v = __shfl_up(pre_tie, o);
      if (lane >= o) { pre += u; pre_tie += v; }
    }
    base = pre - mine;
    tie_base += pre_tie - mine_tie;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool in = many ? key[i] > cut : key[i] >= cut;
      if (in && key[i] != 0u) {
        if (base < 64) cand[base] = static_cast<uint32_t>(e0 + i);
        ++base;
      } else if (many && key[i] == cut) {
        if (tie_base < 64) cand[tie_base] = static_cast<uint32_t>(e0 + i);
        ++tie_base;
      }
    }
    wave_lds_order();
    if (many) n = 64;
    if (lane < n) ec = static_cast<int>(cand[lane]);
    wave_lds_order();
  } else {
    // More than 64 biased keys within the fp32 error of the cut: k rounds of a
    // wave-wide maximum over fp64 keys (rare, and slow).
    uint32_t taken = 0u;
    n = k;                                     // live > 64 >= k
    for (int j = 0; j < k; ++j) {
      double best = -__builtin_inf();
      int be = INT32_MAX;
#pragma unroll 1
      for (int i = 0; i < EPL; ++i) {
        const int e = e0 + i;
        if (i >= per || e >= p.E || ((taken >> i) & 1u)) continue;
        const float f = router_logit(p, t, e);
        const float b = router_bias(p, e);
        if (!(f > -__builtin_inff()) || !(b > -__builtin_inff())) continue;
        const double pr = p.sigmoid ? sigmoid64(f)
                                    : exp(static_cast<double>(f) - static_cast<double>(lmax)) / total64;
        const double v = pr + static_cast<double>(b);
        if (v > best || be == INT32_MAX) { best = v; be = e; }
      }
      double wb = best;
      int we = be;
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) {
        const double v = __shfl_xor(wb, o, 64);
        const int e = __shfl_xor(we, o, 64);
        if (e != INT32_MAX && (we == INT32_MAX || v > wb || (v == wb && e < we))) { wb = v; we = e; }
      }
      if (we == be && be != INT32_MAX) taken |= 1u << (be - e0);
      if (lane == j) ec = we;
    }
  }
  // one candidate per lane: its logit, score and key
  const float lc = ec >= 0 ? router_logit(p, t, ec) : -__builtin_inff();
  double pc = 0.0, kc = -__builtin_inf();
  if (ec >= 0) {
    if (p.sigmoid) {
      pc = sigmoid64(lc);
    } else {
      pc = exp(static_cast<double>(lc) - static_cast<double>(lmax));
      if (p.bias) {
        pc /= total64;
      } else if (!p.renorm) {
        pc /= static_cast<double>(total);
      }
    }
    kc = p.bias ? pc + static_cast<double>(router_bias(p, ec)) : static_cast<double>(lc);
  }
  // rank: candidates with a larger key, or an equal one at a lower index
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t kb = __builtin_bit_cast(uint64_t, kc);
    const uint32_t klo = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(kb)), j);
    const uint32_t khi = __builtin_amdgcn_readlane(static_cast<int>(kb >> 32), j);
    const double kj = __builtin_bit_cast(double, (static_cast<uint64_t>(khi) << 32) | klo);
    const int ej = __builtin_amdgcn_readlane(ec, j);
    rank += (kj > kc || (kj == kc && ej < ec)) ? 1 : 0;
  }
  const bool win = ec >= 0 && rank < k;
  double sum = 1.0;
  if (p.renorm) {
    sum = wave_sum_f(win ? pc : 0.0);
    if (!(sum > 0.0)) sum = 1.0;               // every taken score is zero: weights zero
  }
  const float wc = static_cast<float>(pc / sum * static_cast<double>(p.scale));
  // slot rank -> lane rank
  const int taken_n = n < k ? n : k;
  if (win) cand[rank] = static_cast<uint32_t>(lane);
  wave_lds_order();
  const int src = lane < taken_n ? static_cast<int>(cand[lane]) : lane;
  const int id = __shfl(ec, src, 64);
  const float w = __shfl(wc, src, 64);
  *id_out = lane < taken_n ? id : -1;
  *w_out = lane < taken_n ? w : 0.0f;
  wave_lds_order();
}

}  // namespace cubic
