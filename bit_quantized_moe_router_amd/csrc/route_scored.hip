// Routing by scores: softmax or sigmoid scores over all experts, a choice
// value score + bias, a choice limited to the best groups of experts, the k
// largest choice values, and the (renormalised, scaled) scores of the selected
// experts as weights; then the same permutation as the other router's.
//
// The pages ("Xolotl" card, README "How it works, in one paragraph") give no
// scoring function; the formulas are those of moe_scoring in include/moe.h.
//
// The selection is a comparison of values that lie arbitrarily close, so the
// choice values are formed and compared in 64 bits: two experts with
// different logits then keep their order unless they agree to about 1e-16,
// which a 32-bit score (steps of 6e-8 below 1) would not give.  The vector
// units run 64-bit multiply-adds at the rate of unpacked 32-bit ones, so this
// costs little (an exponential per expert).  Most rows do not need it for every
// expert: 32-bit values with a bound on their error leave a few candidates,
// which are ordered by their 64-bit values; a row that the bound does not
// settle is done in 64 bits as a whole.
//
// What sets the time is the length of a token's chain of dependent steps, not
// its arithmetic (one wave takes a token; its steps were stamped with the
// clock).  Taking the k largest one after the other, each by a maximum over
// the wave, took 770 cycles a round, 6900 of 19200 for one token at 256
// experts, top-8.  Here all candidates are ranked at once.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "moe_internal.h"
#include "topk_common.h"

namespace bqmoe {

// ------------------------------------------------------------- one token
// Order-preserving 64-bit key of a choice value: NaN gets the lowest key of
// all (1; key 0 marks "not in the choice"), -0 and +0 share one.
__device__ __forceinline__ uint64_t order_key64(double v) {
  if (v != v) return 1ull;
  if (v == 0.0) v = 0.0;  // -0 -> +0
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)(((uint64_t)dpp_u32<CTRL>((uint32_t)(u >> 32)) << 32) |
                                          dpp_u32<CTRL>((uint32_t)u)));
}
// Sum over the 64 lanes, the same in every lane (the pairing of wave_sum_lanes).
__device__ __forceinline__ double wave_sum64(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  uint64_t u = (uint64_t)__double_as_longlong(v);
  auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  auto l = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  v = __longlong_as_double((long long)(((uint64_t)h[0] << 32) | l[0])) +
      __longlong_as_double((long long)(((uint64_t)h[1] << 32) | l[1]));
  u = (uint64_t)__double_as_longlong(v);
  h = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  l = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
  return __longlong_as_double((long long)(((uint64_t)h[0] << 32) | l[0])) +
         __longlong_as_double((long long)(((uint64_t)h[1] << 32) | l[1]));
}
// Maximum of a float over the lanes (no NaN among them).
__device__ __forceinline__ float wave_max_lanes(float v) {
  return key_value(wave_allmax_u32(order_key(v)));
}
__device__ __forceinline__ double readlane_f64(double v, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double(
      (long long)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane)
                   << 32) |
                  (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane)));
}

// The score of a logit: m and inv_sum are the row's maximum and 1 / sum of the
// softmax (unused by the sigmoid).  A logit of -inf scores 0 in either.
__device__ __forceinline__ double score_of(const ScoreArgs& S, float l, double m, double inv_sum) {
  if (l == -INFINITY) return 0.0;
  if (S.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
  return exp((double)l - m) * inv_sum;
}

// The two largest of (a1 >= a2) and (b1 >= b2), into a.
__device__ __forceinline__ void merge_top2(uint64_t& a1, uint64_t& a2, uint64_t b1, uint64_t b2) {
  const uint64_t lo = a1 < b1 ? a1 : b1;
  const uint64_t second = a1 < b1 ? b2 : a2;
  a1 = a1 < b1 ? b1 : a1;
  a2 = lo > second ? lo : second;
}

// The value whose order_key64 is `key` (key 1, NaN's, gives a NaN).
__device__ __forceinline__ double key_value64(uint64_t key) {
  return __longlong_as_double((long long)((key >> 63) ? (key & 0x7FFFFFFFFFFFFFFFull) : ~key));
}

// Largest and second largest over the teams of 1 << log2 lanes, in all of their
// lanes (every step pairs lanes that already agree within their halves).
template <int CTRL>
__device__ __forceinline__ void top2_dpp(float& a1, float& a2) {
  const float b1 = __uint_as_float(dpp_u32<CTRL>(__float_as_uint(a1)));
  const float b2 = __uint_as_float(dpp_u32<CTRL>(__float_as_uint(a2)));
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}
__device__ __forceinline__ void team_top2(float& a1, float& a2, int log2) {
  if (log2 >= 1) top2_dpp<0xB1>(a1, a2);
  if (log2 >= 2) top2_dpp<0x4E>(a1, a2);
  if (log2 >= 3) top2_dpp<0x141>(a1, a2);
  if (log2 >= 4) top2_dpp<0x140>(a1, a2);
  for (int o = 16; o < (1 << log2); o <<= 1) {
    const float b1 = __shfl_xor(a1, o, 64), b2 = __shfl_xor(a2, o, 64);
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
  }
}

// The choice by 32-bit values and their error bound (lane l holds experts
// l + 64 i, lg their logits, bs their biases).  False where the bound does not
// settle it: the caller then takes the whole row in 64 bits.  On true, a lane
// with rank < k holds one selected expert: its place in the order, its id and
// its score (up to the softmax's sum where the weights are renormalised).
//
// Every lane's largest value is its head.  Where m heads are at least t, so are
// m values, and all values from t on, compacted into one lane each, hold the k
// largest (m = k, or k + 1 where values have an error).  t is found by
// bisection over the heads' range, with a ballot a step, until m to m + 4 heads
// are left.  There are k to 4 k candidates as a rule; more than 64 are left to
// the 64-bit path.
//
// Errors: the hardware's exponential and reciprocal are good to one unit in
// the last place (2^-23 relative).  Sigmoid, s <= 1: the exponential's argument
// is off by |l| 2^-24, which s (1 - s) |l| <= 0.23 makes 0.12 * 2^-23, its
// result's unit 0.25 * 2^-23, the sum's rounding and the reciprocal's unit
// 1.5 * 2^-23: less than 2^-22.  Softmax of largest score q: p |ln p/q| <= 0.37 q,
// so 0.6 * 2^-23 q, one unit of the exponential, the sum's (64-bit) and the
// product's: less than q 2^-20.  Adding the bias rounds by 2^-24 of the sum.
// Softmax without a bias is ranked by the logits themselves, which has no
// error; its group values are then sums of exponentials with q = 1.
template <int PER>
__device__ bool choose_32(const ScoreArgs& S, const float (&lg)[PER], const float (&bs)[PER],
                          int lane, float* lds, int& rank, int& my_id, double& my_s) {
  const int E = S.E, k = S.k;
  const bool grouped = S.topk_groups < S.n_groups, by_logit = !S.sigmoid && !S.bias;
  // a NaN or an infinite value takes the 64-bit path
  bool odd = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) odd |= !(lg[i] < INFINITY);
  float mx = 0.f, fast_sum = 1.f;
  double inv_sum = 1.0;
  if (!S.sigmoid) {
    mx = lg[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mx = fmaxf(mx, lg[i]);
    mx = wave_max_lanes(mx);
    if (mx == -INFINITY) return false;
    if (S.bias || !S.renorm) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane + 64 * i < E) s += exp((double)lg[i] - (double)mx);
      inv_sum = 1.0 / wave_sum64(s);
      fast_sum = (float)inv_sum;
    }
  }
  // the choice values; unit: their error's bound
  float c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (S.sigmoid)
      c[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * lg[i]));
    else if (by_logit && !grouped)
      c[i] = lg[i];
    else
      c[i] = __builtin_amdgcn_exp2f(1.4426950408889634f * (lg[i] - mx)) * (S.bias ? fast_sum : 1.f);
    if (S.bias) c[i] += bs[i];
    if (lg[i] == -INFINITY) c[i] = -INFINITY;
    odd |= !(c[i] < INFINITY);
  }
  if (__ballot(odd)) return false;
  const float unit = S.sigmoid ? 0x1p-22f : (S.bias ? fast_sum : 1.f) * 0x1p-20f;
  uint64_t kept = ~0ull;
  if (grouped) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i < E) lds[lane + 64 * i] = c[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int ts = 1 << S.team_log2, g = lane >> S.team_log2, gs = S.group_size;
    float a1 = -INFINITY, a2 = -INFINITY;
    if (g < S.n_groups)
#pragma unroll 4
      for (int i = lane & (ts - 1); i < gs; i += ts) {
        const float v = lds[g * gs + i];
        a2 = fmaxf(a2, fminf(a1, v));
        a1 = fmaxf(a1, v);
      }
    team_top2(a1, a2, S.team_log2);
    const float gv = S.group_top == 1 ? a1 : a1 + a2;
    int better = 0;
    for (int h = 0; h < S.n_groups; ++h) {
      const float o =
          __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gv), h << S.team_log2));
      better += (o > gv || (o == gv && h < g)) ? 1 : 0;
    }
    const bool in = g < S.n_groups && better < S.topk_groups;
    kept = __ballot(in);
    // the worst group in and the best one out have to lie clearly apart
    const uint64_t at_lo = __ballot(g < S.n_groups && better == S.topk_groups - 1);
    const uint64_t at_hi = __ballot(g < S.n_groups && better == S.topk_groups);
    const float lo = __int_as_float(__builtin_amdgcn_readlane(
        __float_as_int(gv), (int)__ffsll((unsigned long long)at_lo) - 1));
    const float hi = __int_as_float(__builtin_amdgcn_readlane(
        __float_as_int(gv), (int)__ffsll((unsigned long long)at_hi) - 1));
    if (!(lo - hi > 4.f * unit + 0x1p-21f * fmaxf(fabsf(lo), fabsf(hi)))) return false;
    __builtin_amdgcn_wave_barrier();  // (the values are read; the area is used again)
  }
  uint32_t key[PER], head = 0u;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    const int ge = (int)(((uint32_t)e * S.group_magic) >> 20);  // e / group_size
    const bool out = e >= E || (grouped && !((kept >> (ge << S.team_log2)) & 1));
    key[i] = out ? 0u : order_key(by_logit ? lg[i] : c[i]);
    head = max(head, key[i]);
  }
  const int m = by_logit ? k : k + 1;
  uint32_t t = ~wave_allmax_u32(head ? ~head : 0u);  // the smallest head
  if (__popcll(__ballot(head != 0u)) < m)
    t = 1u;  // fewer heads than m: every value is a candidate
  else
    for (uint32_t hi = wave_allmax_u32(head) + 1u; hi - t > 1u;) {
      const uint32_t mid = t + ((hi - t) >> 1);
      const int cnt = __popcll(__ballot(head >= mid));
      if (cnt >= m)
        t = mid;
      else
        hi = mid;
      if (cnt >= m && cnt <= m + 4) break;
    }
  t = (uint32_t)__builtin_amdgcn_readfirstlane((int)t);
  // the candidates, compacted: id and logit
  int* const cid = reinterpret_cast<int*>(lds);
  float* const cl = lds + 64;
  int n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint64_t at = __ballot(key[i] >= t);
    const int pos = n + __popcll(at & (lane ? (~0ull >> (64 - lane)) : 0ull));
    if (key[i] >= t && pos < 64) {
      cid[pos] = lane + 64 * i;
      cl[pos] = lg[i];
    }
    n += __popcll(at);
  }
  if (n > 64) return false;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const bool cand = lane < n;
  my_id = cid[cand ? lane : 0];
  const float l = cl[cand ? lane : 0];
  my_s = score_of(S, l, (double)mx, inv_sum);
  rank = 0;
  int same = 0;
  if (by_logit) {
    const uint32_t mine = order_key(l);
    for (int j = 0; j < n; ++j) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)mine, j);
      rank += o > mine ? 1 : 0;
      same += o == mine ? 1 : 0;
    }
  } else {
    const double d = l == -INFINITY ? -INFINITY : my_s + (S.bias ? (double)S.bias[my_id] : 0.0);
    for (int j = 0; j < n; ++j) {
      const double o = readlane_f64(d, j);
      rank += o > d ? 1 : 0;
      same += o == d ? 1 : 0;
    }
    // whatever is no candidate is below t by its 32-bit value: the last one
    // chosen has to lie above that by more than the error
    const double edge = t == 1u ? -INFINITY
                                : (double)key_value(t) + (double)unit +
                                      0x1p-23 * fabs((double)key_value(t));
    if (__ballot(cand && rank < k && !(d > edge)) && t != 1u) return false;
  }
  if (__ballot(cand && same > 1)) {  // equal values: the lower index first
    const float v = by_logit ? l : 0.f;
    const double d =
        by_logit ? 0.0
                 : l == -INFINITY ? -INFINITY : my_s + (S.bias ? (double)S.bias[my_id] : 0.0);
    for (int j = 0; j < n; ++j) {
      const int oi = __builtin_amdgcn_readlane(my_id, j);
      const bool eq = by_logit ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j)) == v
                               : readlane_f64(d, j) == d;
      rank += eq && oi < my_id ? 1 : 0;
    }
  }
  if (!cand) rank = 64;
  if (by_logit) {
    // 64-bit scores that run out at 0 are ties, which logits are not
    if (__ballot(rank < k && !(l - mx > -700.f))) return false;
    // a logit of 2^-18 or more is 2^-42 from any other, which l - mx > -700
    // keeps in 64 bits; smaller ones may have one score for two logits
    if (__ballot(rank < k && fabsf(l) < 0x1p-18f)) {
      int small = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        small += __popcll(__ballot(lane + 64 * i < E && fabsf(lg[i]) < 0x1p-18f));
      if (small > 1) return false;
    }
  }
  return true;
}

template <int PER>
__device__ void choose_64(const ScoreArgs& S, const float (&lg)[PER],
                          const float* __restrict__ L, int lane, uint64_t* stage, int& my_id,
                          double& my_s);

// One token by one wave: a lane with rank < k returns one selected expert, its
// place in the order and its weight.  `stage` is max(E, 64) * 8 bytes of LDS of
// the wave's own.
template <int PER>
__device__ __forceinline__ void wave_scored_topk(const ScoreArgs& S, const float* __restrict__ L,
                                                 int lane, uint64_t* stage, int& rank, int& my_id,
                                                 float& my_w) {
  float lg[PER], bs[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    lg[i] = e < S.E ? L[e] : -INFINITY;
  }
  if (S.bias) {
#pragma unroll
    for (int i = 0; i < PER; ++i) bs[i] = S.bias[min(lane + 64 * i, S.E - 1)];
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) bs[i] = 0.f;
  }
  double s;
  __builtin_amdgcn_wave_barrier();  // the last token's staging is read
  if (!choose_32<PER>(S, lg, bs, lane, reinterpret_cast<float*>(stage), rank, my_id, s)) {
    choose_64<PER>(S, lg, L, lane, stage, my_id, s);
    rank = lane;
  }
  if (rank >= S.k) s = 0.0;
  // weights from the scores, without the bias
  if (S.renorm) {
    const double den = wave_sum64(s);
    s = den == 0.0 ? 0.0 : s / den;
  }
  my_w = (float)(s * (double)S.scale);
}

// The whole choice in 64 bits.
template <int PER>
__device__ void choose_64(const ScoreArgs& S, const float (&lg)[PER],
                          const float* __restrict__ L, int lane, uint64_t* stage, int& my_id,
                          double& my_s) {
  const int E = S.E, k = S.k;
  double m = 0.0, inv_sum = 0.0;
  if (!S.sigmoid) {
    float mx = lg[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mx = fmaxf(mx, lg[i]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
    m = (double)mx;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lg[i] != -INFINITY) s += exp((double)lg[i] - m);
    inv_sum = 1.0 / wave_sum64(s);
  }
  uint64_t key[PER];
  int ix[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    ix[i] = e;
    double c = score_of(S, lg[i], m, inv_sum);
    if (S.bias) c += (double)S.bias[e < E ? e : 0];
    if (lg[i] == -INFINITY) c = -INFINITY;  // a masked expert, whatever its bias
    key[i] = e < E ? order_key64(c) : 0ull;
  }
  if (S.topk_groups < S.n_groups) {
    // teams of 64 / 2^ceil(log2 groups) lanes find each group's largest choice values
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i < E) stage[lane + 64 * i] = key[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int ts = 1 << S.team_log2, g = lane >> S.team_log2, gs = S.group_size;
    uint64_t a1 = 0, a2 = 0;
    if (g < S.n_groups)
      for (int i = lane & (ts - 1); i < gs; i += ts) merge_top2(a1, a2, stage[g * gs + i], 0ull);
    for (int o = 1; o < ts; o <<= 1) {
      const uint64_t b1 = __shfl_xor((unsigned long long)a1, o, 64);
      const uint64_t b2 = __shfl_xor((unsigned long long)a2, o, 64);
      merge_top2(a1, a2, b1, b2);
    }
    const uint64_t gv =
        S.group_top == 1 ? a1 : order_key64(key_value64(a1) + key_value64(a2));
    int better = 0;  // groups before this lane's: larger value, or equal and lower index
    for (int h = 0; h < S.n_groups; ++h) {
      const uint64_t o = __shfl((unsigned long long)gv, h << S.team_log2, 64);
      better += (o > gv || (o == gv && h < g)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(g < S.n_groups && better < S.topk_groups);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int ge = (int)(((uint32_t)ix[i] * S.group_magic) >> 20);  // ix / group_size
      if (ix[i] < E && !((kept >> (ge << S.team_log2)) & 1)) key[i] = 0ull;
    }
    __builtin_amdgcn_wave_barrier();
  }
  // each lane sorts its entries (larger key first, indices ascend with i)
#pragma unroll
  for (int p = 0; p < PER; ++p) {
#pragma unroll
    for (int i = p & 1; i + 1 < PER; i += 2) {
      const bool sw = key[i + 1] > key[i] || (key[i + 1] == key[i] && ix[i + 1] < ix[i]);
      const uint64_t ka = key[i], kb = key[i + 1];
      const int ia = ix[i], ib = ix[i + 1];
      key[i] = sw ? kb : ka;
      key[i + 1] = sw ? ka : kb;
      ix[i] = sw ? ib : ia;
      ix[i + 1] = sw ? ia : ib;
    }
  }
  // k rounds: the largest head key, by its upper 32 bits first (one lane
  // usually holds it alone), then its lower ones, then the lowest index
  my_id = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t hi = (uint32_t)(key[0] >> 32), lo = (uint32_t)key[0];
    uint64_t at = __ballot(hi == wave_allmax_u32(hi));
    uint32_t win;
    if (__popcll(at) > 1) {
      const bool in = (at >> lane) & 1;
      const uint32_t lmax = wave_allmax_u32(in ? lo : 0u);
      win = ~wave_allmax_u32(in && lo == lmax ? ~(uint32_t)ix[0] : 0u);
    } else {
      win = (uint32_t)__builtin_amdgcn_readlane(ix[0], (int)__ffsll((unsigned long long)at) - 1);
    }
    const bool pop = (uint32_t)ix[0] == win;
#pragma unroll
    for (int t = 0; t + 1 < PER; ++t) {
      key[t] = pop ? key[t + 1] : key[t];
      ix[t] = pop ? ix[t + 1] : ix[t];
    }
    key[PER - 1] = pop ? 0ull : key[PER - 1];
    my_id = lane == j ? (int)win : my_id;
  }
  my_s = score_of(S, L[my_id], m, inv_sum);
}

// Lanes whose `key` (< 2^bits) equals this lane's, among `active` lanes.
__device__ __forceinline__ uint64_t match_lanes(int key, int bits, uint64_t active) {
  uint64_t peers = active;
  for (int b = 0; b < bits; ++b) {
    const uint64_t m = __ballot((key >> b) & 1);
    peers &= ((key >> b) & 1) ? m : ~m;
  }
  return peers;
}

// Exclusive scan of one value per thread over the block; `tot` holds one int
// per wave, `all` gets the total in every thread.
__device__ __forceinline__ int block_scan(int v, int* tot, int& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(incl, o, 64);
    if (lane >= o) incl += y;
  }
  if (lane == 63) tot[wave] = incl;
  __syncthreads();
  int before = 0, sum = 0;
  for (int w = 0; w < nw; ++w) {
    const int t = tot[w];
    before += w < wave ? t : 0;
    sum += t;
  }
  __syncthreads();
  all = sum;
  return before + incl - v;
}

// The grouped-GEMM tile list (routed experts in id order, then the shared
// expert) from expert tid's row count and offset; every thread of a block of
// at least E calls it.
__device__ __forceinline__ void write_tiles(const ScoreOut& O, int T, int k, int E, int count,
                                            int off, int* tot) {
  const int n = (count + O.tm - 1) / O.tm;
  int ntiles;
  const int first = block_scan(n, tot, ntiles);
  for (int i = 0; i < n; ++i) {
    int32_t* t = O.tiles + 4 * (first + i);
    t[0] = threadIdx.x;
    t[1] = off + i * O.tm;
    t[2] = min(O.tm, count - i * O.tm);
    t[3] = 0;
  }
  const int nsh = O.n_shared ? (T + O.tm - 1) / O.tm : 0;
  for (int i = threadIdx.x; i < nsh; i += blockDim.x) {
    int32_t* t = O.tiles + 4 * (ntiles + i);
    t[0] = -1;
    t[1] = T * k + i * O.tm;
    t[2] = min(O.tm, T - i * O.tm);
    t[3] = 0;
  }
  if (threadIdx.x == 0) O.ctrl[0] = ntiles + nsh;
}

// The decode slot list's header, the shared expert's slot and the empty ones,
// by lane i of a wave (T <= 8).
__device__ __forceinline__ void write_other_slots(const ScoreOut& O, int T, int rows,
                                                  int n_active, int i) {
  const int n_slots = n_active + (O.n_shared ? 1 : 0);
  if (i == 0) O.slots[0] = n_slots;
  if (O.n_shared && i < T) {
    int32_t* rec = O.slots + kSlotRec * (1 + n_active);
    if (i == 0) {
      rec[0] = -1;
      rec[1] = rows;
      rec[2] = T;
      rec[3] = 0;
    }
    rec[kSlotTok + i] = i;
  }
  for (int s = n_slots + i; s < O.max_slots; s += 64)
    for (int j = 0; j < kSlotTok; ++j) O.slots[kSlotRec * (1 + s) + j] = 0;
}

// ------------------------------------------------------------ few tokens
// One block does everything: the waves take the tokens in turn, then (beyond
// 64 rows, or where the tile list is wanted; decode has neither) the rows sit
// 64 to a wave, each wave ranks its rows among themselves by ballots over the
// expert id's bits, and thread e sums the waves' counts of expert e and scans
// them over the experts.  cnt is [chunks][E] in LDS.
//
// Two launches against this one, back to back in a graph, top-8 of 32 / 128 /
// 256 experts: 24 tokens 11.7 / 12.4 / 13.6 us against 9.1 / 10.0 / 11.9, 32
// tokens 11.9 / 12.6 / 13.6 against 11.7 / 12.9 / 15.1; hence the limit of 24.
// Beyond 256 experts a lane holds 8 or 16 values and 16 waves have too few
// registers for them (1024 experts: 11.2 us for one token, 19.3 for eight, 39
// for 32, against 9.8, 12.9 and 16.9 with 8 waves), so the block has 8 waves
// and keeps to 64 rows.
template <int PER, int THREADS>
__global__ __launch_bounds__(THREADS) void k_scored_few(ScoreArgs S, const float* __restrict__ logits,
                                                        int T, ScoreOut O) {
  extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
  __shared__ __attribute__((aligned(16))) int s_row[kScoredFewRows];
  __shared__ int s_tot[THREADS / 64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int E = S.E, k = S.k, rows = T * k;
  if (tid < ((4 - rows) & 3)) s_row[rows + tid] = 0x7FFFFFFF;
  uint64_t* stage = reinterpret_cast<uint64_t*>(sm) + (size_t)wave * S.stage;
  for (int t = wave; t < T; t += THREADS / 64) {
    int j, id;
    float w;
    wave_scored_topk<PER>(S, logits + (size_t)t * E, lane, stage, j, id, w);
    if (j < k) {
      O.ids[t * k + j] = id;
      O.w[t * k + j] = w;
      s_row[t * k + j] = id;
    }
  }
  __syncthreads();
  if (PER > 4 || (rows <= 64 && !O.tiles)) {
    // at most 64 rows, one per lane of wave 0: each row's place from ballots
    // over the bits of the expert ids; thread e counts the rows of expert e and
    // of those before it
    if (wave == 0) {
      const bool act = lane < rows;
      const int id = act ? s_row[lane] : 0;
      uint64_t eq = __ballot(act), less = 0;
      for (int b = S.bits - 1; b >= 0; --b) {
        const bool bit = (id >> b) & 1;
        const uint64_t m1 = __ballot(act && bit);
        less |= bit ? eq & ~m1 : 0ull;
        eq &= bit ? m1 : ~m1;
      }
      const uint64_t below = lane ? (~0ull >> (64 - lane)) : 0ull;
      const int rk = __popcll(eq & below), off = __popcll(less);
      const uint64_t first = __ballot(act && rk == 0);
      const int slot = __popcll(less & first), n_active = __popcll(first);
      if (act) {
        O.perm_tok[off + rk] = lane / k;
        O.inv_row[lane] = off + rk;
        if (O.slots) {
          int32_t* rec = O.slots + kSlotRec * (1 + slot);
          rec[kSlotTok + rk] = lane / k;
          if (rk == 0) {
            rec[0] = id;
            rec[1] = off;
            rec[2] = __popcll(eq);
            rec[3] = O.alt_select && O.alt_select[id] ? 1 : 0;
          }
        }
      }
      if (O.slots) write_other_slots(O, T, rows, n_active, lane);
    }
    for (int e = tid; e < E; e += THREADS) {
      int cnt = 0, off = 0;
#pragma unroll 4
      for (int r = 0; r < rows; r += 4) {
        const int4 o = *reinterpret_cast<const int4*>(s_row + r);  // (padded with no expert)
        cnt += (o.x == e ? 1 : 0) + (o.y == e ? 1 : 0) + (o.z == e ? 1 : 0) + (o.w == e ? 1 : 0);
        off += (o.x < e ? 1 : 0) + (o.y < e ? 1 : 0) + (o.z < e ? 1 : 0) + (o.w < e ? 1 : 0);
      }
      O.counts[e] = cnt;
      O.offsets[e] = off;
    }
    if (tid == 0) O.offsets[E] = rows;
    return;
  }
  const int chunks = (rows + 63) >> 6;
  int* cnt = reinterpret_cast<int*>(sm);
  for (int i = tid; i < chunks * E; i += THREADS) cnt[i] = 0;
  __syncthreads();
  // row r = tid (+ THREADS): its rank among the rows of the same expert in its chunk
  constexpr int RP = THREADS == 256 ? 1 : (kScoredFewRows + THREADS - 1) / THREADS;
  int rk[RP];
#pragma unroll
  for (int q = 0; q < RP; ++q) {
    const int r = q * THREADS + tid;
    const bool act = r < rows;
    const uint64_t active = __ballot(act);
    if (active) {
      const int e = act ? s_row[r] : 0;
      const uint64_t peers = match_lanes(e, S.bits, active);
      const uint64_t lt = lane ? (~0ull >> (64 - lane)) : 0ull;
      rk[q] = __popcll(peers & lt);
      if (act && (peers & lt) == 0) cnt[(r >> 6) * E + e] = __popcll(peers);
    }
  }
  __syncthreads();
  // thread e: counts before each chunk, the expert's total; then offset and slot
  int total = 0;
  if (tid < E)
    for (int c = 0; c < chunks; ++c) {
      const int v = cnt[c * E + tid];
      cnt[c * E + tid] = total;
      total += v;
    }
  int all;
  const int off = block_scan(total, s_tot, all);
  if (tid < E) {
    O.counts[tid] = total;
    O.offsets[tid] = off;
    for (int c = 0; c < chunks; ++c) cnt[c * E + tid] += off;
  }
  if (tid == 0) O.offsets[E] = rows;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < RP; ++q) {
    const int r = q * THREADS + tid;
    if (r < rows) {
      const int pos = cnt[(r >> 6) * E + s_row[r]] + rk[q];
      O.perm_tok[pos] = r / k;
      O.inv_row[r] = pos;
    }
  }
  if (O.tiles) write_tiles(O, T, k, E, tid < E ? total : 0, off, s_tot);
}

// ----------------------------------------------------------- many tokens
// Block b: tokens [b * tb, (b + 1) * tb).  The waves select, then rank the
// block's rows per expert (64-row chunks, contiguous ones to a wave, by
// ballots), giving each row its rank among the block's rows of its expert and
// the block's histogram.  Bound by the issue of the selection's instructions,
// 690 of a wave for a token (8192 tokens of 256 experts, top-8: 16.4 us;
// reading the logits takes 1.8).
template <int PER, int THREADS>
__global__ __launch_bounds__(THREADS) void k_scored_select(ScoreArgs S,
                                                           const float* __restrict__ logits, int T,
                                                           int tb, int32_t* __restrict__ ids,
                                                           float* __restrict__ w,
                                                           uint16_t* __restrict__ hist,
                                                           int32_t* __restrict__ lrank) {
  extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
  constexpr int NW = THREADS / 64;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int E = S.E, k = S.k;
  const int t0 = blockIdx.x * tb, t1 = min(T, t0 + tb);
  uint64_t* stage = reinterpret_cast<uint64_t*>(sm) + (size_t)wave * S.stage;
  int* s_row = reinterpret_cast<int*>(sm + (size_t)NW * S.stage * 8);
  for (int t = t0 + wave; t < t1; t += NW) {
    int j, id;
    float wt;
    wave_scored_topk<PER>(S, logits + (size_t)t * E, lane, stage, j, id, wt);
    if (j < k) {
      ids[(size_t)t * k + j] = id;
      w[(size_t)t * k + j] = wt;
      s_row[(t - t0) * k + j] = id;
    }
  }
  __syncthreads();
  int* cnt = reinterpret_cast<int*>(sm);  // [NW][E], over the staging area
  for (int i = tid; i < NW * E; i += THREADS) cnt[i] = 0;
  __syncthreads();
  const int nrows = (t1 - t0) * k;
  const int nchunk = (nrows + 63) >> 6, per = (nchunk + NW - 1) / NW;
  const int c0 = wave * per, c1 = min(nchunk, c0 + per);
  const size_t r0 = (size_t)t0 * k;
  for (int c = c0; c < c1; ++c) {
    const int r = c * 64 + lane;
    const bool act = r < nrows;
    const int e = act ? s_row[r] : 0;
    const uint64_t peers = match_lanes(e, S.bits, __ballot(act));
    const uint64_t lt = lane ? (~0ull >> (64 - lane)) : 0ull;
    // a wave's LDS accesses complete in program order: all lanes read, then
    // the first lane of each expert writes
    const int base = act ? cnt[wave * E + e] : 0;
    if (act) lrank[r0 + r] = base + __popcll(peers & lt);
    if (act && (peers & lt) == 0) cnt[wave * E + e] = base + __popcll(peers);
  }
  __syncthreads();
  const int Ep = (E + 7) & ~7;
  for (int e = tid; e < Ep; e += THREADS) {
    int run = 0;
    if (e < E)
      for (int v = 0; v < NW; ++v) {
        const int c = cnt[v * E + e];
        cnt[v * E + e] = run;
        run += c;
      }
    hist[(size_t)blockIdx.x * Ep + e] = (uint16_t)run;  // at most 8192 rows a block
  }
  __syncthreads();
  for (int c = c0; c < c1; ++c) {
    const int r = c * 64 + lane;
    if (r < nrows) lrank[r0 + r] += cnt[wave * E + s_row[r]];
  }
}

// Block b places the rows of the select blocks [b * sb, (b + 1) * sb).  Each
// block sums the histogram's columns itself (all of it for the offsets, the
// blocks before its own for its first base), eight 16-bit counts a load: 128 KB
// from L2 at 256 experts and blocks, less than a launch in between would cost
// (4.8 us of this kernel's 7.6 with 32-bit counts one by one).
__global__ __launch_bounds__(1024) void k_scored_place(const int32_t* __restrict__ ids, int T, int E,
                                                       int k, int tb, int sb, int nblk,
                                                       const uint16_t* __restrict__ hist,
                                                       const int32_t* __restrict__ lrank,
                                                       ScoreOut O) {
  __shared__ int s_all[MOE_MAX_EXPERTS], s_base[MOE_MAX_EXPERTS];
  __shared__ int s_tot[16];
  const int tid = threadIdx.x;
  const int b0 = blockIdx.x * sb, b1 = min(nblk, b0 + sb);
  s_all[tid] = 0;
  s_base[tid] = 0;
  __syncthreads();
  // thread = (eight experts, one of `parts` interleaved sets of select blocks); integer sums only
  const int V = (E + 7) / 8, parts = min(1024 / V, 128), part = tid / V, v = tid - part * V;
  if (part < parts) {
    int all[8], base[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) all[j] = base[j] = 0;
#pragma unroll 8
    for (int b = part; b < nblk; b += parts) {
      const u32x4 h = *reinterpret_cast<const u32x4*>(hist + ((size_t)b * V + v) * 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = (int)((h[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
        all[j] += c;
        base[j] += b < b0 ? c : 0;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (8 * v + j < E) {
        atomicAdd(&s_all[8 * v + j], all[j]);
        atomicAdd(&s_base[8 * v + j], base[j]);
      }
  }
  __syncthreads();
  const int total = tid < E ? s_all[tid] : 0;
  int sum;
  const int off = block_scan(total, s_tot, sum);
  if (tid < E) s_base[tid] += off;
  if (blockIdx.x == 0) {
    if (tid < E) {
      O.counts[tid] = total;
      O.offsets[tid] = off;
    }
    if (tid == 0) O.offsets[E] = sum;
    if (O.tiles) write_tiles(O, T, k, E, total, off, s_tot);
  }
  for (int b = b0; b < b1; ++b) {
    __syncthreads();
    const int r0 = b * tb * k, r1 = min(T * k, r0 + tb * k);
    for (int r = r0 + tid; r < r1; r += 1024) {
      const int pos = s_base[ids[r]] + lrank[r];
      O.perm_tok[pos] = r / k;
      O.inv_row[r] = pos;
    }
    if (b + 1 == b1) break;
    __syncthreads();
    if (tid < E) s_base[tid] += hist[(size_t)b * V * 8 + tid];
  }
}

// ------------------------------------------------------------------ launch
static int bits_for(int n) {
  int b = 1;
  while ((1 << b) < n) ++b;
  return b;
}

// tokens per select block: about 256 blocks (one per CU), at least one token
// a wave, and at most 8192 rows (32 KB of LDS)
static int scored_block_tokens(int T, int k, int waves) {
  const int per = (T + 255) / 256, most = 8192 / k / waves * waves;
  const int tb = (per + waves - 1) / waves * waves;
  return tb < most ? tb : most;
}
static int scored_waves(int E) { return E <= 256 ? 16 : 8; }

size_t scored_ws_bytes(const moe_layer* L, int T) {
  const int tb = scored_block_tokens(T, L->top_k, scored_waves(L->n_experts));
  const size_t nblk = ((size_t)T + tb - 1) / tb;
  const size_t hist = 2 * nblk * (((size_t)L->n_experts + 7) & ~size_t(7));
  return ((hist + 255) & ~size_t(255)) + 4 * (size_t)T * L->top_k;
}

int launch_route_scored(const moe_layer* L, const moe_scoring* C, int T, moe_routing* R,
                        uint8_t* scratch, const ScoreOut& out, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  const int E = L->n_experts, k = L->top_k;
  ScoreArgs S{};
  S.bias = C->choice_bias;
  S.scale = C->scale;
  S.E = E;
  S.k = k;
  S.sigmoid = C->score == MOE_SCORE_SIGMOID;
  S.renorm = C->renorm;
  S.n_groups = C->n_groups;
  S.topk_groups = C->topk_groups;
  S.group_top = C->group_top;
  S.group_size = E / C->n_groups;
  S.group_magic = ((1u << 20) + S.group_size - 1) / S.group_size;
  S.team_log2 = 6 - (C->n_groups > 1 ? bits_for(C->n_groups) : 0);
  S.bits = bits_for(E);
  S.stage = E > 64 ? E : 64;
  ScoreOut O = out;
  O.ids = R->topk_ids;
  O.w = R->topk_w;
  O.counts = R->counts;
  O.offsets = R->offsets;
  O.perm_tok = R->perm_tok;
  O.inv_row = R->inv_row;
  const int rows = T * k;
  if (E <= 256 ? T <= kScoredFewTokens : T <= 8 && rows <= 64 && !O.tiles) {
    const int threads = E > 256 ? 512 : T <= 4 ? 256 : 1024;
    const size_t cnt = (size_t)((rows + 63) / 64) * E * 4;
    const size_t stg = (size_t)(threads / 64) * S.stage * 8;
    const size_t lds = cnt > stg ? cnt : stg;
#define BQ_FEW(PER, TH)                                                                       \
  do {                                                                                        \
    const void* f = (const void*)k_scored_few<PER, TH>;                                       \
    if (lds > 65536 - 8192 &&                                                                 \
        hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) !=       \
            hipSuccess)                                                                       \
      return (int)hipErrorInvalidConfiguration;                                               \
    hipLaunchKernelGGL((k_scored_few<PER, TH>), dim3(1), dim3(TH), lds, s, S, R->logits, T, O); \
  } while (0)
    if (threads == 256) {
      if (E <= 64)
        BQ_FEW(1, 256);
      else if (E <= 128)
        BQ_FEW(2, 256);
      else
        BQ_FEW(4, 256);
    } else if (threads == 512) {
      if (E <= 512)
        BQ_FEW(8, 512);
      else
        BQ_FEW(16, 512);
    } else if (E <= 64)
      BQ_FEW(1, 1024);
    else if (E <= 128)
      BQ_FEW(2, 1024);
    else
      BQ_FEW(4, 1024);
#undef BQ_FEW
    return (int)hipGetLastError();
  }
  const int waves = scored_waves(E), tb = scored_block_tokens(T, k, waves);
  const int nblk = (T + tb - 1) / tb;
  uint16_t* hist = (uint16_t*)scratch;
  int32_t* lrank =
      (int32_t*)(scratch + ((2 * (size_t)nblk * ((E + 7) & ~7) + 255) & ~size_t(255)));
  const size_t lds = (size_t)waves * S.stage * 8 + (size_t)tb * k * 4;
#define BQ_SEL(PER, TH)                                                                        \
  do {                                                                                         \
    const void* f = (const void*)k_scored_select<PER, TH>;                                     \
    if (lds > 65536 &&                                                                         \
        hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) !=        \
            hipSuccess)                                                                        \
      return (int)hipErrorInvalidConfiguration;                                                \
    hipLaunchKernelGGL((k_scored_select<PER, TH>), dim3(nblk), dim3(TH), lds, s, S, R->logits, \
                       T, tb, R->topk_ids, R->topk_w, hist, lrank);                            \
  } while (0)
  if (E <= 64)
    BQ_SEL(1, 1024);
  else if (E <= 128)
    BQ_SEL(2, 1024);
  else if (E <= 256)
    BQ_SEL(4, 1024);
  else if (E <= 512)
    BQ_SEL(8, 512);
  else
    BQ_SEL(16, 512);
#undef BQ_SEL
  const int sb = (nblk + 255) / 256;
  hipLaunchKernelGGL(k_scored_place, dim3((nblk + sb - 1) / sb), dim3(1024), 0, s, R->topk_ids, T,
                     E, k, tb, sb, nblk, hist, lrank, O);
  return (int)hipGetLastError();
}

}  // namespace bqmoe
