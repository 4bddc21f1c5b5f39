// score_route.hip -- routing by scores on gfx950: softmax or sigmoid scores, a
// balance bias that takes part in the choice only, expert groups, top-k,
// renormalised weights; and its backward.  (route.hip: top-k of the logits.)
//
//   s_e      = softmax(l)_e or sigmoid(l_e)
//   choice_e = s_e + b_e            (the order of l when nothing is added)
//   group    = its largest choice, or the sum of its two largest
//   the kept_groups best groups stay; idx = the k best choices left
//   w_j      = scale * s_idx[j]  (renormalised: / sum_i s_idx[i])
//
// Ties go to the lower group and the lower expert.  A logit of -inf or NaN
// masks its expert.  Choices are compared in fp64: two scores next to a border
// can differ by less than fp32 tells, and the ids must not depend on that.
// Renormalised weights are formed from the scores divided by the largest
// chosen one (by exponents, before anything can underflow), so they sum to
// scale whatever the logits.
//
// G lanes per token: a wave (64) for few tokens, a 16-lane row for many, as in
// route.hip; lane i holds experts i, i + G, ...  Each of the k rounds: the
// lane's best choice left, the token's maximum by lane moves, then the lowest
// expert that has it.  A few thousand instructions a wave on a few KB: the
// kernel is bound by their latency for few tokens and their number for many.
// 4096 tokens, 256 experts: 3.6 us to launch, read and choose one expert by its
// logit; seven more rounds 2.5, sigmoid scores in fp64 with a bias 1.4, eight
// groups 2.0 (9.6 us in all).
#include <math.h>

#include "ep_internal.h"
#include "lanes.h"

namespace epk {

constexpr int kScoreWaves = 4;       // waves per workgroup
constexpr int kMaxGroups = 64;       // expert groups

struct ScoreRule {
  int32_t sigmoid, groups, kept, top2, renorm;
  float scale;
};

// e^x for x <= 0 in fp64 to about an ulp: x = n ln 2 + r, |r| <= ln 2 / 2, the
// Taylor series of e^r to r^13 (the next term is below 2^-57), times 2^n.
__device__ __forceinline__ double exp_neg(double x) {
  x = fmax(x, -800.0);  // below: 0 (the scaling underflows)
  const double n = rint(x * 1.4426950408889634);
  const double r = __builtin_fma(-n, 2.3190468138462996e-17, __builtin_fma(-n, 0.6931471805599453, x));
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return ldexp(p, (int)n);
}

// 1 / x for x in [1, 2048]: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double recip(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
}

__device__ __forceinline__ double sigmoid_of(double l) {
  const double e = exp_neg(-fabs(l)), r = recip(1.0 + e);
  return l >= 0.0 ? r : e * r;
}

__device__ __forceinline__ double max_d(double a, double b) { return a > b ? a : b; }

// Reductions over a token's G lanes (a 16-lane row or the wave); every lane
// gets the result.
template <int G>
__device__ __forceinline__ double token_max(double v) {
  v = max_d(v, dpp_d<kDppXor1>(v));
  v = max_d(v, dpp_d<kDppXor2>(v));
  v = max_d(v, dpp_d<kDppHalfMirror>(v));
  v = max_d(v, dpp_d<kDppMirror>(v));
  if constexpr (G == 64) {
    double a, b;
    swap16(v, a, b);
    v = max_d(a, b);
    swap32(v, a, b);
    v = max_d(a, b);
  }
  return v;
}
template <int G>
__device__ __forceinline__ double token_sum(double v) {
  return G == 64 ? wave_sum(v) : row_sum(v);
}
template <int G>
__device__ __forceinline__ uint32_t token_min(uint32_t v) {
  return ~(G == 64 ? wave_max(~v) : row_max(~v));
}
// Integers in the order of floats (-0 as 0); kNoChoice is that of -inf.
__device__ __forceinline__ uint32_t choice_key(float f) {
  const int32_t b = __float_as_int(f + 0.0f);
  return (uint32_t)(b ^ (b >> 31 | (int32_t)0x80000000));
}
constexpr uint32_t kNoChoice = 0x007FFFFFu;

template <int G>
__device__ __forceinline__ float token_sum_f(float v) {
  v += __uint_as_float(dpp<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppMirror>(__float_as_uint(v)));
  if constexpr (G == 64) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}
template <int G>
__device__ __forceinline__ float token_max_f(float v) {
  v = fmaxf(v, __uint_as_float(dpp<kDppXor1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kDppXor2>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kDppHalfMirror>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kDppMirror>(__float_as_uint(v))));
  if constexpr (G == 64) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}

// The value of lane J of each 16-lane row (J < 16).
template <int J>
__device__ __forceinline__ uint32_t row_lane(uint32_t v) {
  return dpp<0x150 + J>(v);  // row_newbcast
}

// A logit as the routing reads it: NaN masks like -inf, +inf is the largest float.
__device__ __forceinline__ float clean_logit(float l) {
  return l != l ? -INFINITY : fminf(l, 3.402823466e38f);
}

// LT: float, or uint16_t for bf16
template <typename LT>
__device__ __forceinline__ float logit_value(LT v) {
  if constexpr (sizeof(LT) == 2) return clean_logit(__uint_as_float((uint32_t)v << 16));
  else return clean_logit(v);
}

__device__ __forceinline__ bool masked(float l) { return l == -INFINITY; }

// Top two of two disjoint sets.
__device__ __forceinline__ void join2(double &m1, double &m2, double o1, double o2) {
  m2 = max_d(m1 < o1 ? m1 : o1, max_d(m2, o2));
  m1 = max_d(m1, o1);
}

// LDS written by lanes of this wave is read by others.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Masks the experts of the groups a token may not choose from.  The choices go
// through LDS (sv, the token's own part): `per` lanes share a group, each
// scanning every per-th member, then join; more groups than lanes take several
// passes, which leave their values in gv.
template <int G, int PER>
__device__ __forceinline__ void keep_groups(double (&v)[PER], const ScoreRule &rule, int32_t E,
                                            int sub, double *sv, double *gv) {
  int per = G;
  while (per > 1 && per * rule.groups > G) per >>= 1;
  const int gs = E / rule.groups, pitch = G == 64 ? gs + per : gs;   // (four tokens' LDS has no room for the gap
  // that keeps lanes on other banks: four workgroups a compute unit are worth more)
  const float inv = 1.0f / (float)gs;
  int grp[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = sub + G * i;
    grp[i] = (int)(((float)e + 0.5f) * inv);  // e / gs, exact for E <= 1024
    if (e < E) sv[grp[i] * pitch + e - grp[i] * gs] = v[i];
  }
  wave_fence();
  for (int q0 = 0; q0 < rule.groups; q0 += G / per) {
    const int q = q0 + sub / per;
    double m1 = -INFINITY, m2 = -INFINITY;
    if (q < rule.groups) {
#pragma unroll 4
      for (int i = sub & (per - 1); i < gs; i += per) {
        const double c = sv[q * pitch + i];
        m2 = max_d(m2, m1 < c ? m1 : c);
        m1 = max_d(m1, c);
      }
    }
    if (per > 1) join2(m1, m2, dpp_d<kDppXor1>(m1), dpp_d<kDppXor1>(m2));
    if (per > 2) join2(m1, m2, dpp_d<kDppXor2>(m1), dpp_d<kDppXor2>(m2));
    if (per > 4) join2(m1, m2, dpp_d<kDppHalfMirror>(m1), dpp_d<kDppHalfMirror>(m2));
    if (per > 8) join2(m1, m2, dpp_d<kDppMirror>(m1), dpp_d<kDppMirror>(m2));
    if constexpr (G == 64) {
      double a1, b1, a2, b2;
      if (per > 16) {
        swap16(m1, a1, b1);
        swap16(m2, a2, b2);
        m1 = a1, m2 = a2;
        join2(m1, m2, b1, b2);
      }
      if (per > 32) {
        swap32(m1, a1, b1);
        swap32(m2, a2, b2);
        m1 = a1, m2 = a2;
        join2(m1, m2, b1, b2);
      }
    }
    if (q < rule.groups) gv[q] = rule.top2 && m2 > -INFINITY ? m1 + m2 : m1;
  }
  wave_fence();
  // a group stays if fewer than `kept` come before it; lane `sub` ranks groups
  // sub, sub + G, ...
  uint64_t kept = 0;  // bit g
  for (int q0 = 0; q0 < rule.groups; q0 += G) {
    const int q = q0 + sub;
    const double mine = q < rule.groups ? gv[q] : -INFINITY;
    int rank = 0;
#pragma unroll 8
    for (int p = 0; p < rule.groups; ++p) {
      const double o = gv[p];
      rank += o > mine || (o == mine && p < q) ? 1 : 0;
    }
    const uint64_t b = __ballot(q < rule.groups && rank < rule.kept);
    if constexpr (G == 64) kept = b;  // at most 64 groups
    else kept |= ((b >> (threadIdx.x & 48)) & 0xFFFFull) << q0;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (sub + G * i < E && !((kept >> grp[i]) & 1)) v[i] = -INFINITY;
}

template <typename LT, int G, int PER>
__global__ __launch_bounds__(64 * kScoreWaves) void k_score_route(
    const LT *__restrict__ logits, const float *__restrict__ bias, ScoreRule rule, int32_t T,
    int32_t E, int32_t k, int32_t *__restrict__ idx_out, float *__restrict__ w_out,
    float *__restrict__ scores) {
  constexpr int kTokens = 64 / G;  // of a wave
  __shared__ double s_choice[kScoreWaves * kTokens][G * (PER + (G == 64 ? 1 : 0))];
  __shared__ double s_group[kScoreWaves * kTokens][kMaxGroups];
  const int lane = threadIdx.x & 63, sub = lane & (G - 1), tok = threadIdx.x / G;
  const int64_t t0 = (int64_t)blockIdx.x * (kScoreWaves * kTokens) + tok;
  const bool live = t0 < T;
  if (G == 64 && !live) return;  // the whole wave; no workgroup barrier below
  const int64_t t = live ? t0 : T - 1;  // (G = 16) idle rows keep in step on the last token
  // all loads first, none behind a branch of its own
  LT raw[PER];
  float be[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) raw[i] = logits[t * E + min(sub + G * i, E - 1)];
  if (bias) {
#pragma unroll
    for (int i = 0; i < PER; ++i) be[i] = bias[min(sub + G * i, E - 1)];
  }
  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = sub + G * i < E ? logit_value(raw[i]) : -INFINITY;

  const bool grouped = rule.groups > 1;
  const bool by_logit = !bias && !(grouped && rule.top2);
  const bool want_scores = scores || !by_logit;
  double lmax = 0.0, zinv = 0.0;
  double v[PER];  // scores (a masked expert's come out 0), then choices
  if (rule.sigmoid) {
    if (want_scores) {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = sigmoid_of((double)l[i]);
    }
  } else if (want_scores || !rule.renorm) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);
    m = token_max_f<G>(m);
    lmax = masked(m) ? 0.0 : (double)m;
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = exp_neg((double)l[i] - lmax);
      z += v[i];
    }
    z = token_sum<G>(z);
    zinv = z > 0.0 ? recip(z) : 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] *= zinv;
  }
  if (scores) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (sub + G * i < E && live) scores[t * E + sub + G * i] = (float)v[i];
  }
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = (double)l[i];
  } else if (bias) {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] += (double)be[i];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)  // a bias that is NaN masks too
    v[i] = !masked(l[i]) && v[i] > -INFINITY ? v[i] : -INFINITY;
  if (grouped) keep_groups<G, PER>(v, rule, E, sub, s_choice[tok], s_group[tok]);

  // A round: the lane's best choice left, then the token's, then the lowest
  // expert that has it.  A wave on one token compares choices rounded to fp32
  // first, which keeps their order: one lane alone with the largest has the
  // token's choice, and fp64 and the ids decide only where several have it
  // (4096 tokens, 256 experts: 8.1 -> 6.4 us; four tokens a wave gain nothing).
  int32_t my_e = -1;
  float my_logit = 0.0f;
  if constexpr (G == 64) {
    int2 *const pick = reinterpret_cast<int2 *>(s_group[tok]);   // expert and logit of each choice
    static_assert(kMaxTopK <= kMaxGroups, "the choices fit the groups' values");
    int found = 0;
    for (; found < k; ++found) {
      double b = v[0];
      float bl = l[0];
      int bi = 0;
#pragma unroll
      for (int i = 1; i < PER; ++i) {
        const bool g = v[i] > b;
        b = g ? v[i] : b;
        bl = g ? l[i] : bl;
        bi = g ? i : bi;
      }
      const uint32_t key = choice_key((float)b), top = wave_max(key);
      if (__builtin_amdgcn_readfirstlane(top) <= kNoChoice) break;  // nothing left to choose
      bool mine = key == top;
      const uint64_t have = __ballot(mine);
      if ((have & (have - 1)) != 0) {
        const double best = token_max<G>(mine ? b : -INFINITY);
        const uint32_t e = token_min<G>(mine && b == best ? (uint32_t)(sub + G * bi) : 0xFFFFFFFFu);
        mine = (e & (G - 1)) == (uint32_t)sub;
      }
      if (mine) pick[found] = make_int2(sub + G * bi, __float_as_int(bl));
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = mine && i == bi ? -INFINITY : v[i];
    }
    wave_fence();
    if (sub < found) {
      my_e = pick[sub].x;
      my_logit = __int_as_float(pick[sub].y);
    }
  } else {
    for (int j = 0; j < k; ++j) {
      double b = v[0];
      int bi = 0;
#pragma unroll
      for (int i = 1; i < PER; ++i) {
        const bool g = v[i] > b;
        b = g ? v[i] : b;
        bi = g ? i : bi;
      }
      const double top = token_max<G>(b);
      const bool any = top > -INFINITY;
      if (!__any(any)) break;  // nothing left to choose for any token of the wave
      const uint32_t e = token_min<G>(any && b == top ? (uint32_t)(sub + G * bi) : 0xFFFFFFFFu);
      const int pos = (e & (G - 1)) == (uint32_t)sub ? (int)(e / G) : -1;
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = any && i == pos ? -INFINITY : v[i];
      my_e = sub == j && any ? (int32_t)e : my_e;
    }
    if (my_e >= 0) my_logit = logit_value(logits[t * E + my_e]);
  }

  const bool chosen = my_e >= 0;
  const double my_l = (double)my_logit;
  double w = 0.0;
  if (rule.renorm) {
    // exponents of the scores, up to a common factor: l, or min(l, 0) with 1 + e^-|l| beside it
    const double u = !chosen ? -INFINITY : rule.sigmoid ? fmin(my_l, 0.0) : my_l;
    const double um = token_max<G>(u);
    if (chosen) {
      w = exp_neg(u - um);
      if (rule.sigmoid) w *= recip(1.0 + exp_neg(-fabs(my_l)));
    }
    const double sum = token_sum<G>(w);
    if (chosen) w = w / sum;
  } else if (chosen) {
    w = rule.sigmoid ? sigmoid_of(my_l) : exp_neg(my_l - lmax) * zinv;
  }
  if (live && sub < k) {
    idx_out[t * k + sub] = my_e;
    w_out[t * k + sub] = (float)(w * (double)rule.scale);
  }
}

// ---------------------------------------------------------------------------
// backward: the gradient of the logits from those of the k weights (c = scale)
// and, where given, of the scores.  With p_j the chosen scores over their sum
// and A = sum_i gw_i p_i:
//   renormalised, softmax:  dl_e += c p_j (gw_j - A)          for e = idx[j]
//   renormalised, sigmoid:  dl_e += c p_j (gw_j - A) (1 - s_e)
//   otherwise               ds_e += c gw_j
//   sigmoid:  dl_e += ds_e s_e (1 - s_e);  softmax: dl_e += s_e (ds_e - sum ds s)
// The choice itself has no gradient (nor has the bias).  Entries of -1, ids out
// of range and masked experts carry none; an expert named twice gets the sum.
// DENSE: every expert has a gradient, so all logits are read; otherwise only
// the chosen ones are, and the rest of the row is zeros.  Lanes as in the
// forward: bound by memory for many tokens.

// r[i] += the part of each entry that names expert sub + G * i.
template <int G, int PER, int J>
__device__ __forceinline__ void add_entries(float (&r)[PER], int32_t e, float part, int sub, int k) {
  if constexpr (J < kMaxTopK) {
    if (J < k) {  // wave-uniform
      // entry J sits in lane J of the token's lanes
      uint32_t ej, pj;
      if constexpr (G == 16) {
        ej = row_lane<J>((uint32_t)e);
        pj = row_lane<J>(__float_as_uint(part));
      } else {
        ej = __builtin_amdgcn_readlane((uint32_t)e, J);
        pj = __builtin_amdgcn_readlane(__float_as_uint(part), J);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) r[i] += (uint32_t)(sub + G * i) == ej ? __uint_as_float(pj) : 0.0f;
      add_entries<G, PER, J + 1>(r, e, part, sub, k);
    }
  }
}

template <typename LT, bool DENSE, int G, int PER>
__global__ __launch_bounds__(64 * kScoreWaves) void k_score_route_bwd(
    const LT *__restrict__ logits, const int32_t *__restrict__ idx,
    const float *__restrict__ gw, const float *__restrict__ gs, ScoreRule rule, int32_t T,
    int32_t E, int32_t k, LT *__restrict__ gl, uint32_t *__restrict__ status) {
  const int lane = threadIdx.x & 63, sub = lane & (G - 1);
  const int64_t t0 = (int64_t)blockIdx.x * (kScoreWaves * 64 / G) + threadIdx.x / G;
  const bool live = t0 < T;
  if (G == 64 && !live) return;
  const int64_t t = live ? t0 : T - 1;
  // every load that depends on nothing first
  LT raw[PER];
  float l[PER], ds[PER];
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < PER; ++i) raw[i] = logits[t * E + min(sub + G * i, E - 1)];
#pragma unroll
    for (int i = 0; i < PER; ++i) ds[i] = 0.0f;
    if (gs) {
#pragma unroll
      for (int i = 0; i < PER; ++i) ds[i] = gs[t * E + min(sub + G * i, E - 1)];
    }
  }
  // lane j < k: entry j
  int32_t e = sub < k ? idx[t * k + sub] : -1;
  float g = sub < k ? gw[t * k + sub] * rule.scale : 0.0f;
  const bool out_of_range = e >= E || e < -1;
  if (__any(out_of_range) && lane == 0) atomicOr(status, kFlagIndexRange);
  if (e >= E || e < 0) e = -1;
  const float el = e >= 0 ? logit_value(logits[t * E + e]) : -INFINITY;
  if (masked(el)) e = -1;
  if (e < 0) g = 0.0f;

  float lmax = -INFINITY, zinv = 0.0f;
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      l[i] = sub + G * i < E ? logit_value(raw[i]) : -INFINITY;
      ds[i] = masked(l[i]) ? 0.0f : ds[i];
      lmax = fmaxf(lmax, l[i]);
    }
    if (!rule.sigmoid) {
      lmax = token_max_f<G>(lmax);
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        l[i] = masked(l[i]) ? 0.0f : expf(l[i] - lmax);  // the score's numerator from here on
        z += l[i];
      }
      z = token_sum_f<G>(z);
      zinv = z > 0.0f ? 1.0f / z : 0.0f;
    }
  }

  float part = g;  // what expert e gets: of ds (DENSE without renorm) or of dl
  if (rule.renorm) {
    const float u = e < 0 ? -INFINITY : rule.sigmoid ? fminf(el, 0.0f) : el;
    const float um = token_max_f<G>(u);
    float p = e < 0 ? 0.0f : expf(u - um);
    if (rule.sigmoid && e >= 0) p /= 1.0f + expf(-fabsf(el));
    const float sum = token_sum_f<G>(p);
    p = e >= 0 ? p / sum : 0.0f;
    part = p * (g - token_sum_f<G>(g * p));
    if (rule.sigmoid && e >= 0) part /= 1.0f + expf(el);
  } else if (!DENSE && e >= 0) {  // sigmoid
    part = g / ((1.0f + expf(-el)) * (1.0f + expf(el)));
  }

  float r[PER];  // dl of the chosen (renorm or sparse), or their ds
#pragma unroll
  for (int i = 0; i < PER; ++i) r[i] = 0.0f;
  add_entries<G, PER, 0>(r, e, part, sub, k);
  if constexpr (DENSE) {
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!rule.renorm) ds[i] += r[i];
      if (!rule.sigmoid) {
        l[i] *= zinv;
        dot += ds[i] * l[i];
      }
    }
    if (!rule.sigmoid) dot = token_sum_f<G>(dot);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float v;
      if (!rule.sigmoid) v = l[i] * (ds[i] - dot);
      else v = masked(l[i]) ? 0.0f : ds[i] / ((1.0f + expf(-l[i])) * (1.0f + expf(l[i])));
      r[i] = rule.renorm ? r[i] + v : v;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = sub + G * i;
    if (c >= E || !live) continue;
    if constexpr (sizeof(LT) == 2) gl[t * E + c] = (uint16_t)(pack_bf16x2(r[i], 0.0f) & 0xFFFFu);
    else gl[t * E + c] = r[i];
  }
}

// F(G, PER): a wave per token for few tokens and for more than 256 experts
// (their choices would not fit a row's registers and LDS); a 16-lane row
// otherwise.  "Few" is up to 4096 with more than `many` experts, up to 2048
// below.  Forward, a wave against a row: E = 256 in 8 groups 5.9 and 11.1 us at
// 128 tokens, 9.8 and 11.5 at 4096, 16.3 and 14.4 at 8192; E = 128, softmax: 4.9
// and 5.6 at 4096, 7.4 and 6.2 at 8192; E = 64: 5.2 and 4.9 at 4096.  Backward,
// E = 128: 4.3 and 3.8 at 4096, E = 256: 7.9 and 7.2 at 8192.
constexpr int kManyForward = 64, kManyBackward = 128;
static bool wave_per_token(int32_t T, int32_t E, int many) {
  return E > 256 || T <= (E > many ? 4096 : 2048);
}
#define EP_SCORE_SWITCH(T, E, MANY, F)                           \
  do {                                                           \
    if (wave_per_token(T, E, MANY)) {                            \
      const int per_ = ((E) + 63) / 64;                          \
      if (per_ <= 1) F(64, 1);                                   \
      else if (per_ <= 2) F(64, 2);                              \
      else if (per_ <= 4) F(64, 4);                              \
      else if (per_ <= 8) F(64, 8);                              \
      else F(64, 16);                                            \
    } else {                                                     \
      const int per_ = ((E) + 15) / 16;                          \
      if (per_ <= 2) F(16, 2);                                   \
      else if (per_ <= 4) F(16, 4);                              \
      else if (per_ <= 8) F(16, 8);                              \
      else F(16, 16);                                            \
    }                                                            \
  } while (0)

static ScoreRule score_rule(const ep_route_rule_t &r) {
  return ScoreRule{r.score == EP_SCORE_SIGMOID, r.num_groups, r.kept_groups,
                   r.group_score == EP_GROUP_TOP2, r.renormalise, r.scale};
}

static unsigned score_blocks(int32_t T, int G) {
  const int64_t per = kScoreWaves * 64 / G;
  return (unsigned)((T + per - 1) / per);
}

// T < 2^26, and a launch counts its threads in 32 bits: with a wave a token
// (E > 256) workgroups of 256 threads for four tokens, up to 2^26 - 4 of them.
bool route_scored_fits(const Geometry &g) {
  const int G = wave_per_token(g.T, g.E, kManyForward) ? 64 : 16;
  return g.T < 1 << 26 && (int64_t)score_blocks(g.T, G) * (64 * kScoreWaves) <= (int64_t)UINT32_MAX;
}

hipError_t launch_route_scored(const Geometry &g, const ep_route_rule_t &r, const void *logits,
                               bool bf16, const float *bias, int32_t *idx, float *w, float *scores,
                               hipStream_t s) {
  if (g.T == 0) return hipSuccess;
#define L1(LT, G, P)                                                                            \
  hipLaunchKernelGGL((k_score_route<LT, G, P>), dim3(score_blocks(g.T, G)),                     \
                     dim3(64 * kScoreWaves), 0, s, static_cast<const LT *>(logits), bias,       \
                     score_rule(r), g.T, g.E, g.k, idx, w, scores)
#define L(G, P)                   \
  do {                            \
    if (bf16) L1(uint16_t, G, P); \
    else L1(float, G, P);         \
  } while (0)
  EP_SCORE_SWITCH(g.T, g.E, kManyForward, L);
#undef L
#undef L1
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const Geometry &g, const Workspace &ws,
                                   const ep_route_rule_t &r, const void *logits, bool bf16,
                                   const int32_t *idx, const float *gw, const float *gs, void *gl,
                                   hipStream_t s) {
  if (g.T == 0) return hipSuccess;
  const bool dense = gs || (r.score == EP_SCORE_SOFTMAX && !r.renormalise);
#define L1(LT, D, G, P)                                                                          \
  hipLaunchKernelGGL((k_score_route_bwd<LT, D, G, P>), dim3(score_blocks(g.T, G)),               \
                     dim3(64 * kScoreWaves), 0, s, static_cast<const LT *>(logits), idx, gw, gs, \
                     score_rule(r), g.T, g.E, g.k, static_cast<LT *>(gl), ws.status)
#define L(G, P)                                \
  do {                                         \
    if (bf16 && dense) L1(uint16_t, true, G, P); \
    else if (bf16) L1(uint16_t, false, G, P);  \
    else if (dense) L1(float, true, G, P);     \
    else L1(float, false, G, P);               \
  } while (0)
  EP_SCORE_SWITCH(g.T, g.E, kManyBackward, L);
#undef L
#undef L1
  return hipGetLastError();
}

}  // namespace epk
