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
// One wave per token; lane i holds experts i*PER .. i*PER + PER - 1, so the
// first lane among equals holds the lowest expert.  Each of the k rounds: the
// lane's best choice left, the wave's maximum, a ballot for its first lane.
#include <math.h>

#include "ep_internal.h"
#include "route_impl.h"

namespace epk {

constexpr int kScoreWaves = 4;       // waves per workgroup
constexpr int kMaxGroups = 64;       // expert groups: at least one lane each

struct ScoreRule {
  int32_t sigmoid, groups, kept, top2, renorm;
  float scale;
};

__device__ __forceinline__ double shfl_xor_max(double v, int d) {
  const double o = __shfl_xor(v, d);
  return o > v ? o : v;
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = shfl_xor_max(v, d);
  return v;
}

__device__ __forceinline__ double wave_add(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// A logit as the routing reads it: NaN masks like -inf, +inf is the largest float.
__device__ __forceinline__ float clean_logit(float l) {
  return l != l ? -INFINITY : fminf(l, 3.402823466e38f);
}

__device__ __forceinline__ float load_logit(const void *p, int64_t i, bool bf16) {
  return clean_logit(bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16)
                          : static_cast<const float *>(p)[i]);
}

__device__ __forceinline__ bool masked(float l) { return l == -INFINITY; }

template <int PER>
__global__ __launch_bounds__(64 * kScoreWaves) void k_score_route(
    const void *__restrict__ logits, int32_t bf16, const float *__restrict__ bias, ScoreRule rule,
    int32_t T, int32_t E, int32_t k, int32_t *__restrict__ idx_out, float *__restrict__ w_out,
    float *__restrict__ scores) {
  __shared__ double s_choice[kScoreWaves][64 * PER];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kScoreWaves + wv;
  if (t >= T) return;  // the whole wave; no workgroup barrier below
  const int e0 = lane * PER;
  float l[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = e0 + i < E ? load_logit(logits, t * E + e0 + i, bf16) : -INFINITY;

  const bool grouped = rule.groups > 1;
  const bool by_logit = !bias && !(grouped && rule.top2);
  double lmax = -INFINITY, z = 1.0;
  if (!rule.sigmoid) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);
    lmax = wave_max((double)m);
    if (scores || !rule.renorm || !by_logit) {
      z = 0.0;
#pragma unroll
      for (int i = 0; i < PER; ++i) z += masked(l[i]) ? 0.0 : exp((double)l[i] - lmax);
      z = wave_add(z);
    }
  }
  double v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool in = e0 + i < E, dead = masked(l[i]);
    v[i] = (double)l[i];
    if (scores || !by_logit) {
      const double s = dead ? 0.0
                       : rule.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i]))
                                      : exp((double)l[i] - lmax) / z;
      if (scores && in) scores[t * E + e0 + i] = (float)s;
      if (!by_logit) v[i] = dead ? -INFINITY : bias && in ? s + (double)bias[e0 + i] : s;
    }
    if (!(v[i] > -INFINITY)) v[i] = -INFINITY;  // a bias that is NaN masks too
  }

  if (grouped) {
    double *sv = s_choice[wv];
#pragma unroll
    for (int i = 0; i < PER; ++i) sv[e0 + i] = v[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    // `per` lanes (a power of two) share a group: each scans every per-th member
    int per = 64;
    while (per * rule.groups > 64) per >>= 1;
    const int gs = E / rule.groups, q = lane / per;
    double m1 = -INFINITY, m2 = -INFINITY;
    if (q < rule.groups) {
      for (int i = lane % per; i < gs; i += per) {
        const double c = sv[q * gs + i];
        m2 = fmax(m2, fmin(m1, c));
        m1 = fmax(m1, c);
      }
    }
    for (int d = 1; d < per; d <<= 1) {
      const double o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
      m2 = fmax(fmin(m1, o1), fmax(m2, o2));
      m1 = fmax(m1, o1);
    }
    const double value = rule.top2 && m2 > -INFINITY ? m1 + m2 : m1;
    int rank = 0;
    for (int p = 0; p < rule.groups; ++p) {
      const double o = __shfl(value, p * per);
      rank += o > value || (o == value && p < q) ? 1 : 0;
    }
    // bit q * per: group q stays
    const uint64_t kept = __ballot(q < rule.groups && rank < rule.kept);
    const float inv = 1.0f / (float)gs;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = (int)(((float)(e0 + i) + 0.5f) * inv);  // (e0 + i) / gs, exact for E <= 1024
      if (e0 + i < E && !((kept >> (g * per)) & 1)) v[i] = -INFINITY;
    }
  }

  int32_t my_e = -1;
  float my_l = -INFINITY;
  for (int j = 0; j < k; ++j) {
    double b = v[0];
    int bi = 0;
    float bl = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) {
      const bool g = v[i] > b;
      b = g ? v[i] : b;
      bi = g ? i : bi;
      bl = g ? l[i] : bl;
    }
    const double top = wave_max(b);
    if (!(top > -INFINITY)) break;  // wave-uniform: nothing left to choose
    const int src = __builtin_ctzll(__ballot(b == top));
    const int e = __shfl(e0 + bi, src);
    const float el = __shfl(bl, src);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = lane == src && i == bi ? -INFINITY : v[i];
    my_e = lane == j ? e : my_e;
    my_l = lane == j ? el : my_l;
  }

  const bool chosen = my_e >= 0;
  double w = 0.0;
  if (rule.renorm) {
    // exponents of the scores, up to a common factor: l, or min(l, 0) with 1 + e^-|l| beside it
    const double u = !chosen ? -INFINITY : rule.sigmoid ? fmin((double)my_l, 0.0) : (double)my_l;
    const double um = wave_max(u);
    if (chosen) {
      w = exp(u - um);
      if (rule.sigmoid) w /= 1.0 + exp(-fabs((double)my_l));
    }
    const double sum = wave_add(w);
    if (chosen) w = w / sum * (double)rule.scale;
  } else if (chosen) {
    w = (rule.sigmoid ? 1.0 / (1.0 + exp(-(double)my_l)) : exp((double)my_l - lmax) / z) *
        (double)rule.scale;
  }
  if (lane < k) {
    idx_out[t * k + lane] = my_e;
    w_out[t * k + lane] = (float)w;
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
// the chosen ones are, and the rest of the row is zeros.

template <bool DENSE, int PER>
__global__ __launch_bounds__(64 * kScoreWaves) void k_score_route_bwd(
    const void *__restrict__ logits, int32_t bf16, const int32_t *__restrict__ idx,
    const float *__restrict__ gw, const float *__restrict__ gs, ScoreRule rule, int32_t T,
    int32_t E, int32_t k, void *__restrict__ gl, uint32_t *__restrict__ status) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kScoreWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  // lane j < k: entry j
  int32_t e = lane < k ? idx[t * k + lane] : -1;
  const bool out_of_range = e >= E || e < -1;
  if (__ballot(out_of_range) != 0 && lane == 0) atomicOr(status, kFlagIndexRange);
  if (e >= E) e = -1;
  float el = e >= 0 ? load_logit(logits, t * E + e, bf16) : -INFINITY;
  if (masked(el)) e = -1;
  const float g = e >= 0 ? gw[t * k + lane] * rule.scale : 0.0f;

  float l[PER], lmax = -INFINITY, z = 0.0f;
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = lane + 64 * i;
      l[i] = c < E ? load_logit(logits, t * E + c, bf16) : -INFINITY;
      lmax = fmaxf(lmax, l[i]);
    }
    if (!rule.sigmoid) {
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) lmax = fmaxf(lmax, __shfl_xor(lmax, d));
#pragma unroll
      for (int i = 0; i < PER; ++i) z += masked(l[i]) ? 0.0f : expf(l[i] - lmax);
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) z += __shfl_xor(z, d);
    }
  }

  float part = g;  // what expert e gets: of ds (DENSE without renorm) or of dl
  if (rule.renorm) {
    float um = e < 0 ? -INFINITY : rule.sigmoid ? fminf(el, 0.0f) : el;
    const float u = um;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) um = fmaxf(um, __shfl_xor(um, d));  // k <= 16 lanes
    float p = e < 0 ? 0.0f : expf(u - um);
    if (rule.sigmoid && e >= 0) p /= 1.0f + expf(-fabsf(el));
    float sum = p;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    p = e >= 0 ? p / sum : 0.0f;
    float a = g * p;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) a += __shfl_xor(a, d);
    part = p * (g - a);
    if (rule.sigmoid && e >= 0) part /= 1.0f + expf(el);
  } else if (!DENSE && e >= 0) {  // sigmoid
    const float s = 1.0f / (1.0f + expf(-el));
    part = g * s / (1.0f + expf(el));
  }

  float r[PER];  // dl of the chosen (renorm or sparse), or ds
#pragma unroll
  for (int i = 0; i < PER; ++i) r[i] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl(e, j);
    const float pj = __shfl(part, j);
#pragma unroll
    for (int i = 0; i < PER; ++i) r[i] += lane + 64 * i == ej ? pj : 0.0f;
  }
  if constexpr (DENSE) {
    float ds[PER], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = lane + 64 * i;
      ds[i] = gs && c < E && !masked(l[i]) ? gs[t * E + c] : 0.0f;
      if (!rule.renorm) ds[i] += r[i];
      if (!rule.sigmoid && !masked(l[i])) {
        l[i] = expf(l[i] - lmax) / z;  // the score from here on
        dot += ds[i] * l[i];
      } else if (!rule.sigmoid) {
        l[i] = 0.0f;
      }
    }
    if (!rule.sigmoid) {
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
    }
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
    const int c = lane + 64 * i;
    if (c >= E) continue;
    if (bf16) static_cast<uint16_t *>(gl)[t * E + c] = (uint16_t)(pack_bf16x2(r[i], 0.0f) & 0xFFFFu);
    else static_cast<float *>(gl)[t * E + c] = r[i];
  }
}

#define EP_PER_SWITCH(E, F)          \
  do {                               \
    const int per_ = ((E) + 63) / 64; \
    if (per_ <= 1) F(1);             \
    else if (per_ <= 2) F(2);        \
    else if (per_ <= 4) F(4);        \
    else if (per_ <= 8) F(8);        \
    else F(16);                      \
  } while (0)

static ScoreRule score_rule(const ep_route_rule_t &r) {
  return ScoreRule{r.score == EP_SCORE_SIGMOID, r.num_groups, r.kept_groups,
                   r.group_score == EP_GROUP_TOP2, r.renormalise, r.scale};
}

hipError_t launch_route_scored(const Geometry &g, const ep_route_rule_t &r, const void *logits,
                               bool bf16, const float *bias, int32_t *idx, float *w, float *scores,
                               hipStream_t s) {
  if (g.T == 0) return hipSuccess;
  const unsigned blocks = (unsigned)((g.T + kScoreWaves - 1) / kScoreWaves);
#define L(P)                                                                                   \
  hipLaunchKernelGGL((k_score_route<P>), dim3(blocks), dim3(64 * kScoreWaves), 0, s, logits,   \
                     bf16 ? 1 : 0, bias, score_rule(r), g.T, g.E, g.k, idx, w, scores)
  EP_PER_SWITCH(g.E, L);
#undef L
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const Geometry &g, const Workspace &ws,
                                   const ep_route_rule_t &r, const void *logits, bool bf16,
                                   const int32_t *idx, const float *gw, const float *gs, void *gl,
                                   hipStream_t s) {
  if (g.T == 0) return hipSuccess;
  const unsigned blocks = (unsigned)((g.T + kScoreWaves - 1) / kScoreWaves);
  const bool dense = gs || (r.score == EP_SCORE_SOFTMAX && !r.renormalise);
#define L1(D, P)                                                                                 \
  hipLaunchKernelGGL((k_score_route_bwd<D, P>), dim3(blocks), dim3(64 * kScoreWaves), 0, s, logits, \
                     bf16 ? 1 : 0, idx, gw, gs, score_rule(r), g.T, g.E, g.k, gl, ws.status)
#define L(P)                \
  do {                      \
    if (dense) L1(true, P); \
    else L1(false, P);      \
  } while (0)
  EP_PER_SWITCH(g.E, L);
#undef L
#undef L1
  return hipGetLastError();
}

}  // namespace epk
