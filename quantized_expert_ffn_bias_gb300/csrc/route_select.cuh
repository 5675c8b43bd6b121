// Expert choice of one token by one warp, in the general form of
// colibri_moe_route: sigmoid or softmax scores s, choice by u = s + bias, the
// best groups (largest u or sum of the two largest), then the k largest u,
// weights from s.  Shared by the stand-alone kernel (route.cu) and the layer
// forward (router.cu).
//
// Lane l holds the experts l NV .. l NV + NV - 1, so that a tie goes to the
// lower lane, and so that groups of whole lanes are reduced with a few
// shuffles for all groups at once.  The choice is made in fp32 with approximate
// exponentials on order-preserving integer images, sorted a lane (one
// redux.sync a round).  It is the exact scores' choice all the same: where the
// last kept and the first dropped group or expert are closer than the error of
// the fp32 scores, those around the border are compared by scores in 64 bits
// (computing all of a token's in 64 bits took one warp 35 us and with it the
// call).  Experts whose logit and bias are equal bit for bit tie exactly in
// either form and are no reason for it (16-bit logits tie often); groups whose
// scores are equal are.  The k weights come from fp32 arithmetic on the chosen
// logits (expf, a softmax's sum of approximate terms), within the error that
// the tests derive, or from 64 bits where the chosen scores leave fp32's range.
#pragma once

#include "moe_internal.cuh"

namespace coli {

__device__ __forceinline__ uint32_t route_image(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float route_unimage(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// The value of an image whose low bits were replaced: an infinity's read as a NaN otherwise.
__device__ __forceinline__ float route_unimage_cut(uint32_t k) {
  const float v = route_unimage(k);
  return v == v ? v : (k & 0x80000000u) ? INFINITY : -INFINITY;
}

// Bound on the distance of two approximate scores whose exact order may be the other one, given the token's
// largest score.  A score's error is below s (2^-22 + 2^-22 + 2^-24) for exp2, the quotient and 1 + e, and
// s (1 - s) |z| 2^-23 for the rounded argument of exp2; the latter is largest at the largest score or, where that
// is above 1/2, below 2^-25 ((1 - s) |z| s <= 0.23).  A softmax also carries the sum of up to 32 terms a lane and
// 5 levels (37 * 2^-24), and its arguments z - max enter as x e^-x <= 0.37.  Twice that covers two scores, and a
// quarter is added.  A score below 2^-126 may be flushed to 0 (kFlush: two of them).
__device__ __forceinline__ float route_tol(bool softmax, float smax) {
  constexpr float kFlush = 2.5e-38f;
  if (softmax) return 2.5f * smax * 3.2e-6f + kFlush;
  return 2.5f * smax * (6e-7f + 1.3e-7f * (1.f + fabsf(__logf(fmaxf(smax, 1e-37f))))) + kFlush;
}

__device__ __forceinline__ float route_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A softmax's numerator: all of +infinity share equally, -infinity (also where every logit is) has none.
__device__ __forceinline__ float route_numerator(float z, float m) {
  const float d = m == INFINITY ? (z == INFINITY ? 0.f : -INFINITY) : (m == -INFINITY ? -INFINITY : z - m);
  return route_exp2(d * 1.4426950408889634f);
}
__device__ __forceinline__ float route_sigmoid(float z) {
  return __fdividef(1.f, 1.f + route_exp2(-z * 1.4426950408889634f));
}
// Image of u = s + b (NaN: -infinity's; -0 and +0 are equal).
__device__ __forceinline__ uint32_t route_key(float s, float b) {
  float u = s + b;
  if (!(u == u)) u = -INFINITY;
  return route_image(u + 0.f);
}

// Renormalised weights whose sum is below this are computed again in 64 bits.  Above it a score that fp32 cannot hold
// is less than 2^-66 of the sum, and a softmax's arguments stay above -46.
constexpr float kTinyScores = 8.6736174e-19f;   // 2^-60

// The rare comparisons in 64 bits.  They read the logits and biases again (arguments in arrays would have every
// token store them: 16 us of 33 for 16384 tokens).
struct RouteStats {
  float m, inv;          // softmax: largest logit, 1 / sum
};

// u of one expert in 64 bits; m, sum: the softmax's in 64 bits.
static __device__ __noinline__ double route_exact_score(bool softmax, double m, double sum, float z, float b) {
  const double inf = __longlong_as_double(0x7ff0000000000000ll);
  double s;
  if (softmax) {
    s = m == inf ? (z == INFINITY ? 1.0 : 0.0) : (z == -INFINITY ? 0.0 : exp((double)z - m));
    s = sum > 0.0 ? s / sum : 0.0;
  } else {
    s = 1.0 / (1.0 + exp(-(double)z));
  }
  s += (double)b;
  return s == s ? s : -inf;
}

// Share of this lane's chosen expert in the sum of the warp's chosen scores, in 64 bits; .y: 1, or 0 where all are 0.
// The softmax's own sum cancels.
static __device__ __noinline__ float2 route_ratio(bool softmax, float m, float z, bool chosen) {
  double s = chosen ? route_exact_score(softmax, (double)m, 1.0, z, 0.f) : 0.0, sum = s;
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum > 0.0 ? make_float2((float)(s / sum), 1.f) : make_float2(0.f, 0.f);
}

template <int NV>
struct RouteAgain {
  float z[NV], b[NV];
  uint32_t key[NV];      // images of the fp32 u; 0 past E
  double m, sum;
  bool softmax;
  template <typename Logit>
  __device__ __forceinline__ RouteAgain(const coli_route_desc& r, Logit logit, const float* bias, RouteStats st) {
    const double inf = __longlong_as_double(0x7ff0000000000000ll);
    const int e0 = (int)(threadIdx.x & 31) * NV;
    softmax = r.score == COLI_SCORE_SOFTMAX;
    m = -inf;
    sum = 0.0;
    for (int i = 0; i < NV; ++i) {
      const int e = e0 + i;
      z[i] = e < r.E ? logit(e) : -INFINITY;
      b[i] = bias && e < r.E ? __ldg(bias + e) : 0.f;
      key[i] = e < r.E ? route_key(softmax ? route_numerator(z[i], st.m) * st.inv : route_sigmoid(z[i]), b[i]) : 0u;
      m = fmax(m, (double)z[i]);
    }
    if (!softmax) return;
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int i = 0; i < NV; ++i)
      if (e0 + i < r.E) sum += m == inf ? (z[i] == INFINITY ? 1.0 : 0.0) : (z[i] == -INFINITY ? 0.0 : exp((double)z[i] - m));
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  // Exact scores of the experts in this lane's mask, into u: every lane its next at the same time.
  __device__ __forceinline__ void exact(unsigned which, double (&u)[NV]) const {
    while (__any_sync(0xffffffffu, which)) {
      const int i = which ? __ffs(which) - 1 : 0;
      const double v = route_exact_score(softmax, m, sum, z[i], b[i]);
      if (which) u[i] = v;
      which &= which - 1;
    }
  }
};

// Groups kept (a mask), by exact scores where the fp32 ones are within tol of the border score `a`: lane g
// holds group g's fp32 score.  tol_u: of a single u.
template <int NV, typename Logit>
__device__ __noinline__ unsigned route_groups_exact(const coli_route_desc r, Logit logit, const float* bias,
                                                    RouteStats st, float score, float a, float tol, float tol_u) {
  const int lane = threadIdx.x & 31, G = r.n_group, gsz = r.E / G;
  const double inf = __longlong_as_double(0x7ff0000000000000ll);
  const RouteAgain<NV> x(r, logit, bias, st);
  const bool in = lane < G && score > a + tol, close = lane < G && !in && score >= a - tol;
  const unsigned closes = __ballot_sync(0xffffffffu, close);
  // a close group's second largest u in fp32: experts not below it by more than the tolerance may be among the two
  unsigned which = 0;
  for (unsigned left = closes; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    uint32_t k1 = 0u, k2 = 0u;
    for (int i = 0; i < NV; ++i) {
      const int e = lane * NV + i;
      if (e >= g * gsz && e < (g + 1) * gsz) {
        k2 = max(k2, min(k1, x.key[i]));
        k1 = max(k1, x.key[i]);
      }
    }
    const uint32_t m1 = __reduce_max_sync(0xffffffffu, k1);
    const int first = __ffs(__ballot_sync(0xffffffffu, k1 == m1)) - 1;
    const uint32_t m2 = __reduce_max_sync(0xffffffffu, lane == first ? k2 : k1);
    const float from = route_unimage(r.group_score == COLI_GROUP_TOP2 ? m2 : m1) - tol_u;
    for (int i = 0; i < NV; ++i) {
      const int e = lane * NV + i;
      if (e >= g * gsz && e < (g + 1) * gsz && route_unimage(x.key[i]) >= from) which |= 1u << i;
    }
  }
  double u[NV];
  x.exact(which, u);
  double mine = -inf;
  for (unsigned left = closes; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    double t1 = -inf, t2 = -inf;
    for (unsigned w = which; w; w &= w - 1) {
      const int i = __ffs(w) - 1, e = lane * NV + i;
      if (e < g * gsz || e >= (g + 1) * gsz) continue;
      if (u[i] > t1) { t2 = t1; t1 = u[i]; }
      else t2 = fmax(t2, u[i]);
    }
    auto warp_max = [](double v) {
      for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
      return v;
    };
    double sc = warp_max(t1);
    if (r.group_score == COLI_GROUP_TOP2) {
      const int owner = __ffs(__ballot_sync(0xffffffffu, t1 == sc)) - 1;
      sc += warp_max(lane == owner ? t2 : t1);
      if (!(sc == sc)) sc = -inf;
    }
    if (lane == g) mine = sc;
  }
  int rank = __popc(__ballot_sync(0xffffffffu, in));
  for (unsigned left = closes; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    const double o = __shfl_sync(0xffffffffu, mine, g);
    rank += o > mine || (o == mine && g < lane);
  }
  return __ballot_sync(0xffffffffu, in || (close && rank < r.topk_group));
}

// The picks (lane j < k: the j-th), by exact scores where the fp32 ones are within tol of the last pick's, `a`.
// Those certainly above it are listed here, not taken from the rounds: these went by scores cut to buckets, inside
// which the lower id goes first, so that where a + tol falls into a bucket an expert that is not certain may stand
// among their first picks in the place of one that is.
template <int NV, typename Logit>
__device__ __noinline__ int route_picks_exact(const coli_route_desc r, Logit logit, const float* bias, RouteStats st,
                                              unsigned open, float a, float tol, int pick) {
  const int lane = threadIdx.x & 31, gsz = r.E / r.n_group;
  const RouteAgain<NV> x(r, logit, bias, st);
  unsigned left = 0;                     // this lane's candidates around the border
  int sure = 0;                          // candidates certainly above it (fewer than k): the first picks
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    bool above = false;
    if (e < r.E && ((open >> (e / gsz)) & 1u)) {
      const float v = route_unimage(x.key[i]);
      above = v > a + tol;
      if (!above && v >= a - tol) left |= 1u << i;
    }
    for (unsigned b = __ballot_sync(0xffffffffu, above); b; b &= b - 1)
      if (lane == sure++) pick = (__ffs(b) - 1) * NV + i;
  }
  double u[NV];
  x.exact(left, u);
  for (int j = sure; j < r.k; ++j) {
    double bu = 0.0;
    int be = 0x7fffffff;
    for (int i = 0; i < NV; ++i)
      if (((left >> i) & 1u) && (be == 0x7fffffff || u[i] > bu)) { bu = u[i]; be = lane * NV + i; }
    for (int o = 16; o > 0; o >>= 1) {
      const double u2 = __shfl_xor_sync(0xffffffffu, bu, o);
      const int e2 = __shfl_xor_sync(0xffffffffu, be, o);
      if (e2 != 0x7fffffff && (be == 0x7fffffff || u2 > bu || (u2 == bu && e2 < be))) { bu = u2; be = e2; }
    }
    if (lane == j && be < r.E) pick = be;
    if (be / NV == lane) left &= ~(1u << (be % NV));
  }
  return pick;
}

// Sort a lane's keys, largest first (Batcher's odd-even merge network; past N, keys that are smaller than all).
template <int N>
__device__ __forceinline__ void route_sort(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (j + i + q < N && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
            const uint32_t hi = max(v[j + i], v[j + i + q]), lo = min(v[j + i], v[j + i + q]);
            v[j + i] = hi;
            v[j + i + q] = lo;
          }
}

// z: this lane's logits (experts lane NV + i; NaN already -infinity, past E anything); b: their biases (0 without
// one); bias: where they come from (or NULL); `logit(e)`: the logit of expert e again, by any lane.  topk_idx, topk_w:
// this token's [k]; sel_out (may be NULL): the same ids; near_tie (may be NULL) as colibri_moe_debug_routing
// documents it.
// EXACT = false: returns whether a decision was closer than the scores' error (warp-uniform); its results are then
// to be replaced by route_token_exact's.
template <int NV, bool EXACT, typename Logit>
__device__ __forceinline__ bool route_token(const coli_route_desc& r, const float (&z)[NV], const float (&b)[NV],
                                            const float* bias, Logit logit, int32_t* topk_idx, float* topk_w, int* sel_out,
                                            int32_t* near_tie) {
  const int lane = threadIdx.x & 31;
  const int E = r.E, k = r.k, n_here = E - lane * NV;    // experts of this lane: i < n_here
  const bool softmax = r.score == COLI_SCORE_SOFTMAX;
  // scores
  float s[NV], sum = 0.f;
  RouteStats st{-INFINITY, 0.f};
  if (softmax) {
#pragma unroll
    for (int i = 0; i < NV; ++i) st.m = fmaxf(st.m, i < n_here ? z[i] : -INFINITY);
    st.m = route_unimage(__reduce_max_sync(0xffffffffu, route_image(st.m)));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = i < n_here ? route_numerator(z[i], st.m) : 0.f;
      sum += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    st.inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] *= st.inv;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = route_sigmoid(z[i]);
  }
  // The lane's images of u in order, the low bits giving way to the expert (the lower one the larger): a round of
  // the selection then only compares the lanes' heads.  0: not a candidate (below every image, also -infinity's).
  // kCut: what that may take from a value, relative to it; it enters the tolerances.
  constexpr uint32_t kIdx = NV <= 4 ? 3 : NV <= 8 ? 7 : NV <= 16 ? 15 : 31;
  constexpr float kCut = (float)(kIdx + 1) / 8388608.f;
  uint32_t v[NV];
  float smax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = i < n_here ? (route_key(s[i], b[i]) & ~kIdx) | (kIdx - (uint32_t)i) : 0u;
    smax = fmaxf(smax, i < n_here ? s[i] : 0.f);
  }
  smax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(smax)));
  // groups of whole lanes (a power of two of them) are reduced by shuffles from the sorted lists; other groups one
  // by one, and the lists are sorted when the closed groups are out of them
  const bool grouped = r.topk_group < r.n_group;
  const int gsz = E / r.n_group, lanes = gsz / NV;
  const bool whole = lanes * NV == gsz && (lanes & (lanes - 1)) == 0;
  if (!grouped || whole) route_sort<NV>(v);
  const float tol_s = route_tol(softmax, smax);
  bool tie = false, again = false;       // a decision closer than kNearTie, than the scores' error

  // groups
  unsigned open = 0xffffffffu;           // kept groups
  if (grouped) {
    const int G = r.n_group;
    const bool top2 = r.group_score == COLI_GROUP_TOP2;
    uint32_t t1 = 0u, t2 = 0u;           // a group's two largest images
    int mine = lane;                     // this lane's group, or the group whose scores it holds
    if (whole) {
      t1 = v[0];
      t2 = NV > 1 ? v[1] : 0u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        if (o < lanes) {
          const uint32_t a1 = __shfl_xor_sync(0xffffffffu, t1, o), a2 = __shfl_xor_sync(0xffffffffu, t2, o);
          t2 = max(min(t1, a1), max(t2, a2));
          t1 = max(t1, a1);
        }
      }
      mine = lane >> (31 - __clz(lanes));
    } else {
      for (int g = 0; g < G; ++g) {
        uint32_t a1 = 0u, a2 = 0u;
        const int lo = g * gsz - lane * NV;      // the group's experts among this lane's: lo <= i < lo + gsz
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int at = (int)(kIdx - (v[i] & kIdx));
          if (v[i] && at >= lo && at < lo + gsz) {
            a2 = max(a2, min(a1, v[i]));
            a1 = max(a1, v[i]);
          }
        }
        const uint32_t m1 = __reduce_max_sync(0xffffffffu, a1);
        const int owner = __ffs(__ballot_sync(0xffffffffu, a1 == m1)) - 1;
        const uint32_t m2 = __reduce_max_sync(0xffffffffu, lane == owner ? a2 : a1);
        if (lane == g) {
          t1 = m1;
          t2 = m2;
        }
      }
    }
    float sc = -INFINITY, mag = 0.f;
    if (mine < G) {
      sc = route_unimage_cut(t1);
      mag = fabsf(sc);
      if (top2) {
        const float second = route_unimage_cut(t2);
        mag = fmaxf(mag, fabsf(second));
        sc += second;
        if (!(sc == sc)) sc = -INFINITY;
      }
      sc += 0.f;
      if (!(mag < INFINITY)) mag = 0.f;
    }
    int rank = 0;
    for (int g = 0; g < G; ++g) {
      const float o = __shfl_sync(0xffffffffu, sc, whole ? g * lanes : g);
      rank += o > sc || (o == sc && g < mine);
    }
    if (mine >= G) rank = 64;
    // the last kept and the first dropped score
    const float a = __shfl_sync(0xffffffffu, sc, __ffs(__ballot_sync(0xffffffffu, rank == r.topk_group - 1)) - 1);
    const float c = __shfl_sync(0xffffffffu, sc, __ffs(__ballot_sync(0xffffffffu, rank == r.topk_group)) - 1);
    const float gap = a == c ? 0.f : a - c;
    mag = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mag)));
    const float tol = 2.f * tol_s + (1e-6f + 3.f * kCut) * mag;   // each term and sum rounds by 2^-24 of mag or 2 mag
    tie = gap < kNearTie + 4.f * kCut * mag;
    // lane g holds group g's score and whether it is kept
    const int from = whole ? (lane * lanes) & 31 : lane;
    const float score = __shfl_sync(0xffffffffu, sc, from);
    open = __ballot_sync(0xffffffffu, __shfl_sync(0xffffffffu, rank, from) < r.topk_group && lane < G);
    again = gap <= tol && a > -INFINITY;
    if (EXACT && again)
      open = route_groups_exact<NV>(r, logit, bias, st, score, a, tol, tol_s + (5e-7f + 1.5f * kCut) * mag);
    if (whole) {
      if (!(mine < G && ((open >> (mine & 31)) & 1u)))
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = 0u;
    } else {
      const float per = 1.0f / (float)gsz;       // (e + 1/2) / gsz is exact enough for e < 1024
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int g = (int)(((float)(lane * NV + (int)(kIdx - (v[i] & kIdx))) + 0.5f) * per);
        if (!((open >> (g & 31)) & 1u)) v[i] = 0u;
      }
      route_sort<NV>(v);
    }
  }

  // the k largest: every round the warp takes the best head (ties: the lower lane, the lower expert) and the
  // winning lane moves its list up
  uint32_t kth = 0u;
  int pick = -1;
  for (int j = 0; j < k; ++j) {
    kth = __reduce_max_sync(0xffffffffu, v[0]);
    // heads that differ only in the expert's bits are equal scores: the lower lane goes first
    const int owner = __ffs(__ballot_sync(0xffffffffu, (v[0] | kIdx) == (kth | kIdx))) - 1;
    const int e = __shfl_sync(0xffffffffu, lane * NV + (int)(kIdx - (v[0] & kIdx)), owner);
    if (lane == j) pick = e;
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i + 1 < NV; ++i) v[i] = v[i + 1];
      v[NV - 1] = 0u;
    }
  }
  const uint32_t nxt = __reduce_max_sync(0xffffffffu, v[0]);   // best of those left (0: none)
  if (nxt) {
    const float a = route_unimage(kth & ~kIdx), c = route_unimage(nxt & ~kIdx);
    const float gap = a == c ? 0.f : a - c;
    const float tol = tol_s + (2e-7f + 1.5f * kCut) * fabsf(a);
    tie |= gap < kNearTie + 2.f * kCut * fabsf(a);
    bool close = gap <= tol && fabsf(a) < INFINITY;     // infinite u are exact, and tol is infinite there
    if (close) {
      // unless every candidate around the border has the last pick's logit and bias: those tie exactly
      const int e_k = __shfl_sync(0xffffffffu, pick, k - 1);
      const float zk = logit(e_k), bk = bias ? __ldg(bias + e_k) : 0.f;
      bool other = false;
#pragma unroll 1
      for (int i = 0; i < NV && i < n_here; ++i) {
        const int e = lane * NV + i;
        const float ze = logit(e), be = bias ? __ldg(bias + e) : 0.f;
        const float ue = (softmax ? route_numerator(ze, st.m) * st.inv : route_sigmoid(ze)) + be;
        other |= fabsf(ue - a) <= 2.f * tol && (ze != zk || be != bk) && ((open >> (e / gsz)) & 1u);
      }
      close = __any_sync(0xffffffffu, other);
    }
    again |= close;
    if (EXACT && close)
      pick = route_picks_exact<NV>(r, logit, bias, st, open, a, tol, pick);
  }
  if (near_tie && lane == 0) *near_tie = tie ? 1 : 0;

  // ascending ids: rank of each pick among the picks; weights from the chosen logits, rounded
  int rank = 0;
  for (int i = 0; i < k; ++i) rank += __shfl_sync(0xffffffffu, pick, i) < pick;
  float w = 0.f;
  if (lane < k) {
    const float l = logit(pick);
    if (softmax) w = sum > 0.f ? expf(st.m == INFINITY ? (l == INFINITY ? 0.f : -INFINITY) : l - st.m) / sum : 0.f;
    else w = 1.0f / (1.0f + expf(-l));
  }
  float total = 1.f;
  if (r.renorm) {
    total = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  // chosen scores near or below fp32's range: their ratios are taken in 64 bits (unless every chosen logit is -infinity)
  if (r.renorm && total < kTinyScores && __any_sync(0xffffffffu, lane < k && logit(pick) > -INFINITY)) {
    again = true;
    if constexpr (EXACT) {
      const float2 ratio = route_ratio(softmax, st.m, lane < k ? logit(pick) : -INFINITY, lane < k);
      w = ratio.x;
      total = ratio.y;
    }
  }
  if (lane < k) {
    topk_idx[rank] = pick;
    topk_w[rank] = total > 0.f ? r.scale * w / total : 0.f;
    if (sel_out) sel_out[rank] = pick;
  }
  __syncwarp();
  return again;
}

// The same with exact decisions, for the few tokens that need it: from the start, out of line and last, so that it
// costs the other tokens neither registers nor stores (calls amid the selection cost every token 130 instructions).
template <int NV, typename Logit>
__device__ __noinline__ void route_token_exact(const coli_route_desc r, const float* bias, Logit logit,
                                               int32_t* topk_idx, float* topk_w, int* sel_out, int32_t* near_tie) {
  const int lane = threadIdx.x & 31;
  float z[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    z[i] = e < r.E ? logit(e) : -INFINITY;
    b[i] = bias && e < r.E ? __ldg(bias + e) : 0.f;
  }
  route_token<NV, true>(r, z, b, bias, logit, topk_idx, topk_w, sel_out, near_tie);
}

}  // namespace coli
