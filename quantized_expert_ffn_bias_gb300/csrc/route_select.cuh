// Expert choice of one token by one warp, in the general form of
// colibri_moe_route: sigmoid or softmax scores s, choice by u = s + bias, the
// best groups (largest u or sum of the two largest), then the k largest u,
// weights from s.  Shared by the stand-alone kernel (route.cu) and the layer
// forward (router.cu).
//
// The choice is made in fp32 on order-preserving integer images (one
// redux.sync a round), and is exact all the same: where the last kept and the
// first dropped group or expert are closer than the error of the fp32 scores,
// the warp makes the choice again with scores in 64 bits.  Experts whose logit
// and bias are equal bit for bit tie exactly in either form and are no reason
// for it (16-bit logits tie often).
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

// Bounds on the distance of two fp32 scores whose exact order may be the other one, relative to the
// token's largest s: expf is within 2 ulp, 1 + e, the quotient and s + bias round once each (sigmoid:
// 4 * 2^-23 a score, times two scores, doubled); a softmax also carries z - max (x e^-x 2^-24 at most)
// and the sum of up to 32 terms a lane and 5 levels (38 * 2^-24).
constexpr float kRouteTolSigmoid = 2e-6f, kRouteTolSoftmax = 1.2e-5f;

// The choice again in 64 bits.  z: this lane's logits (experts lane + 32 i).  Returns lane j < k's pick
// in descending order of u.
template <int NV>
__device__ __noinline__ int route_pick_exact(const coli_route_desc& r, const float* zin, const float* bias) {
  const int lane = threadIdx.x & 31;
  const int nv = (r.E + 31) / 32, gsz = r.E / r.n_group;
  const double inf = __longlong_as_double(0x7ff0000000000000ll);
  auto warp_max = [](double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  };
  double u[NV], m = -inf, sum = 0.0;
  for (int i = 0; i < nv; ++i) {
    u[i] = lane + 32 * i < r.E ? (double)zin[i] : -inf;
    m = fmax(m, u[i]);
  }
  if (r.score == COLI_SCORE_SOFTMAX) {
    m = warp_max(m);
    for (int i = 0; i < nv; ++i) {
      u[i] = m == inf ? (u[i] == inf ? 1.0 : 0.0) : (u[i] == -inf ? 0.0 : exp(u[i] - m));
      sum += u[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  for (int i = 0; i < nv; ++i) {
    const int e = lane + 32 * i;
    u[i] = r.score == COLI_SCORE_SOFTMAX ? (sum > 0.0 ? u[i] / sum : 0.0) : 1.0 / (1.0 + exp(-u[i]));
    if (bias && e < r.E) u[i] += (double)bias[e];
    if (!(u[i] == u[i]) || e >= r.E) u[i] = -inf;
  }
  unsigned open = 0xffffffffu;
  if (r.topk_group < r.n_group) {
    double mine = -inf;
    for (int g = 0; g < r.n_group; ++g) {
      double t1 = -inf, t2 = -inf;
      for (int i = 0; i < nv; ++i) {
        const int e = lane + 32 * i;
        if (e >= r.E || e / gsz != g) continue;
        if (u[i] > t1) { t2 = t1; t1 = u[i]; }
        else t2 = fmax(t2, u[i]);
      }
      double sc = warp_max(t1);
      if (r.group_score == COLI_GROUP_TOP2) {
        const int owner = __ffs(__ballot_sync(0xffffffffu, t1 == sc)) - 1;
        sc += warp_max(lane == owner ? t2 : t1);
        if (!(sc == sc)) sc = -inf;
      }
      if (lane == g) mine = sc;
    }
    int rank = 0;
    for (int g = 0; g < r.n_group; ++g) {
      const double o = __shfl_sync(0xffffffffu, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    open = __ballot_sync(0xffffffffu, lane < r.n_group && rank < r.topk_group);
  }
  unsigned left = 0;                     // this lane's experts that can still be picked
  for (int i = 0; i < nv; ++i) {
    const int e = lane + 32 * i;
    if (e < r.E && ((open >> (e / gsz)) & 1u)) left |= 1u << i;
  }
  int pick = -1;
  for (int j = 0; j < r.k; ++j) {
    double bu = -inf;
    int be = 0x7fffffff;
    for (int i = 0; i < nv; ++i)
      if ((left >> i) & 1u)
        if (be == 0x7fffffff || u[i] > bu) { bu = u[i]; be = lane + 32 * i; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double u2 = __shfl_xor_sync(0xffffffffu, bu, o);
      const int e2 = __shfl_xor_sync(0xffffffffu, be, o);
      if (e2 != 0x7fffffff && (be == 0x7fffffff || u2 > bu || (u2 == bu && e2 < be))) { bu = u2; be = e2; }
    }
    if (lane == j) pick = be;
    if ((be & 31) == lane) left &= ~(1u << (be >> 5));
  }
  return pick;
}

// z: this lane's logits (experts lane + 32 i, NaN already -infinity).  topk_idx, topk_w: this token's [k];
// sel_out (may be NULL): the same ids; near_tie (may be NULL) as colibri_moe_debug_routing documents it.
template <int NV>
__device__ __forceinline__ void route_token(const coli_route_desc& r, const float (&z)[NV], const float* bias,
                                            int32_t* topk_idx, float* topk_w, int* sel_out, int32_t* near_tie) {
  const int lane = threadIdx.x & 31;
  const int E = r.E, k = r.k, gsz = E / r.n_group;
  const bool softmax = r.score == COLI_SCORE_SOFTMAX;
  // scores
  float s[NV];
  if (softmax) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, lane + 32 * i < E ? z[i] : -INFINITY);
    m = route_unimage(__reduce_max_sync(0xffffffffu, route_image(m)));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = lane + 32 * i < E ? (m == INFINITY ? (z[i] == INFINITY ? 1.f : 0.f) : (z[i] == -INFINITY ? 0.f : expf(z[i] - m)))
                               : 0.f;
      sum += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = lane + 32 * i < E ? 1.0f / (1.0f + expf(-z[i])) : 0.f;
  }
  uint32_t key[NV];                      // image of u; 0: not a candidate (below every image, also -infinity's)
  float smax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    float u = s[i] + (bias && e < E ? __ldg(bias + e) : 0.f);
    if (!(u == u)) u = -INFINITY;
    u += 0.f;                            // -0 and +0 are equal scores
    key[i] = e < E ? route_image(u) : 0u;
    smax = fmaxf(smax, s[i]);
  }
  smax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(smax)));
  const float tol_s = (softmax ? kRouteTolSoftmax : kRouteTolSigmoid) * smax;
  bool again = false, tie = false;       // a decision closer than the scores' error; closer than kNearTie

  // groups
  unsigned open = 0xffffffffu;
  if (r.topk_group < r.n_group) {
    float mine = -INFINITY, mag = 0.f;   // lane g: group g's score, the larger magnitude of its terms
    for (int g = 0; g < r.n_group; ++g) {
      uint32_t t1 = 0u, t2 = 0u;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e >= g * gsz && e < (g + 1) * gsz) {
          t2 = max(t2, min(t1, key[i]));
          t1 = max(t1, key[i]);
        }
      }
      const uint32_t m1 = __reduce_max_sync(0xffffffffu, t1);
      float sc = route_unimage(m1), mg = fabsf(sc);
      if (r.group_score == COLI_GROUP_TOP2) {
        const int owner = __ffs(__ballot_sync(0xffffffffu, t1 == m1)) - 1;
        const float second = route_unimage(__reduce_max_sync(0xffffffffu, lane == owner ? t2 : t1));
        mg = fmaxf(mg, fabsf(second));
        sc += second;
        if (!(sc == sc)) sc = -INFINITY;
      }
      if (lane == g) {
        mine = sc + 0.f;
        mag = mg < INFINITY ? mg : 0.f;
      }
    }
    int rank = 0;
    for (int g = 0; g < r.n_group; ++g) {
      const float o = __shfl_sync(0xffffffffu, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    if (lane >= r.n_group) rank = 64;
    open = __ballot_sync(0xffffffffu, rank < r.topk_group);
    const unsigned last = __ballot_sync(0xffffffffu, rank == r.topk_group - 1);
    const unsigned next = __ballot_sync(0xffffffffu, rank == r.topk_group);
    const float a = __shfl_sync(0xffffffffu, mine, __ffs(last) - 1), b = __shfl_sync(0xffffffffu, mine, __ffs(next) - 1);
    const float gap = a == b ? 0.f : a - b;
    mag = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mag)));
    again = gap <= 2.f * tol_s + 1e-6f * mag && a > -INFINITY;   // each term and each sum rounds by 2^-24 of mag or 2 mag
    tie = gap < kNearTie;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((open >> (e / gsz)) & 1u)) key[i] = 0u;
    }
  }

  // the k largest: every round the warp takes the best lane candidate and the winning lane rescans
  uint32_t full[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) full[i] = key[i];
  auto lane_best = [&](uint32_t& bk, int& bi) {
    bk = 0u;
    bi = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > bk) { bk = key[i]; bi = i; }
  };
  uint32_t bk, kth = 0u;
  int bi, pick = -1;
  lane_best(bk, bi);
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, bk);
    const int e = (int)__reduce_min_sync(0xffffffffu, bk == m ? (unsigned)(lane + 32 * bi) : 0x7fffffffu);
    if (lane == j) pick = e;
    kth = m;
    if ((e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == (e >> 5)) key[i] = 0u;
      lane_best(bk, bi);
    }
  }
  const uint32_t nxt = __reduce_max_sync(0xffffffffu, bk);     // best of those left (0: none)
  if (nxt) {
    const float a = route_unimage(kth), b = route_unimage(nxt);
    const float gap = a == b ? 0.f : a - b;
    const float tol = tol_s + 5e-7f * fabsf(a);
    tie |= gap < kNearTie;
    if (!again && gap <= tol && a > -INFINITY) {
      // close: unless every candidate around the border has the last pick's logit and bias
      const int e_k = __shfl_sync(0xffffffffu, pick, k - 1);
      float zk = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == (e_k >> 5)) zk = z[i];
      zk = __shfl_sync(0xffffffffu, zk, e_k & 31);
      const float bk_ = bias ? __ldg(bias + e_k) : 0.f;
      bool other = false;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (full[i] && fabsf(route_unimage(full[i]) - a) <= 2.f * tol)
          other |= z[i] != zk || (bias && __ldg(bias + e) != bk_);
      }
      again = __any_sync(0xffffffffu, other);
    }
  }
  if (again) {
    float zc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) zc[i] = z[i];
    pick = route_pick_exact<NV>(r, zc, bias);
  }
  if (near_tie && lane == 0) *near_tie = tie ? 1 : 0;

  // ascending ids: rank of each pick among the picks, then weights from s
  int rank = 0;
  for (int i = 0; i < k; ++i) rank += __shfl_sync(0xffffffffu, pick, i) < pick;
  float my = 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = __shfl_sync(0xffffffffu, pick, j);
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i == (e >> 5)) v = s[i];
    v = __shfl_sync(0xffffffffu, v, e & 31);
    if (lane == j) my = v;
  }
  float sum = 1.f;
  if (r.renorm) {
    sum = lane < k ? my : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (lane < k) {
    topk_idx[rank] = pick;
    topk_w[rank] = sum > 0.f ? r.scale * my / sum : 0.f;
    if (sel_out) sel_out[rank] = pick;
  }
  __syncwarp();
}

}  // namespace coli
