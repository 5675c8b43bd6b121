// Routing to experts from given logits (colibri_moe_route): one warp per token,
// the token's E logits in registers (NV a lane).  "25GB RAM runs 744B GLM-5.2"
// page (pwwt.cn), section 3.1: DeepSeek-V3 style router; the selection itself
// is in route_select.cuh.
#include "plan.h"
#include "route_select.cuh"

namespace coli {

constexpr int kRouteWarps = 4;

struct RouteCall {
  coli_route_desc r;
  int T;
  const void* logits;
  long long stride;
  const float* bias;
  int32_t* idx;
  float* w;
};

template <int LT>
__device__ __forceinline__ float route_load(const void* p, size_t i) {
  float v;
  if constexpr (LT == COLI_X_F32) v = __ldg(static_cast<const float*>(p) + i);
  else if constexpr (LT == COLI_X_BF16)
    v = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16);
  else v = __half2float(__ushort_as_half(__ldg(static_cast<const uint16_t*>(p) + i)));
  return v == v ? v : -INFINITY;
}

// VEC: rows and biases start on 16-byte borders and E is a multiple of NV, so a lane's experts are whole vectors.
template <int LT, int NV, bool VEC>
__global__ void __launch_bounds__(kRouteWarps * 32, NV <= 8 ? 8 : 4) route_kernel(const __grid_constant__ RouteCall c) {
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= c.T) return;
  float z[NV], b[NV];
  const size_t row = (size_t)t * c.stride;
  const int e0 = lane * NV;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    z[i] = -INFINITY;
    b[i] = 0.f;
  }
  if constexpr (VEC) {
    if (e0 < c.r.E) {
      if constexpr (LT == COLI_X_F32) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(c.logits) + row + e0 + i));
          z[i] = v.x; z[i + 1] = v.y; z[i + 2] = v.z; z[i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(c.logits) + row + e0 + i));
          const uint32_t h[4] = {v.x & 0xFFFFu, v.x >> 16, v.y & 0xFFFFu, v.y >> 16};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            z[i + j] = LT == COLI_X_BF16 ? __uint_as_float(h[j] << 16) : __half2float(__ushort_as_half((uint16_t)h[j]));
        }
      }
      if (c.bias)
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(c.bias + e0 + i));
          b[i] = v.x; b[i + 1] = v.y; b[i + 2] = v.z; b[i + 3] = v.w;
        }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (!(z[i] == z[i])) z[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < c.r.E) {
        z[i] = route_load<LT>(c.logits, row + e0 + i);
        if (c.bias) b[i] = __ldg(c.bias + e0 + i);
      }
  }
  const void* logits = c.logits;
  auto logit = [=](int e) { return route_load<LT>(logits, row + e); };
  int32_t* idx = c.idx + (size_t)t * c.r.k;
  float* w = c.w + (size_t)t * c.r.k;
  if (route_token<NV, false>(c.r, z, b, c.bias, logit, idx, w, nullptr, nullptr))
    route_token_exact<NV>(c.r, c.bias, logit, idx, w, nullptr, nullptr);
}

template <int LT, int NV>
static void launch_route_nv(const RouteCall& c, cudaStream_t st) {
  const int blocks = c.T / kRouteWarps + (c.T % kRouteWarps ? 1 : 0);
  const int size = LT == COLI_X_F32 ? 4 : 2;
  const bool vec = c.r.E % NV == 0 && aligned(c.logits, 16) && c.stride * size % 16 == 0 && aligned(c.bias, 16);
  if (vec) route_kernel<LT, NV, true><<<blocks, kRouteWarps * 32, 0, st>>>(c);
  else route_kernel<LT, NV, false><<<blocks, kRouteWarps * 32, 0, st>>>(c);
}

template <int LT>
static void launch_route_lt(const RouteCall& c, cudaStream_t st) {
  if (c.r.E <= 128) launch_route_nv<LT, 4>(c, st);
  else if (c.r.E <= 256) launch_route_nv<LT, 8>(c, st);
  else if (c.r.E <= 384) launch_route_nv<LT, 12>(c, st);
  else if (c.r.E <= 512) launch_route_nv<LT, 16>(c, st);
  else launch_route_nv<LT, 32>(c, st);
}

coli_status check_route_desc(const coli_route_desc& r, const char* who) {
  if (r.E < 1 || r.k < 1) return fail(COLI_EINVAL, "%s: E and k must be positive", who);
  if (r.E > kMaxE) return fail(COLI_EUNSUPPORTED, "%s: E=%d exceeds %d", who, r.E, kMaxE);
  if (r.score != COLI_SCORE_SIGMOID && r.score != COLI_SCORE_SOFTMAX)
    return fail(COLI_EINVAL, "%s: unknown score %d", who, r.score);
  if (r.n_group < 1 || r.n_group > 32 || r.E % r.n_group)
    return fail(COLI_EINVAL, "%s: n_group=%d is not a divisor of E=%d up to 32", who, r.n_group, r.E);
  if (r.topk_group < 1 || r.topk_group > r.n_group)
    return fail(COLI_EINVAL, "%s: topk_group=%d outside [1, %d]", who, r.topk_group, r.n_group);
  if (r.group_score != COLI_GROUP_TOP2 && r.group_score != COLI_GROUP_MAX)
    return fail(COLI_EINVAL, "%s: unknown group_score %d", who, r.group_score);
  if (r.topk_group < r.n_group && r.group_score == COLI_GROUP_TOP2 && r.E / r.n_group < 2)
    return fail(COLI_EINVAL, "%s: groups of one expert have no two largest scores", who);
  if (r.k > kMaxK || r.k > r.E / r.n_group * r.topk_group)
    return fail(COLI_EINVAL, "%s: k=%d exceeds %d or the experts of the kept groups", who, r.k, kMaxK);
  if (r.renorm != 0 && r.renorm != 1) return fail(COLI_EINVAL, "%s: renorm must be 0 or 1", who);
  if (!(r.scale == r.scale)) return fail(COLI_EINVAL, "%s: scale is NaN", who);
  return COLI_OK;
}

}  // namespace coli

using namespace coli;

extern "C" {

coli_status colibri_moe_route(const coli_route_desc* desc, int T, const void* logits, int ltype,
                              long long logit_stride, const float* bias, int32_t* topk_idx, float* topk_w,
                              void* stream) {
  if (!desc) return fail(COLI_EINVAL, "route: null description");
  const coli_status rc = check_route_desc(*desc, "route");
  if (rc != COLI_OK) return rc;
  if (T < 0) return fail(COLI_EINVAL, "route: T=%d is negative", T);
  if (ltype != COLI_X_BF16 && ltype != COLI_X_F32 && ltype != COLI_X_F16)
    return fail(COLI_EUNSUPPORTED, "route: unknown logit type %d", ltype);
  if (logit_stride < desc->E) return fail(COLI_EINVAL, "route: logit_stride is smaller than E");
  if (T == 0) return COLI_OK;
  if (!logits || !topk_idx || !topk_w) return fail(COLI_EINVAL, "route: null pointer");
  if (!aligned(logits, ltype == COLI_X_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return fail(COLI_EALIGN, "route: a pointer is not aligned to its elements");
  const RouteCall c{*desc, T, logits, logit_stride, bias, topk_idx, topk_w};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (ltype == COLI_X_F32) launch_route_lt<COLI_X_F32>(c, st);
  else if (ltype == COLI_X_BF16) launch_route_lt<COLI_X_BF16>(c, st);
  else launch_route_lt<COLI_X_F16>(c, st);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "route");
}

coli_status colibri_moe_set_route(coli_moe_plan_t* plan, const coli_route_desc* desc) {
  if (!plan) return fail(COLI_EINVAL, "set_route: null plan");
  if (!desc) {
    plan->routed = 0;
    return COLI_OK;
  }
  const coli_status rc = check_route_desc(*desc, "set_route");
  if (rc != COLI_OK) return rc;
  if (desc->E != plan->desc.E || desc->k != plan->desc.k)
    return fail(COLI_EINVAL, "set_route: E=%d, k=%d are not the plan's (%d, %d)", desc->E, desc->k, plan->desc.E,
                plan->desc.k);
  plan->route = *desc;
  plan->routed = 1;
  return COLI_OK;
}

}  // extern "C"
