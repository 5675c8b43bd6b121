// Rotary positions: of any part of any heads, and of the rows that go into the
// paged cache.  "25GB RAM runs 744B GLM-5.2" page (pwwt.cn), section 3.2: 64 of
// the 576 cached values carry the positions.
//
// A pair (a, b) at position t turns by the angle t f_j.  Frequencies are kept in
// units of 2^-64 turns: the product with the position modulo 2^64 is the exact
// fraction of a turn, at any position, with one integer multiplication; its sine
// and cosine then need no range reduction.
#include <cmath>

#include "plan.h"

namespace coli {

constexpr int kRopeThreads = 128, kRopeItems = 4;   // pieces (of a row) a thread, all loads in flight at once
constexpr int kRopeMaxDim = 256;

// (amplitude cos, amplitude sin) of position * freq
__device__ __forceinline__ float2 rope_turn(int32_t position, unsigned long long freq, float amplitude) {
  const unsigned long long phase = (unsigned long long)(long long)position * freq;
  // in half turns, -1 .. 1: the conversion keeps 24 bits of small angles too
  const float x = __ll2float_rn((long long)phase) * 1.0842021724855044e-19f;   // 2^-63
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}
__device__ __forceinline__ float2 rope_rotate(float a, float b, float2 t) {
  return make_float2(fmaf(a, t.x, -b * t.y), fmaf(a, t.y, b * t.x));
}

template <typename T>
__device__ __forceinline__ float2 rope_unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 rope_unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 rope_unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t rope_pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t rope_pack<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t rope_pack<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float rope_load(const T* p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return rope_unpack<T>(*reinterpret_cast<const uint16_t*>(p)).x;
}
template <typename T>
__device__ __forceinline__ void rope_store(T* p, float v) {
  if constexpr (sizeof(T) == 4) *p = v;
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)rope_pack<T>(v, 0.f);
}

struct RopeArgs {
  int n, H, pairs;
  int tokens, heads, pieces;         // of a CTA: tokens, heads; of a head: pieces
  FastDiv by_pieces, by_heads;
  float amplitude;
  const int32_t *n_valid, *position;
  const unsigned long long* freq;
  const uint8_t* x;
  uint8_t* out;
  long long x_tok, x_head, out_tok, out_head;    // elements
};

// BYTES of a vector, as the alignment allows: 16, 8, 4, or 0: values one by one.
template <int BYTES>
struct RopeVec {
  alignas(BYTES ? BYTES : 4) uint32_t w[BYTES ? BYTES / 4 : 1];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
};

// A piece is a vector (in the half layout one of either half), or one pair.  A CTA takes some tokens and heads; its threads'
// pieces are loaded first, the tokens' sines and cosines computed meanwhile, once for all heads.
// A copy in its traffic, 128 bytes a head of 64 16-bit values read and written: 8192 tokens of 64 heads take 22.0 us, 6.1 TB/s
// (24.1 with 256 threads a CTA; with those 26.2 by two pieces a thread and 29.0 by eight).  One token: 2.3 us.
template <typename T, bool HALF, int BYTES>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs p) {
  extern __shared__ __align__(16) float2 turn[];           // [tokens][pairs]
  constexpr int kV = BYTES ? BYTES / (int)sizeof(T) : 1;   // values of a vector
  constexpr int kPairs = BYTES && !HALF ? kV / 2 : kV;     // pairs of a piece
  static_assert(kPairs > 0, "whole pairs");
  const int tid = threadIdx.x;
  const int tok0 = blockIdx.x * p.tokens, head0 = blockIdx.y * p.heads;
  const int tokens = min(p.tokens, p.n - tok0), heads = min(p.heads, p.H - head0);
  const int valid = p.n_valid ? *p.n_valid : p.n;          // (awaited where the results are written)
  const int items = p.tokens * p.heads * p.pieces;
  const T* x = reinterpret_cast<const T*>(p.x);
  T* out = reinterpret_cast<T*>(p.out);

  RopeVec<BYTES> lo[kRopeItems], hi[kRopeItems];
  float a[kRopeItems], b[kRopeItems];                    // BYTES = 0
  int tok[kRopeItems], pair[kRopeItems];
  long long at[kRopeItems];
  // One round (the host takes no more items than that).  A loop all the same, since it keeps the compiler from mixing the loads
  // with the sines and cosines, for which it takes more registers: written straight 8192 tokens take 25.0 us, not 22.6 (heads
  // of 40 in the half layout 24.1, not 20.4; the straight form held to 8 or 9 CTAs an SM 24.8 and 24.4).
  for (int i0 = 0; i0 < items; i0 += kRopeThreads * kRopeItems) {
#pragma unroll
    for (int k = 0; k < kRopeItems; ++k) {
      const int i = i0 + k * kRopeThreads + tid, row = p.by_pieces(i), c = (i - row * p.pieces) * kPairs;
      const int t = p.by_heads(row), h = row - t * p.heads;
      tok[k] = -1;
      if (i >= items || t >= tokens || h >= heads) continue;
      tok[k] = t;
      pair[k] = c;
      const T* src = x + (tok0 + t) * p.x_tok + (head0 + h) * p.x_head + (HALF ? c : 2 * c);
      at[k] = (tok0 + t) * p.out_tok + (head0 + h) * p.out_head + (HALF ? c : 2 * c);
      if constexpr (BYTES) {
        lo[k].load(src);
        if (HALF) hi[k].load(src + p.pairs);
      } else {
        a[k] = rope_load(src);
        b[k] = rope_load(src + (HALF ? p.pairs : 1));
      }
    }
    if (i0 == 0) {
      for (int i = tid; i < tokens * p.pairs; i += kRopeThreads) {
        const int t = i / p.pairs, j = i - t * p.pairs;
        turn[i] = rope_turn(p.position[tok0 + t], p.freq[j], p.amplitude);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kRopeItems; ++k) {
      if (tok[k] < 0 || tok0 + tok[k] >= valid) continue;
      const float2* w = turn + tok[k] * p.pairs + pair[k];
      T* dst = out + at[k];
      if constexpr (!BYTES) {
        const float2 r = rope_rotate(a[k], b[k], w[0]);
        rope_store(dst, r.x);
        rope_store(dst + (HALF ? p.pairs : 1), r.y);
      } else {
        uint32_t* u = lo[k].w;
        uint32_t* v = hi[k].w;
        constexpr int kWords = BYTES / 4;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            uint32_t &f = HALF ? u[i] : u[2 * i], &g = HALF ? v[i] : u[2 * i + 1];
            const float2 z = rope_rotate(__uint_as_float(f), __uint_as_float(g), w[i]);
            f = __float_as_uint(z.x);
            g = __float_as_uint(z.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            if constexpr (HALF) {
              const float2 f = rope_unpack<T>(u[i]), g = rope_unpack<T>(v[i]);
              const float2 y = rope_rotate(f.x, g.x, w[2 * i]), z = rope_rotate(f.y, g.y, w[2 * i + 1]);
              u[i] = rope_pack<T>(y.x, z.x);
              v[i] = rope_pack<T>(y.y, z.y);
            } else {
              const float2 f = rope_unpack<T>(u[i]), z = rope_rotate(f.x, f.y, w[i]);
              u[i] = rope_pack<T>(z.x, z.y);
            }
          }
        }
        if (HALF) hi[k].store(dst + p.pairs);
        lo[k].store(dst);
      }
    }
  }
}

// ------------------------------------------------------------------ append with norm and rotation
// A warp takes a row: a lane holds 16 of its latent values and one pair of its rotary ones.  Nothing waits for *n_valid,
// slots or positions before the row's loads are in flight.  A copy in its traffic (75.8 MB for 32768 rows: 16.3 us, 4.65 TB/s;
// with four rows a warp 19.1, two 18.6, one 17.6, and one with 40 registers, so that 48 warps an SM fit, 16.3).  192 rows: 2.2 us.
constexpr int kArWarps = 4;
static_assert(COLI_KV_VALUE == 32 * 16 && COLI_KV_ROTARY == 64, "16 values and a pair a lane");

struct AppendRopeArgs {
  int n, page_size, n_pages;
  FastDiv by_page;
  long long page_stride;                          // elements
  float eps, amplitude;
  const int32_t *n_valid, *position, *slot;
  const unsigned long long* freq;
  const uint16_t *latent, *rope;
  long long latent_stride, rope_stride;           // elements
  const float* gain;
  uint16_t* cache;
};

template <typename T, bool HALF>
__global__ void __launch_bounds__(kArWarps * 32, 12) kv_append_rope_kernel(const AppendRopeArgs p) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kArWarps + (threadIdx.x >> 5);
  if (row >= p.n) return;
  const uint4* src = reinterpret_cast<const uint4*>(p.latent + row * p.latent_stride);
  uint4 v[2] = {src[lane], src[32 + lane]};
  const uint16_t* rs = p.rope + row * p.rope_stride;
  const uint32_t rot = HALF ? (uint32_t)rs[lane] | ((uint32_t)rs[lane + 32] << 16) : *reinterpret_cast<const uint32_t*>(rs + 2 * lane);
  const int slot = p.slot[row], position = p.position[row];
  const unsigned long long freq = p.freq[lane];
  const int page = p.by_page(max(slot, 0));
  if ((p.n_valid && row >= *p.n_valid) || slot < 0 || page >= p.n_pages) return;       // (the same in every lane)
  uint16_t* dst = p.cache + page * p.page_stride + (long long)(slot - page * p.page_size) * COLI_KV_WIDTH;
  if (p.gain) {
    uint32_t* w = &v[0].x;
    auto squares = [&](float s) {                      // sum of the row's (s x)^2
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = rope_unpack<T>(w[i]);
        sum = fmaf(f.x * s, f.x * s, fmaf(f.y * s, f.y * s, sum));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      return sum * (1.0f / COLI_KV_VALUE);
    };
    float s = 1.f, mean = squares(1.f) + p.eps;
    if (!(mean > 1e-30f && mean < 1e36f)) {
      // squares or eps that leave fp32's range: the row times a power of two near 1 / its largest value.  Up only where squares
      // are small, and then no further than 2^60 where there is an eps (below 1e-30; it decides); else down by 2^30 at least,
      // so that the sum with an eps of any size is finite
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = rope_unpack<T>(w[i]);
        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = (int)(__float_as_uint(top) >> 23) - 127;
      const int most = mean >= 1e36f ? -30 : p.eps > 0.f ? 60 : 126;
      s = __uint_as_float((uint32_t)(max(-126, min(-e, most)) + 127) << 23);
      mean = squares(s) + p.eps * s * s;
    }
    const float by = 1.0f / sqrtf(mean);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 g = *reinterpret_cast<const float4*>(p.gain + (i >> 1) * 256 + lane * 8 + (i & 1) * 4);
      const float2 a = rope_unpack<T>(w[2 * i]), b = rope_unpack<T>(w[2 * i + 1]);
      w[2 * i] = rope_pack<T>(a.x * s * by * g.x, a.y * s * by * g.y);
      w[2 * i + 1] = rope_pack<T>(b.x * s * by * g.z, b.y * s * by * g.w);
    }
  }
  reinterpret_cast<uint4*>(dst)[lane] = v[0];
  reinterpret_cast<uint4*>(dst)[32 + lane] = v[1];
  const float2 f = rope_unpack<T>(rot);
  const float2 z = rope_rotate(f.x, f.y, rope_turn(position, freq, p.amplitude));
  const uint32_t two = rope_pack<T>(z.x, z.y);
  if (HALF) {
    dst[COLI_KV_VALUE + lane] = (uint16_t)two;
    dst[COLI_KV_VALUE + 32 + lane] = (uint16_t)(two >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(dst + COLI_KV_VALUE + 2 * lane) = two;
  }
}

static coli_status check_rope_desc(const coli_rope_desc* d, const char* who) {
  if (!d) return fail(COLI_EINVAL, "%s: null description of the rotation", who);
  if (d->dim < 2 || d->dim > kRopeMaxDim || d->dim % 2)
    return fail(COLI_EINVAL, "%s: dim=%d must be even, from 2 to %d", who, d->dim, kRopeMaxDim);
  if (d->layout != COLI_ROPE_INTERLEAVED && d->layout != COLI_ROPE_HALF)
    return fail(COLI_EINVAL, "%s: unknown layout %d", who, d->layout);
  if (!std::isfinite(d->amplitude)) return fail(COLI_EINVAL, "%s: amplitude is not finite", who);
  return COLI_OK;
}

template <typename T, bool HALF>
static void rope_launch(const RopeArgs& a, int bytes, dim3 grid, size_t smem, cudaStream_t st) {
  constexpr int kLeast = sizeof(T) == 4 && !HALF ? 8 : 4;  // bytes of the smallest vector of whole pairs
  auto k = bytes == 16 ? rope_kernel<T, HALF, 16> : bytes == 8 ? rope_kernel<T, HALF, 8>
                       : bytes == 4 ? rope_kernel<T, HALF, kLeast> : rope_kernel<T, HALF, 0>;
  k<<<grid, kRopeThreads, smem, st>>>(a);
}

}  // namespace coli

using namespace coli;

extern "C" {

coli_status colibri_rope_frequencies(const coli_rope_desc* desc, uint64_t* freq) {
  const coli_status rc = check_rope_desc(desc, "rope_frequencies");
  if (rc != COLI_OK) return rc;
  if (!freq) return fail(COLI_EINVAL, "rope_frequencies: null pointer");
  const coli_rope_desc& d = *desc;
  if (!(d.base > 1.0) || !std::isfinite(d.base)) return fail(COLI_EINVAL, "rope_frequencies: base must be above 1 and finite");
  if (d.scaling < COLI_ROPE_NONE || d.scaling > COLI_ROPE_YARN)
    return fail(COLI_EINVAL, "rope_frequencies: unknown scaling %d", d.scaling);
  if (d.scaling != COLI_ROPE_NONE && (!(d.factor >= 1.0) || !std::isfinite(d.factor)))
    return fail(COLI_EINVAL, "rope_frequencies: factor must be at least 1 and finite");
  const double pi = 3.14159265358979323846;
  double low = 0, high = 0;
  if (d.scaling == COLI_ROPE_YARN) {
    if (!(d.original_len > 0) || !std::isfinite(d.original_len))
      return fail(COLI_EINVAL, "rope_frequencies: original_len must be positive and finite");
    if (!(d.beta_slow > 0) || !(d.beta_fast > d.beta_slow) || !std::isfinite(d.beta_fast))
      return fail(COLI_EINVAL, "rope_frequencies: need beta_fast > beta_slow > 0, finite");
    auto pair_of = [&](double turns) { return d.dim * std::log(d.original_len / (turns * 2 * pi)) / (2 * std::log(d.base)); };
    low = std::fmax(std::floor(pair_of(d.beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(d.beta_slow)), d.dim - 1.0);
    if (!(high > low)) high = low + 0.001;
  }
  for (int j = 0; j < d.dim / 2; ++j) {
    const double e = -2.0 * j / d.dim;
    double f = std::pow(d.base, e);
    if (d.scaling == COLI_ROPE_LINEAR) f /= d.factor;
    if (d.scaling == COLI_ROPE_NTK && d.dim > 2) f *= std::pow(d.factor, e * d.dim / (d.dim - 2.0));
    if (d.scaling == COLI_ROPE_YARN) {
      const double g = std::fmin(std::fmax((j - low) / (high - low), 0.0), 1.0);
      f = f * (1 - g) + f / d.factor * g;
    }
    freq[j] = (uint64_t)std::nearbyint(std::ldexp(f / (2 * pi), 64));       // (f <= 1: below 2^62)
  }
  return COLI_OK;
}

coli_status colibri_rope(const coli_rope_desc* desc, int dtype, int n_tokens, const int32_t* n_valid, int H,
                         const int32_t* position, const uint64_t* freq, const void* x, long long x_token_stride,
                         long long x_head_stride, void* out, long long out_token_stride, long long out_head_stride,
                         void* stream) {
  const coli_status rc = check_rope_desc(desc, "rope");
  if (rc != COLI_OK) return rc;
  if (n_tokens < 0 || H < 1) return fail(COLI_EINVAL, "rope: need n_tokens >= 0 and H >= 1");
  if (H > 1024) return fail(COLI_EUNSUPPORTED, "rope: H=%d exceeds 1024 heads", H);
  if (dtype != COLI_X_BF16 && dtype != COLI_X_F16 && dtype != COLI_X_F32)
    return fail(COLI_EUNSUPPORTED, "rope: bf16, fp16 or fp32 (dtype %d)", dtype);
  if (n_tokens == 0) return COLI_OK;
  if (!position || !freq || !x || !out) return fail(COLI_EINVAL, "rope: null pointer");
  const int size = dtype == COLI_X_F32 ? 4 : 2;
  if (!aligned(position, 4) || !aligned(n_valid, 4) || !aligned(freq, 8) || !aligned(x, size) || !aligned(out, size))
    return fail(COLI_EALIGN, "rope: position and n_valid 4-byte, freq 8-byte alignment, x and out that of their elements");
  const long long xt = n_tokens > 1 ? x_token_stride : 0, xh = H > 1 ? x_head_stride : 0;
  const long long ot = n_tokens > 1 ? out_token_stride : 0, oh = H > 1 ? out_head_stride : 0;
  if (xt < 0 || xh < 0) return fail(COLI_EINVAL, "rope: a stride of x is negative");
  if ((n_tokens > 1 && ot < desc->dim) || (H > 1 && oh < desc->dim)) return fail(COLI_EINVAL, "rope: outputs overlap (strides of out)");
  if (x == out && (xt != ot || xh != oh)) return fail(COLI_EINVAL, "rope: in place, but with other strides of out than of x");
  RopeArgs a;
  const bool half = desc->layout == COLI_ROPE_HALF;
  // the largest vector that strides, addresses and the row's pieces are whole multiples of (2763 tokens of 128 heads of 64
  // values: by 16 bytes 16.4 us, 8 bytes 22.1, 4 bytes 24.4, value by value 58.7)
  const unsigned long long mixed = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out) |
                                   (unsigned long long)(xt * size) | (unsigned long long)(xh * size) |
                                   (unsigned long long)(ot * size) | (unsigned long long)(oh * size) |
                                   (unsigned long long)((half ? desc->dim / 2 : desc->dim) * size);
  int bytes = mixed % 16 == 0 ? 16 : mixed % 8 == 0 ? 8 : mixed % 4 == 0 ? 4 : 0;
  if (bytes == 4 && size == 4 && !half) bytes = 0;         // (half a pair)
  const int values = bytes ? bytes / size : 1, pairs = bytes && !half ? values / 2 : values;     // of a piece
  a.n = n_tokens;
  a.H = H;
  a.pairs = desc->dim / 2;
  a.pieces = a.pairs / pairs;
  const int room = kRopeThreads * kRopeItems;
  a.heads = a.pieces * H <= room ? H : room / a.pieces;      // (at most 128 pieces)
  a.tokens = room / (a.pieces * a.heads);
  if (a.tokens > 32) a.tokens = 32;
  a.by_pieces.set(a.pieces);
  a.by_heads.set(a.heads);
  a.amplitude = desc->amplitude;
  a.n_valid = n_valid;
  a.position = position;
  a.freq = reinterpret_cast<const unsigned long long*>(freq);
  a.x = static_cast<const uint8_t*>(x);
  a.out = static_cast<uint8_t*>(out);
  a.x_tok = xt;
  a.x_head = xh;
  a.out_tok = ot;
  a.out_head = oh;
  const dim3 grid(n_tokens / a.tokens + (n_tokens % a.tokens ? 1 : 0), (H + a.heads - 1) / a.heads);
  const size_t smem = (size_t)a.tokens * a.pairs * sizeof(float2);           // (at most 32 KB)
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == COLI_X_BF16) half ? rope_launch<__nv_bfloat16, true>(a, bytes, grid, smem, st) : rope_launch<__nv_bfloat16, false>(a, bytes, grid, smem, st);
  else if (dtype == COLI_X_F16) half ? rope_launch<__half, true>(a, bytes, grid, smem, st) : rope_launch<__half, false>(a, bytes, grid, smem, st);
  else half ? rope_launch<float, true>(a, bytes, grid, smem, st) : rope_launch<float, false>(a, bytes, grid, smem, st);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "rope");
}

coli_status colibri_kv_append_rope(const coli_kv_desc* desc, const coli_rope_desc* rope_desc, int n_tokens,
                                   const int32_t* n_valid, const void* latent, long long latent_stride,
                                   const float* gain, float eps, const void* rope, long long rope_stride,
                                   const int32_t* position, const uint64_t* freq, const int32_t* slot, void* cache,
                                   void* stream) {
  coli_status rc = check_kv_desc(desc, "kv_append_rope");
  if (rc == COLI_OK) rc = check_rope_desc(rope_desc, "kv_append_rope");
  if (rc != COLI_OK) return rc;
  if (rope_desc->dim != COLI_KV_ROTARY) return fail(COLI_EINVAL, "kv_append_rope: dim=%d, cached rows have 64 rotary values", rope_desc->dim);
  if (desc->dtype != COLI_X_BF16 && desc->dtype != COLI_X_F16)
    return fail(COLI_EUNSUPPORTED, "kv_append_rope: the cache holds bf16 or fp16 (dtype %d)", desc->dtype);
  if (n_tokens < 0) return fail(COLI_EINVAL, "kv_append_rope: n_tokens=%d is negative", n_tokens);
  if (gain && !(eps >= 0.f && eps <= 3.402823466e38f)) return fail(COLI_EINVAL, "kv_append_rope: eps must be at least 0 and finite");
  if (n_tokens == 0) return COLI_OK;
  if (!latent || !rope || !slot || !cache || !position || !freq) return fail(COLI_EINVAL, "kv_append_rope: null pointer");
  if (latent_stride < 0 || rope_stride < 0) return fail(COLI_EINVAL, "kv_append_rope: a stride is negative");
  if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(cache, 16) || !aligned(gain, 16) || latent_stride % 8 || rope_stride % 8)
    return fail(COLI_EALIGN, "kv_append_rope: latent, rope, gain and cache 16-byte aligned, strides multiples of 8");
  if (!aligned(slot, 4) || !aligned(n_valid, 4) || !aligned(position, 4) || !aligned(freq, 8))
    return fail(COLI_EALIGN, "kv_append_rope: slot, n_valid, position or freq misaligned");
  AppendRopeArgs a;
  a.n = n_tokens;
  a.page_size = desc->page_size;
  a.n_pages = desc->n_pages;
  a.by_page.set(desc->page_size);
  a.page_stride = desc->page_stride;
  a.eps = eps;
  a.amplitude = rope_desc->amplitude;
  a.n_valid = n_valid;
  a.position = position;
  a.slot = slot;
  a.freq = reinterpret_cast<const unsigned long long*>(freq);
  a.latent = static_cast<const uint16_t*>(latent);
  a.rope = static_cast<const uint16_t*>(rope);
  a.latent_stride = latent_stride;
  a.rope_stride = rope_stride;
  a.gain = gain;
  a.cache = static_cast<uint16_t*>(cache);
  const int grid = n_tokens / kArWarps + (n_tokens % kArWarps ? 1 : 0);
  const bool half = rope_desc->layout == COLI_ROPE_HALF, bf16 = desc->dtype == COLI_X_BF16;
  auto k = bf16 ? (half ? kv_append_rope_kernel<__nv_bfloat16, true> : kv_append_rope_kernel<__nv_bfloat16, false>)
                : (half ? kv_append_rope_kernel<__half, true> : kv_append_rope_kernel<__half, false>);
  k<<<grid, kArWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "kv_append_rope");
}

}  // extern "C"
