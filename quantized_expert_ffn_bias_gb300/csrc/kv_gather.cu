// Rows of whole requests out of the paged cache, side by side: what the
// up-projection to keys and values of every head reads.  "25GB RAM runs 744B
// GLM-5.2" page (pwwt.cn), section 3.2: 576 cached values a token (512 latent,
// 64 rotary).
//
// A copy, bound by HBM for large batches.  Every CTA scans the lengths into its
// own shared memory, then its warps take four rows at a time (nine full rounds
// of 16-byte pieces, all loads in flight before the first store), round after
// round; the next round's pages are looked up while the rows are on their way.
#include "plan.h"

namespace coli {

constexpr int kKgWarps = 8, kKgThreads = kKgWarps * 32, kKgRows = 4, kKgPieces = COLI_KV_WIDTH * 2 / 16;
constexpr int kKgRounds = kKgRows * kKgPieces / 32, kKgMaxB = 8192;
static_assert(kKgRounds * 32 == kKgRows * kKgPieces, "whole rounds");

struct GatherArgs {
  int B, n_rows, page_size, max_pages, n_pages;
  FastDiv by_page;
  long long page_stride;               // bytes
  const int32_t *seq_len, *table;
  const uint8_t* cache;
  int32_t *k_start, *status;
  uint8_t *latent, *rope;
  long long latent_stride, rope_stride;     // bytes
};

__global__ void __launch_bounds__(kKgThreads) kv_gather_kernel(const GatherArgs p) {
  extern __shared__ int starts[];      // [B + 1] first row of each request, at most n_rows
  __shared__ unsigned warp_tot[kKgWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // sums that stop at n_rows + 1 (one more than there is room for is as good as any)
  const unsigned cap = (unsigned)p.n_rows + 1u;
  unsigned carry = 0;
  int bits = 0;
  for (int b0 = 0; b0 < p.B; b0 += kKgThreads) {
    const int b = b0 + tid;
    unsigned v = 0;
    if (b < p.B) {
      const int s = p.seq_len[b];
      if (s < 0) bits |= COLI_DEV_KV_TABLE_FULL;
      v = min((unsigned)max(s, 0), cap);
    }
    unsigned inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = min(inc + n, cap);          // (both at most 2^31: no wrap)
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    unsigned base = carry, all = carry;
#pragma unroll
    for (int w = 0; w < kKgWarps; ++w) {
      if (w < warp) base = min(base + warp_tot[w], cap);
      all = min(all + warp_tot[w], cap);
    }
    if (b < p.B) starts[b + 1] = (int)min(base + inc, (unsigned)p.n_rows);
    carry = all;
    __syncthreads();
  }
  if (tid == 0) starts[0] = 0;
  if (carry == cap) bits |= COLI_DEV_KV_TOKENS;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.B; b += kKgThreads) p.k_start[b] = starts[b];
  const int n = starts[p.B];

  // lanes 0..3 of a warp: where row (first + lane) lies, -1 where it has no page
  auto find = [&](int first) {
    long long from = -1;
    const int row = first + lane;
    if (lane < kKgRows && row < n) {
      int l = 0, h = p.B;                              // last request that starts at or before the row: it has rows
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (starts[mid] <= row) l = mid;
        else h = mid;
      }
      const int key = row - starts[l], col = p.by_page(key);
      const int page = col < p.max_pages ? p.table[(size_t)l * p.max_pages + col] : -1;
      if (page >= 0 && page < p.n_pages) from = page * p.page_stride + (long long)(key - col * p.page_size) * (COLI_KV_WIDTH * 2);
      else bits |= COLI_DEV_KV_BAD_PAGE;
    }
    return from;
  };
  const long long step = (long long)gridDim.x * kKgWarps * kKgRows;
  long long row0 = ((long long)blockIdx.x * kKgWarps + warp) * kKgRows;
  long long from = row0 < n ? find((int)row0) : -1;
  for (; row0 < n; row0 += step) {
    uint4 v[kKgRounds];
#pragma unroll
    for (int i = 0; i < kKgRounds; ++i) {
      const int piece = i * 32 + lane, r = piece / kKgPieces, c = piece - r * kKgPieces;
      const long long at = __shfl_sync(0xffffffffu, from, r);
      v[i] = make_uint4(0, 0, 0, 0);
      if (at >= 0) v[i] = *reinterpret_cast<const uint4*>(p.cache + at + c * 16);
    }
    if (row0 + step < n) from = find((int)(row0 + step));
#pragma unroll
    for (int i = 0; i < kKgRounds; ++i) {
      const int piece = i * 32 + lane, r = piece / kKgPieces, c = piece - r * kKgPieces;
      const long long row = row0 + r;
      if (row >= n) continue;
      if (c < COLI_KV_VALUE * 2 / 16) *reinterpret_cast<uint4*>(p.latent + row * p.latent_stride + c * 16) = v[i];
      else *reinterpret_cast<uint4*>(p.rope + row * p.rope_stride + (c - COLI_KV_VALUE * 2 / 16) * 16) = v[i];
    }
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace coli

using namespace coli;

extern "C" {

coli_status colibri_kv_gather(const coli_kv_desc* desc, int B, int n_rows, const int32_t* seq_len,
                              const int32_t* block_table, const void* cache, int32_t* k_start, void* latent,
                              long long latent_stride, void* rope, long long rope_stride, int32_t* status, void* stream) {
  const coli_status rc = check_kv_desc(desc, "kv_gather");
  if (rc != COLI_OK) return rc;
  if (B < 1 || n_rows < 0) return fail(COLI_EINVAL, "kv_gather: need B >= 1 and n_rows >= 0");
  if (B > kKgMaxB) return fail(COLI_EUNSUPPORTED, "kv_gather: B=%d exceeds %d requests", B, kKgMaxB);
  if (n_rows > 0x7fffffff - 4096) return fail(COLI_EUNSUPPORTED, "kv_gather: n_rows exceeds 2^31 - 4096");
  if (!seq_len || !block_table || !cache || !k_start || !status || (n_rows > 0 && (!latent || !rope)))
    return fail(COLI_EINVAL, "kv_gather: null pointer");
  if (!aligned(seq_len, 4) || !aligned(block_table, 4) || !aligned(k_start, 4) || !aligned(status, 4))
    return fail(COLI_EALIGN, "kv_gather: a pointer is not 4-byte aligned");
  if (!aligned(cache, 16) || !aligned(latent, 16) || !aligned(rope, 16))
    return fail(COLI_EALIGN, "kv_gather: cache, latent and rope 16-byte aligned");
  if (n_rows > 1) {
    if (latent_stride < COLI_KV_VALUE || rope_stride < COLI_KV_ROTARY)
      return fail(COLI_EINVAL, "kv_gather: strides of at least 512 (latent) and 64 (rope)");
    if (latent_stride % 8 || rope_stride % 8) return fail(COLI_EALIGN, "kv_gather: strides must be multiples of 8 elements");
  }
  GatherArgs a;
  a.B = B;
  a.n_rows = n_rows;
  a.page_size = desc->page_size;
  a.max_pages = desc->max_pages;
  a.n_pages = desc->n_pages;
  a.by_page.set(desc->page_size);
  a.page_stride = desc->page_stride * 2;
  a.seq_len = seq_len;
  a.table = block_table;
  a.cache = static_cast<const uint8_t*>(cache);
  a.k_start = k_start;
  a.status = status;
  a.latent = static_cast<uint8_t*>(latent);
  a.rope = static_cast<uint8_t*>(rope);
  a.latent_stride = latent_stride * 2;
  a.rope_stride = rope_stride * 2;
  // CTAs that stay: each scans the lengths once
  constexpr int kRows = kKgWarps * kKgRows, kMost = 152 * 4;
  const int want = n_rows / kRows + 1;
  kv_gather_kernel<<<want < kMost ? want : kMost, kKgThreads, (size_t)(B + 1) * 4, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "kv_gather");
}

}  // extern "C"
