// Paged cache of compressed keys: the bookkeeping of one step (block tables,
// positions, slots, on the GPU from the requests' lengths) and the writing of
// its rows.  "25GB RAM runs 744B GLM-5.2" page (pwwt.cn), section 3.2: MLA
// attention keeps 576 values a token (512 latent, 64 rotary).
//
// Step: one thread-block cluster of 8 CTAs, one launch.  Every CTA scans all
// requests (freed pages, wanted pages, new tokens) into its own shared memory;
// finished requests push their pages, a cluster barrier makes the pushes
// visible and ends every CTA's reading of the inputs (so the outputs may be
// the inputs' arrays), then the new pages, the token rows and the requests'
// results are dealt over the cluster's threads.  What bounds it is latency:
// the launch, the loads of the lengths and of a token's page, the scan's
// barriers (one scan where everything can be served, sums in 32 bits where
// the sizes allow it: 14.3 -> 10.5 us a call for 500 requests of 13,000 tokens,
// a median; a process's calls from Python move it by 2 us).
#include "plan.h"

namespace coli {

constexpr int kStepCtas = 8, kStepThreads = 1024, kStepMaxB = 8192;

struct StepArgs {
  coli_kv_desc d;
  int B, n_tokens;
  const int32_t *new_len, *seq_len, *held;
  int32_t *table, *free_pages;
  const int32_t* free_count;
  int32_t *seq_out, *held_out, *count_out, *q_start, *position, *slot, *status;
  FastDiv by_page;
};

template <typename I>
struct Sum3 {
  I a, b, c;
};

// Block-wide exclusive sums of three values a thread (1024 threads); *total: the block's sums.
template <typename I>
__device__ __forceinline__ Sum3<I> scan3(Sum3<I> v, Sum3<I>* warp_tot, Sum3<I>* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto warp_inc = [lane](Sum3<I> x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sum3<I> n{__shfl_up_sync(0xffffffffu, x.a, o), __shfl_up_sync(0xffffffffu, x.b, o),
                      __shfl_up_sync(0xffffffffu, x.c, o)};
      if (lane >= o) {
        x.a += n.a;
        x.b += n.b;
        x.c += n.c;
      }
    }
    return x;
  };
  const Sum3<I> inc = warp_inc(v);
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const Sum3<I> w = warp_tot[lane], wi = warp_inc(w);
    warp_tot[lane] = Sum3<I>{wi.a - w.a, wi.b - w.b, wi.c - w.c};
    if (lane == 31) *total = wi;
  }
  __syncthreads();
  const Sum3<I> base = warp_tot[warp];
  return Sum3<I>{base.a + inc.a - v.a, base.b + inc.b - v.b, base.c + inc.c - v.c};
}

// Last i in [0, n) with first[i] <= x (first ascending, first[0] <= x).
__device__ __forceinline__ int last_at_most(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// I: type of the sums (64 bits where 8192 requests of wrong lengths could leave 32).
template <typename I>
__global__ void __launch_bounds__(kStepThreads, 1) kv_step_kernel(const StepArgs p) {
  extern __shared__ int step_sm[];
  const int B = p.B;
  int* qs = step_sm;                 // [B + 1] first token row
  int* pp = qs + B + 1;              // [B + 1] first new page
  int* seq = pp + B + 1;             // [B] tokens before the step
  int* hold = seq + B;               // [B] pages before the step
  int* add = hold + B;               // [B] new tokens; -1: finished; -2: lengths that are not valid
  int* back = add + B;               // [B] first place of a finished request's pages among those that return
  __shared__ Sum3<I> warp_tot[32], total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x, ps = p.d.page_size;
  const int count_in = *p.free_count;
  int bits = 0;
  // pages for n more tokens (seq + n <= max_pages * page_size < 2^31)
  auto need_of = [&](int s, int n, int h) { return max(0, p.by_page((int)((unsigned)s + n + ps - 1)) - h); };

  // sums over the requests: pages that return, pages wanted, tokens wanted
  Sum3<I> carry{0, 0, 0};
  for (int base = 0; base < B; base += kStepThreads) {
    const int b = base + tid;
    Sum3<I> v{0, 0, 0};
    if (b < B) {
      const int n = p.new_len[b], s = p.seq_len[b];
      int h = p.held[b];
      const bool fine = h >= 0 && h <= p.d.max_pages;
      if (!fine) h = 0;
      int a;
      if (n < 0) {
        a = -1;
        v.a = h;
        if (!fine) bits |= COLI_DEV_KV_TABLE_FULL;
      } else if (fine && s >= 0 && s <= (long long)h * ps && (long long)s + n <= (long long)p.d.max_pages * ps) {
        a = n;
        v.b = need_of(s, n, h);
        v.c = (I)min(n, p.n_tokens) + (n > p.n_tokens);      // (more than there is room for is as good as all of it)
      } else {
        a = -2;
        bits |= COLI_DEV_KV_TABLE_FULL;
      }
      seq[b] = s;
      hold[b] = h;
      add[b] = a;
    }
    const Sum3<I> e = scan3(v, warp_tot, &total);
    if (b < B) {
      back[b] = (int)min((long long)(carry.a + e.a), (long long)p.d.n_pages);
      pp[b] = (int)min((long long)(carry.b + e.b), 0x7fffffffLL);
      qs[b] = (int)min((long long)(carry.c + e.c), 0x7fffffffLL);
    }
    carry.a += total.a;
    carry.b += total.b;
    carry.c += total.c;
    __syncthreads();
  }
  const int count0 = max(0, min(count_in, p.d.n_pages));
  // more pages than the cache has can only come from wrong inputs: they are dropped
  const int avail = (int)min((long long)p.d.n_pages, (long long)count0 + carry.a);
  if ((long long)count0 + carry.a > p.d.n_pages || count_in != count0) bits |= COLI_DEV_KV_BAD_PAGE;
  // push the finished requests' pages (a warp per request, dealt over the cluster)
  if (carry.a > 0)
    for (int b = rank * 32 + warp; b < B; b += kStepCtas * 32) {
      if (add[b] != -1) continue;
      // eight loads on their way at a time: a long request has hundreds of pages
      const int n = min((long long)hold[b], p.d.n_pages - ((long long)count0 + back[b]));
      const int32_t* from = p.table + (size_t)b * p.d.max_pages;
      int32_t* to = p.free_pages + ((long long)count0 + back[b]);
      for (int i0 = lane; i0 < n; i0 += 8 * 32) {
        int32_t page[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + j * 32 < n) page[j] = from[i0 + j * 32];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + j * 32 < n) to[i0 + j * 32] = page[j];
      }
    }
  int n_new = (int)min((long long)carry.b, 0x7fffffffLL), n_rows = (int)min((long long)carry.c, 0x7fffffffLL);
  if (carry.b > avail || carry.c > p.n_tokens) {
    // Not everything can be served: a request is when what it and those before it ask for is there (the sums so
    // far); the served ones' sums follow.
    __syncthreads();
    Sum3<I> given{0, 0, 0};
    for (int base = 0; base < B; base += kStepThreads) {
      const int b = base + tid;
      int need = 0, want = 0;
      if (b < B && add[b] >= 0) {
        need = need_of(seq[b], add[b], hold[b]);
        want = add[b];
        const bool pages = need > 0 && (long long)pp[b] + need > avail;
        const bool rows = want > 0 && (long long)qs[b] + want > p.n_tokens;
        if (pages) bits |= COLI_DEV_KV_NO_PAGES;
        if (rows) bits |= COLI_DEV_KV_TOKENS;
        if (pages || rows) {
          need = want = 0;
          add[b] = -2;
        }
      }
      const Sum3<I> e = scan3(Sum3<I>{0, (I)need, (I)want}, warp_tot, &total);
      if (b < B) {
        pp[b] = (int)(given.b + e.b);
        qs[b] = (int)(given.c + e.c);
      }
      given.b += total.b;
      given.c += total.c;
      __syncthreads();
    }
    n_new = (int)given.b;
    n_rows = (int)given.c;
  }
  if (tid == 0) {
    pp[B] = n_new;
    qs[B] = n_rows;
  }
  // every CTA has read the inputs, every push is visible
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();

  const int gtid = rank * kStepThreads + tid, gthreads = kStepCtas * kStepThreads;
  auto popped = [&](int i) { return __ldcg(p.free_pages + (avail - 1 - i)); };   // the i-th new page
  for (int i = gtid; i < n_rows; i += gthreads) {
    const int b = last_at_most(qs, B, i);
    const int pos = seq[b] + (i - qs[b]), col = p.by_page(pos);
    const int page = col < hold[b] ? p.table[(size_t)b * p.d.max_pages + col] : popped(pp[b] + col - hold[b]);
    const bool in = page >= 0 && page < p.d.n_pages;
    if (!in) bits |= COLI_DEV_KV_BAD_PAGE;
    p.position[i] = pos;
    p.slot[i] = in ? page * ps + (pos - col * ps) : -1;
  }
  for (int j = gtid; j < n_new; j += gthreads) {
    const int b = last_at_most(pp, B, j);
    p.table[(size_t)b * p.d.max_pages + hold[b] + (j - pp[b])] = popped(j);
  }
  for (int b = gtid; b < B; b += gthreads) {
    const bool dead = add[b] == -1;
    p.q_start[b] = qs[b];
    p.seq_out[b] = dead ? 0 : seq[b] + (qs[b + 1] - qs[b]);
    p.held_out[b] = dead ? 0 : hold[b] + (pp[b + 1] - pp[b]);
  }
  if (gtid == 0) {
    p.q_start[B] = n_rows;
    *p.count_out = avail - n_new;
  }
  if (bits) atomicOr(p.status, bits);
}

// ------------------------------------------------------------------ append
// A copy, bound by HBM for large batches (75.5 MB for 32768 rows), by the launch for small ones.  A row has 72
// pieces of 16 bytes, so four rows are nine full rounds of a warp, all of whose loads are in flight before the
// first store; the rows' slots are read once, by four lanes.
constexpr int kAppendWarps = 8, kAppendRows = 4, kRowPieces = COLI_KV_WIDTH * 2 / 16;
constexpr int kAppendRounds = kAppendRows * kRowPieces / 32;
static_assert(kAppendRounds * 32 == kAppendRows * kRowPieces, "whole rounds");

struct AppendArgs {
  int n, page_size, n_pages;
  FastDiv by_page;
  long long page_stride;             // bytes
  const int32_t* n_valid;
  const uint8_t *latent, *rope;
  long long latent_stride, rope_stride;   // bytes
  const int32_t* slot;
  uint8_t* cache;
};

__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(const AppendArgs p) {
  const int lane = threadIdx.x & 31;
  const int row0 = (blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) * kAppendRows;
  const int n = p.n_valid ? min(p.n, *p.n_valid) : p.n;
  if (row0 >= n) return;
  // lanes 0..3: where the rows go (-1: nowhere)
  long long to = -1;
  if (lane < kAppendRows && row0 + lane < n) {
    const int s = p.slot[row0 + lane], page = p.by_page(max(s, 0));
    if (s >= 0 && page < p.n_pages) to = page * p.page_stride + (long long)(s - page * p.page_size) * (COLI_KV_WIDTH * 2);
  }
  uint4 v[kAppendRounds];
#pragma unroll
  for (int i = 0; i < kAppendRounds; ++i) {
    const int piece = i * 32 + lane, r = piece / kRowPieces, c = piece - r * kRowPieces, row = row0 + r;
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < n)
      v[i] = c < COLI_KV_VALUE * 2 / 16
                 ? *reinterpret_cast<const uint4*>(p.latent + row * p.latent_stride + c * 16)
                 : *reinterpret_cast<const uint4*>(p.rope + row * p.rope_stride + (c - COLI_KV_VALUE * 2 / 16) * 16);
  }
#pragma unroll
  for (int i = 0; i < kAppendRounds; ++i) {
    const int piece = i * 32 + lane, r = piece / kRowPieces, c = piece - r * kRowPieces;
    const long long at = __shfl_sync(0xffffffffu, to, r);
    if (at >= 0) *reinterpret_cast<uint4*>(p.cache + at + c * 16) = v[i];
  }
}

coli_status check_kv_desc(const coli_kv_desc* d, const char* who) {
  if (!d) return fail(COLI_EINVAL, "%s: null description", who);
  if (d->page_size < 1 || d->max_pages < 1 || d->n_pages < 1)
    return fail(COLI_EINVAL, "%s: page_size, max_pages and n_pages must be positive", who);
  if ((long long)d->n_pages * d->page_size > 0x7fffffffLL)
    return fail(COLI_EUNSUPPORTED, "%s: n_pages * page_size exceeds 2^31 - 1 slots", who);
  if ((long long)d->max_pages * d->page_size > 0x7fffffffLL)
    return fail(COLI_EUNSUPPORTED, "%s: max_pages * page_size exceeds 2^31 - 1 keys", who);
  if (d->page_stride % COLI_KV_WIDTH || d->page_stride < (long long)d->page_size * COLI_KV_WIDTH)
    return fail(COLI_EINVAL, "%s: page_stride must be a multiple of %d, at least a page's rows", who, COLI_KV_WIDTH);
  return COLI_OK;
}

}  // namespace coli

using namespace coli;

extern "C" {

coli_status colibri_kv_step(const coli_kv_desc* desc, int B, int n_tokens, const int32_t* new_len,
                            const int32_t* seq_len, const int32_t* held, int32_t* block_table, int32_t* free_pages,
                            const int32_t* free_count, int32_t* seq_len_out, int32_t* held_out,
                            int32_t* free_count_out, int32_t* q_start, int32_t* position, int32_t* slot,
                            int32_t* status, void* stream) {
  const coli_status rc = check_kv_desc(desc, "kv_step");
  if (rc != COLI_OK) return rc;
  if (B < 1 || n_tokens < 0) return fail(COLI_EINVAL, "kv_step: need B >= 1 and n_tokens >= 0");
  if (B > kStepMaxB) return fail(COLI_EUNSUPPORTED, "kv_step: B=%d exceeds %d requests", B, kStepMaxB);
  const void* ptrs[] = {new_len, seq_len, held, block_table, free_pages, free_count, seq_len_out, held_out,
                        free_count_out, q_start, status};
  for (const void* q : ptrs) {
    if (!q) return fail(COLI_EINVAL, "kv_step: null pointer");
    if (!aligned(q, 4)) return fail(COLI_EALIGN, "kv_step: a pointer is not 4-byte aligned");
  }
  if (n_tokens > 0 && (!position || !slot)) return fail(COLI_EINVAL, "kv_step: null pointer");
  if (!aligned(position, 4) || !aligned(slot, 4)) return fail(COLI_EALIGN, "kv_step: a pointer is not 4-byte aligned");
  StepArgs a{*desc, B, n_tokens, new_len, seq_len, held, block_table, free_pages, free_count, seq_len_out,
             held_out, free_count_out, q_start, position, slot, status, {}};
  a.by_page.set(desc->page_size);
  const bool wide = (long long)B * desc->max_pages > 0x3fffffffLL || (long long)B * ((long long)n_tokens + 1) > 0x3fffffffLL;
  auto kern = wide ? kv_step_kernel<long long> : kv_step_kernel<int>;
  const size_t smem = (size_t)(6 * B + 2) * 4;
  cudaError_t ce = cudaSuccess;
  if (smem > 40 * 1024)
    ce = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (6 * kStepMaxB + 2) * 4);
  if (ce != cudaSuccess) return cuda_fail(ce, "kv_step");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kStepCtas);
  cfg.blockDim = dim3(kStepThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kStepCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ce = cudaLaunchKernelEx(&cfg, kern, a);
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "kv_step");
}

coli_status colibri_kv_append(const coli_kv_desc* desc, int n_tokens, const int32_t* n_valid, const void* latent,
                              long long latent_stride, const void* rope, long long rope_stride, const int32_t* slot,
                              void* cache, void* stream) {
  const coli_status rc = check_kv_desc(desc, "kv_append");
  if (rc != COLI_OK) return rc;
  if (n_tokens < 0) return fail(COLI_EINVAL, "kv_append: n_tokens=%d is negative", n_tokens);
  if (n_tokens == 0) return COLI_OK;
  if (!latent || !rope || !slot || !cache) return fail(COLI_EINVAL, "kv_append: null pointer");
  if (latent_stride < 0 || rope_stride < 0) return fail(COLI_EINVAL, "kv_append: a stride is negative");
  if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(cache, 16) || latent_stride % 8 || rope_stride % 8)
    return fail(COLI_EALIGN, "kv_append: latent, rope and cache 16-byte aligned, strides multiples of 8");
  if (!aligned(slot, 4) || !aligned(n_valid, 4)) return fail(COLI_EALIGN, "kv_append: slot or n_valid misaligned");
  AppendArgs a;
  a.n = n_tokens;
  a.page_size = desc->page_size;
  a.n_pages = desc->n_pages;
  a.page_stride = desc->page_stride * 2;
  a.n_valid = n_valid;
  a.latent = static_cast<const uint8_t*>(latent);
  a.rope = static_cast<const uint8_t*>(rope);
  a.latent_stride = latent_stride * 2;
  a.rope_stride = rope_stride * 2;
  a.slot = slot;
  a.cache = static_cast<uint8_t*>(cache);
  a.by_page.set(desc->page_size);
  constexpr int kRows = kAppendWarps * kAppendRows;
  kv_append_kernel<<<n_tokens / kRows + (n_tokens % kRows ? 1 : 0), kAppendWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "kv_append");
}

}  // extern "C"
