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
// the launch, two dependent loads a token and the scans' barriers.
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
};

struct Sum3 {
  long long a, b, c;
};

// Block-wide exclusive sums of three values a thread (1024 threads); *total: the block's sums.
__device__ __forceinline__ Sum3 scan3(Sum3 v, Sum3* warp_tot, Sum3* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto warp_inc = [lane](long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += n;
    }
    return x;
  };
  Sum3 inc{warp_inc(v.a), warp_inc(v.b), warp_inc(v.c)};
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const Sum3 w = warp_tot[lane];
    const Sum3 wi{warp_inc(w.a), warp_inc(w.b), warp_inc(w.c)};
    warp_tot[lane] = Sum3{wi.a - w.a, wi.b - w.b, wi.c - w.c};
    if (lane == 31) *total = wi;
  }
  __syncthreads();
  const Sum3 base = warp_tot[warp];
  const Sum3 r{base.a + inc.a - v.a, base.b + inc.b - v.b, base.c + inc.c - v.c};
  __syncthreads();
  return r;
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

__global__ void __launch_bounds__(kStepThreads, 1) kv_step_kernel(const StepArgs p) {
  extern __shared__ int step_sm[];
  int* qs = step_sm;                 // [B + 1] first token row
  int* pp = qs + p.B + 1;            // [B + 1] first new page (before that: first freed page)
  int* seq = pp + p.B + 1;           // [B] tokens before the step
  int* hold = seq + p.B;             // [B] pages before the step
  __shared__ Sum3 warp_tot[32], total;
  __shared__ int s_count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x, ps = p.d.page_size, B = p.B;
  if (tid == 0) s_count = *p.free_count;

  // a request's lengths: what it frees, asks for, and whether it can be served at all
  struct Req {
    int add, seq, held;
    long long need;
    bool dead, ok, wrong;
  };
  auto request = [&](int b) {
    Req r;
    const int n = p.new_len[b];
    r.seq = p.seq_len[b];
    r.held = p.held[b];
    r.dead = n < 0;
    const bool fine = r.held >= 0 && r.held <= p.d.max_pages;
    if (!fine) r.held = 0;
    const long long after = (long long)r.seq + (n > 0 ? n : 0), pages = (after + ps - 1) / ps;
    r.ok = fine && !r.dead && r.seq >= 0 && r.seq <= (long long)r.held * ps && pages <= p.d.max_pages;
    r.wrong = !r.ok && !(fine && r.dead);
    r.add = r.ok ? n : 0;
    r.need = r.ok && pages > r.held ? pages - r.held : 0;
    return r;
  };
  int bits = 0;

  // scan 1: pages freed, pages wanted, tokens wanted
  Sum3 carry{0, 0, 0};
  for (int base = 0; base < B; base += kStepThreads) {
    const int b = base + tid;
    Req r{};
    if (b < B) r = request(b);
    const Sum3 v{b < B && r.dead ? r.held : 0, r.need, r.add};
    const Sum3 e = scan3(v, warp_tot, &total);
    if (b < B) {
      seq[b] = r.seq;
      hold[b] = r.held;
      pp[b] = (int)min(carry.a + e.a, (long long)p.d.n_pages);
    }
    carry.a += total.a;
    carry.b += total.b;
    carry.c += total.c;
    __syncthreads();
  }
  const int count0 = max(0, min(s_count, p.d.n_pages));
  // more pages than the cache has can only come from wrong inputs: they are dropped
  const int avail = (int)min((long long)p.d.n_pages, count0 + carry.a);
  if (count0 + carry.a > p.d.n_pages || s_count != count0) bits |= COLI_DEV_KV_BAD_PAGE;
  // push the finished requests' pages (a warp per request, dealt over the cluster)
  for (int b = rank * 32 + warp; b < B; b += kStepCtas * 32) {
    if (p.new_len[b] >= 0) continue;
    for (int i = lane; i < hold[b]; i += 32) {
      const long long at = (long long)count0 + pp[b] + i;
      if (at < p.d.n_pages) p.free_pages[at] = p.table[(size_t)b * p.d.max_pages + i];
    }
  }
  const bool all_fit = carry.b <= avail && carry.c <= p.n_tokens;
  __syncthreads();                   // pp's freed pages are read

  // scan 2: what is served.  A request is served when what it and those before it ask for is there.
  Sum3 ask{0, 0, 0}, given{0, 0, 0};
  for (int base = 0; base < B; base += kStepThreads) {
    const int b = base + tid;
    Req r{};
    if (b < B) r = request(b);
    bool serve = b < B && r.ok;
    if (!all_fit) {
      const Sum3 e = scan3(Sum3{0, r.need, r.add}, warp_tot, &total);
      if (serve && r.need > 0 && ask.b + e.b + r.need > avail) { serve = false; bits |= COLI_DEV_KV_NO_PAGES; }
      if (b < B && r.ok && r.add > 0 && ask.c + e.c + r.add > p.n_tokens) { serve = false; bits |= COLI_DEV_KV_TOKENS; }
      ask.b += total.b;
      ask.c += total.c;
      __syncthreads();
    }
    if (b < B && r.wrong) bits |= COLI_DEV_KV_TABLE_FULL;
    const Sum3 e = scan3(Sum3{0, serve ? r.need : 0, serve ? r.add : 0}, warp_tot, &total);
    if (b < B) {
      pp[b] = (int)(given.b + e.b);
      qs[b] = (int)(given.c + e.c);
    }
    given.b += total.b;
    given.c += total.c;
    __syncthreads();
  }
  if (tid == 0) {
    pp[B] = (int)given.b;
    qs[B] = (int)given.c;
  }
  // every CTA has read the inputs, every push is visible
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");

  const int gtid = rank * kStepThreads + tid, gthreads = kStepCtas * kStepThreads;
  auto popped = [&](int i) { return __ldcg(p.free_pages + (avail - 1 - i)); };   // the i-th new page
  const int n_new = pp[B], n_rows = qs[B];
  for (int j = gtid; j < n_new; j += gthreads) {
    const int b = last_at_most(pp, B, j);
    p.table[(size_t)b * p.d.max_pages + hold[b] + (j - pp[b])] = popped(j);
  }
  for (int i = gtid; i < n_rows; i += gthreads) {
    const int b = last_at_most(qs, B, i);
    const int pos = seq[b] + (i - qs[b]), col = pos / ps;
    const int page = col < hold[b] ? p.table[(size_t)b * p.d.max_pages + col] : popped(pp[b] + col - hold[b]);
    const bool in = page >= 0 && page < p.d.n_pages;
    if (!in) bits |= COLI_DEV_KV_BAD_PAGE;
    p.position[i] = pos;
    p.slot[i] = in ? page * ps + pos % ps : -1;
  }
  for (int b = gtid; b < B; b += gthreads) {
    const bool dead = p.new_len[b] < 0;
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
// A copy: 72 16-byte pieces a row, one a thread and pass, kAppendUnroll passes' loads in flight.  Bound by
// HBM for large batches, by the launch for small ones.
constexpr int kAppendThreads = 256, kAppendUnroll = 4, kRowPieces = COLI_KV_WIDTH * 2 / 16;

struct AppendArgs {
  int n, page_size, n_pages;
  long long page_stride;             // bytes
  const int32_t* n_valid;
  const uint8_t *latent, *rope;
  long long latent_stride, rope_stride;   // bytes
  const int32_t* slot;
  uint8_t* cache;
};

__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs p) {
  const int n = p.n_valid ? max(0, min(p.n, *p.n_valid)) : p.n;
  const long long pieces = (long long)n * kRowPieces, step = (long long)gridDim.x * kAppendThreads;
  for (long long i0 = (long long)blockIdx.x * kAppendThreads + threadIdx.x; i0 < pieces; i0 += kAppendUnroll * step) {
    uint4 v[kAppendUnroll];
    uint8_t* to[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
      const long long i = i0 + u * step;
      to[u] = nullptr;
      if (i >= pieces) continue;
      const int row = (int)(i / kRowPieces), c = (int)(i - (long long)row * kRowPieces);
      const int s = __ldg(p.slot + row);
      v[u] = c < COLI_KV_VALUE * 2 / 16
                 ? *reinterpret_cast<const uint4*>(p.latent + row * p.latent_stride + c * 16)
                 : *reinterpret_cast<const uint4*>(p.rope + row * p.rope_stride + (c - COLI_KV_VALUE * 2 / 16) * 16);
      const int page = s / p.page_size;
      if (s >= 0 && page < p.n_pages)
        to[u] = p.cache + page * p.page_stride + (long long)(s - page * p.page_size) * (COLI_KV_WIDTH * 2) + c * 16;
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = v[u];
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
  const StepArgs a{*desc, B, n_tokens, new_len, seq_len, held, block_table, free_pages, free_count, seq_len_out,
                   held_out, free_count_out, q_start, position, slot, status};
  const size_t smem = (size_t)(4 * B + 2) * 4;
  cudaError_t ce = cudaSuccess;
  if (smem > 40 * 1024)
    ce = cudaFuncSetAttribute(kv_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (4 * kStepMaxB + 2) * 4);
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
  ce = cudaLaunchKernelEx(&cfg, kv_step_kernel, a);
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
  const long long pieces = (long long)n_tokens * kRowPieces;
  const long long want = (pieces + kAppendThreads - 1) / kAppendThreads;
  const int grid = (int)(want < 152 * 8 ? want : 152 * 8);
  kv_append_kernel<<<grid, kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "kv_append");
}

}  // extern "C"
