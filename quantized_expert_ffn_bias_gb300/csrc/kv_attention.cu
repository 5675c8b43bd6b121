// Attention of new tokens over the paged compressed cache ("25GB RAM runs 744B
// GLM-5.2" page (pwwt.cn), section 3.2: 576 cached values a token; section 3.3:
// sparse attention over the selected keys):
//   out[n][h] = sum_j p_j v[j],  p = softmax_j(scale * q[n][h] . k[j]),
// k[j] the cached row of key j (576 values), v[j] its first 512.
//
// Every head of a token shares the cached row, so a tile of 64 (token, head)
// rows and 128 keys is two dense contractions of the same 128 cached rows, and
// the tile is loaded once for both (tcgen05, operands in shared memory, fp32
// accumulators in tensor memory):
//   S^T[128 keys][64 rows]  = K Q^T    (K as it lies: keys are the MMA's M)
//   O^T[512][64 rows]      += V^T P^T  (V^T is the same tile read transposed)
// What bounds a tile is shared memory: its MMAs read 408 KB of operands (A and B of 68 MMAs, 4 and 2 KB each), loads and
// P^T write 160 KB, 4,550 cycles at 128 bytes a cycle of the 5,080 that it takes where the rows come from L2.
// The transposed form is what makes it fit: O^T takes 256 of the 512 TMEM
// columns, where 128 rows of O would take all of them, and each thread of the
// softmax holds one key's 64 scores, so that its weights are one 128-byte row
// of the P^T operand.  Shared memory: 144 KB of cached rows, 72 KB of queries;
// P^T takes the place of the rotary part, which only S^T reads.
//
// Softmax: per row a reference m (log2 units) that is raised, with the sums and
// O^T rescaled, only when a score exceeds it by 8 (fp16: 15, see at_top): a tile
// needs no reduction over its keys (they lie across lanes).  References are
// whole numbers, so that raising one rounds nothing.  Each thread sums its own
// key's weights; the sums are reduced once at the end.
//
// Work: units (row tiles of one request, or of one token where keys are
// selected) with their key tiles, dealt in equal runs of key tiles to one CTA
// per SM (or gang of CTAs).  A unit cut by a border leaves partial results in
// the workspace, which the join kernel adds up in order.
#include <atomic>

#include "plan.h"

namespace coli {

constexpr int kAtW = COLI_KV_WIDTH, kAtV = COLI_KV_VALUE;
constexpr int kAtKeys = 128;                       // keys a tile (MMA M of S^T, TMEM lanes)
constexpr int kAtRows = 64;                        // (token, head) rows a unit (MMA N)
constexpr int kAtBoxBytes = kAtKeys * 128;         // 64 columns of a key tile, 128-byte swizzle
constexpr int kAtQBoxBytes = kAtRows * 128;        // 64 columns of the queries
constexpr int kAtBoxes = kAtW / 64;                // 9: eight of values, one rotary
constexpr int kAtLoadWarps = 2;                    // loader warps that copy rows themselves (one issues TMA loads)
constexpr int kAtLaneKeys = kAtKeys / (32 * kAtLoadWarps);   // keys of a tile a copying lane looks up
constexpr int kAtSmWarps = 8;                      // softmax warps: two per TMEM sub-partition, 32 rows each
constexpr int kAtSmThreads = kAtSmWarps * 32, kAtHalf = kAtRows / 2;
constexpr int kAtFirstLoad = 2 + kAtSmWarps;       // warp 0 loads; copying loaders go on from here
constexpr int at_threads(bool tma) { return (1 + kAtSmWarps + (tma ? 1 : kAtLoadWarps)) * 32; }
constexpr int kAtMinBox = 64;                      // fewest key rows of a TMA box (see the kernel)
constexpr int kAtMaxCtas = 160;                    // CTAs the workspace has room for
constexpr int kAtMaxB = 8192, kAtMaxH = 1024;
constexpr int kAtMaxDevices = 64;                  // devices whose properties are kept between calls
constexpr size_t kAtSmem = (size_t)kAtBoxes * (kAtBoxBytes + kAtQBoxBytes) + 1024;
constexpr int kAtPart = kAtRows * kAtV;            // floats of a partial O
// A reference makes the largest weight 2^(top - 1) .. 2^top; growth to 2^(top + kAtGrow) raises it.  bf16 has fp32's
// range; fp16 ends at 2^16 and loses bits below 2^-14 (all below 2^-25), so its weights take the upper part.
constexpr float kAtGrow = 8.f;
__host__ __device__ constexpr float at_top(bool bf16) { return bf16 ? 0.f : 7.f; }
constexpr uint32_t kAtSCol = 256;                  // TMEM column of S^T (O^T: 0..255)

// A unit: the work of one gang of CTAs, 64 rows each, over the same keys.
struct __align__(16) AtUnit {
  int b;              // request
  int row0, row_end;  // (token * H + head) rows; member m of the gang has row0 + 64 m ..
  int first;          // key tiles of the units before it
  int tiles;          // its key tiles
  int shift;          // position of a row's token: shift + row / H
  int seq;            // tokens of the request in the cache
  int pad;
};

// 64 rows of a unit cut by borders: its parts are those of CTAs cta, cta + gang, ...
struct __align__(16) AtJoin {
  int row0, row_end;
  int cta, parts;
  int slot;     // of the first part (the others': 2 * their CTA)
  int gang;
  int pad[2];
};

struct AtArgs {
  coli_kv_desc d;
  FastDiv by_page, by_heads;         // page_size, H
  int B, n_tokens, H, topk;
  float scale_log2;
  int rows_per_page;                 // cached rows from a page to the next (page_stride / 576)
  int box, box_log2;                 // TMA loads: key rows of a box (a power of two, divides the page size and 128)
  long long q_tok, q_head;           // query strides, bytes
  const uint8_t *q, *cache;
  const int32_t *table, *q_start, *seq_len, *sel;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int32_t* cta_status;               // [kAtMaxCtas] what each CTA saw
  AtUnit* units;                     // unit u of run r at u + r
  AtJoin* joins;                     // [kAtMaxCtas] written by every CTA (parts = 0: none)
  float* part;                       // [2 kAtMaxCtas] partial O, in the order the main kernel's threads hold it (at_part)
  float2* part_ml;                   // [2 kAtMaxCtas][64] reference, sum
  unsigned long long wait_ns;
  int withhold;                      // failure-path test: 1: CTA 0's first copies never count as complete
};

// Place of row c (a multiple of four: four rows follow one another) and value v in a partial O.  A thread of
// the main kernel holds many rows of one value, so neighbouring values of four rows lie together.
__host__ __device__ constexpr int at_part(int c, int v) { return ((c >> 2) * kAtV + v) * 4; }

// Borders of G <= kAtMaxCtas equal runs of the W key tiles: floor(W j / G), without leaving 32 bits.  The
// remainder's part is below kAtMaxCtas^2, where the fp32 quotient of x + 1/2 is exact.
struct AtCuts {
  int q, r;
  float inv;
  __device__ __forceinline__ AtCuts(int W, int G) : q(W / G), r(W - q * G), inv(1.0f / (float)G) {}
  __device__ __forceinline__ int operator()(int j) const { return q * j + (int)(((float)(r * j) + 0.5f) * inv); }
};

// ------------------------------------------------------------------ plan
// Every CTA finds its own run of the work from the lengths (a kernel of its own took 7 us, most of it launch and
// loads).  Rows come in tiles of 64: a request's T H rows, or, where keys are selected, a token's heads.
// Row tiles of the same keys may go to a gang of CTAs that take the same key tiles at about the same time, so
// that a tile comes from memory once and from L2 for the others of the gang: 24 requests of three tokens read
// 589 MB of 236 MB unique without gangs, their row tiles being dealt to CTAs at unrelated times.  A gang costs
// CTAs (whole gangs only) and idle members (rows that do not fill it), so the size is chosen by an estimate:
// time of the longest run of key tiles, or of the tiles' bytes from memory, whichever is longer.
constexpr int kAtGangs = 6;
__host__ __device__ constexpr int at_gang(int i) { return i < 4 ? i + 1 : i * 2 - 2; }   // 1, 2, 3, 4, 6, 8
constexpr float kAtTileNs = 2700.f;                // a key tile on one SM (measured)
constexpr float kAtTileMemNs = 23.f;               // 147 KB at the memory's measured copy rate
constexpr int kAtL2Tiles = 400;                    // 59 MB: unique tiles that stay in L2 between row tiles

struct AtRun {
  int gang, run;         // CTAs a gang, this CTA's gang
  int beg, end, unit0;   // its key tiles, the unit of the first
  int prefetch;          // 1: the keys exceed what stays in L2
  int wrong;             // 1: q_start does not ascend
  int status;            // what is wrong with the lengths (COLI_DEV_KV_*)
};

// `sm`: shared memory for 3 B + 2 ints, free again when the call returns.  Every thread of the CTA calls it.
// unit_sm receives the run's first unit.  The code runs once a launch, and what it costs is mostly fetching it:
// loops are kept rolled and each step is written once.
__device__ __forceinline__ AtRun at_plan(const AtArgs& p, int* sm, AtUnit* unit_sm) {
  int* qs = sm;                      // [B + 1] q_start
  int* base = qs + p.B + 1;          // [B + 1] first unit of each request
  int* seq = base + p.B + 1;         // [B]
  __shared__ int warp_tot[32], total, s_unit0, s_flags[3];
  __shared__ unsigned sums[kAtGangs + 1];
  const int tid = threadIdx.x, nthr = blockDim.x, B = p.B, max_ctas = gridDim.x;
  if (tid <= kAtGangs) sums[tid] = 0;
  if (tid < 3) s_flags[tid] = 0;
#pragma unroll 1
  for (int b = tid; b <= B; b += nthr) {
    qs[b] = p.q_start[b];
    if (b < B) seq[b] = max(0, p.seq_len[b]);
  }
  __syncthreads();
  const int heads = (p.H + kAtRows - 1) / kAtRows;
  const int most = p.d.max_pages * p.d.page_size;      // (at most 2^31 - 1: checked by the host)
  const int sel_tiles = (p.topk + kAtKeys - 1) / kAtKeys;
  auto row_of_batch = [&](int i) { return max(0, min(qs[i], p.n_tokens)); };      // rows outside the batch do not exist
  // Requests: row tiles over the same keys (a row tile group), how many such groups, key tiles of each.  Sums of
  // key tiles stay below 2^31 (checked by the host).
  struct Req {
    int n, rows;
    unsigned tiles;
  };
  auto request = [&](int b) {
    Req r;
    const int T = max(0, row_of_batch(b + 1) - row_of_batch(b));
    r.n = p.sel ? T : min(T, 1);
    r.rows = p.sel ? heads : (T * p.H + kAtRows - 1) / kAtRows;        // (n_tokens * H < 2^31 - 64)
    const int keys = min(seq[b], most);
    r.tiles = (unsigned)r.n * (unsigned)(p.sel ? sel_tiles : max(1, (int)(((unsigned)keys + kAtKeys - 1) / kAtKeys)));
    return r;
  };
  // eight threads a request: one for each gang size, one for the unique key tiles, one idle
  {
    const int g = tid & 7, size = g < kAtGangs ? at_gang(g) : 1 << 30;
    const unsigned third = size == 3 ? 0x55555556u : 0x2AAAAAABu;      // of x < 2^31: x / 3, x / 6
    unsigned s = 0;
    bool down = false, many = false, beyond = false;
#pragma unroll 1
    for (int b = tid >> 3; b < B; b += nthr >> 3) {
      const Req q = request(b);
      down |= qs[b + 1] < qs[b];                       // not ascending: nothing is computed
      many |= q.n && q.rows > 1;                       // a gang is of use where row tiles share keys
      beyond |= q.n && seq[b] > most;                  // keys without a place in the block table: left out
      const unsigned x = (unsigned)(q.rows + size - 1);
      s += q.tiles * (g >= kAtGangs ? 1u : (size == 3 || size == 6) ? __umulhi(x, third) : x >> (31 - __clz(size)));
    }
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if ((tid & 31) <= kAtGangs && s) atomicAdd(&sums[tid & 7], s);
    if (down) s_flags[0] = 1;
    if (many) s_flags[1] = 1;
    if (beyond) s_flags[2] = 1;
  }
  __syncthreads();
  AtRun r;
  r.wrong = s_flags[0];
  r.status = (s_flags[0] ? COLI_DEV_KV_TOKENS : 0) | (s_flags[2] ? COLI_DEV_KV_BAD_PAGE : 0);
  r.gang = 1;
  r.prefetch = sums[kAtGangs] > (unsigned)kAtL2Tiles;
  if (s_flags[1]) {
    float best = INFINITY;
#pragma unroll 1
    for (int g = 0; g < kAtGangs && at_gang(g) <= max_ctas; ++g) {
      const float runs = (float)(max_ctas / at_gang(g));
      const float mem = (float)(r.prefetch ? sums[g] : sums[kAtGangs]);
      const float cost = fmaxf(ceilf(__fdividef((float)sums[g], runs)) * kAtTileNs, mem * kAtTileMemNs);
      if (cost < best) {
        best = cost;
        r.gang = at_gang(g);
      }
    }
  }
  const int gang = r.gang, gang_rows = gang * kAtRows;
  r.run = blockIdx.x / gang;
  const int member = blockIdx.x - r.run * gang;
  r.beg = r.end = 0;

  // Two sums over the CTA's threads share this loop: pass 0, units of each request; pass 1, key tiles of each
  // unit (only their total, needed where one round does not see every unit); pass 2, the run's own units.
  int n_units = 0, W = 0, G = 0, n = B, before = 0;   // before: where the run before this one begins
  bool opens = false;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    int carry = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += nthr) {
      const int i = i0 + tid;
      int v = 0;
      AtUnit un;
      if (i < n && pass == 0) {
        const Req q = request(i);
        v = q.n * (gang == 1 ? q.rows : (q.rows + gang - 1) / gang);
      } else if (i < n) {
        int l = 0, h = B;                              // last b with base[b] <= i
#pragma unroll 1
        while (h - l > 1) {
          const int mid = (l + h) >> 1;
          if (base[mid] <= i) l = mid;
          else h = mid;
        }
        const int q0 = row_of_batch(l), q1 = row_of_batch(l + 1);
        un.b = l;
        un.seq = seq[l];
        un.shift = un.seq - qs[l + 1];                 // seq - (qs[l + 1] - qs[l]) - qs[l]
        un.pad = 0;
        if (p.sel) {
          const int per = (heads + gang - 1) / gang, j = i - base[l], tok = q0 + (per == 1 ? j : j / per);
          un.row0 = tok * p.H + (per == 1 ? 0 : j % per) * gang_rows;
          un.row_end = (tok + 1) * p.H;
          v = sel_tiles;
        } else {
          un.row0 = q0 * p.H + (i - base[l]) * gang_rows;
          un.row_end = q1 * p.H;
          const long long keys = (long long)un.shift + p.by_heads(min(un.row_end - 1, un.row0 + gang_rows - 1)) + 1;
          v = max(1, (int)(((unsigned)max(0ll, min(keys, (long long)most)) + kAtKeys - 1) / kAtKeys));
        }                                              // (a unit without keys still writes its rows: one tile)
        un.tiles = v;
      }
      const int e = carry + block_exclusive_scan(v, warp_tot, &total);
      carry += total;
      if (pass == 0 && i < B) base[i] = e;
      if (pass == 2) {
        if (i0 == 0) {
          if (W == 0) W = total;
          G = min(max_ctas / gang, W);
          // The longest run decides the time, so no more runs than it needs (512 tiles over 152 CTAs and over 128
          // both take four rounds): fewer parts to write and join.  Units of equal length: whole runs a unit.
          if (G > 0) {
            const int longest = (W + G - 1) / G;
            int runs = (W + longest - 1) / longest;
            if (n_units <= nthr && n_units <= G && __syncthreads_and(v == 0 || v * n_units == W)) {
              const int whole = n_units * (G / n_units);
              if ((W + whole - 1) / whole == longest) runs = whole;
            }
            G = runs;
          }
          if (r.run < G) {
            const AtCuts cut(W, G);
            before = r.run > 0 ? cut(r.run - 1) : 0;
            r.beg = cut(r.run);
            r.end = cut(r.run + 1);
          }
        }
        un.first = e;
        const int last = e + v;
        if (v && e < r.end && last > r.beg) {
          p.units[i + r.run] = un;
          if (e <= r.beg) {
            s_unit0 = i;
            *unit_sm = un;
            // a run that begins with the first border inside its unit lists the join of its member's rows
            const int row0 = un.row0 + member * kAtRows;
            opens = r.run > 0 && e < r.beg && before <= e && row0 < un.row_end;
            if (opens) {
              const AtCuts cut(W, G);
              int m = r.run;                           // runs run - 1 .. m - 1 begin before the unit's end
#pragma unroll 1
              for (int h = G; m < h;) {
                const int mid = (m + h) >> 1;
                if (cut(mid) < last) m = mid + 1;
                else h = mid;
              }
              AtJoin jn;
              jn.row0 = row0;
              jn.row_end = min(row0 + kAtRows, un.row_end);
              jn.cta = (r.run - 1) * gang + member;
              jn.gang = gang;
              jn.parts = m - (r.run - 1);
              jn.slot = 2 * jn.cta + (before < e ? 1 : 0);
              jn.pad[0] = jn.pad[1] = 0;
              p.joins[blockIdx.x] = jn;
            }
          }
        }
      }
      __syncthreads();
      if (pass == 2 && carry >= r.end) break;          // the units that follow are other runs'
    }
    if (pass == 0) {
      n = n_units = r.wrong ? 0 : carry;
      if (n_units <= nthr) pass = 1;                   // one round sees every unit: no need of pass 1
    } else if (pass == 1) {
      W = carry;
    }
  }
  if (!__syncthreads_or(opens) && tid == 0) p.joins[blockIdx.x].parts = 0;
  r.unit0 = s_unit0;
  return r;
}

// ------------------------------------------------------------------ main kernel

// 16 bytes of global memory into shared memory, asynchronously; `bar` counts this thread once its copies so far have landed.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Operand read transposed (MN-major), 128-byte swizzle: the operand's M (or N) runs along the 128-byte rows,
// 64 elements an atom, the next 64 `mn_bytes` further; K runs down the rows, 8 an atom of 1024 bytes.
__device__ __forceinline__ uint64_t umma_desc_sw128_mn(uint32_t saddr, uint32_t mn_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(mn_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ float at_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t at_pack(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Barrier of the softmax warps; with `or`: whether any thread's pred is true.
__device__ __forceinline__ void sm_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kAtSmThreads) : "memory"); }
__device__ __forceinline__ bool sm_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "n"(kAtSmThreads)
      : "memory");
  return r != 0;
}

// Reduce v[32] over the warp's lanes; lane l ends with the result of column l.
template <typename F>
__device__ __forceinline__ float warp_columns(const float (&v)[32], F op) {
  const int lane = threadIdx.x & 31;
  float w[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) w[i] = v[i];
  // fold: a lane keeps the half of the columns that its bit chooses and gives the other half away
#pragma unroll
  for (int n = 16; n >= 1; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? w[n + i] : w[i], give = up ? w[i] : w[n + i];
      w[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, n));
    }
  }
  return w[0];
}

// MMAs of a K-step sequence, both operands in shared memory, issued by one elected lane of a converged warp
// (descriptors then stay in uniform registers: 36 MMAs took 4,900 cycles to issue from a single-lane branch).
// Step s adds s * sa (sb) to the descriptor of A (B), in units of 16 bytes; acc = 0: the first overwrites.
template <int STEPS, int SA, int SB>
__device__ __forceinline__ void umma_steps(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  static_assert(STEPS == 4 || STEPS == 8, "");
  if constexpr (STEPS == 8) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "add.u64 a1, %1, %5;\n\tadd.u64 a2, a1, %5;\n\tadd.u64 a3, a2, %5;\n\tadd.u64 a4, a3, %5;\n\t"
        "add.u64 a5, a4, %5;\n\tadd.u64 a6, a5, %5;\n\tadd.u64 a7, a6, %5;\n\t"
        "add.u64 b1, %2, %6;\n\tadd.u64 b2, b1, %6;\n\tadd.u64 b3, b2, %6;\n\tadd.u64 b4, b3, %6;\n\t"
        "add.u64 b5, b4, %6;\n\tadd.u64 b6, b5, %6;\n\tadd.u64 b7, b6, %6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(SA), "n"(SB)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "add.u64 a1, %1, %5;\n\tadd.u64 a2, a1, %5;\n\tadd.u64 a3, a2, %5;\n\t"
        "add.u64 b1, %2, %6;\n\tadd.u64 b2, b1, %6;\n\tadd.u64 b3, b2, %6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "n"(SA), "n"(SB)
        : "memory");
  }
}

// Arrive on `bar` when the MMAs issued so far are complete (one elected lane of a converged warp).
__device__ __forceinline__ void umma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// TMA: key tiles arrive as TMA boxes of p.box = 64 or 128 rows (pages of whole boxes, every key up to the
// position) and the queries as one box a 64 columns (token and head rows evenly spaced); otherwise two warps
// copy row by row (cp.async), from pages of any size, for selected keys and for queries of any strides.  A TMA
// load costs its issuing warp about 60 cycles whatever its rows: a chunk of 500 tokens over 6,000 keys takes 407,
// 412, 468 and 601 us with boxes of 128, 64, 32 and 16 rows, 426 us with copies; a gathering TMA load of four rows a
// coordinate measured 83 cycles for 512 bytes, 12.5 us a tile of 128 keys.
template <bool BF16, bool TMA>
__global__ void __launch_bounds__(at_threads(TMA), 1)
    kv_attention_kernel(const AtArgs p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t full[5], empty[4], q_full, q_empty, s_full, p_ready, o_full;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, cta_status;
  __shared__ AtUnit unit_sm;                           // the run's first unit
  __shared__ uint32_t key_ok[2][4];                    // bit i of word w: key 32 w + i of the tile is there
  __shared__ uint32_t key_fin[2][4];                   // bit i of word w of a half: key 32 w + i has a finite score there
  __shared__ __align__(16) float ref[kAtRows], fac[kAtRows], keep[kAtRows], red[4][kAtRows];   // ref: the negated references
  __shared__ __align__(16) int lim[kAtRows];           // last key position each row sees (dense)
  __shared__ int has_ref[kAtRows];                     // the row has seen a key
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem + kAtBoxes * kAtBoxBytes;
  uint8_t* rot = smem + 8 * kAtBoxBytes;               // rotary part of the keys, then P^T
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_v = &abort_flag;

  if (TMA && warp == 0 && lane == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&qmap);
  }
  if (threadIdx.x == 0) {
    // copying warps: one arrival a thread, and one a warp for key_ok (with the rotary box)
    // (an arrival too many for a withheld stage; a test of it where the copies are issued costs 3 % of short runs)
    for (int i = 0; i < 5; ++i)
      mbar_init(&full[i], (TMA ? 1 : kAtLoadWarps * 32 + (i == 4 ? kAtLoadWarps : 0)) + (i == 0 && blockIdx.x == 0 ? p.withhold : 0));
    for (int i = 0; i < 4; ++i) mbar_init(&empty[i], 1);
    mbar_init(&q_full, TMA ? 1 : kAtLoadWarps * 32);
    mbar_init(&q_empty, 1);
    mbar_init(&s_full, 1);
    mbar_init(&p_ready, kAtSmWarps);
    mbar_init(&o_full, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  griddep_wait();                                      // the launch may overlap the kernel before; its results not
  const AtRun plan = at_plan(p, reinterpret_cast<int*>(smem), &unit_sm);
  const int cta = blockIdx.x, beg = plan.beg, end = plan.end, unit0 = plan.unit0;
  const int my_rows = (cta - plan.run * plan.gang) * kAtRows;    // this member's rows of a unit begin there
  const AtUnit* units = p.units + plan.run;
  if (threadIdx.x == 0) cta_status = plan.status;
  // (the plan's use of shared memory ends before the TMA and MMA use of it)
  fence_proxy_async_smem();
  __syncthreads();
  auto fail_wait = [&]() {
    atomicOr(&cta_status, COLI_DEV_WAIT_TIMEOUT);
    atomicExch(&abort_flag, 1);
  };

  if (warp == 0 || warp >= kAtFirstLoad) {
    // ---------------------------------------------------------------- loader
    const int lw = warp == 0 ? 0 : warp - kAtFirstLoad + 1;           // copying: this warp's keys of a tile start at 32 kAtLaneKeys lw
    bool ok = true;
    int it = 0, un = 0;
    // it, un: tiles begun, units whose queries are on their way, when the loop ends; the last tile's barriers d < given
    // have copies on their way
    int given = 5;
    const int n_box = TMA ? kAtKeys >> p.box_log2 : 0;       // boxes of 64 columns a tile
    for (int at = beg, u = unit0; ok && at < end; ++u) {
      const AtUnit ut = u == unit0 ? unit_sm : units[u];
      const int t0 = at - ut.first, t1 = min(end - ut.first, ut.tiles);
      const int row0 = ut.row0 + my_rows;
      if (row0 >= ut.row_end) {                        // this member has no rows of the unit
        at = ut.first + t1;
        continue;
      }
      const int tok = p.by_heads(row0);
      const int seen = p.sel ? min(ut.seq, ut.shift + tok + 1) : ut.seq;   // keys before this are there
      const int32_t* table = p.table + (size_t)ut.b * p.d.max_pages;
      const int32_t* sel = p.sel + (size_t)tok * p.topk;
      // Where a key's row is, in two steps a tile apart, so that their loads are on the way before a tile's
      // copies queue up: the key (TMA: the first of box l; copying: key 32 j + l of the warp's), then its page.
      constexpr int kRows = TMA ? 1 : kAtLaneKeys;
      int key[kRows], next[kRows], page[kRows];       // tile t + 1's keys, tile t + 2's, tile t + 1's pages
      auto find_key = [&](int t, int (&key)[kRows]) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          if constexpr (TMA) {
            key[j] = t * kAtKeys + (lane & (n_box - 1)) * p.box;
          } else {
            key[j] = t * kAtKeys + (lw * kAtLaneKeys + j) * 32 + lane;
            if (p.sel) key[j] = key[j] < p.topk ? sel[key[j]] : -1;
          }
        }
      };
      auto find_page = [&]() {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const int col = p.by_page(max(key[j], 0));
          page[j] = key[j] >= 0 && key[j] < seen && col < p.d.max_pages ? table[col] : -1;
        }
      };
      // the row; false where there is none (then row 0, whose values meet weights of 0)
      auto row_of = [&](int j, long long& row) {
        row = 0;
        if (key[j] < 0 || key[j] >= seen) return false;
        if (page[j] < 0 || page[j] >= p.d.n_pages) {
          atomicOr(&cta_status, COLI_DEV_KV_BAD_PAGE);
          return false;
        }
        row = (long long)page[j] * p.rows_per_page + (key[j] - p.by_page(key[j]) * p.d.page_size);
        return true;
      };
      long long row[kRows];
      bool there[kRows];
      find_key(t0, key);
      find_page();
#pragma unroll
      for (int j = 0; j < kRows; ++j) there[j] = row_of(j, row[j]);
      find_key(t0 + 1, key);
      // queries
      if (un > 0 && !mbar_wait(&q_empty, (un - 1) & 1, p.wait_ns)) { ok = false; break; }
      if constexpr (TMA) {
        if (lane == 0) mbar_arrive_expect_tx(&q_full, (uint32_t)(kAtBoxes * kAtQBoxBytes));
        __syncwarp();
        // rows past the unit's last are other rows' or, behind the tensor, zeros: computed, not written
        if (lane < kAtBoxes) tma_load_2d_nohint(qs + lane * kAtQBoxBytes, &qmap, lane * 64, row0, &q_full);
      } else {
        // eight lanes a row and box: 16 bytes each
        const int c = lane & 7;
#pragma unroll 1
        for (int i = 0; i < kAtRows / (4 * kAtLoadWarps); ++i) {
          const int r = (i * kAtLoadWarps + lw) * 4 + (lane >> 3);
          const int gr = min(row0 + r, ut.row_end - 1);
          const uint8_t* src = p.q + p.by_heads(gr) * p.q_tok + (gr - p.by_heads(gr) * p.H) * p.q_head + c * 16;
          uint8_t* dst = qs + r * 128 + ((c ^ (r & 7)) << 4);
#pragma unroll
          for (int x = 0; x < kAtBoxes; ++x) copy16(dst + x * kAtQBoxBytes, src + x * 128);
        }
        copies_arrive(&q_full);
      }
      for (int t = t0; t < t1; ++t, ++it) {
        if (*abort_v) { ok = false; break; }
        // which keys are there, in key order
        uint32_t mine[kRows] = {};
        if constexpr (TMA) {
          // box j holds keys j box .. (j + 1) box - 1, there up to `seen`
          const unsigned boxes = __ballot_sync(0xffffffffu, there[0]);
          if (lane < 4) {
            mine[0] = (boxes >> ((lane * 32) >> p.box_log2)) & 1u ? 0xffffffffu : 0u;
            const int left = seen - (t * kAtKeys + lane * 32);
            if (left < 32) mine[0] &= left <= 0 ? 0u : (1u << left) - 1u;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kRows; ++j) mine[j] = __ballot_sync(0xffffffffu, there[j]);
        }
        // copying: the rows of the eight lanes a key, once a tile
        const uint8_t* src[TMA ? 1 : 8 * kRows];
        if constexpr (!TMA) {
#pragma unroll
          for (int i = 0; i < 8 * kRows; ++i)
            src[i] = p.cache + __shfl_sync(0xffffffffu, row[i >> 3], (i & 7) * 4 + (lane >> 3)) * (kAtW * 2) + (lane & 7) * 16;
        }
        if (t + 1 < t1) {
          find_page();
          find_key(t + 2, next);
        }
        // pairs of value boxes as the previous tile's products free them, then the rotary box
#pragma unroll 1
        for (int d = 0; d < 4 && ok; ++d) {
          if (it > 0 && !mbar_wait(&empty[d], (it - 1) & 1, p.wait_ns)) { ok = false; given = d; break; }
          if constexpr (TMA) {
            if (d == 0 && lane < 4) key_ok[it & 1][lane] = mine[0];
            if (lane == 0) mbar_arrive_expect_tx(&full[d], (uint32_t)(2 * kAtBoxBytes));
            __syncwarp();
            // lanes 0 .. n_box - 1: the first 64 columns, the next n_box lanes: the other 64
            if (lane < 2 * n_box) {
              const int x = 2 * d + (lane >= n_box), j = lane & (n_box - 1);
              tma_load_2d_nohint(smem + x * kAtBoxBytes + j * p.box * 128, &kmap, x * 64, (int)row[0], &full[d]);
            }
          } else {
            if (d == 0 && lane == 0)
#pragma unroll
              for (int j = 0; j < kRows; ++j) key_ok[it & 1][lw * kRows + j] = mine[j];
#pragma unroll
            for (int i = 0; i < 8 * kRows; ++i) {      // eight lanes a key
              const int k = lw * 32 * kRows + i * 4 + (lane >> 3);
              uint8_t* dst = smem + k * 128 + (((lane & 7) ^ (k & 7)) << 4);
              copy16(dst + (2 * d) * kAtBoxBytes, src[i] + (2 * d) * 128);
              copy16(dst + (2 * d + 1) * kAtBoxBytes, src[i] + (2 * d + 1) * 128);
            }
            copies_arrive(&full[d]);
          }
        }
        if (!ok) { ++it; break; }
        if constexpr (TMA) {
          if (lane == 0) mbar_arrive_expect_tx(&full[4], (uint32_t)kAtBoxBytes);
          __syncwarp();
          if (lane < n_box) tma_load_2d_nohint(rot + lane * p.box * 128, &kmap, 8 * 64, (int)row[0], &full[4]);
        } else {
#pragma unroll
          for (int i = 0; i < 8 * kRows; ++i) {
            const int k = lw * 32 * kRows + i * 4 + (lane >> 3);
            copy16(rot + k * 128 + (((lane & 7) ^ (k & 7)) << 4), src[i] + 8 * 128);
          }
          copies_arrive(&full[4]);
          if (lane == 0) mbar_arrive(&full[4]);        // key_ok is written
        }
        if (t + 1 < t1) {
#pragma unroll
          for (int j = 0; j < kRows; ++j) {
            there[j] = row_of(j, row[j]);
            key[j] = next[j];
          }
          // the next tile is on its way to L2 while this one is worked on (its place in shared memory is taken)
          if (!plan.prefetch) {
          } else if constexpr (TMA) {
            for (int i = lane; i < kAtBoxes * n_box; i += 32)      // (i and the lane have the same box of rows)
              tma_prefetch_2d(&kmap, (i >> (7 - p.box_log2)) * 64, (int)row[0]);
          } else {
#pragma unroll
            for (int j = 0; j < kRows; ++j)
              if (there[j])
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.cache + row[j] * (kAtW * 2)),
                             "n"(kAtW * 2)
                             : "memory");
          }
        }
      }
      at = ut.first + t1;
      ++un;
    }
    if (!ok) fail_wait();
    // Copies in flight land before the CTA leaves, whichever role gave up: this warp may have issued its last ones long
    // before.  A barrier's phase before the awaited one is complete: its copies were waited for by way of `empty`.
    if constexpr (!TMA) asm volatile("cp.async.wait_all;" ::: "memory");
    if (TMA && lane == 0) {
      if (un > 0) mbar_wait(&q_full, (un - 1) & 1, kWaitLimitNs);
#pragma unroll 1
      for (int d = 0; d < 5; ++d) {
        const int t = it - (d < given ? 1 : 2);
        if (t >= 0) mbar_wait(&full[d], t & 1, d == 0 && p.withhold ? 1000000ull : kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (the warp stays converged; its waits
    // are the suspending ones: polling takes issue slots from the softmax warps beside it, chunk 1.72 -> 1.69 ms)
    const uint32_t fmt = BF16 ? (1u << 7) | (1u << 10) : 0u;
    const uint32_t idesc = (1u << 4) | fmt | ((uint32_t)(kAtRows >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    const uint32_t idesc_t = idesc | (1u << 15) | (1u << 16);            // both operands MN-major
    const uint64_t kd = umma_desc_sw128(smem_u32(smem)), qd = umma_desc_sw128(smem_u32(qs));
    const uint64_t vd = umma_desc_sw128_mn(smem_u32(smem), kAtBoxBytes);
    const uint64_t pd = umma_desc_sw128_mn(smem_u32(rot), kAtBoxBytes);
    bool ok = true;
    int it = 0, un = 0;
    for (int at = beg, u = unit0; ok && at < end; ++u) {
      const AtUnit ut = u == unit0 ? unit_sm : units[u];
      const int t0 = at - ut.first, t1 = min(end - ut.first, ut.tiles);
      at = ut.first + t1;
      if (ut.row0 + my_rows >= ut.row_end) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(&q_full, un & 1, p.wait_ns));
      if (!TMA) fence_proxy_async_smem();              // the copies are ordinary writes; the MMA reads by the async proxy
      for (int t = t0; ok && t < t1; ++t, ++it) {
        // S^T: nine boxes of 64 columns, four steps of 16 each
#pragma unroll
        for (int x = 0; x < kAtBoxes; ++x) {
          if ((x & 1) == 0) {
            ok = ok && mbar_wait(&full[x >> 1], it & 1, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!TMA) fence_proxy_async_smem();
            tc_fence_after();
          }
          if (ok)
            umma_steps<4, 2, 2>(tmem + kAtSCol, kd + (uint64_t)(x * (kAtBoxBytes >> 4)),
                                qd + (uint64_t)(x * (kAtQBoxBytes >> 4)), idesc, x ? 1u : 0u);
        }
        if (!ok) break;
        umma_commit_elect(&s_full);
        if (t + 1 == t1) umma_commit_elect(&q_empty);
        ok = ok && mbar_wait(&p_ready, it & 1, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // O^T: four blocks of 128 values, eight steps of 16 keys each
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          umma_steps<8, 128, 128>(tmem + (uint32_t)(d * kAtRows), vd + (uint64_t)(2 * d * (kAtBoxBytes >> 4)), pd,
                                  idesc_t, t > t0 ? 1u : 0u);
          umma_commit_elect(&empty[d]);
        }
      }
      if (!ok) break;
      umma_commit_elect(&o_full);
      ++un;
    }
    // What was issued ends before tensor memory is freed, whichever role gave up: the last unit's products and then
    // those of a unit left in its middle (committed after that wait: a barrier's phases are awaited one by one).
    if (un > 0) mbar_wait(&o_full, (un - 1) & 1, kWaitLimitNs);
    if (!ok) {
      if (lane == 0) fail_wait();
      umma_commit_elect(&o_full);
      mbar_wait(&o_full, un & 1, kWaitLimitNs);
    }
  } else {
    // ---------------------------------------------------------------- softmax and output (warps 2 ..)
    const int sp = warp & 3;                           // TMEM sub-partition: keys 32 sp .. 32 sp + 31 of a tile
    const int half = (warp - 2) >> 2, c0 = half * kAtHalf;   // this warp's 32 rows of the unit
    const int me = sp * 32 + lane;                     // this thread's key of a tile, value of a block of O^T
    const int id = threadIdx.x - 64;                   // thread among the softmax warps
    const uint32_t trow = tmem + ((uint32_t)(sp * 32) << 16) + (uint32_t)c0;
    int it = 0, un = 0;
    for (int at = beg, u = unit0; at < end; ++u) {
      const AtUnit ut = u == unit0 ? unit_sm : units[u];
      const int t0 = at - ut.first, t1 = min(end - ut.first, ut.tiles);
      at = ut.first + t1;
      const int row0 = ut.row0 + my_rows;
      if (row0 >= ut.row_end) continue;
      const bool whole = t0 == 0 && t1 == ut.tiles;
      const int slot = 2 * cta + (u == unit0 ? 0 : 1);
      if (id < kAtRows) {
        lim[id] = p.sel ? 0x7fffffff : ut.shift + p.by_heads(min(row0 + id, ut.row_end - 1));
        ref[id] = 0.f;
        has_ref[id] = 0;
      }
      const int seen_all = ut.shift + p.by_heads(row0);      // every row sees the keys up to this one
      float l[kAtHalf];                                // sums of this key's weights
#pragma unroll
      for (int c = 0; c < kAtHalf; ++c) l[c] = 0.f;
      sm_sync();
      bool ok = true, unset = true;                    // unset: some row has no reference yet
      for (int t = t0; t < t1; ++t, ++it) {
        // (the rotary box's barrier orders the loader's key_ok before this read)
        ok = mbar_wait(&full[4], it & 1, p.wait_ns) && mbar_wait(&s_full, it & 1, p.wait_ns);
        tc_fence_after();
        float x[kAtHalf];
        {
          uint32_t r[2][16];
          tmem_ld16_issue(trow + kAtSCol, r[0]);
          tmem_ld16_issue(trow + kAtSCol + 16, r[1]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < kAtHalf; ++c) x[c] = __uint_as_float(r[c >> 4][c & 15]);
        }
        const uint32_t kw = key_ok[it & 1][sp];
        const bool there = (kw >> lane) & 1u;
        const int key = t * kAtKeys + me;
        // some row does not see some key of this warp (the same in both halves)
        const bool masked = p.sel ? kw != 0xffffffffu : (t * kAtKeys + sp * 32 + 31 > seen_all || kw != 0xffffffffu);
        if (masked) {
          bool fin = false;
#pragma unroll
          for (int c = 0; c < kAtHalf; ++c) fin |= fabsf(x[c]) < INFINITY;
          const unsigned fw = __ballot_sync(0xffffffffu, fin);
          if (lane == 0) key_fin[half][sp] = fw;
        }
        // distance to the references
#pragma unroll
        for (int c = 0; c < kAtHalf; c += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&ref[c0 + c]);
          x[c] = fmaf(x[c], p.scale_log2, m.x);
          x[c + 1] = fmaf(x[c + 1], p.scale_log2, m.y);
          x[c + 2] = fmaf(x[c + 2], p.scale_log2, m.z);
          x[c + 3] = fmaf(x[c + 3], p.scale_log2, m.w);
        }
        if (masked) {                                  // (after the scale, which may be 0 or negative)
#pragma unroll
          for (int c = 0; c < kAtHalf; c += 4) {
            const int4 lm = *reinterpret_cast<const int4*>(&lim[c0 + c]);
            if (!there || (!p.sel && key > lm.x)) x[c] = -INFINITY;
            if (!there || (!p.sel && key > lm.y)) x[c + 1] = -INFINITY;
            if (!there || (!p.sel && key > lm.z)) x[c + 2] = -INFINITY;
            if (!there || (!p.sel && key > lm.w)) x[c + 3] = -INFINITY;
          }
        }
        // does any score exceed its row's reference by more than kAtGrow?
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kAtHalf; c += 4)
          top = fmaxf(fmaxf(fmaxf(top, x[c]), fmaxf(x[c + 1], x[c + 2])), x[c + 3]);
        if (sm_any(top > kAtGrow + at_top(BF16) || unset || !ok)) {
          if (sm_any(!ok)) { ok = false; break; }
          red[sp][c0 + lane] = warp_columns(x, [](float a, float b) { return fmaxf(a, b); });
          sm_sync();
          bool none = false;
          if (id < kAtRows) {
            const float g = ceilf(fmaxf(fmaxf(red[0][id], red[1][id]), fmaxf(red[2][id], red[3][id]))) - at_top(BF16);
            const bool raise = g > kAtGrow || (!has_ref[id] && g > -INFINITY);
            fac[id] = raise ? g : 0.f;                 // by how much
            // what that leaves of the sums so far: a first reference may lie far below 0, but they are 0 (or NaN) then
            keep[id] = raise && has_ref[id] ? at_exp2(-g) : 1.f;
            if (raise) {
              ref[id] -= g;
              has_ref[id] = 1;
            }
            none = !has_ref[id];
          }
          unset = sm_any(none);
#pragma unroll
          for (int c = 0; c < kAtHalf; ++c) {
            x[c] -= fac[c0 + c];
            l[c] *= keep[c0 + c];
          }
          if (t > t0) {                                // (the first tile's products overwrite O^T)
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {              // four blocks of O^T, 16 rows at a time
              const uint32_t col = (uint32_t)((i >> 1) * kAtRows + (i & 1) * 16);
              uint32_t r[16];
              tmem_ld16_issue(trow + col, r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                r[j] = __float_as_uint(__uint_as_float(r[j]) * keep[c0 + (i & 1) * 16 + j]);
              tmem_st16(trow + col, r);
            }
            tmem_st_wait();
          }
        }
        // weights, their sums, and the key's half of its row of P^T (64 weights = 128 bytes, swizzled)
        uint8_t* prow = rot + me * 128;
#pragma unroll
        for (int c = 0; c < kAtHalf; c += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = at_exp2(x[c + 2 * i]), b = at_exp2(x[c + 2 * i + 1]);
            l[c + 2 * i] += a;
            l[c + 2 * i + 1] += b;
            w[i] = at_pack<BF16>(a, b);
          }
          *reinterpret_cast<uint4*>(prow + ((((c0 + c) >> 3) ^ (me & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // a key whose every score is not finite holds an infinity or a NaN: its values must not meet the zero
        // weights of the rows that do not see it
        if (masked && !(((key_fin[0][sp] | key_fin[1][sp]) >> lane) & 1u)) {
#pragma unroll 1
          for (int i = half * 32; i < half * 32 + 32; ++i)
            *reinterpret_cast<uint4*>(smem + (i >> 3) * kAtBoxBytes + me * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready);
      }
      if (!ok) {
        fail_wait();
        break;
      }
      // -------------------------------------------------------------- the unit's rows
      ok = mbar_wait(&o_full, un & 1, p.wait_ns);
      tc_fence_after();
      red[sp][c0 + lane] = warp_columns(l, [](float a, float b) { return a + b; });
      if (sm_any(!ok)) {
        fail_wait();
        break;
      }
      if (id < kAtRows) {
        const float sum = (red[0][id] + red[1][id]) + (red[2][id] + red[3][id]);
        if (whole) {
          fac[id] = sum == 0.f ? 0.f : 1.0f / sum;
          const int row = row0 + id;
          if (p.lse && row < ut.row_end)
            p.lse[row] = sum == 0.f ? -INFINITY : (log2f(sum) - ref[id]) * 0.693147180559945309f;
        } else {
          p.part_ml[(size_t)slot * kAtRows + id] = make_float2(has_ref[id] ? -ref[id] : -INFINITY, sum);
        }
      }
      sm_sync();
      const int rows = min(kAtRows, ut.row_end - row0) - c0;    // of this half
      float* part = p.part + (size_t)slot * kAtPart;
      uint16_t* out = p.out + (size_t)(row0 + c0) * kAtV;
#pragma unroll 1
      for (int d = 0; d < 4; ++d) {
        uint32_t r[2][16];
        tmem_ld16_issue(trow + d * kAtRows, r[0]);
        tmem_ld16_issue(trow + d * kAtRows + 16, r[1]);
        tmem_ld_wait();
        if (whole) {
          // lanes 2 i and 2 i + 1 hold neighbouring values of a row: they trade halves of two rows
#pragma unroll
          for (int i = 0; i < kAtHalf; i += 2) {
            const float a = __uint_as_float(r[i >> 4][i & 15]) * fac[c0 + i];
            const float b = __uint_as_float(r[i >> 4][(i & 15) + 1]) * fac[c0 + i + 1];
            const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : b, 1);
            const int c = i + (lane & 1);
            const uint32_t two = (lane & 1) ? at_pack<BF16>(got, b) : at_pack<BF16>(a, got);
            if (c < rows) *reinterpret_cast<uint32_t*>(out + (size_t)c * kAtV + d * 128 + (me & ~1)) = two;
          }
        } else {
#pragma unroll
          for (int i = 0; i < kAtHalf; i += 4)
            if (i < rows)
              *reinterpret_cast<float4*>(part + at_part(c0 + i, d * 128 + me)) =
                  make_float4(__uint_as_float(r[i >> 4][i & 15]), __uint_as_float(r[i >> 4][(i & 15) + 1]),
                              __uint_as_float(r[i >> 4][(i & 15) + 2]), __uint_as_float(r[i >> 4][(i & 15) + 3]));
        }
      }
      tc_fence_before();
      sm_sync();                                       // everyone is done with ref, fac, red
      ++un;
    }
  }
  griddep_launch_dependents();                         // (earlier, the join's CTAs would take slots from the next call's)
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.cta_status[cta] = cta_status;
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// ------------------------------------------------------------------ join
// Adds up the parts of every cut unit, in order.  A task is four rows of a unit: 64 values where the parts are
// many (eight thread groups take every eighth part each, then meet in shared memory), all 512 where they are
// few (the values of the first parts are then loaded before their weights are known).
constexpr float kAtLowest = -3.402823466e38f;      // below every reference; a part whose row saw no key has -infinity
constexpr int kAtJoinThreads = 512, kAtJoinCtas = 304, kAtJoinFew = 8;
__host__ __device__ constexpr int at_join_tasks(int parts) { return parts <= 0 ? 0 : parts <= kAtJoinFew ? 16 : 128; }

template <bool BF16>
__global__ void __launch_bounds__(kAtJoinThreads, 2) kv_attention_join_kernel(const AtArgs p, int ctas) {
  __shared__ __align__(16) float wgt[kAtMaxCtas][4];    // a part's reference, then its weight, for each row of the task
  __shared__ float sum[kAtMaxCtas][4];
  __shared__ float inv[4];
  __shared__ float4 meet[7][64];
  __shared__ int starts[8 * 32 + 1], warp_tot[32], total;  // first task of each CTA's join
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the cut units' rows, listed; the main kernel's CTAs' status
  static_assert(kAtMaxCtas <= 8 * 32, "a thread each");
  const int parts = tid < ctas ? p.joins[tid].parts : 0;
  const int bits = blockIdx.x == 0 && tid < ctas ? p.cta_status[tid] : 0;
  const int start = block_exclusive_scan(at_join_tasks(parts), warp_tot, &total);
  if (tid < 8 * 32) starts[tid] = start;
  if (blockIdx.x == 0) {
    const int timed = __syncthreads_or(bits & COLI_DEV_WAIT_TIMEOUT), page = __syncthreads_or(bits & COLI_DEV_KV_BAD_PAGE);
    const int order = __syncthreads_or(bits & COLI_DEV_KV_TOKENS);
    if (tid == 0)
      *p.status = (timed ? COLI_DEV_WAIT_TIMEOUT : 0) | (page ? COLI_DEV_KV_BAD_PAGE : 0) | (order ? COLI_DEV_KV_TOKENS : 0);
  }
  __syncthreads();
  const int n_tasks = total;
  for (int task = blockIdx.x; task < n_tasks; task += gridDim.x) {
    int j = 0, h = 8 * 32;                              // last CTA whose join starts at or before the task
    while (h - j > 1) {
      const int mid = (j + h) >> 1;
      if (starts[mid] <= task) j = mid;
      else h = mid;
    }
    const AtJoin jn = p.joins[j];
    const int sub = task - starts[j];
    const int n = jn.parts;
    const bool few = n <= kAtJoinFew;
    const int c = (few ? sub : sub >> 3) * 4, rows = jn.row_end - jn.row0 - c;
    if (rows <= 0) continue;
    auto slot = [&](int i) { return (size_t)(i ? 2 * (jn.cta + i * jn.gang) : jn.slot); };
    auto add = [](float4& a, const float4 w, const float4 o) {
      a.x = fmaf(w.x, o.x, a.x);
      a.y = fmaf(w.y, o.y, a.y);
      a.z = fmaf(w.z, o.z, a.z);
      a.w = fmaf(w.w, o.w, a.w);
    };
    auto write = [&](const float4 a, const float4 by, int val) {
      const float r[4] = {a.x * by.x, a.y * by.y, a.z * by.z, a.w * by.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < rows) p.out[(size_t)(jn.row0 + c + i) * kAtV + val] = (uint16_t)at_pack<BF16>(r[i], 0.f);
    };
    auto lse = [&](float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f; };
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (few) {
      // the values of the first parts, and all references and sums, on their way at the same time
      constexpr int kAhead = 4;
      float4 o[kAhead];
      const float* src = p.part + at_part(c, tid);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < n) o[i] = *reinterpret_cast<const float4*>(src + slot(i) * kAtPart);
      float2 ml = make_float2(0.f, 0.f);
      if (tid < 4 * n) ml = p.part_ml[slot(tid >> 2) * kAtRows + c + (tid & 3)];
      __syncthreads();                                  // the previous task's weights are read
      if (tid < 4 * n) {
        wgt[tid >> 2][tid & 3] = ml.x;
        sum[tid >> 2][tid & 3] = ml.y;
      }
      __syncthreads();
      if (tid < 4) {                                    // thread r: the parts' weights for row c + r
        float m = kAtLowest, l = 0.f;
        for (int i = 0; i < n; ++i) m = fmaxf(m, wgt[i][tid]);
        for (int i = 0; i < n; ++i) {
          const float w = at_exp2(wgt[i][tid] - m);
          wgt[i][tid] = w;
          l += w * sum[i][tid];
        }
        inv[tid] = l == 0.f ? 0.f : 1.0f / l;
        if (p.lse && tid < rows) p.lse[jn.row0 + c + tid] = lse(m, l);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < n) add(acc, *reinterpret_cast<const float4*>(&wgt[i][0]), o[i]);
      for (int i = kAhead; i < n; ++i)
        add(acc, *reinterpret_cast<const float4*>(&wgt[i][0]), *reinterpret_cast<const float4*>(src + slot(i) * kAtPart));
      write(acc, make_float4(inv[0], inv[1], inv[2], inv[3]), tid);
      continue;
    }
    __syncthreads();                                    // the previous task's weights are read
    for (int i = tid; i < n * 4; i += kAtJoinThreads) {
      const float2 ml = p.part_ml[slot(i >> 2) * kAtRows + c + (i & 3)];
      wgt[i >> 2][i & 3] = ml.x;
      sum[i >> 2][i & 3] = ml.y;
    }
    __syncthreads();
    if (warp < 4) {                                     // warp w: the parts' weights for row c + w
      float m = kAtLowest;
      for (int i = lane; i < n; i += 32) m = fmaxf(m, wgt[i][warp]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float l = 0.f;
      for (int i = lane; i < n; i += 32) {
        const float w = at_exp2(wgt[i][warp] - m);
        wgt[i][warp] = w;
        l += w * sum[i][warp];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) {
        inv[warp] = l == 0.f ? 0.f : 1.0f / l;
        if (p.lse && warp < rows && (sub & 7) == 0) p.lse[jn.row0 + c + warp] = lse(m, l);
      }
    }
    __syncthreads();
    const int grp = tid >> 6, v = tid & 63, val = (sub & 7) * 64 + v;
    const float* src = p.part + at_part(c, val);
#pragma unroll 4
    for (int i = grp; i < n; i += 8)
      add(acc, *reinterpret_cast<const float4*>(&wgt[i][0]), *reinterpret_cast<const float4*>(src + slot(i) * kAtPart));
    if (grp) meet[grp - 1][v] = acc;
    __syncthreads();
    if (grp) continue;
#pragma unroll
    for (int g = 0; g < 7; ++g) add(acc, make_float4(1.f, 1.f, 1.f, 1.f), meet[g][v]);
    write(acc, make_float4(inv[0], inv[1], inv[2], inv[3]), val);
  }
}

// ------------------------------------------------------------------ host side

struct AtWs {
  size_t cta_status, units, joins, part, part_ml, total;
  long long max_units;
};

static AtWs at_ws(int B, int n_tokens, int H) {
  AtWs w;
  // dense: sum over requests of ceil(T H / 64); selected keys: n_tokens * ceil(H / 64)
  const long long dense = (long long)n_tokens * H / kAtRows + B + 1;
  const long long sel = (long long)n_tokens * ((H + kAtRows - 1) / kAtRows);
  w.max_units = dense > sel ? dense : sel;
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  w.cta_status = take(kAtMaxCtas * sizeof(int32_t));
  w.units = take((size_t)(w.max_units + kAtMaxCtas) * sizeof(AtUnit));
  w.joins = take((size_t)kAtMaxCtas * sizeof(AtJoin));
  w.part = take((size_t)2 * kAtMaxCtas * kAtPart * sizeof(float));
  w.part_ml = take((size_t)2 * kAtMaxCtas * kAtRows * sizeof(float2));
  w.total = off;
  return w;
}

// Rows of 576 elements, boxes of 64 columns and `box` rows, 128-byte swizzle.
static CUresult at_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, bool bf16, const void* base,
                       long long rows, int box_rows) {
  const cuuint64_t gdim[2] = {(cuuint64_t)kAtW, (cuuint64_t)rows};
  const cuuint64_t gstr[1] = {(cuuint64_t)kAtW * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                const_cast<void*>(base), gdim, gstr, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <bool BF16, bool TMA>
static cudaError_t at_launch(const AtArgs& a, const CUtensorMap& kmap, const CUtensorMap& qmap, int ctas,
                             int dev, cudaStream_t st) {
  static_assert((size_t)(3 * kAtMaxB + 2) * sizeof(int) + 1024 <= kAtSmem, "the plan's arrays");
  // once a device: setting it again costs as much as a tenth of a launch
  static std::atomic<bool> set[kAtMaxDevices];
  cudaError_t e = cudaSuccess;
  if (dev >= kAtMaxDevices || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kv_attention_kernel<BF16, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAtSmem);
    if (e != cudaSuccess) return e;
    if (dev < kAtMaxDevices) set[dev].store(true, std::memory_order_relaxed);
  }
  e = launch_pdl(kv_attention_kernel<BF16, TMA>, dim3(ctas), dim3(at_threads(TMA)), kAtSmem, st, a, kmap, qmap);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_attention_join_kernel<BF16>, dim3(kAtJoinCtas), dim3(kAtJoinThreads), 0, st, a, ctas);
}

// Failure-path testing (colibri_kv_debug_inject): of the calls of this thread.
static thread_local struct {
  int flags = 0;
  unsigned long long wait_ns = kWaitLimitNs;
} at_inject;

}  // namespace coli

using namespace coli;

extern "C" {

coli_status colibri_kv_attention_workspace_size(int B, int n_tokens, int H, size_t* bytes) {
  if (!bytes || B < 1 || n_tokens < 0 || H < 1) return fail(COLI_EINVAL, "kv_attention_workspace_size: bad argument");
  if ((long long)n_tokens * H > 0x7fffffffLL)
    return fail(COLI_EUNSUPPORTED, "kv_attention_workspace_size: n_tokens * H exceeds 2^31 - 1 rows");
  *bytes = at_ws(B, n_tokens, H).total;
  return COLI_OK;
}

coli_status colibri_kv_attention(const coli_kv_desc* desc, int B, int n_tokens, int H, float scale, const void* q,
                                 long long q_token_stride, long long q_head_stride, const void* cache,
                                 const int32_t* block_table, const int32_t* q_start, const int32_t* seq_len,
                                 const int32_t* topk_idx, int topk, void* out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const coli_status rc = check_kv_desc(desc, "kv_attention");
  if (rc != COLI_OK) return rc;
  if (B < 1 || n_tokens < 0 || H < 1) return fail(COLI_EINVAL, "kv_attention: need B, H >= 1 and n_tokens >= 0");
  if (B > kAtMaxB || H > kAtMaxH) return fail(COLI_EUNSUPPORTED, "kv_attention: at most 8192 requests of 1024 heads");
  if (desc->dtype != COLI_X_BF16 && desc->dtype != COLI_X_F16)
    return fail(COLI_EUNSUPPORTED, "kv_attention: the cache holds bf16 or fp16 (dtype %d)", desc->dtype);
  const float scale_log2 = scale * 1.4426950408889634f;    // (beyond 2.36e38 not finite either)
  if (!(scale_log2 - scale_log2 == 0.f)) return fail(COLI_EINVAL, "kv_attention: scale is not finite, or its product with log2(e) is not");
  if (topk_idx && topk < 1) return fail(COLI_EINVAL, "kv_attention: topk must be positive with topk_idx");
  if ((long long)n_tokens * H > 0x7fffffffLL - 1024)       // (row numbers of a last, partial gang of row tiles)
    return fail(COLI_EUNSUPPORTED, "kv_attention: n_tokens * H exceeds 2^31 - 1024 rows");
  if (topk_idx && topk > 1 << 30) return fail(COLI_EUNSUPPORTED, "kv_attention: topk exceeds 2^30");
  const long long per_page = desc->page_stride / COLI_KV_WIDTH;
  const long long cached = (desc->n_pages - 1LL) * per_page + desc->page_size;
  if (cached > 0x7fffffffLL) return fail(COLI_EUNSUPPORTED, "kv_attention: the cache exceeds 2^31 - 1 rows");
  if (n_tokens == 0) return COLI_OK;
  if (!q || !cache || !block_table || !q_start || !seq_len || !out || !workspace)
    return fail(COLI_EINVAL, "kv_attention: null pointer");
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return fail(COLI_EALIGN, "kv_attention: q, cache and out 16-byte, workspace 256-byte alignment");
  if (!aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(seq_len, 4) || !aligned(topk_idx, 4) || !aligned(lse, 4))
    return fail(COLI_EALIGN, "kv_attention: a pointer is not 4-byte aligned");
  const long long ts = n_tokens > 1 ? q_token_stride : 0, hs = H > 1 ? q_head_stride : 0;
  if (ts < 0 || hs < 0 || (n_tokens > 1 && ts == 0) || (H > 1 && hs == 0))
    return fail(COLI_EINVAL, "kv_attention: query strides must be positive");
  if (ts % 8 || hs % 8) return fail(COLI_EALIGN, "kv_attention: query strides must be multiples of 8 elements");
  const AtWs w = at_ws(B, n_tokens, H);
  if (workspace_bytes < w.total)
    return fail(COLI_EWORKSPACE, "kv_attention: workspace %zu bytes < required %zu", workspace_bytes, w.total);
  const long long tiles = topk_idx ? (topk + kAtKeys - 1LL) / kAtKeys
                                   : ((long long)desc->max_pages * desc->page_size + kAtKeys - 1) / kAtKeys;
  if (w.max_units * tiles > 0x7fffffffLL)
    return fail(COLI_EUNSUPPORTED, "kv_attention: %lld units of up to %lld key tiles exceed 2^31 - 1",
                w.max_units, tiles);
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  static std::atomic<int> known_sms[kAtMaxDevices];
  if (ce == cudaSuccess && dev < kAtMaxDevices) sms = known_sms[dev].load(std::memory_order_relaxed);
  if (ce == cudaSuccess && !sms) {
    ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (ce == cudaSuccess && dev < kAtMaxDevices) known_sms[dev].store(sms, std::memory_order_relaxed);
  }
  if (ce != cudaSuccess) return cuda_fail(ce, "kv_attention: device query");
  const bool bf16 = desc->dtype == COLI_X_BF16;
  // TMA boxes where pages are whole boxes and query rows evenly spaced; else the copying kernel
  int box = kAtKeys;
  while (desc->page_size % box) box /= 2;
  const bool tma = !topk_idx && box >= kAtMinBox && (H == 1 || hs == kAtW) && (n_tokens == 1 || ts == (long long)H * kAtW);
  CUtensorMap kmap = {}, qmap = {};
  if (tma) {
    auto encode = get_encode();
    if (!encode) return fail(COLI_ECUDA, "kv_attention: cuTensorMapEncodeTiled is not available");
    CUresult r = at_map(encode, &kmap, bf16, cache, cached, box);
    if (r != CUDA_SUCCESS) return fail(COLI_ECUDA, "kv_attention: cache tensor map (%d)", (int)r);
    r = at_map(encode, &qmap, bf16, q, (long long)n_tokens * H, kAtRows);
    if (r != CUDA_SUCCESS) return fail(COLI_ECUDA, "kv_attention: query tensor map (%d)", (int)r);
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AtArgs a;
  a.d = *desc;
  a.B = B;
  a.n_tokens = n_tokens;
  a.H = H;
  a.topk = topk_idx ? topk : 0;
  a.scale_log2 = scale_log2;
  a.rows_per_page = (int)per_page;
  a.box = box;
  a.box_log2 = 0;
  while ((1 << a.box_log2) < box) ++a.box_log2;
  a.by_page.set(desc->page_size);
  a.by_heads.set(H);
  a.q_tok = ts * 2;
  a.q_head = hs * 2;
  a.q = static_cast<const uint8_t*>(q);
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = block_table;
  a.q_start = q_start;
  a.seq_len = seq_len;
  a.sel = topk_idx;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.cta_status = reinterpret_cast<int32_t*>(ws + w.cta_status);
  a.units = reinterpret_cast<AtUnit*>(ws + w.units);
  a.joins = reinterpret_cast<AtJoin*>(ws + w.joins);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  a.wait_ns = at_inject.wait_ns;
  a.withhold = at_inject.flags & COLI_INJECT_WITHHOLD_STAGE ? 1 : 0;
  const int ctas = sms < kAtMaxCtas ? sms : kAtMaxCtas;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tma) ce = bf16 ? at_launch<true, true>(a, kmap, qmap, ctas, dev, st) : at_launch<false, true>(a, kmap, qmap, ctas, dev, st);
  else ce = bf16 ? at_launch<true, false>(a, kmap, qmap, ctas, dev, st) : at_launch<false, false>(a, kmap, qmap, ctas, dev, st);
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "kv_attention: launch");
}

coli_status colibri_kv_debug_inject(int flags, double wait_limit_ms) {
  if (flags & ~COLI_INJECT_WITHHOLD_STAGE) return fail(COLI_EINVAL, "kv_debug_inject: unknown flag bits 0x%x", flags);
  if (!(wait_limit_ms == wait_limit_ms)) return fail(COLI_EINVAL, "kv_debug_inject: wait limit is NaN");
  at_inject.flags = flags;
  // between a microsecond and the ordinary limit
  at_inject.wait_ns = wait_limit_ms > 0 && wait_limit_ms * 1e6 < (double)kWaitLimitNs
                          ? (unsigned long long)(wait_limit_ms * 1e6) : kWaitLimitNs;
  if (at_inject.wait_ns < 1000) at_inject.wait_ns = 1000;
  return COLI_OK;
}

coli_status colibri_kv_check_status(const void* workspace, int32_t* device_status, void* stream) {
  if (!workspace || !device_status) return fail(COLI_EINVAL, "kv_check_status: null argument");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  cudaError_t ce = cudaMemcpyAsync(&v, workspace, 4, cudaMemcpyDeviceToHost, st);
  if (ce == cudaSuccess) ce = cudaStreamSynchronize(st);
  if (ce != cudaSuccess) return cuda_fail(ce, "kv_check_status");
  *device_status = v;
  if (v) return fail(COLI_EDEVICE, "kv_attention device status 0x%x (wait timeout = 2, bad page = 64)", v);
  return COLI_OK;
}

}  // extern "C"
