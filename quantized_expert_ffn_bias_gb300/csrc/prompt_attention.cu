// Attention of prompts in the expanded form of latent attention ("25GB RAM
// runs 744B GLM-5.2" page (pwwt.cn), section 3.2: 576 cached values a token,
// of which 64 carry the rotary positions): the latent rows have been projected
// up to keys and values of every head, and
//   out[n][h] = sum_j p_j v[j][h],
//   p = softmax_j(scale * (q[n][h][:128] . k[j][h] + q[n][h][128:] . r[j])),
// r[j] the rotary key that all heads share.  A (row, key, head) costs 320
// multiply-adds here and 1088 in the absorbed form over the cache, which in
// turn reads 1152 bytes a key where this one reads 512 a head: prompts and
// chunks belong here, single tokens there.
//
// A pair of CTAs (a cluster, one on each SM of a TPC) takes 512 rows of one head as two row tiles of 256, 128 rows of
// either in each CTA, and walks the keys in tiles of 128 (tcgen05 with cta_group::2, fp32 accumulators in tensor memory):
//   S_x[256 rows][128 keys] = Q_x [K | R]^T   (12 products of depth 16)
//   O_x[256 rows][128]     += P_x V           (8 products; P_x takes S_x's place in tensor memory as 16-bit weights)
// Each CTA holds half of a key tile (64 keys of K and R, 64 of V's 128 columns: 40 KB), so three tiles fit beside the
// queries' 96 KB, and each product reads half the operand bytes of a CTA's own; with whole tiles in each CTA (1.6 of them
// fitted) the products waited 1,000 of 4,260 cycles a tile for keys and values.
// While the softmax warps of one row tile work, the tensor cores take the other's products: PV_0(t), S_0(t + 1),
// PV_1(t), S_1(t + 1), ...  A thread of the softmax holds a whole row of S, so that sums need no other thread.
//
// Softmax: per row a reference m (log2 units, a whole number; at first that of scores near 0).  A tile takes its weights
// against the reference as it is, without looking for the largest score; only where a row's weights sum to more than 2^15,
// or those of its first keys to less than 2^-6 (fp16: 32, so that weights down to 2^-29 of the sum count), are the scores
// read again, their maximum taken and the reference (with the sum and O) moved.  Looking for the maximum first cost 8 % of a
// prompt of 8192.  That branch is written for size: with scores of normal spread hardly a tile takes it; a first key that scores
// 12 above the rest costs 8192 tokens 2 %, the batch below 12 %, scores that rise by 20 along the keys 15 and 34 %.
//
// Work: units with their key tiles, dealt in equal runs to the pairs.  A unit is 512 rows of one head, or, for the last rows
// of a request where they are 256 at most, those of two heads, one to either row tile: with one row tile the tensor cores
// wait while its softmax runs (7 tokens over 20,018 keys, 16 heads: 66 us, by two heads 59; 45 to 48 by now).  A unit cut by a
// border leaves partial results in the workspace, which the join kernel adds up in order.
//
// What bounds it: a prompt of 8192 tokens and 64 heads takes 795 to 815 us on a GPU that has not been busy (1.71 PFLOP/s, 87 % of
// the measured burst rate of bf16 products; 930 us at the power limit, where those reach 1.73): a step of both row tiles takes
// 3,000 cycles, its products 2,560; the rest is the way from one row tile's softmax (1,050 cycles) to its next scores, a
// chain of 3,000 cycles that two row tiles do not quite hide.  A unit costs about 10,000 cycles beside its steps (first
// scores, last products, rows out, instructions that were not used for a while), which is most of what a batch of short
// prompts pays: 12 of 209 to 1484 tokens, 32 heads, 155 us: 88 for 55 steps a pair, 15 for the call, 52 for 9.3 units.
#include <atomic>
#include <type_traits>

#include "plan.h"

namespace coli {

constexpr int kPaQk = COLI_PROMPT_KEY + COLI_PROMPT_ROTARY, kPaV = COLI_PROMPT_VALUE;
static_assert(kPaQk == 192 && kPaV == 128, "three boxes of 64 columns of queries and keys, two of values");
constexpr int kPaTile = 128;                       // rows of a CTA in a row tile, keys of a key tile
constexpr int kPaRows = 4 * kPaTile;               // rows of a unit
constexpr int kPaCtaRows = kPaRows / 2;
constexpr int kPaKeyBox = 64 * 128;                // 64 columns of 64 keys
constexpr int kPaValues = kPaTile * 128;           // 64 columns of 128 values' rows
constexpr int kPaKeys3 = 3 * kPaKeyBox;            // a CTA's K and R of a tile
constexpr int kPaStage = kPaKeys3 + kPaValues;     // its part of a key tile
constexpr int kPaStages = 3;
constexpr int kPaQBytes = 3 * kPaTile * 128;       // its part of a row tile's queries
constexpr int kPaOutStage = 8 * 64;                // a warp's place for results on their way out
constexpr int kPaSmWarps = 8;                      // softmax: warps 0..3 row tile 0, 4..7 row tile 1
constexpr int kPaLoader = 8, kPaMma = 9, kPaCheck = 10, kPaCheckWarps = 2;
constexpr int kPaThreads = (kPaCheck + kPaCheckWarps) * 32;
constexpr size_t kPaSmem = 2 * (size_t)kPaQBytes + (size_t)kPaStages * kPaStage + kPaSmWarps * kPaOutStage;
static_assert(kPaSmem + 6 * 1024 <= 232448, "with the kernel's own arrays");
constexpr int kPaMasked = 6;                       // key tiles of a unit of which some row does not see some key: 5, or 3 of two heads
constexpr int kPaMaxCtas = 160;                    // CTAs the workspace has room for
constexpr int kPaMaxB = 8192, kPaMaxH = 1024;
constexpr int kPaMaxDevices = 64;
constexpr int kPaPart = kPaCtaRows * kPaV;         // floats of a CTA's partial O
// A reference that is set by the largest weight makes that 2^(top - 1) .. 2^top.  It is set, or raised, where a tile's weights
// against the one so far sum to more than kPaSumLimit, or those of a row's first keys to less than pa_first.  bf16 has fp32's
// range; fp16 ends at 2^16 and loses bits below 2^-14, so its weights take the upper part.
__host__ __device__ constexpr float pa_top(bool bf16) { return bf16 ? 0.f : 7.f; }
constexpr float kPaSumLimit = 32768.f;             // a row's weights of a tile sum to at most this,
__host__ __device__ constexpr float pa_first(bool bf16) { return bf16 ? 1.f / 64 : 32.f; }   // those of its first keys to at least this
constexpr float kPaLowest = -3.402823466e38f;      // reference of a part in which the row has no finite score, below all others
constexpr uint32_t kPaOCol = 256;                  // TMEM columns: S_0 0.., S_1 128.., O_0 256.., O_1 384..

// A unit cut by borders: its parts are those of pairs pair, pair + 1, ...
struct __align__(16) PaJoin {
  int row0, rows;   // first row of the batch, rows
  int h, heads;     // first head; 2: two heads of the same rows
  int pair, parts;
  int which;        // of the first pair's two partial results (the others': the first)
  int first;        // rows from this one on see a key
};

struct PaArgs {
  int B, n_tokens, n_keys, H;
  float scale_log2;
  const int32_t *q_start, *k_start;
  const uint8_t* v;                  // the values (read again where one is not finite)
  long long v_tok, v_head;           // their strides, bytes
  uint16_t* out;
  float* lse;
  int32_t* status;
  int32_t* cta_status;               // [kPaMaxCtas]
  PaJoin* joins;                     // [kPaMaxCtas / 2] one a pair, written by it (parts = 0: none)
  float* part;                       // [2 kPaMaxCtas] partial O (pa_slot, pa_part)
  float2* part_ml;                   // [2 kPaMaxCtas][256] reference (-infinity: no values written), sum
  unsigned long long wait_ns;
  int withhold;                      // failure-path test: 1: no pair's first keys ever count as there
};

struct PaMaps {
  CUtensorMap q, k, r, v;
};

// Partial results: two a pair (of its run's first unit, of its last), a half in each CTA.  A CTA's row i is row
// rank 128 + i % 128 of row tile i / 128.
__host__ __device__ constexpr size_t pa_slot(int pair, int which, int rank) { return ((size_t)pair * 2 + which) * 2 + rank; }
// Place of row r and value c (a multiple of four) in one: neighbouring rows' four values lie together, as a warp's
// threads hold them.
__host__ __device__ constexpr int pa_part(int r, int c) { return ((c >> 2) * kPaCtaRows + r) * 4; }

// ------------------------------------------------------------------ plan
// Every CTA finds its pair's run of the work from the lengths.  A request's T new rows over L keys come in blocks of 512;
// block j (1, 2, ...) sees keys up to its last row: max(1, a + 4 j) tiles with a = ceil((L - T) / 128), the last block all
// of them.  Units are (request, head, block), block fastest, so that neighbouring pairs work on the same head's keys; a last
// block of at most 256 rows comes behind them, two heads a unit.
// What a unit costs beside its tiles (its rows' way out, the first softmax: about 10,000 cycles, a tile 3,100) is dealt with
// them: a unit's places are kPaUnitCost and then its tiles; a border among the first is one before its first tile.
// The code runs once a launch and what it costs is mostly fetching it: 32 bits, few divisions, each step written once.
constexpr int kPaUnitCost = 3;
constexpr int kPaTilesPerBlock = kPaRows / kPaTile;
__device__ __forceinline__ int pa_blocks(int T) { return (int)(((unsigned)T + kPaRows - 1) / kPaRows); }
// blocks that units take head by head; 1 more where the last one goes by two heads
__device__ __forceinline__ bool pa_short(int T) { return (unsigned)(T - 1) % kPaRows < (unsigned)kPaRows / 2; }
__device__ __forceinline__ int pa_key_tiles(int keys) { return max(1, (keys + kPaTile - 1) >> 7); }
// Places of the first n of nb blocks, saturating (a sum that does not fit 31 bits is refused).
__device__ __noinline__ unsigned pa_before(int T, int L, int nb, int n) {
  const int a = (L - T + kPaTile - 1) >> 7;
  const int m = min(n, nb - 1);
  const int flat = a < 0 ? min(m, -a / kPaTilesPerBlock) : 0;        // blocks whose rows see nothing: one tile each
  const long long s = flat + (long long)(m - flat) * a +
                      (long long)(kPaTilesPerBlock / 2) * ((long long)m * (m + 1) - (long long)flat * (flat + 1)) +
                      (n == nb ? pa_key_tiles(L) : 0) + (long long)kPaUnitCost * n;
  return (unsigned)min(s, 0x7fffffffll);
}

// Borders of G <= kPaMaxCtas equal runs of the W places: floor(W j / G), without leaving 32 bits.  The
// remainder's part is below kPaMaxCtas^2, where the fp32 quotient of x + 1/2 is exact.
struct PaCuts {
  int q, r;
  float inv;
  __device__ __forceinline__ PaCuts(int W, int G) : q(W / G), r(W - q * G), inv(1.0f / (float)G) {}
  __device__ __forceinline__ int operator()(int j) const { return q * j + (int)(((float)(r * j) + 0.5f) * inv); }
};

struct __align__(16) PaUnit {
  int b, h, blk;
  int nb;            // blocks that go head by head; block nb goes by two heads
  int q0, T, k0, L;
  int first;         // places of the units before it
  int tiles;
  // The tiles of it between two borders.
  __device__ __forceinline__ int from(int beg) const { return max(0, beg - first - kPaUnitCost); }
  __device__ __forceinline__ int to(int end) const { return min(end - first - kPaUnitCost, tiles); }
};

struct PaRun {
  int beg, end;
  int status;
};

// Where a warp is: a unit and its part [t0, t1) of the run.  In shared memory, filled by one lane; the code that fills it
// stands once (no inlining): every role's own copy of it made the kernel 139 KB, more than the instruction cache, and a
// unit's first tile cost 5,000 cycles in place of 1,500.
struct __align__(16) PaAt {
  PaUnit u;
  int live;          // 0: behind the run's last
  int opening;       // the run's first
  int whole;         // all of the unit's tiles
  int t0;
  int two;           // row tile 1 has the rows of tile 0 and the next head
  int heads;         // key tiles a step: 2 where there are two heads
  int row0;          // its first row of the request
  int shift;         // the last key that row i of the request sees: shift + i
  int rows[2];       // rows of either row tile
  int n[2];          // key tiles of row tile x in the part
  int all;           // the larger
  int masked;        // first tile of which some row does not see some key
  __device__ __forceinline__ int first_row(int x) const { return row0 + (two ? 0 : x * 2 * kPaTile); }
};

__device__ __forceinline__ void pa_tiles(PaUnit& u) {
  const int rows = u.T - u.blk * kPaRows;              // of the request from the block's first on
  u.tiles = pa_key_tiles(rows <= kPaRows ? u.L : u.L - rows + kPaRows);
}
// The unit after u (of the same or a later request; the caller has not reached the end of the work).
__device__ __noinline__ void pa_next(const PaArgs& p, PaUnit& u) {
  u.first += kPaUnitCost + u.tiles;
  if (u.blk == u.nb) {
    u.h += 2;
  } else if (++u.blk == u.nb) {
    u.blk = 0;
    ++u.h;
  }
  if (u.h >= p.H) {
    u.h = 0;
    if (u.blk < u.nb && pa_short(u.T)) {
      u.blk = u.nb;
    } else {
      do {
        if (u.b + 1 >= p.B) return;
        ++u.b;
        u.q0 = p.q_start[u.b];
        u.T = p.q_start[u.b + 1] - u.q0;
        u.k0 = p.k_start[u.b];
        u.L = p.k_start[u.b + 1] - u.k0;
      } while (u.T == 0);
      u.nb = pa_blocks(u.T) - (pa_short(u.T) ? 1 : 0);
      u.blk = 0;
    }
  }
  pa_tiles(u);
}

// a: the part that begins at place `at` (of a.u) of a run that ends at `end`.
__device__ __noinline__ void pa_part(const PaArgs& p, PaAt& a, int at, int end) {
  const PaUnit& u = a.u;
  const int t0 = u.from(at), t1 = u.to(end);
  a.live = t1 > 0;                                     // (else the border lies before its first tile)
  a.t0 = t0;
  a.whole = t0 == 0 && t1 == u.tiles;
  const int row0 = u.blk * kPaRows, shift = u.L - u.T;
  const bool two = u.blk == u.nb;
  a.row0 = row0;
  a.shift = shift;
  a.two = two;
  a.heads = two && u.h + 1 < p.H ? 2 : 1;
  int all = 0;
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {
    const int from = row0 + (two ? 0 : x * 2 * kPaTile);
    const int rows = two && x >= a.heads ? 0 : max(0, min(2 * kPaTile, u.T - from));
    const int seen = rows > 0 ? (shift + from + rows + kPaTile - 1) >> 7 : 0;
    const int n = max(0, min(t1, seen) - t0);
    a.rows[x] = rows;
    a.n[x] = n;
    all = max(all, n);
  }
  a.all = all;
  a.masked = max(0, (shift + row0 + 1) >> 7);
}
// b: the part after a.
__device__ __noinline__ void pa_advance(const PaArgs& p, const PaAt& a, PaAt& b, int end) {
  b = a;
  b.opening = 0;
  const int at = a.u.first + kPaUnitCost + a.u.tiles;
  b.live = 0;
  if (at >= end) return;
  pa_next(p, b.u);
  pa_part(p, b, at, end);
}

constexpr int kPaWhole = 3;                // units of at most so many tiles are not cut: a join costs more (20 requests of 100 over 400 keys,
                                           // 32 heads: 63.6 us, with 4 66.9; 4 prompts of 300, 64 heads: 44.6, with 2 46.5)

// Every thread of the CTA calls it.  Each thread sums a stretch of the requests.  found: shared memory; found[0] receives
// the unit of the run's first place.
__device__ __forceinline__ PaRun pa_plan(const PaArgs& p, PaUnit* found) {
  __shared__ unsigned warp_tot[kPaThreads / 32];
  __shared__ int s_longest;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kPaThreads - 1) / kPaThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  if (tid == 0) s_longest = 0;
  bool wrong = false;
  unsigned sum = 0;
  int longest = 0;
  unsigned by_head = 0;                                // of the request looked at last: a head's places
  auto tiles_of = [&](int b, int& q0, int& T, int& k0, int& L) {
    const int q1 = p.q_start[b + 1], k1 = p.k_start[b + 1];
    q0 = p.q_start[b];
    k0 = p.k_start[b];
    if (q0 < 0 || q1 < q0 || q1 > p.n_tokens || k0 < 0 || k1 < k0 || k1 > p.n_keys) {
      wrong = true;
      return 0u;
    }
    T = q1 - q0;
    L = k1 - k0;
    if (T == 0) return 0u;
    const int nb = pa_blocks(T), shrt = pa_short(T) ? 1 : 0;
    by_head = pa_before(T, L, nb, nb - shrt);
    return (unsigned)min((unsigned long long)by_head * p.H + (shrt ? (unsigned long long)(kPaUnitCost + pa_key_tiles(L)) * ((p.H + 1) >> 1) : 0ull),
                         0x7fffffffull);
  };
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    int q0, T, k0, L;
    const unsigned t = tiles_of(b, q0, T, k0, L);
    sum = min(sum + t, 0x7fffffffu);
    if (t) longest = max(longest, pa_key_tiles(L));
  }
  unsigned inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = min(inc + n, 0x7fffffffu);
  }
  if (lane == 31) warp_tot[warp] = inc;
  longest = __reduce_max_sync(0xffffffffu, longest);
  wrong = __syncthreads_or(wrong);
  if (lane == 0 && longest) atomicMax(&s_longest, longest);
  unsigned total = 0, base = 0;
#pragma unroll 1
  for (int w = 0; w < kPaThreads / 32; ++w) {
    if (w == warp) base = total;
    total = min(total + warp_tot[w], 0x7fffffffu);
  }
  base += inc - sum;
  wrong |= total > 0x7fff0000u;                        // (room for sums with it)
  PaRun r;
  r.status = wrong ? COLI_DEV_KV_TOKENS : 0;
  r.beg = r.end = 0;
  const int W = wrong ? 0 : (int)total, pair = blockIdx.x >> 1;
  if ((blockIdx.x & 1) == 0 && tid == 0) p.joins[pair].parts = 0;
  // The longest run decides the time, so no more runs than it needs: fewer parts to write and join.
  int G = min((int)gridDim.x >> 1, W);
  if (pair >= G) return r;
  const int most = (W + G - 1) / G;
  G = (W + most - 1) / most;
  if (pair >= G) return r;
  const PaCuts cut(W, G);
  r.beg = cut(pair);
  r.end = cut(pair + 1);
  // the units of the run's first place and, where short units are not cut, of the next run's: found by the thread whose
  // requests hold it
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int x = k ? r.end : r.beg;
    if (k && (s_longest > kPaWhole || x >= W)) break;
    __syncthreads();
    if (x >= (int)base && x < (int)(base + sum)) {
      PaUnit u;
      int rest = x - (int)base, b = b0;
#pragma unroll 1
      for (;; ++b) {
        const int t = (int)tiles_of(b, u.q0, u.T, u.k0, u.L);
        if (rest < t) break;
        rest -= t;
      }
      u.b = b;
      const int blocks = pa_blocks(u.T), unit = (int)by_head;
      u.nb = blocks - (pa_short(u.T) ? 1 : 0);
      if (rest < unit * p.H) {                         // (the sum fits 31 bits)
        u.h = rest / unit;
        rest -= u.h * unit;
        int i = 0, n = u.nb;                           // last block with before(block) <= rest
#pragma unroll 1
        while (n - i > 1) {
          const int mid = (i + n) >> 1;
          if ((int)pa_before(u.T, u.L, blocks, mid) <= rest) i = mid;
          else n = mid;
        }
        u.blk = i;
        rest -= (int)pa_before(u.T, u.L, blocks, i);
      } else {
        rest -= unit * p.H;
        const int tiles = kPaUnitCost + pa_key_tiles(u.L);
        u.blk = u.nb;
        u.h = rest / tiles * 2;
        rest -= (u.h >> 1) * tiles;
      }
      u.first = x - rest;
      pa_tiles(u);
      found[k] = u;
    }
    __syncthreads();                                   // (the first round's make s_longest known, too)
    if (k && found[1].from(x) > 0) r.end = found[1].first + kPaUnitCost + found[1].tiles;
  }
  if (s_longest <= kPaWhole) {
    // short units are not cut: a run takes those that begin in it
    if (found[0].from(r.beg) > 0) {
      r.beg = found[0].first + kPaUnitCost + found[0].tiles;
      __syncthreads();
      if (tid == 0) pa_next(p, found[0]);
    }
    return r;
  }
  // a run that begins with the first border inside its unit lists the join
  const PaUnit& u = found[0];
  if ((blockIdx.x & 1) == 0 && tid == 0 && pair > 0 && u.from(r.beg) > 0 && u.from(cut(pair - 1)) == 0) {
    int m = pair;
    while (m < G && cut(m) < u.first + kPaUnitCost + u.tiles) ++m;     // runs pair - 1 .. m - 1 begin before the unit's end
    PaJoin jn;
    jn.row0 = u.q0 + u.blk * kPaRows;
    jn.rows = min(kPaRows, u.T - u.blk * kPaRows);
    jn.h = u.h;
    jn.heads = u.blk == u.nb && u.h + 1 < p.H ? 2 : 1;
    jn.pair = pair - 1;
    jn.parts = m - (pair - 1);
    jn.which = cut(pair - 1) < u.first ? 1 : 0;
    jn.first = u.T - u.L - u.blk * kPaRows;
    p.joins[pair] = jn;
  }
  return r;
}

// ------------------------------------------------------------------ main kernel

// Address of the same place of shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* at, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_store(uint32_t at, uint32_t v) {
  asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same where only tensor memory is handed over: tcgen05.wait::st and fence::before_thread_sync come before it and order it,
// so that the arrival itself needs none (a release for the cluster waits for every store: 1,000 cycles a tile).
__device__ __forceinline__ void cluster_arrive_tmem(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_fence() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Wait for a phase, at most about limit_ns, suspended by the hardware for 20 us at a time.  For the cluster: nearly every
// barrier counts copies, products or arrivals of either CTA.
// (What comes after the first look stands once: it is called from twenty places.)
constexpr uint32_t kPaSuspendNs = 20000;
__device__ __forceinline__ bool pa_look(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kPaSuspendNs)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool pa_wait_on(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
  const unsigned long long t0 = globaltimer();
  for (;;) {
    if (pa_look(bar, parity)) return true;
    if (globaltimer() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
  return pa_look(smem_u32(bar), parity) || pa_wait_on(smem_u32(bar), parity, limit_ns);
}

// TMA loads of a pair: into this CTA's shared memory, counted on a barrier of either CTA.
__device__ __forceinline__ void tma_pair_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_pair_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Operand read transposed (MN-major), 128-byte swizzle: 64 elements of N an atom of 8 K rows, the next 8 of K 1024 bytes
// further (an operand here has one atom of N a CTA).
__device__ __forceinline__ uint64_t pa_desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kPaValues >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ float pa_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 32 consecutive TMEM columns of this warp's 32 lanes -> registers (issue only)
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// registers -> 8 consecutive TMEM columns
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
constexpr int kPaChunk = 16;                       // columns of scores at a time (32: 2 % slower)
// registers -> 32 consecutive TMEM columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// Uses of the registers stay behind the wait.
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t* r) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Four products of depth 16 of a pair of CTAs, both operands in shared memory, issued by one elected lane of a converged
// warp; acc = 0: the first overwrites.
__device__ __forceinline__ void pa_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with A in tensor memory (8 columns a step) and B MN-major (16 rows of 128 bytes a step).
__device__ __forceinline__ void pa_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.u64 b1, %2, 128;\n\tadd.u64 b2, %2, 256;\n\tadd.u64 b3, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a2], b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a3], b3, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on `bar` in both CTAs when the products issued so far are complete (one elected lane of a converged warp).
__device__ __forceinline__ void pa_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\telect.sync _|e, 0xffffffff;\n\tmov.b16 m, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

// The same in this CTA alone.
__device__ __forceinline__ void pa_commit_here(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// What a row's sums are multiplied by: 0 where it sees no key; NaN where every key that it sees scores -infinity, as the softmax
// has it.
__device__ __forceinline__ float pa_share(float l, bool sees) { return l == 0.f ? (sees ? __int_as_float(0x7fffffff) : 0.f) : 1.0f / l; }

// Of a 32-bit word of two 16-bit values: whether either is an infinity or a NaN, and the word with those as 0.
template <bool BF16>
__device__ __forceinline__ bool pa_not_finite(uint32_t half) {
  constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  return (half & e) == e;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pa_finite_part(uint32_t w) {
  return (pa_not_finite<BF16>(w) ? 0u : w & 0xffffu) | (pa_not_finite<BF16>(w >> 16) ? 0u : w & 0xffff0000u);
}

template <bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const __grid_constant__ PaArgs p, const __grid_constant__ PaMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // Barriers of the first CTA, for its product issuer: what is there in both CTAs.
  __shared__ uint64_t q_full[2], k_full[kPaStages], v_full[kPaStages], v_ok[kPaStages], p_ready[2];
  // Barriers of either CTA: what the products are done with; values that the check awaits.
  __shared__ uint64_t q_empty[2], k_empty[kPaStages], v_empty[kPaStages], s_full[2], o_full[2], v_here[kPaStages], drained;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, cta_status, any_bad;      // any_bad: `bad` has been written
  // Keys (bits of two words, for either half) of the masked tiles whose values are not all finite in the columns of either
  // CTA, of four units, written only where there are any: the third word then is the unit's number plus one.  done: units
  // whose output each warp of either CTA has written.
  __shared__ uint32_t bad[2][4][kPaMasked][2][3], done[2][kPaSmWarps];
  uint8_t* smem = smem_raw;                            // (aligned as declared: the kernel's own arrays take whole KB before it)
  uint8_t* qsm = smem + kPaStages * kPaStage;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;                     // of this CTA in its pair (clusters are two neighbouring blocks)
  volatile int* abort_v = &abort_flag;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_ready[x], 8);
      mbar_init(&o_full[x], 1);
    }
    for (int i = 0; i < kPaStages; ++i) {
      mbar_init(&k_full[i], 1 + (i == 0 ? p.withhold : 0));     // (an arrival too many for a withheld stage)
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&v_here[i], 1);
      mbar_init(&v_ok[i], 2 * kPaCheckWarps);
    }
    mbar_init(&drained, 1);
    abort_flag = any_bad = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 2 * kPaSmWarps) (&done[0][0])[threadIdx.x] = 0;
  if (threadIdx.x < 2 * 4 * kPaMasked * 2) (&bad[0][0][0][0][0])[threadIdx.x * 3 + 2] = 0;
  if (warp == kPaLoader && lane == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.r);
    prefetch_tensormap(&maps.v);
  }
  if (warp == kPaMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                      // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  griddep_wait();                                      // the launch may overlap the kernel before; its results not
  __shared__ PaUnit found[2];
  __shared__ PaAt places[kPaThreads / 32][2];          // where each warp is, and what comes next
  int end;
  {
    const PaRun run = pa_plan(p, found);
    end = run.end;
    if (threadIdx.x == 0) cta_status = run.status;
    __syncthreads();
    if (lane == 0) {
      PaAt& a = places[warp][0];
      a.live = 0;
      if (run.beg < end) {
        a.u = found[0];
        pa_part(p, a, run.beg, end);
        a.opening = 1;
      }
    }
  }
  __syncthreads();
  int now = 0;
  bool looked = false;
  auto look_ahead = [&]() {                            // once a part, where the warp waits anyway
    if (lane == 0) pa_advance(p, places[warp][now], places[warp][now ^ 1], end);
    looked = true;
    __syncwarp();
  };
  auto next_part = [&]() {
    if (!looked) look_ahead();
    looked = false;
    now ^= 1;
    __syncwarp();
  };
  auto fail_wait = [&]() {
    atomicOr(&cta_status, COLI_DEV_WAIT_TIMEOUT);
    atomicExch(&abort_flag, 1);
  };

  if (warp == kPaLoader) {
    // ---------------------------------------------------------------- loader
    bool ok = true;
    unsigned tile = 0, q_used = 0, q_phase = 0;        // key tiles begun; bit x: row tile x's queries were loaded, parity
    auto wait = [&](uint64_t* bar, unsigned phase) { ok = __all_sync(0xffffffffu, pa_wait(bar, phase & 1, p.wait_ns)); };
    for (; ok && places[warp][now].live; next_part()) {
      const PaAt& a = places[warp][now];
      const int steps = a.all * a.heads, heads = a.heads, masked = a.masked, k0 = a.u.k0;
#pragma unroll 1
      for (int i = 0; ok && i < steps; ++i, ++tile) {
        if (__any_sync(0xffffffffu, *abort_v)) { ok = false; break; }
        const int t = a.t0 + (heads == 2 ? i >> 1 : i), head = a.u.h + (heads == 2 ? i & 1 : 0);
        const unsigned s = tile % kPaStages, use = tile / kPaStages;
        uint8_t* dst = smem + s * kPaStage;
        const int key = k0 + t * kPaTile;
        if (use > 0) wait(&k_empty[s], use - 1);
        if (!ok) break;
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&k_full[s], (uint32_t)(2 * kPaKeys3));
          const uint32_t bar = cluster_addr(&k_full[s], 0);
          tma_pair_3d(dst, &maps.k, 0, head, key + rank * 64, bar);
          tma_pair_3d(dst + kPaKeyBox, &maps.k, 64, head, key + rank * 64, bar);
          tma_pair_2d(dst + 2 * kPaKeyBox, &maps.r, 0, key + rank * 64, bar);
        }
        __syncwarp();
        if (i == 0) {                                  // the queries: rows past the unit's last are other rows' or, behind
#pragma unroll 1
          for (int x = 0; ok && x < 2; ++x) {          // the tensor, zeros: computed, not written
            if (a.n[x] == 0) continue;
            if ((q_used >> x) & 1) wait(&q_empty[x], q_phase >> x);
            if (!ok) break;
            q_phase ^= q_used & (1u << x);
            q_used |= 1u << x;
            if (lane < 3) {
              if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&q_full[x], (uint32_t)(2 * kPaQBytes));
              tma_pair_3d(qsm + x * kPaQBytes + lane * (kPaTile * 128), &maps.q, lane * 64, a.u.h + (a.two ? x : 0),
                          a.u.q0 + a.first_row(x) + rank * kPaTile, cluster_addr(&q_full[x], 0));
            }
            __syncwarp();
          }
          look_ahead();                                // and the next unit's on their way to L2
          const PaAt& b = places[warp][now ^ 1];
          if (ok && b.live && lane < 6) {
            const int x = lane / 3;
            tma_prefetch_3d(&maps.q, (lane % 3) * 64, min(b.u.h + (b.two ? x : 0), p.H - 1),
                            b.u.q0 + b.first_row(x) + rank * kPaTile);
          }
          __syncwarp();
        }
        if (ok && use > 0) wait(&v_empty[s], use - 1);
        if (!ok) break;
        if (lane == 0) {
          uint32_t bar = cluster_addr(&v_full[s], 0);
          if (t >= masked) {                           // these values go through the check: it says when they are ready
            mbar_arrive_expect_tx(&v_here[s], (uint32_t)kPaValues);
            if (rank == 0) mbar_arrive(&v_full[s]);
            bar = smem_u32(&v_here[s]);
          } else if (rank == 0) {
            mbar_arrive_expect_tx(&v_full[s], (uint32_t)(2 * kPaValues));
          }
          tma_pair_3d(dst + kPaKeys3, &maps.v, rank * 64, head, key, bar);
        }
        __syncwarp();
      }
    }
    // the products' last arrivals come before the CTA leaves
#pragma unroll 1
    for (unsigned s = 0; s < kPaStages; ++s) {
      if (!ok || tile <= s) continue;
      wait(&k_empty[s], (tile - s - 1) / kPaStages);
      if (ok) wait(&v_empty[s], (tile - s - 1) / kPaStages);
    }
#pragma unroll 1
    for (int x = 0; x < 2; ++x)
      if (ok && ((q_used >> x) & 1)) wait(&q_empty[x], q_phase >> x);
    if (!ok) fail_wait();
  } else if (warp == kPaMma) {
    // ---------------------------------------------------------------- product issuer (the warp stays converged)
    if (rank == 0) {
      const uint32_t idesc = BF16 ? umma_idesc_bf16(256, 128) : umma_idesc_f16(256, 128);
      const uint32_t idesc_v = idesc | (1u << 16);     // B MN-major
      const uint64_t kd = umma_desc_sw128(smem_u32(smem)), qd = umma_desc_sw128(smem_u32(qsm));
      const uint64_t vd = pa_desc_mn(smem_u32(smem + kPaKeys3));
      bool ok = true;
      // parities, bit x or s: of q_full, p_ready, v_ok
      unsigned tile = 0, q_phase = 0, p_phase = 0, checked = 0;
      auto wait = [&](uint64_t* bar, unsigned phase) {
        ok = __all_sync(0xffffffffu, ok && pa_wait(bar, phase & 1, p.wait_ns));
        return ok;
      };
      for (; ok && places[warp][now].live; next_part()) {
        const PaAt& a = places[warp][now];
        const int n0 = a.n[0], n1 = a.n[1], all = a.all, heads = a.heads, masked = a.masked - a.t0;
        // (the row tiles' code written out: rolled up it is 9 KB less, and 8192 tokens take 852 us, not 815)
        // Step i: row tile by row tile, the products with the values of tile i (i = -1: none) and the scores of tile i + 1
#pragma unroll 1
        for (int i = -1; ok && i < all; ++i) {
#pragma unroll
          for (int x = 0; ok && x < 2; ++x) {
            const int n = x ? n1 : n0;
            const uint32_t sx = tmem + x * kPaTile;
            if (i >= 0 && i < n) {
              const unsigned j = tile + i * heads + (heads == 2 ? x : 0), s = j % kPaStages;
              // the values, or, where some row does not see some key, the values after their check.  (Every phase of a
              // barrier is awaited or, v_full's of a checked tile, known to be over: a parity tells neighbours apart.)
              if (x == 0 || heads == 2 || i >= n0) {   // (else row tile 0 waited for them)
                if (i >= masked) {
                  ok = __all_sync(0xffffffffu, pa_wait(&v_ok[s], (checked >> s) & 1, p.wait_ns));
                  checked ^= 1u << s;
                } else {
                  wait(&v_full[s], j / kPaStages);
                }
              }
              if (!wait(&p_ready[x], p_phase >> x)) break;
              p_phase ^= 1u << x;
              tc_fence_after();
              const uint64_t v = vd + (uint64_t)((s * kPaStage) >> 4);
              pa_mma_ts(sx + kPaOCol, sx, v, idesc_v, i ? 1u : 0u);
              pa_mma_ts(sx + kPaOCol, sx + 32, v + (uint64_t)(kPaValues / 2 >> 4), idesc_v, 1u);
              if (heads == 2 || x == 1 || i >= n1) pa_commit(&v_empty[s]);       // (else row tile 1 is yet to read them)
              if (i + 1 == n) pa_commit(&o_full[x]);
            }
            if (i + 1 < n) {
              const unsigned j = tile + (i + 1) * heads + (heads == 2 ? x : 0), s = j % kPaStages;
              if (i < 0) {
                if (!wait(&q_full[x], q_phase >> x)) break;
                q_phase ^= 1u << x;
              }
              if ((x == 0 || heads == 2 || i + 1 >= n0) && !wait(&k_full[s], j / kPaStages)) break;
              tc_fence_after();
              const uint64_t k = kd + (uint64_t)((s * kPaStage) >> 4), q = qd + (uint64_t)((x * kPaQBytes) >> 4);
#pragma unroll
              for (int c = 0; c < 3; ++c)
                pa_mma_ss(sx, q + (uint64_t)(c * (kPaTile * 128) >> 4), k + (uint64_t)(c * kPaKeyBox >> 4), idesc, c ? 1u : 0u);
              pa_commit(&s_full[x]);
              if (i + 2 == n) pa_commit(&q_empty[x]);
              if (heads == 2 || x == 1 || i + 1 >= n1) pa_commit(&k_empty[s]);
            }
          }
        }
        tile += all * heads;
      }
      if (!ok && lane == 0) fail_wait();
      __syncwarp();
      // what was issued ends before tensor memory is freed, whichever role gave up
      pa_commit_here(&drained);
      pa_wait(&drained, 0, kWaitLimitNs);
    }
  } else if (warp >= kPaCheck) {
    // ---------------------------------------------------------------- check of the values of masked tiles
    // A row's weight for a key that it does not see is 0, and 0 times an infinity or a NaN is a NaN: such values
    // become 0 in shared memory before the product, and the rows that do see the key add them in the end.  Only the
    // tiles that cross the diagonal are looked at, by either CTA in its columns.
    const int half = warp - kPaCheck;                  // of the tile's keys
    const volatile uint32_t* done_v = &done[0][0];
    // the warps that write the rows have read what `bad` holds of four units before
    auto free_again = [&](unsigned uu) {
      if (uu < 4) return true;
      const unsigned long long from = globaltimer();
      while (__any_sync(0xffffffffu, (int)(done_v[lane & (2 * kPaSmWarps - 1)] - (uu - 3)) < 0))
        if (__any_sync(0xffffffffu, globaltimer() - from > p.wait_ns)) return false;
      cluster_fence();                                 // (their reads come before the writes to come)
      return true;
    };
    bool ok = true;
    unsigned tile = 0, checked = 0, uu = 0;
    for (; ok && places[warp][now].live; next_part()) {
      const PaAt& a = places[warp][now];
      if (a.all == 0) continue;
      const int heads = a.heads, steps = a.all * heads, ahead = (a.t0 - a.masked) * heads;     // of the masked tiles
      look_ahead();
#pragma unroll 1
      for (int i = max(0, -ahead); ok && i < steps; ++i) {
        const unsigned s = (tile + i) % kPaStages;
        ok = __all_sync(0xffffffffu, pa_wait(&v_here[s], (checked >> s) & 1, p.wait_ns));
        checked ^= 1u << s;
        if (!ok) break;
        uint8_t* box = smem + s * kPaStage + kPaKeys3 + half * (kPaValues / 2);
        uint32_t flags[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint8_t* row = box + (k * 32 + lane) * 128;
          uint32_t top = 0;                            // the largest magnitude of either half of the words
#pragma unroll
          for (int c = 0; c < 8; ++c) {                // (the lanes' rows meet the banks evenly by the rotation)
            const uint4 w = *reinterpret_cast<const uint4*>(row + (((c + lane) & 7) << 4));
            top = __vmaxu2(__vmaxu2(top, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
            top = __vmaxu2(__vmaxu2(top, w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
          }
          const bool wrong = pa_not_finite<BF16>(top) || pa_not_finite<BF16>(top >> 16);
          flags[k] = __ballot_sync(0xffffffffu, wrong);
          if (wrong) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint4* w = reinterpret_cast<uint4*>(row + (c << 4));
              *w = make_uint4(pa_finite_part<BF16>(w->x), pa_finite_part<BF16>(w->y), pa_finite_part<BF16>(w->z),
                              pa_finite_part<BF16>(w->w));
            }
          }
        }
        if (flags[0] | flags[1]) {
          ok = free_again(uu);
          if (!ok) break;
          if (lane < 2) cluster_store(cluster_addr(&any_bad, lane), 1);
          if (lane < 6) {                              // three words into either CTA
            const int w = lane % 3;
            cluster_store(cluster_addr(&bad[rank][uu & 3][ahead + i][half][w], lane / 3),
                          w == 2 ? uu + 1 : w == 1 ? flags[1] : flags[0]);
          }
          fence_proxy_async_smem();
          cluster_fence();
          __syncwarp();
        }
        // (a release also where nothing was written: the copy that this warp waited for is handed on)
        if (lane == 0) cluster_arrive(cluster_addr(&v_ok[s], 0));
      }
      tile += steps;
      ++uu;
    }
    if (!ok && lane == 0) fail_wait();
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int x = warp >> 2, sp = warp & 3;            // row tile, TMEM sub-partition
    const uint32_t ts = tmem + ((uint32_t)(sp * 32) << 16) + (uint32_t)(x * kPaTile), to = ts + kPaOCol;
    const int warp_row = rank * kPaTile + sp * 32, in_tile = warp_row + lane;      // of the row tile's 256
    const uint32_t ready = cluster_addr(&p_ready[x], 0);
    uint8_t* stage = qsm + 2 * kPaQBytes + warp * kPaOutStage;
    unsigned it = 0, un = 0, uu = 0;
    bool ok = true;
    for (; ok && places[warp][now].live; next_part()) {
      const PaAt& a = places[warp][now];
      const int n = a.n[x], t0 = a.t0;
      const bool mine = in_tile < a.rows[x], any = warp_row < a.rows[x];     // rows past the last are not written
      const int lim = a.shift + min(a.first_row(x) + in_tile, a.u.T - 1);    // the last key this row sees
      const int lim0 = a.shift + a.first_row(x) + warp_row;      // of the warp's first row
      float m = -pa_top(BF16), l = 0.f;                // reference, sum of the weights
      bool has = false;                                // the row has seen a key
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++it) {
        ok = __all_sync(0xffffffffu, pa_wait(&s_full[x], it & 1, p.wait_ns));
        if (!ok) break;
        tc_fence_after();
        const int key0 = (t0 + i) * kPaTile, rel = lim - key0;       // the tile's columns up to rel are seen
        // the tile's weights against the reference as it is; false where the sum tells that it does not serve
        auto weights = [&](auto all_seen) {
          uint32_t w[kPaTile / 2];
          const float2 by = make_float2(p.scale_log2, p.scale_log2), off = make_float2(-m, -m);
          float2 sum = make_float2(0.f, 0.f);
          // (the next chunk of scores is on its way while one is worked on)
          uint32_t r[2][kPaChunk];
          tmem_ld16_issue(ts, r[0]);
          tmem_ld_done<kPaChunk>(r[0]);
#pragma unroll
          for (int c = 0; c < kPaTile; c += kPaChunk) {
            uint32_t(&a)[kPaChunk] = r[(c / kPaChunk) & 1];
            uint32_t(&b)[kPaChunk] = r[(c / kPaChunk + 1) & 1];
            if (c + kPaChunk < kPaTile) tmem_ld16_issue(ts + c + kPaChunk, b);
#pragma unroll
            for (int j = 0; j < kPaChunk; j += 2) {
              const float2 d = ffma2(make_float2(__uint_as_float(a[j]), __uint_as_float(a[j + 1])), by, off);
              float2 e = make_float2(pa_exp2(d.x), pa_exp2(d.y));
              if constexpr (!decltype(all_seen)::value) {
                if (c + j > rel) e.x = 0.f;
                if (c + j + 1 > rel) e.y = 0.f;
              }
              sum = fadd2(sum, e);
              w[(c + j) / 2] = pa_pack<BF16>(e.x, e.y);
            }
            if (c + kPaChunk < kPaTile) tmem_ld_done<kPaChunk>(b);
          }
          const float add = sum.x + sum.y;
          const bool off_range = !(add <= kPaSumLimit) || (!has && rel >= 0 && !(add >= pa_first(BF16)));
          if (__any_sync(0xffffffffu, mine && off_range)) return false;
          l += add;
          has |= rel >= 0;
#pragma unroll
          for (int c = 0; c < kPaTile / 2; c += 32) tmem_st32(ts + c, w + c);
          return true;
        };
        bool fine = true;
        if (any) {
          if (key0 > lim0 + 31) {                      // no row of the warp sees any of these keys
            uint32_t zero[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) zero[j] = 0u;
            tmem_st32(ts, zero);
            tmem_st32(ts + 32, zero);
          } else if (key0 + kPaTile - 1 <= lim0) {
            fine = weights(std::true_type());
          } else {
            fine = weights(std::false_type());
          }
        }
        if (!fine) {
          // the maximum, a reference that serves, and the weights against it.  Rare: small code, the scores read twice
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kPaTile; c += 16) {
            uint32_t r[16];
            tmem_ld16_issue(ts + c, r);
            tmem_ld_done<16>(r);
#pragma unroll
            for (int j = 0; j < 16; ++j) {             // (masks after the scale, which may be 0 or negative)
              const float d = fmaf(__uint_as_float(r[j]), p.scale_log2, -m);
              top = fmaxf(top, c + j > rel ? -INFINITY : d);
            }
          }
          const float g = ceilf(top) - pa_top(BF16);
          const bool move = has ? g > 0.f : g > -INFINITY;
          // what that leaves of the sums so far: a first reference may lie far from 0, but they are 0 (or NaN) then
          const float keep = move && has ? pa_exp2(-g) : 1.f;
          // (the distance to the old reference is taken first: a product with the scale may lie far beyond their difference)
          const float by = move ? g : 0.f;
          l *= keep;
          if (i > 0 && __any_sync(0xffffffffu, keep != 1.f)) {     // (the first tile's products overwrite O)
#pragma unroll 1
            for (int c = 0; c < kPaV; c += 16) {
              uint32_t o[16];
              tmem_ld16_issue(to + c, o);
              tmem_ld_done<16>(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
              tmem_st16(to + c, o);
            }
          }
          float add = 0.f;
#pragma unroll 1
          for (int c = 0; c < kPaTile; c += 16) {      // (a chunk's weights take columns that are read already)
            uint32_t r[16], w[8];
            tmem_ld16_issue(ts + c, r);
            tmem_ld_done<16>(r);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float d[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                d[k] = c + j + k > rel ? 0.f : pa_exp2(fmaf(__uint_as_float(r[j + k]), p.scale_log2, -m) - by);
                add += d[k];
              }
              w[j / 2] = pa_pack<BF16>(d[0], d[1]);
            }
            tmem_st8(ts + c / 2, w);
          }
          m += by;
          has |= move;
          l += add;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(&p_ready[x]);     // (prompts of many units: 1 % over the way of the other CTA)
          else cluster_arrive_tmem(ready);
        }
      }
      // -------------------------------------------------------------- the unit's rows
      look_ahead();
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu, pa_wait(&o_full[x], un & 1, p.wait_ns));
        ++un;
      }
      if (!ok) break;
      tc_fence_after();
      const int masked = a.masked, head = a.u.h + (a.two ? x : 0), row = a.first_row(x) + in_tile;
      if (masked < t0 + n && *(volatile int*)&any_bad) {
        // values that were taken out of masked tiles are added to the rows that see them (rare: small code)
        const int e0 = max(masked, t0) - masked, e1 = t0 + n - masked, step = a.heads, mine_of = a.two ? x : 0;
        bool here = false;
        for (int e = e0; e < e1; ++e)
          here |= bad[lane & 1][uu & 3][e * step + mine_of][lane >> 1 & 1][2] == uu + 1;
        if (__any_sync(0xffffffffu, here)) {
#pragma unroll 1
          for (int e = e0 * 128; e < e1 * 128; ++e) {
            const int w = (e >> 7) * step + mine_of;
            uint32_t word = 0;
            for (int src = 0; src < 2; ++src) {
              const uint32_t* b = bad[src][uu & 3][w][(e >> 6) & 1];
              if (b[2] == uu + 1) word |= b[(e >> 5) & 1];
            }
            if (!((word >> (e & 31)) & 1u)) continue;
            const int key = masked * kPaTile + e;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v + (a.u.k0 + (long long)key) * p.v_tok + head * p.v_head);
#pragma unroll 1
            for (int c = 0; c < kPaV; c += 16) {
              uint32_t o[16];
              tmem_ld16_issue(to + c, o);
              tmem_ld_done<16>(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint32_t b = v[c + j];
                const float val = BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
                if (pa_not_finite<BF16>(b) && key <= lim) o[j] = __float_as_uint(__uint_as_float(o[j]) + val);
              }
              tmem_st16(to + c, o);
              tmem_st_wait();
            }
          }
        }
      }
      if (any) {
        const float by = pa_share(l, lim >= 0);
        const bool whole = a.whole;
        const size_t slot = pa_slot(blockIdx.x >> 1, a.opening ? 0 : 1, rank), row0 = (size_t)(a.u.q0 + row - lane) * p.H + head;
        const int in_cta = x * kPaTile + sp * 32 + lane;
        if (mine && whole && p.lse)
          p.lse[row0 + (size_t)lane * p.H] = l == 0.f ? -INFINITY : (log2f(l) + m) * 0.693147180559945309f;
        if (mine && !whole) p.part_ml[slot * kPaCtaRows + in_cta] = make_float2(has || l != 0.f ? m : n > 0 ? kPaLowest : -INFINITY, l);
        const int rows = a.rows[x] - warp_row;
        // eight rows of 64 bytes at a time by way of shared memory, so that a store covers eight lines (a row a lane: 32)
        const int r = lane >> 2;
        uint8_t* out = reinterpret_cast<uint8_t*>(p.out + (row0 + (size_t)r * p.H) * kPaV) + (lane & 3) * 16;
        const size_t row8 = (size_t)p.H * (8 * kPaV * 2);
        uint8_t* mine8 = stage + (lane & 7) * 64;
        const uint8_t* read8 = stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4);
        float* po = p.part + slot * kPaPart;
#pragma unroll 1
        for (int c = 0; c < kPaV; c += 32) {
          uint32_t o[32];
          tmem_ld32_issue(to + c, o);
          tmem_ld_done<32>(o);
          if (n == 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
          }
          if (whole) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j] = pa_pack<BF16>(__uint_as_float(o[2 * j]) * by, __uint_as_float(o[2 * j + 1]) * by);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if ((lane >> 3) == g) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  *reinterpret_cast<uint4*>(mine8 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
              }
              __syncwarp();
              const uint4 w = *reinterpret_cast<const uint4*>(read8);
              if (g * 8 + r < rows) *reinterpret_cast<uint4*>(out + g * row8 + c * 2) = w;
              __syncwarp();
            }
          } else if (n > 0 && mine) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(po + pa_part(in_cta, c + j)) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
      }
      tc_fence_before();
      if (*(volatile int*)&any_bad) cluster_fence();   // (the check writes `bad` again when it knows that it has been read)
      __syncwarp();                                    // (every lane has read `bad`)
      uu += a.all > 0;
      if (lane < 2) cluster_store(cluster_addr(&done[rank][warp], lane), uu);
    }
    if (!ok && lane == 0) fail_wait();
  }
  griddep_launch_dependents();                         // (earlier, the join's CTAs would take slots from the next call's)
  tc_fence_before();
  __syncthreads();
  if (abort_flag) {
    // copies may be on their way that no wait tells of: they end long before this does
    const unsigned long long from = globaltimer();
    while (globaltimer() - from < 1000000ull) {}
  }
  if (threadIdx.x == 0) p.cta_status[blockIdx.x] = cta_status;
  cluster_sync();                                      // the pair's products, copies and arrivals are over in both CTAs
  if (warp == kPaMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// ------------------------------------------------------------------ join
// Adds up the parts of every cut unit, in order.  A task is 32 rows of a unit (a row a lane, 16 values a warp).
constexpr int kPaJoinThreads = 256, kPaJoinCtas = 608, kPaAhead = 3;

template <bool BF16>
__global__ void __launch_bounds__(kPaJoinThreads) prompt_attention_join_kernel(const PaArgs p, int ctas) {
  __shared__ int starts[kPaJoinThreads], warp_tot[32], total;        // first task of each pair's join
  __shared__ PaJoin joins[kPaMaxCtas / 2];
  static_assert(kPaMaxCtas <= kPaJoinThreads, "a thread each");
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int tasks = 0;
  if (tid < ctas / 2) {
    const PaJoin jn = p.joins[tid];
    joins[tid] = jn;
    if (jn.parts > 0) tasks = (jn.rows + 31) / 32 * jn.heads;
  }
  const int bits = blockIdx.x == 0 && tid < ctas ? p.cta_status[tid] : 0;
  starts[tid] = block_exclusive_scan(tasks, warp_tot, &total);
  if (blockIdx.x == 0) {
    const int timed = __syncthreads_or(bits & COLI_DEV_WAIT_TIMEOUT), order = __syncthreads_or(bits & COLI_DEV_KV_TOKENS);
    if (tid == 0) *p.status = (timed ? COLI_DEV_WAIT_TIMEOUT : 0) | (order ? COLI_DEV_KV_TOKENS : 0);
  }
  __syncthreads();
  const int n_tasks = total;
  for (int task = blockIdx.x; task < n_tasks; task += gridDim.x) {
    int j = 0, h = kPaJoinThreads;                     // last pair whose join starts at or before the task
    while (h - j > 1) {
      const int mid = (j + h) >> 1;
      if (starts[mid] <= task) j = mid;
      else h = mid;
    }
    const PaJoin& jn = joins[j];
    const int n = jn.parts, per = (jn.rows + 31) / 32, sub = task - starts[j], second = jn.heads == 2 && sub >= per ? 1 : 0;
    const int r = (sub - second * per) * 32 + lane, c0 = warp * 16;        // (a second head's rows are row tile 1's)
    if (r >= jn.rows) continue;
    const int rank = (r >> 7) & 1, i_cta = ((r >> 8) + second) * kPaTile + (r & 127);
    float m = kPaLowest, l = 0.f;
    float4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    // three parts at a time, all of their loads in flight at once, against a maximum that grows
    for (int i0 = 0; i0 < n; i0 += kPaAhead) {
      float2 ml[kPaAhead];
      float4 o[kPaAhead][4];
#pragma unroll
      for (int k = 0; k < kPaAhead; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (i0 + k < n) {
          const size_t slot = pa_slot(jn.pair + i0 + k, i0 + k ? 0 : jn.which, rank);
          ml[k] = p.part_ml[slot * kPaCtaRows + i_cta];
#pragma unroll
          for (int c = 0; c < 4; ++c) o[k][c] = *reinterpret_cast<const float4*>(p.part + slot * kPaPart + pa_part(i_cta, c0 + 4 * c));
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kPaAhead; ++k) top = fmaxf(top, ml[k].x);
      const float keep = pa_exp2(m - top);
      m = top;
      l *= keep;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = make_float4(acc[c].x * keep, acc[c].y * keep, acc[c].z * keep, acc[c].w * keep);
#pragma unroll
      for (int k = 0; k < kPaAhead; ++k) {
        const float w = pa_exp2(ml[k].x - m);
        l += w * ml[k].y;
        if (ml[k].x != -INFINITY) {                    // (else no values were written; 0 times one that is not finite stays a NaN)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            acc[c].x = fmaf(w, o[k][c].x, acc[c].x);
            acc[c].y = fmaf(w, o[k][c].y, acc[c].y);
            acc[c].z = fmaf(w, o[k][c].z, acc[c].z);
            acc[c].w = fmaf(w, o[k][c].w, acc[c].w);
          }
        }
      }
    }
    const float by = pa_share(l, r >= jn.first);
    const size_t row = (size_t)(jn.row0 + r) * p.H + jn.h + second;
    if (p.lse && warp == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      uint4 w;
      w.x = pa_pack<BF16>(acc[c].x * by, acc[c].y * by);
      w.y = pa_pack<BF16>(acc[c].z * by, acc[c].w * by);
      w.z = pa_pack<BF16>(acc[c + 1].x * by, acc[c + 1].y * by);
      w.w = pa_pack<BF16>(acc[c + 1].z * by, acc[c + 1].w * by);
      *reinterpret_cast<uint4*>(p.out + row * kPaV + c0 + 4 * c) = w;
    }
  }
}

// ------------------------------------------------------------------ host side

struct PaWs {
  size_t cta_status, joins, part, part_ml, total;
};

static PaWs pa_ws() {
  PaWs w;
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  w.cta_status = take(kPaMaxCtas * sizeof(int32_t));
  w.joins = take((size_t)(kPaMaxCtas / 2) * sizeof(PaJoin));
  w.part = take((size_t)2 * kPaMaxCtas * kPaPart * sizeof(float));
  w.part_ml = take((size_t)2 * kPaMaxCtas * kPaCtaRows * sizeof(float2));
  w.total = off;
  return w;
}

// [rows][heads][cols] of 16-bit values with strides in elements; boxes of 64 columns of one head and `box` rows,
// 128-byte swizzle.  (The stride of an axis of one is not read.)
static CUresult pa_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, bool bf16, const void* base, int cols,
                       int heads, long long head_stride, long long rows, long long row_stride, int box) {
  const cuuint64_t gdim[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t gstr[2] = {(cuuint64_t)(heads > 1 ? head_stride : cols) * 2, (cuuint64_t)(rows > 1 ? row_stride : cols) * 2};
  const cuuint32_t bdim[3] = {64, 1, (cuuint32_t)box};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                const_cast<void*>(base), gdim, gstr, bdim, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}
static CUresult pa_map_rope(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* m, bool bf16, const void* base,
                            long long rows, long long row_stride) {
  const cuuint64_t gdim[2] = {(cuuint64_t)COLI_PROMPT_ROTARY, (cuuint64_t)rows};
  const cuuint64_t gstr[1] = {(cuuint64_t)(rows > 1 ? row_stride : COLI_PROMPT_ROTARY) * 2};
  const cuuint32_t bdim[2] = {64, (cuuint32_t)kPaTile / 2};
  const cuuint32_t es[2] = {1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                const_cast<void*>(base), gdim, gstr, bdim, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <bool BF16>
static cudaError_t pa_launch(const PaArgs& a, const PaMaps& maps, int ctas, int dev, cudaStream_t st) {
  // once a device: setting it again costs as much as a tenth of a launch
  static std::atomic<bool> set[kPaMaxDevices];
  cudaError_t e = cudaSuccess;
  if (dev >= kPaMaxDevices || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(prompt_attention_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPaSmem);
    if (e != cudaSuccess) return e;
    if (dev < kPaMaxDevices) set[dev].store(true, std::memory_order_relaxed);
  }
  e = launch_pdl(prompt_attention_kernel<BF16>, dim3(ctas), dim3(kPaThreads), kPaSmem, st, a, maps);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be tasks
  const long long tasks = (long long)a.n_tokens * a.H / 32 + ctas;
  return launch_pdl(prompt_attention_join_kernel<BF16>, dim3(tasks < kPaJoinCtas ? (int)tasks : kPaJoinCtas),
                    dim3(kPaJoinThreads), 0, st, a, ctas);
}

}  // namespace coli

using namespace coli;

extern "C" {

coli_status colibri_prompt_attention_workspace_size(int B, int n_tokens, int n_keys, int H, size_t* bytes) {
  if (!bytes || B < 1 || n_tokens < 0 || n_keys < 0 || H < 1)
    return fail(COLI_EINVAL, "prompt_attention_workspace_size: bad argument");
  *bytes = pa_ws().total;
  return COLI_OK;
}

coli_status colibri_prompt_attention(int dtype, int B, int n_tokens, int n_keys, int H, float scale, const void* q,
                                     long long q_token_stride, long long q_head_stride, const void* k,
                                     long long k_token_stride, long long k_head_stride, const void* k_rope,
                                     long long rope_stride, const void* v, long long v_token_stride,
                                     long long v_head_stride, const int32_t* q_start, const int32_t* k_start, void* out,
                                     float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 1 || n_tokens < 0 || n_keys < 0 || H < 1)
    return fail(COLI_EINVAL, "prompt_attention: need B, H >= 1 and n_tokens, n_keys >= 0");
  if (B > kPaMaxB || H > kPaMaxH) return fail(COLI_EUNSUPPORTED, "prompt_attention: at most 8192 requests of 1024 heads");
  if (dtype != COLI_X_BF16 && dtype != COLI_X_F16)
    return fail(COLI_EUNSUPPORTED, "prompt_attention: bf16 or fp16 (dtype %d)", dtype);
  const float scale_log2 = scale * 1.4426950408889634f;    // (beyond 2.36e38 not finite either)
  if (!(scale_log2 - scale_log2 == 0.f))
    return fail(COLI_EINVAL, "prompt_attention: scale is not finite, or its product with log2(e) is not");
  if (n_tokens > 0x7fffffff - 4096 || n_keys > 0x7fffffff - 4096)
    return fail(COLI_EUNSUPPORTED, "prompt_attention: n_tokens or n_keys exceeds 2^31 - 4096");
  if (n_tokens == 0) return COLI_OK;
  if (!q || !q_start || !k_start || !out || !workspace || (n_keys > 0 && (!k || !k_rope || !v)))
    return fail(COLI_EINVAL, "prompt_attention: null pointer");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(k_rope, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return fail(COLI_EALIGN, "prompt_attention: q, k, k_rope, v and out 16-byte, workspace 256-byte alignment");
  if (!aligned(q_start, 4) || !aligned(k_start, 4) || !aligned(lse, 4))
    return fail(COLI_EALIGN, "prompt_attention: a pointer is not 4-byte aligned");
  const struct { long long stride; bool read; } strides[] = {
      {q_token_stride, n_tokens > 1}, {q_head_stride, H > 1}, {k_token_stride, n_keys > 1}, {k_head_stride, n_keys > 0 && H > 1},
      {rope_stride, n_keys > 1}, {v_token_stride, n_keys > 1}, {v_head_stride, n_keys > 0 && H > 1}};
  for (const auto& s : strides) {
    if (!s.read) continue;
    if (s.stride <= 0) return fail(COLI_EINVAL, "prompt_attention: strides must be positive");
    if (s.stride % 8) return fail(COLI_EALIGN, "prompt_attention: strides must be multiples of 8 elements");
    if (s.stride >= 1LL << 38) return fail(COLI_EUNSUPPORTED, "prompt_attention: a stride exceeds 2^38 elements");
  }
  const PaWs w = pa_ws();
  if (workspace_bytes < w.total)
    return fail(COLI_EWORKSPACE, "prompt_attention: workspace %zu bytes < required %zu", workspace_bytes, w.total);
  int dev = 0, sms = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  static std::atomic<int> known_sms[kPaMaxDevices];
  if (ce == cudaSuccess && dev < kPaMaxDevices) sms = known_sms[dev].load(std::memory_order_relaxed);
  if (ce == cudaSuccess && !sms) {
    ce = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (ce == cudaSuccess && dev < kPaMaxDevices) known_sms[dev].store(sms, std::memory_order_relaxed);
  }
  if (ce != cudaSuccess) return cuda_fail(ce, "prompt_attention: device query");
  const bool bf16 = dtype == COLI_X_BF16;
  auto encode = get_encode();
  if (!encode) return fail(COLI_ECUDA, "prompt_attention: cuTensorMapEncodeTiled is not available");
  PaMaps maps;
  CUresult r = pa_map(encode, &maps.q, bf16, q, kPaQk, H, q_head_stride, n_tokens, q_token_stride, kPaTile);
  // without keys no tile is loaded: the queries stand in
  const bool keys = n_keys > 0;
  if (r == CUDA_SUCCESS)
    r = pa_map(encode, &maps.k, bf16, keys ? k : q, COLI_PROMPT_KEY, H, keys ? k_head_stride : q_head_stride,
               keys ? n_keys : 1, k_token_stride, kPaTile / 2);
  if (r == CUDA_SUCCESS) r = pa_map_rope(encode, &maps.r, bf16, keys ? k_rope : q, keys ? n_keys : 1, rope_stride);
  if (r == CUDA_SUCCESS)
    r = pa_map(encode, &maps.v, bf16, keys ? v : q, kPaV, H, keys ? v_head_stride : q_head_stride, keys ? n_keys : 1,
               v_token_stride, kPaTile);
  if (r != CUDA_SUCCESS) return fail(COLI_ECUDA, "prompt_attention: tensor map (%d)", (int)r);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PaArgs a;
  a.B = B;
  a.n_tokens = n_tokens;
  a.n_keys = n_keys;
  a.H = H;
  a.scale_log2 = scale_log2;
  a.q_start = q_start;
  a.k_start = k_start;
  a.v = static_cast<const uint8_t*>(v);
  a.v_tok = v_token_stride * 2;
  a.v_head = H > 1 ? v_head_stride * 2 : 0;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.cta_status = reinterpret_cast<int32_t*>(ws + w.cta_status);
  a.joins = reinterpret_cast<PaJoin*>(ws + w.joins);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  const KvInject inject = kv_inject();
  a.wait_ns = inject.wait_ns;
  a.withhold = inject.flags & COLI_INJECT_WITHHOLD_STAGE ? 1 : 0;
  const int ctas = (sms < kPaMaxCtas ? sms : kPaMaxCtas) & ~1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ce = bf16 ? pa_launch<true>(a, maps, ctas, dev, st) : pa_launch<false>(a, maps, ctas, dev, st);
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "prompt_attention: launch");
}

}  // extern "C"
