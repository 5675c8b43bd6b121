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
// A CTA takes 256 rows of one head as two tiles of 128 and walks the keys in
// tiles of 128 (tcgen05, fp32 accumulators in tensor memory):
//   S_x[128 rows][128 keys] = Q_x [K | R]^T   (12 products of depth 16)
//   O_x[128 rows][128]     += P_x V           (8 products; P_x takes S_x's place in tensor memory as 16-bit weights)
// While the softmax warps of one row tile work, the tensor cores take the other's products: PV_0(t), S_0(t + 1),
// PV_1(t), S_1(t + 1), ...  A thread of the softmax holds a whole row of S, so that maxima and sums need no other
// thread.
//
// Softmax: per row a reference m (log2 units, a whole number) that is raised, with the sum and O rescaled, only when it
// has to be: a tile whose every key is seen takes its weights against the reference as it is, without looking for the
// largest score; only where a row's weights sum to more than 2^15 (or the tile is a unit's first, or masked) are the scores
// read again, their maximum taken and the reference raised (where a score exceeds it by 8, or the sum was too large).
//
// Work: units (256 rows of one head, or of a gang of CTAs that walk the same keys) with their key tiles, in the order
// request, head, rows, dealt in equal runs of key tiles.  A unit cut by a border leaves partial results in the
// workspace, which the join kernel adds up in order.
#include <atomic>

#include "plan.h"

namespace coli {

constexpr int kPaQk = COLI_PROMPT_KEY + COLI_PROMPT_ROTARY, kPaV = COLI_PROMPT_VALUE;
static_assert(kPaQk == 192 && kPaV == 128, "three boxes of 64 columns of queries and keys, two of values");
constexpr int kPaTile = 128;                       // rows of a row tile, keys of a key tile
constexpr int kPaRows = 2 * kPaTile;               // rows a CTA takes of a unit
constexpr int kPaSlotBytes = kPaTile * 128;        // 64 columns of 128 keys (K, R), or 128 columns of 64 keys (V)
constexpr int kPaSlots = 8;                        // ring of slots: K, K, R, V, V of tile after tile
constexpr int kPaQBytes = 3 * kPaTile * 128;       // a row tile's queries
constexpr size_t kPaSmem = 2 * (size_t)kPaQBytes + (size_t)kPaSlots * kPaSlotBytes + 1024;
constexpr int kPaSmWarps = 8;                      // softmax: warps 0..3 row tile 0, 4..7 row tile 1
constexpr int kPaLoader = 8, kPaMma = 9, kPaCheck = 10, kPaCheckWarps = 2;
constexpr int kPaThreads = (kPaCheck + kPaCheckWarps) * 32;
constexpr int kPaMaxCtas = 160;                    // CTAs the workspace has room for
constexpr int kPaMaxB = 8192, kPaMaxH = 1024;
constexpr int kPaMaxDevices = 64;
constexpr int kPaPart = kPaRows * kPaV;            // floats of a partial O
constexpr float kPaGrow = 8.f;
constexpr float kPaSumLimit = 32768.f;             // a row's weights of one tile sum to at most this, or its reference is looked at
// A reference makes the largest weight 2^(top - 1) .. 2^top; growth to 2^(top + kPaGrow) raises it.  bf16 has fp32's
// range; fp16 ends at 2^16 and loses bits below 2^-14, so its weights take the upper part.
__host__ __device__ constexpr float pa_top(bool bf16) { return bf16 ? 0.f : 7.f; }
constexpr uint32_t kPaOCol = 256;                  // TMEM columns: S_0 0.., S_1 128.., O_0 256.., O_1 384..

// 256 rows of a unit cut by borders: its parts are those of CTAs cta, cta + gang, ...
struct __align__(16) PaJoin {
  int row0, rows;   // first row of the batch, rows
  int h;
  int cta, parts, gang;
  int slot;         // of the first part (the others': 2 * their CTA)
  int pad;
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
  PaJoin* joins;                     // [kPaMaxCtas] written by every CTA (parts = 0: none)
  float* part;                       // [2 kPaMaxCtas] partial O (pa_part)
  float2* part_ml;                   // [2 kPaMaxCtas][256] reference, sum
  unsigned long long wait_ns;
  int withhold;                      // failure-path test: 1: CTA 0's first copy never counts as complete
};

struct PaMaps {
  CUtensorMap q, k, r, v;
};

// Place of row r and value c (a multiple of four) in a partial O: neighbouring rows' four values lie together, as a
// warp's threads hold them.
__host__ __device__ constexpr int pa_part(int r, int c) { return ((c >> 2) * kPaRows + r) * 4; }

// ------------------------------------------------------------------ plan
// Every CTA finds its own run of the work from the lengths.  A request's new rows come in blocks of 256 * gang;
// block j of a request (1, 2, ...) sees keys up to its last row: max(1, a + 2 gang j) tiles with
// a = ceil((keys - rows) / 128), the last block all of them.  Units are (request, head, block), block fastest.
// Members of a gang take 256 rows each of the same keys at about the same time, so that a key tile comes from memory
// once for all of them: a CTA alone takes 80 KB a tile in about the time that memory needs for 152 of those.
struct PaRequest {
  int T, L, nb, a, g2;     // new rows, keys, blocks, see above, 2 * gang
  __device__ __forceinline__ PaRequest(int T_, int L_, int gang) : T(T_), L(L_), g2(2 * gang) {
    const int rows = kPaRows * gang;
    nb = (int)(((long long)T + rows - 1) / rows);
    a = (L - T + kPaTile - 1) >> 7;
  }
  // tiles of the first n blocks
  __device__ __forceinline__ long long before(int n) const {
    const int m = min(n, nb - 1);
    long long s = 0;
    if (m > 0) {
      const int flat = a < 0 ? min(m, -a / g2) : 0;        // blocks whose rows see nothing: one tile each
      s = flat + (long long)(m - flat) * a + (long long)g2 * (((long long)m * (m + 1) - (long long)flat * (flat + 1)) / 2);
    }
    if (n == nb && nb > 0) s += max(1, (L + kPaTile - 1) >> 7);
    return s;
  }
};

// A unit as its CTA (member `mem` of the gang) sees it.
struct PaUnit {
  int b, h, blk, nb;
  int q0, T, k0, L;
  long long first;   // key tiles of the units before it
  int tiles;
};

struct PaRun {
  int gang, member;
  long long beg, end;
  PaUnit unit0;      // that of `beg`
  int status;
};

__device__ __forceinline__ void pa_open(const PaArgs& p, PaUnit& u, int b, int gang) {
  u.b = b;
  u.q0 = p.q_start[b];
  u.T = p.q_start[b + 1] - u.q0;
  u.k0 = p.k_start[b];
  u.L = p.k_start[b + 1] - u.k0;
  u.nb = (int)(((long long)u.T + kPaRows * gang - 1) / (kPaRows * gang));
}
__device__ __forceinline__ void pa_tiles(PaUnit& u, int gang) {
  const int last = (int)min((long long)u.T, ((long long)u.blk + 1) * (kPaRows * gang));
  u.tiles = max(1, (u.L - u.T + last + kPaTile - 1) >> 7);
}
// The unit after u (of the same or a later request; the caller has not reached the end of the work).
__device__ __forceinline__ void pa_next(const PaArgs& p, PaUnit& u, int gang) {
  u.first += u.tiles;
  if (++u.blk == u.nb) {
    u.blk = 0;
    if (++u.h == p.H) {
      u.h = 0;
      do {
        if (u.b + 1 >= p.B) return;
        pa_open(p, u, u.b + 1, gang);
      } while (u.T == 0);
    }
  }
  pa_tiles(u, gang);
}

// What a part [t0, t1) of a unit is for this member.
struct PaPart {
  int row0, rows;    // its first row of the request, its rows (<= 0: none)
  int shift;         // the last key that row i of the request sees: shift + i
  int n[2];          // key tiles of row tile x in the part
  int all;           // the larger
  __device__ __forceinline__ PaPart(const PaUnit& u, int gang, int member, int t0, int t1) {
    const long long at = ((long long)u.blk * gang + member) * kPaRows;
    rows = (int)max(-1ll, min((long long)kPaRows, u.T - at));
    row0 = rows > 0 ? (int)at : 0;
    shift = u.L - u.T;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = min(kPaTile, rows - x * kPaTile);
      const int seen = r > 0 ? (shift + row0 + x * kPaTile + r + kPaTile - 1) >> 7 : 0;
      n[x] = max(0, min(t1, seen) - t0);
    }
    all = max(n[0], n[1]);
  }
  // first tile of which some row does not see some key
  __device__ __forceinline__ int masked() const { return max(0, (shift + row0 + 1) >> 7); }
};

constexpr float kPaTileNs = 1650.f;        // a key tile for 256 rows on one SM (measured)
constexpr float kPaTileMemNs = 12.1f;      // 82 KB at the memory's measured copy rate
constexpr long long kPaL2Keys = 100000;    // (key, head) pairs that stay in L2 between row blocks: 51 MB of keys and values
constexpr int kPaWhole = 4;                // units of at most so many tiles are not cut: a join costs more

// `sm`: shared memory for 16 (B + 1) bytes, free again when the call returns.  Every thread of the CTA calls it.
__device__ __forceinline__ PaRun pa_plan(const PaArgs& p, uint8_t* sm) {
  long long* first = reinterpret_cast<long long*>(sm);               // [B + 1] key tiles of the requests before
  int* qs = reinterpret_cast<int*>(first + p.B + 1);                 // [B + 1]
  int* ks = qs + p.B + 1;                                            // [B + 1]
  __shared__ long long sums[4], warp_tot[kPaThreads / 32 + 1];
  __shared__ int s_wrong, s_longest;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.B;
  if (tid < 4) sums[tid] = 0;
  if (tid == 0) s_wrong = s_longest = 0;
#pragma unroll 1
  for (int b = tid; b <= B; b += kPaThreads) {
    qs[b] = p.q_start[b];
    ks[b] = p.k_start[b];
  }
  __syncthreads();
  {
    bool wrong = false;
    long long s1 = 0, s2 = 0, s4 = 0, keys = 0;
    int longest = 0;
#pragma unroll 1
    for (int b = tid; b < B; b += kPaThreads) {
      const int q0 = qs[b], q1 = qs[b + 1], k0 = ks[b], k1 = ks[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > p.n_tokens || k0 < 0 || k1 < k0 || k1 > p.n_keys) {
        wrong = true;
      } else if (q1 > q0) {
        const PaRequest r1(q1 - q0, k1 - k0, 1), r2(q1 - q0, k1 - k0, 2), r4(q1 - q0, k1 - k0, 4);
        s1 += r1.before(r1.nb);
        s2 += r2.before(r2.nb);
        s4 += r4.before(r4.nb);
        keys += k1 - k0;
        longest = max(longest, max(1, (k1 - k0 + kPaTile - 1) >> 7));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      s4 += __shfl_xor_sync(0xffffffffu, s4, o);
      keys += __shfl_xor_sync(0xffffffffu, keys, o);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0 && longest) {
      atomicAdd(reinterpret_cast<unsigned long long*>(&sums[0]), (unsigned long long)s1);
      atomicAdd(reinterpret_cast<unsigned long long*>(&sums[1]), (unsigned long long)s2);
      atomicAdd(reinterpret_cast<unsigned long long*>(&sums[2]), (unsigned long long)s4);
      atomicAdd(reinterpret_cast<unsigned long long*>(&sums[3]), (unsigned long long)keys);
      atomicMax(&s_longest, longest);
    }
    if (wrong) s_wrong = 1;
  }
  __syncthreads();
  PaRun r;
  r.status = s_wrong ? COLI_DEV_KV_TOKENS : 0;
  r.gang = 1;
  if (sums[3] * p.H > kPaL2Keys) {
    float best = INFINITY;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int g = 1 << i;
      if (g > (int)gridDim.x) break;
      const float w = (float)sums[i] * (float)p.H;
      const float cost = fmaxf(w / (float)((int)gridDim.x / g) * kPaTileNs, w * kPaTileMemNs);
      if (cost < best) {
        best = cost;
        r.gang = g;
      }
    }
  }
  const int gang = r.gang, run = blockIdx.x / gang;
  r.member = blockIdx.x - run * gang;
  r.beg = r.end = 0;
  // key tiles of the requests before each
  long long carry = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < B; b0 += kPaThreads) {
    const int b = b0 + tid;
    long long v = 0;
    if (b < B && !s_wrong) {
      const PaRequest q(qs[b + 1] - qs[b], ks[b + 1] - ks[b], gang);
      v = q.before(q.nb) * p.H;
    }
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    if (tid == 0) {
      long long s = 0;
#pragma unroll 1
      for (int w = 0; w < kPaThreads / 32; ++w) {
        const long long t = warp_tot[w];
        warp_tot[w] = s;
        s += t;
      }
      warp_tot[kPaThreads / 32] = s;
    }
    __syncthreads();
    if (b < B) first[b] = carry + warp_tot[warp] + inc - v;
    carry += warp_tot[kPaThreads / 32];
    __syncthreads();
  }
  if (tid == 0) first[B] = carry;
  __syncthreads();
  const long long W = carry;
  if (tid == 0) p.joins[blockIdx.x].parts = 0;
  if (W == 0) return r;
  // The longest run decides the time, so no more runs than it needs: fewer parts to write and join.
  long long G = min((long long)((int)gridDim.x / gang), W);
  const long long longest = (W + G - 1) / G;
  G = (W + longest - 1) / longest;
  if (run >= G) return r;
  auto cut = [&](long long j) { return W * j / G; };       // (W < 2^44, G < 2^8)
  auto locate = [&](long long x) {
    int l = 0, h = B;                                      // last b with first[b] <= x: it has rows
#pragma unroll 1
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (first[mid] <= x) l = mid;
      else h = mid;
    }
    PaUnit u;
    u.b = l;
    u.q0 = qs[l];
    u.T = qs[l + 1] - qs[l];
    u.k0 = ks[l];
    u.L = ks[l + 1] - ks[l];
    const PaRequest q(u.T, u.L, gang);
    u.nb = q.nb;
    const long long per = q.before(q.nb);
    long long rest = x - first[l];
    u.h = (int)(rest / per);
    rest -= u.h * per;
    int i = 0, n = q.nb;                                   // last block with before(block) <= rest
#pragma unroll 1
    while (n - i > 1) {
      const int mid = (i + n) >> 1;
      if (q.before(mid) <= rest) i = mid;
      else n = mid;
    }
    u.blk = i;
    u.first = x - rest + q.before(i);
    pa_tiles(u, gang);
    return u;
  };
  r.beg = cut(run);
  r.end = cut(run + 1);
  r.unit0 = locate(r.beg);
  if (s_longest <= kPaWhole) {
    // short units are not cut: a run takes those that begin in it
    auto up = [&](long long x) {
      if (x == W) return W;
      const PaUnit u = locate(x);
      return u.first == x ? x : u.first + u.tiles;
    };
    r.beg = up(r.beg);
    r.end = up(r.end);
    if (r.beg < r.end) r.unit0 = locate(r.beg);
    return r;
  }
  // a run that begins with the first border inside its unit lists the join of its member's rows
  if (tid == 0 && run > 0 && r.unit0.first < r.beg) {
    const PaUnit& u = r.unit0;
    const long long before = cut(run - 1);
    const PaPart part(u, gang, r.member, 0, u.tiles);
    if (before <= u.first && part.rows > 0) {
      int m = run;
      while (m < G && cut(m) < u.first + u.tiles) ++m;     // runs run - 1 .. m - 1 begin before the unit's end
      PaJoin jn;
      jn.row0 = u.q0 + part.row0;
      jn.rows = part.rows;
      jn.h = u.h;
      jn.cta = (run - 1) * gang + r.member;
      jn.parts = m - (run - 1);
      jn.gang = gang;
      jn.slot = 2 * jn.cta + (before < u.first ? 1 : 0);
      jn.pad = 0;
      p.joins[blockIdx.x] = jn;
    }
  }
  return r;
}

// ------------------------------------------------------------------ main kernel

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Operand read transposed (MN-major), 128-byte swizzle: 64 elements of N an atom of 8 K rows, the next 64 `mn_bytes`
// further, the next 8 of K 1024 bytes further.
__device__ __forceinline__ uint64_t pa_desc_mn(uint32_t saddr, uint32_t mn_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(mn_bytes >> 4) << 16;
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

// Four products of depth 16, both operands in shared memory, issued by one elected lane of a converged warp; acc = 0:
// the first overwrites.
__device__ __forceinline__ void pa_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
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
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on `bar` when the products issued so far are complete (one elected lane of a converged warp).
__device__ __forceinline__ void pa_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

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
__global__ void __launch_bounds__(kPaThreads, 1) prompt_attention_kernel(const PaArgs p, const __grid_constant__ PaMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t full[kPaSlots], empty[kPaSlots], q_full[2], q_empty[2], s_full[2], p_ready[2], o_full[2], v_full[2][2], v_ok[2], drained;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, cta_status;
  // keys of the masked tiles (at most three a unit) whose values are not all finite, of four units; done: units whose
  // output each softmax warp has written
  __shared__ uint32_t bad[4][3][4], done[kPaSmWarps];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qsm = smem + kPaSlots * kPaSlotBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_v = &abort_flag;

  if (threadIdx.x == 0) {
    // (an arrival too many for a withheld stage)
    for (int i = 0; i < kPaSlots; ++i) {
      mbar_init(&full[i], 1 + (i == 0 && blockIdx.x == 0 ? p.withhold : 0));
      mbar_init(&empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_ready[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&v_full[x][0], 1);
      mbar_init(&v_full[x][1], 1);
      mbar_init(&v_ok[x], kPaCheckWarps);
    }
    mbar_init(&drained, 1);
    for (int i = 0; i < kPaSmWarps; ++i) done[i] = 0;
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kPaLoader && lane == 0) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.r);
    prefetch_tensormap(&maps.v);
  }
  if (warp == kPaMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  griddep_wait();                                      // the launch may overlap the kernel before; its results not
  const PaRun run = pa_plan(p, smem);
  const int gang = run.gang, member = run.member;
  if (threadIdx.x == 0) cta_status = run.status;
  // (the plan's use of shared memory ends before the TMA use of it)
  fence_proxy_async_smem();
  __syncthreads();
  auto fail_wait = [&]() {
    atomicOr(&cta_status, COLI_DEV_WAIT_TIMEOUT);
    atomicExch(&abort_flag, 1);
  };

  if (warp == kPaLoader) {
    // ---------------------------------------------------------------- loader
    bool ok = true;
    unsigned pos = 0;                                  // slots filled so far
    unsigned checked[2] = {0, 0};                      // slots of values that go through the check, of either half
    int un[2] = {0, 0};                                // units whose queries are on their way
    PaUnit u = run.unit0;
    for (long long at = run.beg; ok && at < run.end; pa_next(p, u, gang)) {
      const int t0 = (int)(at - u.first), t1 = (int)min(run.end - u.first, (long long)u.tiles);
      at = u.first + t1;
      const PaPart part(u, gang, member, t0, t1);
      if (part.all == 0) continue;
      const int masked = part.masked();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || part.n[x] == 0) continue;
        if (un[x] > 0) ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[x], (un[x] - 1) & 1, p.wait_ns));
        if (!ok) continue;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[x], (uint32_t)kPaQBytes);
          // rows past the unit's last are other rows' or, behind the tensor, zeros: computed, not written
          for (int i = 0; i < 3; ++i)
            tma_load_3d(qsm + x * kPaQBytes + i * (kPaTile * 128), &maps.q, i * 64, u.h, u.q0 + part.row0 + x * kPaTile, &q_full[x]);
        }
        __syncwarp();
        ++un[x];
      }
      for (int t = t0; ok && t < t0 + part.all; ++t) {
        if (__any_sync(0xffffffffu, *abort_v)) { ok = false; break; }
        const int key = u.k0 + t * kPaTile;
        const bool check = t >= masked;                // its values then count on v_full, which the check awaits
#pragma unroll 1
        for (int i = 0; i < 5; ++i, ++pos) {
          const unsigned s = pos % kPaSlots;
          if (pos >= kPaSlots) ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], (pos / kPaSlots - 1) & 1, p.wait_ns));
          if (!ok) break;
          if (lane == 0) {
            uint8_t* dst = smem + s * kPaSlotBytes;
            uint64_t* bar = &full[s];
            if (check && i >= 3) {
              mbar_arrive(bar);
              bar = &v_full[(i == 3 ? checked[0] : checked[1]) & 1][i - 3];
            }
            mbar_arrive_expect_tx(bar, (uint32_t)kPaSlotBytes);
            if (i < 2) {
              tma_load_3d(dst, &maps.k, i * 64, u.h, key, bar);
            } else if (i == 2) {
              tma_load_2d_nohint(dst, &maps.r, 0, key, bar);
            } else {                                   // 64 keys: two boxes of 64 values
              tma_load_3d(dst, &maps.v, 0, u.h, key + (i - 3) * 64, bar);
              tma_load_3d(dst + kPaSlotBytes / 2, &maps.v, 64, u.h, key + (i - 3) * 64, bar);
            }
          }
          __syncwarp();
          checked[0] += check && i == 3;
          checked[1] += check && i == 4;
        }
      }
    }
    if (!ok) fail_wait();
    // Copies in flight land before the CTA leaves, whichever role gave up.  A slot's phases before its last are
    // complete: it was filled again only after its use.
    if (lane == 0) {
      for (int x = 0; x < 2; ++x)
        if (un[x] > 0) mbar_wait(&q_full[x], (un[x] - 1) & 1, kWaitLimitNs);
      for (unsigned s = 0; s < kPaSlots; ++s)
        if (pos > s) mbar_wait(&full[s], ((pos - s - 1) / kPaSlots) & 1, s == 0 && p.withhold ? 1000000ull : kWaitLimitNs);
      for (int h = 0; h < 2; ++h)
        for (unsigned j = 0; j < 2; ++j)
          if (checked[h] > j) mbar_wait(&v_full[j][h], ((checked[h] - j - 1) / 2) & 1, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kPaMma) {
    // ---------------------------------------------------------------- product issuer (the warp stays converged)
    const uint32_t idesc = BF16 ? umma_idesc_bf16(128, 128) : umma_idesc_f16(128, 128);
    const uint32_t idesc_v = idesc | (1u << 16);       // B MN-major
    const uint64_t kd = umma_desc_sw128(smem_u32(smem)), qd = umma_desc_sw128(smem_u32(qsm));
    const uint64_t vd = pa_desc_mn(smem_u32(smem), kPaSlotBytes / 2);
    bool ok = true;
    unsigned pos = 0;                                  // slots consumed before this unit's tile
    unsigned checked = 0, un[2] = {0, 0}, it[2] = {0, 0};
    auto wait = [&](uint64_t* bar, unsigned phase) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar, phase & 1, p.wait_ns));
      return ok;
    };
    PaUnit u = run.unit0;
    for (long long at = run.beg; ok && at < run.end; pa_next(p, u, gang)) {
      const int t0 = (int)(at - u.first), t1 = (int)min(run.end - u.first, (long long)u.tiles);
      at = u.first + t1;
      const PaPart part(u, gang, member, t0, t1);
      if (part.all == 0) continue;
      const int masked = part.masked();
      // S of row tile x and key tile i of the part, whose slots begin at `from`
      auto scores = [&](int x, int i, unsigned from, bool wait_keys) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const unsigned s = (from + c) % kPaSlots;
          if (wait_keys) {
            if (!wait(&full[s], (from + c) / kPaSlots)) return;
            tc_fence_after();
          }
          pa_mma_ss(tmem + x * kPaTile, qd + (uint64_t)((x * kPaQBytes + c * (kPaTile * 128)) >> 4),
                    kd + (uint64_t)(s * (kPaSlotBytes >> 4)), idesc, c ? 1u : 0u);
        }
        pa_commit(&s_full[x]);
        if (i + 1 == part.n[x]) pa_commit(&q_empty[x]);
      };
      auto release = [&](unsigned from, int n) {
        for (int c = 0; c < n; ++c) pa_commit(&empty[(from + c) % kPaSlots]);
      };
      bool fresh = true;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || part.n[x] == 0) continue;
        if (!wait(&q_full[x], un[x])) continue;
        ++un[x];
        scores(x, 0, pos, fresh);
        fresh = false;
      }
      if (!ok) break;
      release(pos, 3);
      for (int i = 0; ok && i < part.all; ++i, pos += 5) {
        const unsigned vpos = pos + 3, next = pos + 5;
        // the values, or, where some row does not see some key, the values after their check.  (Every phase of a
        // barrier is awaited or, for the value slots of a checked tile, known to be over: a parity tells neighbours apart.)
        if (t0 + i >= masked) {
          wait(&v_ok[checked & 1], checked >> 1);
          ++checked;
        } else {
          wait(&full[vpos % kPaSlots], vpos / kPaSlots);
          wait(&full[(vpos + 1) % kPaSlots], (vpos + 1) / kPaSlots);
        }
        if (!ok) break;
        fresh = true;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || i >= part.n[x]) continue;
          if (!wait(&p_ready[x], it[x])) continue;
          ++it[x];
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c)
            pa_mma_ts(tmem + kPaOCol + x * kPaTile, tmem + x * kPaTile + c * 32,
                      vd + (uint64_t)(((vpos + c) % kPaSlots) * (kPaSlotBytes >> 4)), idesc_v, i || c ? 1u : 0u);
          if (i + 1 < part.n[x]) {
            scores(x, i + 1, next, fresh);
            fresh = false;
          } else {
            pa_commit(&o_full[x]);
          }
        }
        if (!ok) break;
        release(vpos, 2);
        if (i + 1 < part.all) release(next, 3);
      }
    }
    if (!ok && lane == 0) fail_wait();
    __syncwarp();
    // what was issued ends before tensor memory is freed, whichever role gave up
    pa_commit(&drained);
    mbar_wait(&drained, 0, kWaitLimitNs);
  } else if (warp >= kPaCheck) {
    // ---------------------------------------------------------------- check of the values of masked tiles
    // A row's weight for a key that it does not see is 0, and 0 times an infinity or a NaN is a NaN: such values
    // become 0 in shared memory before the product, and the rows that do see the key add them in the end.  Only the
    // tiles that cross the diagonal are looked at.
    const int half = warp - kPaCheck;                  // of the tile's keys
    volatile uint32_t* done_v = done;
    // the softmax warps have read what `bad` holds of four units before
    auto free_again = [&](unsigned uu) {
      if (uu < 4) return true;
      const unsigned long long from = globaltimer();
      while (__any_sync(0xffffffffu, (int)(done_v[lane & (kPaSmWarps - 1)] - (uu - 3)) < 0))
        if (__any_sync(0xffffffffu, globaltimer() - from > p.wait_ns)) return false;
      return true;
    };
    bool ok = true;
    unsigned pos = 0, checked = 0, uu = 0;
    PaUnit u = run.unit0;
    for (long long at = run.beg; ok && at < run.end; pa_next(p, u, gang)) {
      const int t0 = (int)(at - u.first), t1 = (int)min(run.end - u.first, (long long)u.tiles);
      at = u.first + t1;
      const PaPart part(u, gang, member, t0, t1);
      if (part.all == 0) continue;
      const int masked = part.masked();
      if (masked < t0 + part.all) ok = free_again(uu);
      for (int i = max(0, masked - t0); ok && i < part.all; ++i) {
        const unsigned v = pos + 5 * i + 3 + half, s = v % kPaSlots;
        ok = __all_sync(0xffffffffu, mbar_wait(&v_full[checked & 1][half], (checked >> 1) & 1, p.wait_ns));
        if (!ok) break;
        uint8_t* box = smem + s * kPaSlotBytes;
        uint32_t flags[2];
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          uint8_t* row = box + (k * 32 + lane) * 128;  // and the same row of the second box
          uint32_t top = 0;                            // the largest magnitude of either half of the words
#pragma unroll
          for (int c = 0; c < 16; ++c) {               // (the lanes' rows meet the banks evenly by the rotation)
            const uint4 w = *reinterpret_cast<const uint4*>(row + (c >> 3) * (kPaSlotBytes / 2) + (((c + lane) & 7) << 4));
            top = __vmaxu2(__vmaxu2(top, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
            top = __vmaxu2(__vmaxu2(top, w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
          }
          const bool wrong = pa_not_finite<BF16>(top) || pa_not_finite<BF16>(top >> 16);
          flags[k] = __ballot_sync(0xffffffffu, wrong);
          if (wrong) {
#pragma unroll 1
            for (int c = 0; c < 16; ++c) {
              uint4* w = reinterpret_cast<uint4*>(row + (c >> 3) * (kPaSlotBytes / 2) + ((c & 7) << 4));
              *w = make_uint4(pa_finite_part<BF16>(w->x), pa_finite_part<BF16>(w->y), pa_finite_part<BF16>(w->z),
                              pa_finite_part<BF16>(w->w));
            }
          }
        }
        if (lane == 0) {
          bad[uu & 3][t0 + i - masked][half * 2] = flags[0];
          bad[uu & 3][t0 + i - masked][half * 2 + 1] = flags[1];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ok[checked & 1]);
        ++checked;
      }
      pos += 5 * part.all;
      ++uu;
    }
    if (!ok && lane == 0) fail_wait();
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int x = warp >> 2, sp = warp & 3;            // row tile, TMEM sub-partition
    const uint32_t ts = tmem + ((uint32_t)(sp * 32) << 16) + (uint32_t)(x * kPaTile), to = ts + kPaOCol;
    const int in_unit = x * kPaTile + sp * 32 + lane;  // this thread's row of the CTA's 256
    unsigned it = 0, un = 0, uu = 0;
    bool ok = true;
    PaUnit u = run.unit0;
    for (long long at = run.beg; at < run.end; pa_next(p, u, gang)) {
      const int t0 = (int)(at - u.first), t1 = (int)min(run.end - u.first, (long long)u.tiles);
      const bool opening = at == run.beg, whole = t0 == 0 && t1 == u.tiles;
      at = u.first + t1;
      const PaPart part(u, gang, member, t0, t1);
      const int n = part.n[x];
      if (part.rows <= x * kPaTile) {
        uu += part.all > 0;
        if (lane == 0) *const_cast<volatile uint32_t*>(&done[warp]) = uu;
        continue;
      }
      const bool mine = in_unit < part.rows;           // rows past the last are not written
      const int row = part.row0 + in_unit;             // of the request
      const int lim = part.shift + min(row, u.T - 1);  // the last key it sees
      const int lim0 = part.shift + part.row0 + x * kPaTile + sp * 32;      // of the warp's first row
      float m = 0.f, l = 0.f;                          // reference, sum of the weights
      bool has = false;                                // the row has seen a key
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++it) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[x], it & 1, p.wait_ns));
        if (!ok) break;
        tc_fence_after();
        const int key0 = (t0 + i) * kPaTile;
        bool slow = key0 + kPaTile - 1 > lim0 || __any_sync(0xffffffffu, !has);
        float grow = kPaGrow;                          // by how much a score exceeds a reference that is raised
        if (!slow) {
          // every key is seen: weights against the reference as it is; the sum tells whether it still serves
          uint32_t w[kPaTile / 2];
          const float2 by = make_float2(p.scale_log2, p.scale_log2), off = make_float2(-m, -m);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < kPaTile; c += 32) {
            uint32_t r[32];
            tmem_ld32_issue(ts + c, r);
            tmem_ld_done<32>(r);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 d = ffma2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), by, off);
              const float2 e = make_float2(pa_exp2(d.x), pa_exp2(d.y));
              sum = fadd2(sum, e);
              w[(c + j) / 2] = pa_pack<BF16>(e.x, e.y);
            }
          }
          const float add = sum.x + sum.y;
          slow = __any_sync(0xffffffffu, !(add <= kPaSumLimit));
          grow = 0.f;
          if (!slow) {
            l += add;
#pragma unroll
            for (int c = 0; c < kPaTile / 2; c += 32) tmem_st32(ts + c, w + c);
          }
        }
        if (slow) {
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kPaTile; c += 32) {
            uint32_t r[32];
            tmem_ld32_issue(ts + c, r);
            tmem_ld_done<32>(r);
#pragma unroll
            for (int j = 0; j < 32; ++j) {             // (masks after the scale, which may be 0 or negative)
              const float d = fmaf(__uint_as_float(r[j]), p.scale_log2, -m);
              top = fmaxf(top, key0 + c + j > lim ? -INFINITY : d);
            }
          }
          const float g = ceilf(top) - pa_top(BF16);
          const bool raise = g > grow || (!has && g > -INFINITY);
          // what that leaves of the sums so far: a first reference may lie far below 0, but they are 0 (or NaN) then
          const float keep = raise && has ? pa_exp2(-g) : 1.f;
          // (the distance to the old reference is taken first: a product with the scale may lie far beyond their difference)
          const float by = raise ? g : 0.f;
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
          float s0 = 0.f, s1 = 0.f;
#pragma unroll 1
          for (int c = 0; c < kPaTile; c += 32) {      // (a chunk's weights take columns that are read already)
            uint32_t r[32], w[16];
            tmem_ld32_issue(ts + c, r);
            tmem_ld_done<32>(r);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float d[2];
#pragma unroll
              for (int k = 0; k < 2; ++k)
                d[k] = key0 + c + j + k > lim ? 0.f : pa_exp2(fmaf(__uint_as_float(r[j + k]), p.scale_log2, -m) - by);
              s0 += d[0];
              s1 += d[1];
              w[j / 2] = pa_pack<BF16>(d[0], d[1]);
            }
            tmem_st16(ts + c / 2, w);
          }
          m += by;
          has |= raise;
          l += s0 + s1;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[x]);
      }
      // -------------------------------------------------------------- the unit's rows
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[x], un & 1, p.wait_ns));
        ++un;
      }
      if (!ok) break;
      tc_fence_after();
      const int slot = 2 * (int)blockIdx.x + (opening ? 0 : 1);
      const int masked = part.masked();
      // values that were taken out of masked tiles (keys of this row tile only: the others' products come first)
      uint32_t any_bad = 0;
      for (int t = max(masked, t0); t < t0 + n; ++t)
#pragma unroll
        for (int w = 0; w < 4; ++w) any_bad |= bad[uu & 3][t - masked][w];
      float by = 1.f;
      if (whole) {
        by = l == 0.f ? 0.f : 1.0f / l;
        if (mine && p.lse) p.lse[(size_t)(u.q0 + row) * p.H + u.h] = l == 0.f ? -INFINITY : (log2f(l) + m) * 0.693147180559945309f;
      } else if (mine) {
        p.part_ml[(size_t)slot * kPaRows + in_unit] = make_float2(has || l != 0.f ? m : -INFINITY, l);
      }
      uint16_t* out = p.out + ((size_t)(u.q0 + row) * p.H + u.h) * kPaV;
      float* po = p.part + (size_t)slot * kPaPart;
#pragma unroll 1
      for (int c = 0; c < kPaV; c += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32_issue(to + c, o);
          tmem_ld_done<32>(o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        if (any_bad) {
#pragma unroll 1
          for (int e = (max(masked, t0) - masked) * 128; e < (t0 + n - masked) * 128; ++e) {
            if (!((bad[uu & 3][e >> 7][(e >> 5) & 3] >> (e & 31)) & 1u)) continue;
            const int key = masked * kPaTile + e;
            if (!mine || key > lim) continue;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(p.v + (u.k0 + (long long)key) * p.v_tok + u.h * p.v_head) + c;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t b = v[j];
              const float val = BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
              if (pa_not_finite<BF16>(b)) o[j] = __float_as_uint(__uint_as_float(o[j]) + val);
            }
          }
        }
        if (!mine) continue;
        if (whole) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pa_pack<BF16>(__uint_as_float(o[j + 2 * k]) * by, __uint_as_float(o[j + 2 * k + 1]) * by);
            *reinterpret_cast<uint4*>(out + c + j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (n > 0) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint4*>(po + pa_part(in_unit, c + j)) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();                                    // (every lane has read `bad`)
      uu += part.all > 0;
      if (lane == 0) *const_cast<volatile uint32_t*>(&done[warp]) = uu;
    }
    if (!ok && lane == 0) fail_wait();
  }
  griddep_launch_dependents();                         // (earlier, the join's CTAs would take slots from the next call's)
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.cta_status[blockIdx.x] = cta_status;
  if (warp == kPaMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// ------------------------------------------------------------------ join
// Adds up the parts of every cut unit, in order.  A task is 32 rows of a unit (a row a lane, 16 values a warp).
constexpr float kPaLowest = -3.402823466e38f;      // below every reference; a part whose row saw no key has -infinity
constexpr int kPaJoinThreads = 256, kPaJoinCtas = 304;

template <bool BF16>
__global__ void __launch_bounds__(kPaJoinThreads) prompt_attention_join_kernel(const PaArgs p, int ctas) {
  __shared__ int starts[kPaJoinThreads], warp_tot[32], total;        // first task of each CTA's join
  static_assert(kPaMaxCtas <= kPaJoinThreads, "a thread each");
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool listed = tid < ctas && p.joins[tid].parts > 0;
  const int bits = blockIdx.x == 0 && tid < ctas ? p.cta_status[tid] : 0;
  starts[tid] = block_exclusive_scan(listed ? (p.joins[tid].rows + 31) / 32 : 0, warp_tot, &total);
  if (blockIdx.x == 0) {
    const int timed = __syncthreads_or(bits & COLI_DEV_WAIT_TIMEOUT), order = __syncthreads_or(bits & COLI_DEV_KV_TOKENS);
    if (tid == 0) *p.status = (timed ? COLI_DEV_WAIT_TIMEOUT : 0) | (order ? COLI_DEV_KV_TOKENS : 0);
  }
  __syncthreads();
  const int n_tasks = total;
  for (int task = blockIdx.x; task < n_tasks; task += gridDim.x) {
    int j = 0, h = kPaJoinThreads;                     // last CTA whose join starts at or before the task
    while (h - j > 1) {
      const int mid = (j + h) >> 1;
      if (starts[mid] <= task) j = mid;
      else h = mid;
    }
    const PaJoin jn = p.joins[j];
    const int r = (task - starts[j]) * 32 + lane, c0 = warp * 16;
    if (r >= jn.rows) continue;
    auto slot = [&](int i) { return (size_t)(i ? 2 * (jn.cta + i * jn.gang) : jn.slot); };
    float m = kPaLowest, l = 0.f;
#pragma unroll 4
    for (int i = 0; i < jn.parts; ++i) m = fmaxf(m, p.part_ml[slot(i) * kPaRows + r].x);
    float4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < jn.parts; ++i) {
      const float2 ml = p.part_ml[slot(i) * kPaRows + r];
      const float* src = p.part + slot(i) * kPaPart;
      const float w = pa_exp2(ml.x - m);
      l += w * ml.y;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 o = *reinterpret_cast<const float4*>(src + pa_part(r, c0 + 4 * c));
        if (w != 0.f) {                                // (a part without keys has written no values)
          acc[c].x = fmaf(w, o.x, acc[c].x);
          acc[c].y = fmaf(w, o.y, acc[c].y);
          acc[c].z = fmaf(w, o.z, acc[c].z);
          acc[c].w = fmaf(w, o.w, acc[c].w);
        }
      }
    }
    const float by = l == 0.f ? 0.f : 1.0f / l;
    const size_t row = (size_t)(jn.row0 + r) * p.H + jn.h;
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
  w.joins = take((size_t)kPaMaxCtas * sizeof(PaJoin));
  w.part = take((size_t)2 * kPaMaxCtas * kPaPart * sizeof(float));
  w.part_ml = take((size_t)2 * kPaMaxCtas * kPaRows * sizeof(float2));
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
  const cuuint32_t bdim[2] = {64, (cuuint32_t)kPaTile};
  const cuuint32_t es[2] = {1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                const_cast<void*>(base), gdim, gstr, bdim, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <bool BF16>
static cudaError_t pa_launch(const PaArgs& a, const PaMaps& maps, int ctas, int dev, cudaStream_t st) {
  static_assert((size_t)(kPaMaxB + 1) * 16 + 1024 <= kPaSmem, "the plan's arrays");
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
  return launch_pdl(prompt_attention_join_kernel<BF16>, dim3(kPaJoinCtas), dim3(kPaJoinThreads), 0, st, a, ctas);
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
               keys ? n_keys : 1, k_token_stride, kPaTile);
  if (r == CUDA_SUCCESS) r = pa_map_rope(encode, &maps.r, bf16, keys ? k_rope : q, keys ? n_keys : 1, rope_stride);
  if (r == CUDA_SUCCESS)
    r = pa_map(encode, &maps.v, bf16, keys ? v : q, kPaV, H, keys ? v_head_stride : q_head_stride, keys ? n_keys : 1,
               v_token_stride, kPaTile / 2);
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
  const int ctas = sms < kPaMaxCtas ? sms : kPaMaxCtas;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ce = bf16 ? pa_launch<true>(a, maps, ctas, dev, st) : pa_launch<false>(a, maps, ctas, dev, st);
  return ce == cudaSuccess ? COLI_OK : cuda_fail(ce, "prompt_attention: launch");
}

}  // extern "C"
