// sv_attend.cuh - attention over the 4-bit cache: parameters, the split of a
// call's work over CTAs, masks and scores, shared by the kernels; internal.
//
// A unit of work is a tile of query rows (of the step's tokens and the
// heads of one key/value head) against the slots that its request sees.  The slots come in
// chunks; all chunks of all units, laid end to end, are cut into equal shares,
// one a CTA, so that ragged lengths and few long requests keep every SM busy alike.
// A CTA walks its share's pieces (runs of chunks of one unit).  A piece that
// is not a whole unit leaves its rows' running max, sum and weighted values in
// the workspace, and a second kernel joins a unit's pieces in order.  Which
// CTA does what depends on the lengths alone, so results do not vary from run to run.
#pragma once

#include "sv_cache.cuh"
#include "sv_launch.h"

namespace sv {

// Weights are 2^(score - reference), the largest of a row 2^15 (few rows) or 2^7 to 2^15 (many): fp16's
// least step of 2^-24 is 2^-39 or 2^-31 of it.
constexpr float kFewShift = 15.f;
// Scores are taken times their factor and less the reference in one step, which keeps places of the
// product that a max in 32 bits has lost: 2^-11 at a reference of 2^14, 1 (a weight of 2^16, none of
// fp16's) at 2^24, and all of the weight at 2^28. From kFar on the product is rounded first, so that
// exponents are differences of 32-bit scores.
constexpr float kFar = 16384.f;
constexpr float kLeast = -3.402823466e38f;  // in place of a max of -inf
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && m != -INFINITY; }
__device__ __forceinline__ float far_exponent(float s, float f, float m, float shift) {
  return __fadd_rn(__fsub_rn(__fmul_rn(s, f), fmaxf(m, kLeast)), shift);
}
// The log-sum-exp of weights 2^(x - m + shift), x in units of log2, that add up to l.
__device__ __forceinline__ float log_sum(float m, float l, float shift) {
  return l == 0.f ? -INFINITY : (m + (log2f(l) - shift)) * 0.6931471805599453f;
}

struct AttendParams {
  CacheView cache;
  const void* q;             // [B, N, Hq, D] at element strides
  long long qb, qn, qh;
  void* out;                 // [B, N, Hq, D]
  float* out_lse;            // [B, N, Hq] or null
  int* out_status;           // [B] or null
  const int* lens;           // [B] slots in use, the step's own among them
  const int* q_lens;         // [B] tokens of the step, or null (N)
  const int* parent;         // request b's tree at parent + b * parent_stride, or null (a chain)
  int parent_stride;
  const float* slopes;       // [Hq] or null
  int B, N, Hq, group;       // group = Hq / Hkv
  int window;                // 0: none
  float scale, softcap;      // softcap 0: none
  // the split
  int rows;                  // query rows of a unit
  int chunk;                 // slots of a chunk
  int least;                 // chunks that are worth a CTA
  int* desc;                 // [G][4] the split unit that begins in each CTA's share: b, head, row tile, pieces
  int* late;                 // [G] whether a wait in the CTA ran out, or null
  float shift;               // exponent of the weight of a score that equals a partial row's max
  unsigned long long wait_ns;  // limit of the waits
  float* part;               // [2 G][rows][D + 4] unfinished rows: values, max or reference, sum
  float* fold;               // [G] second sums of the fp32 calls
};

// What a request's arguments come to.
struct Request {
  int len, nq, base;  // slots, tokens of the step, slot of the first of them
  int lo;             // first slot that any of them sees
  int chunks, tiles;  // of each of its units; units of a head
  bool ok;
};

__device__ __forceinline__ Request request_of(const AttendParams& p, int b) {
  Request r;
  r.len = p.lens[b];
  r.nq = p.q_lens ? p.q_lens[b] : p.N;
  r.ok = r.nq >= 0 && r.nq <= p.N && r.len >= r.nq &&
         r.len <= ((long long)p.cache.M << p.cache.shift);
  if (!r.ok) {  // (its rows come out as rows that see nothing)
    r.len = 0;
    r.nq = p.N;
  }
  r.base = r.len - r.nq;
  r.lo = 0;
  if (!r.ok) {
    r.base = 0;
  } else if (p.window > 0) {
    r.lo = max(0, r.base - (p.window - 1));
  }
  r.tiles = (r.nq * p.group + p.rows - 1) / p.rows;
  r.chunks = r.tiles == 0 ? 0 : max(1, (r.len + p.chunk - 1) / p.chunk - r.lo / p.chunk);
  return r;
}

__device__ __forceinline__ long long work_of(const AttendParams& p, int b) {
  const Request r = request_of(p, b);
  return (long long)r.chunks * r.tiles * p.cache.Hkv;
}

// The CTA's share [begin, end) of the call's chunks, and the request and offset in
// it where the share begins.  Every thread of the block (T of them) takes part.
struct Share {
  long long begin, end, total;
  int b;          // request of `begin`
  long long at;   // `begin` counted from that request's first chunk
  int G;          // CTAs with a share
};

template <int T>
__device__ __forceinline__ long long block_scan(long long x, long long* smem, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) smem[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    if (w < warp) before += smem[w];
    all += smem[w];
  }
  *total = all;
  return x + before;
}

// smem: T / 32 + 2 long longs.
template <int T>
__device__ __forceinline__ Share find_share(const AttendParams& p, int cta, int ctas,
                                            long long* smem) {
  const int t = threadIdx.x;
  const long long first = t < p.B ? work_of(p, t) : 0;
  long long total, part;
  const long long first_scan = block_scan<T>(first, smem, &total), first_total = total;
  for (int b0 = T; b0 < p.B; b0 += T) {
    block_scan<T>(b0 + t < p.B ? work_of(p, b0 + t) : 0, smem, &part);
    total += part;
  }
  // `least` chunks a CTA, but a CTA for every unit: a CTA walks its units one after the other
  long long want = (total + p.least - 1) / p.least;
  if (want < ctas) {
    long long units = 0;
    for (int b = 0; b < p.B; b += T) {
      long long some = 0;
      if (b + t < p.B) {
        const Request r = request_of(p, b + t);
        some = (long long)r.tiles * p.cache.Hkv;
      }
      block_scan<T>(some, smem, &part);
      units += part;
    }
    if (units > want) want = units;
  }
  Share s;
  s.total = total;
  s.G = (int)(want < ctas ? want : ctas);
  s.begin = s.end = s.at = 0;
  s.b = 0;
  if (cta < s.G) {
    s.begin = total * cta / s.G;
    s.end = total * (cta + 1) / s.G;
  }
  long long* found = smem + T / 32;
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += T) {
    const long long work = b0 == 0 ? first : b0 + t < p.B ? work_of(p, b0 + t) : 0;
    part = first_total;
    const long long scan = b0 == 0 ? first_scan : block_scan<T>(work, smem, &part);
    const long long from = before + scan - work;
    if (from <= s.begin && s.begin < from + work) {
      found[0] = b0 + t;
      found[1] = s.begin - from;
    }
    before += part;
  }
  __syncthreads();
  if (s.begin < s.end) {
    s.b = (int)found[0];
    s.at = found[1];
  }
  __syncthreads();
  return s;
}

// A walk over the chunks of a share.
struct Walk {
  Request r;
  int b, h, tile, c;  // the chunk's request, head, row tile, and place in the unit
  long long left;     // chunks from here on
  Walk() = default;
  __device__ __forceinline__ Walk(const AttendParams& p, const Share& s)
      : r(request_of(p, s.b)), b(s.b), left(s.end - s.begin) {
    const int unit = (int)(s.at / r.chunks);
    c = (int)(s.at - (long long)unit * r.chunks);
    h = unit / r.tiles;
    tile = unit - h * r.tiles;
  }
  // n chunks on, which are of one unit
  __device__ __forceinline__ void skip(const AttendParams& p, int n) {
    left -= n;
    c += n;
    if (c == r.chunks) next_unit(p);
  }
  __device__ __forceinline__ void next_unit(const AttendParams& p) {
    c = 0;
    if (++tile < r.tiles) return;
    tile = 0;
    if (++h < p.cache.Hkv) return;
    h = 0;
    while (left > 0) {
      r = request_of(p, ++b);
      if (r.tiles > 0) break;
    }
  }
};

// How many CTAs' shares meet the unit [u0, u1) of whose chunks CTA `cta` holds the first.
__device__ __forceinline__ int pieces_of(const Share& s, int cta, long long u1) {
  int n = 1;
  while (s.total * (cta + n) / s.G < u1) ++n;
  return n;
}

// A request's tree in shared memory: which nodes each node sees (bits), and its depth.  The
// parents and whether they are no tree lie elsewhere, where they are needed no longer than it
// takes to build.
struct TreeView {
  int *mem, *scratch;  // [N] depths, [N][words] bits; [N + 1]
  int N, words;
  __device__ __forceinline__ TreeView(void* at, void* build, int n)
      : mem(static_cast<int*>(at)), scratch(static_cast<int*>(build)), N(n), words((n + 31) / 32) {}
  __device__ __forceinline__ int& depth(int n) const { return mem[n]; }
  __device__ __forceinline__ int& parent(int n) const { return scratch[n + 1]; }
  __device__ __forceinline__ int& bad() const { return scratch[0]; }
  __device__ __forceinline__ int& bits(int n, int w) const { return mem[N + n * words + w]; }
  __device__ __forceinline__ bool sees(int n, int other) const {
    return bits(n, other >> 5) >> (other & 31) & 1;
  }
};
inline size_t tree_bytes(int N) { return (size_t)N * (1 + (N + 31) / 32) * sizeof(int); }

// Builds it with the block's T threads; false when the parents are no tree.
template <int T>
__device__ __forceinline__ bool build_tree(const AttendParams& p, int b, int nq,
                                           const TreeView& tree) {
  const int t = threadIdx.x;
  __syncthreads();
  if (t == 0) tree.bad() = 0;
  __syncthreads();
  const int* parent = p.parent + (long long)b * p.parent_stride;
  for (int n = t; n < nq; n += T) {
    const int up = n ? parent[n - 1] : -1;
    tree.parent(n) = up;
    if (n && (up < 0 || up >= n)) tree.bad() = 1;
  }
  __syncthreads();
  const bool bad = tree.bad() != 0;
  if (bad) {
    __syncthreads();
    return false;
  }
  for (int n = t; n < nq; n += T) {
    for (int w = 0; w < tree.words; ++w) tree.bits(n, w) = 0;
    int d = -1;
    for (int at = n; at >= 0; at = tree.parent(at), ++d) tree.bits(n, at >> 5) |= 1 << (at & 31);
    tree.depth(n) = d;
  }
  __syncthreads();
  return true;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
  return d;
}

// A pair of scales (64 s in fp16) and -9 / 8 of them.
struct Scale2 {
  uint32_t s, off;
  __device__ __forceinline__ Scale2() {}
  // The two bytes of `word` that the low bits of the selector name.
  __device__ __forceinline__ Scale2(uint32_t word, uint32_t sel) {
    set(__byte_perm(word, 0, sel) * 128u + 0x04000400u);
  }
  __device__ __forceinline__ void set(uint32_t pair) {
    s = pair;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(off) : "r"(pair), "r"(0xbc80bc80u));
  }
};
constexpr uint32_t kPair01 = 0x4140, kPair23 = 0x4342;

// The 8 values of a word, pairs (2 i, 2 i + 1) in x[i].  A code in the low four bits of an fp16
// number of exponent 2^4 is 16 + c / 64, one four bits up in one of 2^0 it is 1 + c / 64: two of
// four pairs need no shift, and one shift serves the other two.  (16 + 8 / 64) 64 s would
// not be exact, so those pairs take a subtraction and a product.
__device__ __forceinline__ void decode_word(uint32_t w, const Scale2& sc, uint32_t (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t y = i == 0 ? w : w >> 8;
    const uint32_t low = and_or(y, 0x000f000fu, 0x4c004c00u);
    const uint32_t high = and_or(y, 0x00f000f0u, 0x3c003c00u);
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(low), "r"(0xcc08cc08u));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x[2 * i]) : "r"(d), "r"(sc.s));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(x[2 * i + 1]) : "r"(high), "r"(sc.s), "r"(sc.off));
  }
}

// tanh by one exponential; off by 2^-22 of 1, whatever its size.
__device__ __forceinline__ float tanh_fast(float x) {
  return 1.f - __fdividef(2.f, ex2(x * (2.f * kLog2e)) + 1.f);
}

// cap * tanh(x) of scores.  The fast form is off by 2^-22 cap: 2^-13 of a score's unit at most where it is
// taken.  One branch for a chunk's scores: a branch each took 93 us instead of 91 for 5 tokens of 16
// requests (up to 8192 slots, 8 heads of 256, two query heads each).
constexpr float kFastCap = 512.f;
template <bool EXACT, class F>
__device__ __forceinline__ void cap_all(float cap, F each) {
  if (EXACT || cap > kFastCap)
    each([=](float x) { return cap * tanhf(x); });
  else
    each([=](float x) { return cap * tanh_fast(x); });
}
// What takes a sum of a row's products, of q scaled down by `down`, to a capped score's tanh, or without a
// cap to units of log2. (A cap may be subnormal; scores of 0 stay 0. The scale meets `down` first: times
// log2 e by itself it can be infinity.)
__device__ __forceinline__ float score_factor(const AttendParams& p, float down) {
  return p.softcap > 0.f ? down * fminf(fabsf(p.scale) / p.softcap, 3e38f)
                         : down * fabsf(p.scale) * kLog2e;
}

// Joins the pieces of split units (launched behind either kernel).
cudaError_t launch_join(const AttendParams& p, int D, int dtype, int ctas, int units,
                        cudaStream_t stream);

// The kernel for tiles of few rows and the one for many (tensor memory); they fill in the split.
struct AttendPlan {
  int rows, chunk, least, ctas;
  int fold;  // bytes of a CTA's second sums
  float shift;
};
cudaError_t plan_few(int D, int dtype, int rows, AttendPlan* plan);
cudaError_t launch_few(const AttendParams& p, int D, int dtype, const AttendPlan& plan,
                       cudaStream_t stream);
cudaError_t plan_many(int rows, AttendPlan* plan);
cudaError_t launch_many(const AttendParams& p, int D, const AttendPlan& plan, cudaStream_t stream);
// launch_many's kernel of 128 rows a tile.
cudaError_t launch_rows(const AttendParams& p, int D, const AttendPlan& plan, cudaStream_t stream);

}  // namespace sv
