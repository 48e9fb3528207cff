// sv_attend.cu - attention of a step's tokens over the 4-bit cache
// (spec_cache_attention): the kernel for few query rows, the join of split
// units, and the entry point.
//
// Few rows (a token or a few drafts of a group of heads): bound by HBM, if the
// decoding of the codes keeps up.  So nothing decoded passes through shared memory: a
// warp's lanes take the cache's words, copied ahead asynchronously, into the registers of the tensor
// instruction's fragments (m16n8k16) and decode them there, 11 instructions a word of 8.
//   S^T = K Q^T   A = 16 slots x 16 dimensions of keys in fp16, B = 8 query rows.
//                 The order of the dimensions is free as long as Q's agrees: the
//                 four lanes of a slot each take a quarter of its row, which is
//                 one 16-byte load and one scale a slot at D = 128.
//   O^T += V^T P^T  A = 16 dimensions x 16 slots of values in fp16, B = the weights.
//                 A lane takes 4 neighbouring slots (two pairs of the fragment) of D / 8
//                 dimensions; the halves of two slots' words are merged
//                 (prmt) so that a masked shift leaves the same dimension of both.
// Eight rows a tile leave no half of the tensor instruction empty, as rows on
// its 16-side would.  The weights move from the result's layout to the operand's by
// movmatrix.  Scores are sums of exact products in 32 bits; weights are rounded to fp16
// (2^-11 of each, against 2^-8 of the bf16 result; fp32 calls add a second
// fp16 number for the rest, of the weights and of Q).
//
// Each of the four warps of a CTA walks its own chunks of 32 slots with its own
// running max and sum; the warps join at the end of a piece.
// Measured: a token of 256 requests of up to 4096 slots (4 heads a group, 8 groups of 128) 216 us, 4.0 TB/s;
// issue slots 60 % used, the tensor pipe busy in 76 % of the cycles, 16 warps an SM.  The first form, without
// shared memory's ring of 3 stages a warp, took 317.
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/spec_verify.h"
#include "sv_attend.cuh"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

constexpr int kFewThreads = 128;
constexpr int kFewWarps = kFewThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NW words of shared memory, aligned to them.
template <int NW>
__device__ __forceinline__ void load_words(const char* p, uint32_t (&w)[NW]) {
  if constexpr (NW == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (NW == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < NW / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

// 16 slots of a head in shared memory: key codes, value codes, their scales.  A lane takes (g =
// lane / 4, t = lane % 4) a quarter of the keys of slots 4 (g / 2) + g % 2 and two on, and an eighth of
// the values of slots 4 t .. 4 t + 3.  Every four rows a gap of 32 bytes (64 for keys of
// 32-byte rows) keeps those loads off each other's banks.
template <int D>
struct Tile {
  static constexpr int kRow = D / 2, kKeyGap = D == 64 ? 64 : 0, kValueGap = 32;
  static constexpr int kValues = 16 * kRow + 4 * kKeyGap;            // offset of the values
  static constexpr int kScales = kValues + 16 * kRow + 4 * kValueGap;  // and of the scales
  static constexpr int kScaleBytes = D / 2;                          // of the keys (16 D / 32)
  static constexpr int kBytes = kScales + 2 * kScaleBytes;
  static constexpr int KW = D / 32, VW = D / 64;  // words a lane takes of a slot
  static __device__ __forceinline__ constexpr int key(int n) { return n * kRow + (n >> 2) * kKeyGap; }
  static __device__ __forceinline__ constexpr int value_step(int n) {
    return n * kRow + (n >> 2) * kValueGap;
  }
  static __device__ __forceinline__ int value(int n) { return kValues + value_step(n); }
};

__device__ __forceinline__ void copy16(uint32_t dst, const char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Queues the copies of KT tiles of page `id` from `token` on (`head`: the head's keys in page 0); a
// page that is none, or past the last slot in use (-1), gives keys of NaN and values that are finite.
template <int D, int KT>
__device__ __forceinline__ void queue_tiles(const CacheView& c, const char* head, int block,
                                            int id, int token, char* stage) {
  const int lane = lane_id();
  constexpr int kPer = D / 32;       // 16-byte units of a row, and of a tile's scales
  constexpr int kUnits = KT * kPer;  // of the tiles' scales
  const int unit = lane % kUnits;
  char* scales = stage + unit / kPer * Tile<D>::kBytes + Tile<D>::kScales + unit % kPer * 16 +
                 (lane < kUnits ? 0 : Tile<D>::kScaleBytes);
  if ((unsigned)id >= (unsigned)c.pages) {
    const uint32_t x = lane < kUnits ? kNanScale * 0x01010101u : 0u;
    if (lane < 2 * kUnits) *reinterpret_cast<uint4*>(scales) = make_uint4(x, x, x, x);
    return;
  }
  const char* base = head + (unsigned long long)(unsigned)id * c.page_stride;
  const char* k = base + (token * (D / 2) + lane * 16);
  const char* v = k + block;
  // (a lane's rows are a multiple of 4 apart: constants from its first)
  constexpr int kApart = 32 / kPer, kRows = D / 64;
  static_assert(kApart % 4 == 0, "");
  const int row = lane / kPer, x = lane % kPer * 16;
  const uint32_t key = smem_u32(stage) + Tile<D>::key(row) + x;
  const uint32_t value = smem_u32(stage) + Tile<D>::value(row) + x;
#pragma unroll
  for (int i = 0; i < KT * kRows; ++i) {
    const int at = i / kRows * Tile<D>::kBytes, n = i % kRows * kApart;
    copy16(key + (at + Tile<D>::key(n)), k + i * 512);
    copy16(value + (at + Tile<D>::value_step(n)), v + i * 512);
  }
  if (lane < 2 * kUnits)
    copy16(smem_u32(scales), base + (((D / 2) << c.shift) + token * (D / kGroup) + unit * 16 +
                                     (lane < kUnits ? 0 : block)));
}

template <int D, int NT, int NS>
struct Query {  // B fragments of NT tiles of 8 rows, NS fp16 parts each
  uint32_t b[NT][NS][D / 16][2];
};

// S^T of 16 slots: s[n] = {slot, row 2 t}, {slot, row 2 t + 1}, and the same two slots on.
template <int D, int NT, int NS>
__device__ __forceinline__ void scores(const char* tile, const Query<D, NT, NS>& q,
                                       float (&s)[NT][4]) {
  const int lane = lane_id(), g = lane / 4, t = lane % 4;
  const uint32_t sel = (g & 1) * 0x0101u;
#pragma unroll
  for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
  using Q = Tile<D>;
  uint32_t k[2][Q::KW];
  const char* row = tile + Q::key(4 * (g >> 1) + (g & 1)) + t * (D / 8);
  load_words<Q::KW>(row, k[0]);
  load_words<Q::KW>(row + 2 * Q::kRow, k[1]);
  const char* scales = tile + Q::kScales + t * (D / 4) / kGroup * 16 + 4 * (g >> 1);
  Scale2 s0, s1;
#pragma unroll
  for (int w = 0; w < Q::KW; ++w) {
    if (w % 4 == 0) {
      const uint32_t four = *reinterpret_cast<const uint32_t*>(scales + w / 4 * 16);
      s0 = Scale2(four, 0x4040 + sel);
      s1 = Scale2(four, 0x4242 + sel);
    }
    uint32_t x0[4], x1[4];
    decode_word(k[0][w], s0, x0);
    decode_word(k[1][w], s1, x1);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t a[4] = {x0[2 * half], x1[2 * half], x0[2 * half + 1], x1[2 * half + 1]};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < NS; ++i)
          mma_f16(s[n], a, q.b[n][i][2 * w + half][0], q.b[n][i][2 * w + half][1]);
    }
  }
}

// O^T += V^T P^T of 16 slots; P: operand fragments, NP fp16 parts.  Slots whose bit of `dead` (of
// the lane's four) is set count as zeros whatever they hold.
template <int D, int NT, int NP>
__device__ __forceinline__ void values(const char* tile, const uint32_t (&P)[NT][NP][2],
                                       uint32_t dead, float (&o)[NT][D / 16][4]) {
  const int lane = lane_id(), g = lane / 4, t = lane % 4;
  using Q = Tile<D>;
  const uint32_t four = *reinterpret_cast<const uint32_t*>(
      tile + Q::kScales + Q::kScaleBytes + g * (D / 8) / kGroup * 16 + 4 * t);
  Scale2 sa(four, kPair01), sb(four, kPair23);
  if (dead) {
    sa.set(sa.s & ~((dead & 1) * 0xffffu | (dead >> 1 & 1) * 0xffff0000u));
    sb.set(sb.s & ~((dead >> 2 & 1) * 0xffffu | (dead >> 3 & 1) * 0xffff0000u));
  }
  uint32_t v[4][Q::VW];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    load_words<Q::VW>(tile + Q::value(4 * t) + i * Q::kRow + g * (D / 16), v[i]);
#pragma unroll
  for (int w = 0; w < Q::VW; ++w) {
    uint32_t x[4][4];
    decode_word(__byte_perm(v[0][w], v[1][w], 0x5410), sa, x[0]);
    decode_word(__byte_perm(v[0][w], v[1][w], 0x7632), sa, x[1]);
    decode_word(__byte_perm(v[2][w], v[3][w], 0x5410), sb, x[2]);
    decode_word(__byte_perm(v[2][w], v[3][w], 0x7632), sb, x[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a[4] = {x[0][i], x[1][i], x[2][i], x[3][i]};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < NP; ++k) mma_f16(o[n][4 * w + i], a, P[n][k][0], P[n][k][1]);
    }
  }
}

// Dimension of o[n][i][0] (and of [1]; [2] and [3] hold the next one).
template <int D>
__device__ __forceinline__ int dim_of(int i) {
  return (lane_id() / 4) * (D / 8) + 8 * (i / 4) + 2 * (i % 4);
}

template <typename T>
__device__ __forceinline__ float2 load2(const T* p);
template <>
__device__ __forceinline__ float2 load2(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}
template <>
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(bf16_lo(w), bf16_hi(w));
}

// The rows' operand fragments in fp16.  A row is scaled by a power of two that takes its
// largest value to [2^14, 2^15): bf16 values are then exact down to 2^-28 of it, and
// fp32 values, in two parts, good to 2^-24 of themselves; what is lost below is 2^-39 of the
// largest.  unscale[n][e] (of rows 2 t and 2 t + 1) takes the scores back.
template <int D, int NT, int NS, typename T>
__device__ __forceinline__ void load_query(const AttendParams& p, int b, int h, int row0, int rows,
                                           Query<D, NT, NS>& q, float (&unscale)[NT][2]) {
  const int lane = lane_id(), g = lane / 4, t = lane % 4;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = row0 + 8 * n + g;
    const bool ok = row < rows;
    const int i = row / p.group, j = row - i * p.group;
    const T* src = static_cast<const T*>(p.q) + b * p.qb + i * p.qn +
                   (long long)(h * p.group + j) * p.qh + t * (D / 4);
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < D / 8; ++k) {
      const float2 x = ok ? load2<T>(src + 2 * k) : make_float2(0.f, 0.f);
      top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
    // 2^(14 - e) for top in [2^e, 2^(e + 1)); rows of nothing larger than 2^-98 by 2^112
    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -98), 127);
    float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    if (!is_finite(top)) up = qnan();  // (infinities as NaN: their products with codes of 0 are)
    if (p.scale < 0.f) up = -up;       // scores go on with the scale's magnitude
    const float down = __uint_as_float((uint32_t)(127 + e - 14) << 23);
    unscale[n][0] = __shfl_sync(kAll, down, 8 * t);
    unscale[n][1] = __shfl_sync(kAll, down, 8 * t + 4);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int x2 = 0; x2 < 2; ++x2) {
        float2 x = ok ? load2<T>(src + 4 * k + 2 * x2) : make_float2(0.f, 0.f);
        x.x *= up;
        x.y *= up;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const uint32_t w = pack_f16(x.x, x.y);
          q.b[n][s][k][x2] = w;
          const float2 got = unpack_f16(w);
          x.x -= got.x;
          x.y -= got.y;
        }
      }
  }
}

// What the lanes of a warp keep of their rows (2 t and 2 t + 1 of each tile).
template <int D, int NT>
struct Rows {
  float ref[NT][2], l[NT][2];  // the weights' reference (log2), the lane's part of the sum
  float o[NT][D / 16][4];
};

struct Where {  // of a tile's rows: the step's token and its position, a slope
  int node[2], pos[2];
  float slope[2];
};

// Shared memory of a CTA: the scan, each warp's stages (the warps' rows of a
// finished piece take their place), a tree where the call has one.
constexpr int kStages = 3;
template <int D>
__host__ __device__ constexpr int few_tiles() {  // of 16 slots, a chunk
  return D == 256 ? 1 : 2;
}
constexpr int kFewScan = 64;
static_assert(sizeof(long long) * (kFewWarps + 2) <= kFewScan, "");
template <int D, int NT>
__host__ __device__ constexpr int few_ring() {
  const int ring = kFewWarps * kStages * few_tiles<D>() * Tile<D>::kBytes;
  const int rows = kFewWarps * 8 * NT * (D + 4) * (int)sizeof(float);
  return ring > rows ? ring : rows;
}
// The tensor instruction cuts its sums off: 2^-24 of them a product of 16 slots or so, always towards 0,
// which was 2^-12 of the result over 131072 slots of one CTA. bf16, whose half step is 2^-9 and more, leaves
// it at that. In fp32 calls a thread adds what it has of the weighted values to a second sum in the workspace, by
// ordinary additions, every 256 products (2048 slots of the warp, 8192 of the unit), and starts again
// from 0: some 2^-17. 64 tokens of up to 8192 slots (8 heads of 128) take 136 us, 132 without; every 64 products
// cost 9 %, products that start from 0 in every tile 6 %, second sums in shared memory a CTA an SM for
// trees of more than 160 nodes.
template <int D>
__host__ __device__ constexpr int fold_chunks() {
  return 128 / few_tiles<D>();
}
template <int D, int NT, typename T>
__host__ __device__ constexpr int few_fold() {  // a thread's sums and their references
  return sizeof(T) == 4 ? kFewThreads * NT * (D / 4 + 2) * (int)sizeof(float) : 0;
}
template <int D, int NT>
struct Fold {
  float* at;  // the thread's first word; word i is kFewThreads i on
  __device__ __forceinline__ float& word(int i) const { return at[i * kFewThreads]; }
  static constexpr int kPer = D / 4 + 2;  // of a tile: its sums, two references
  // sum = sum (`first`: 0) + o, o = 0
  __device__ __forceinline__ void add(Rows<D, NT>& acc, bool first) const {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float g = factor(n, e, acc.ref[n][e], first);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int x = e; x < 4; x += 2) {
            float& sum = word(n * kPer + 4 * i + x);
            sum = first ? acc.o[n][i][x] : fmaf(sum, g, acc.o[n][i][x]);
            acc.o[n][i][x] = 0.f;
          }
        word(n * kPer + D / 4 + e) = acc.ref[n][e];
      }
  }
  // o = sum + o
  __device__ __forceinline__ void take(Rows<D, NT>& acc) const {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float g = factor(n, e, acc.ref[n][e], false);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int x = e; x < 4; x += 2)
            acc.o[n][i][x] = fmaf(word(n * kPer + 4 * i + x), g, acc.o[n][i][x]);
      }
  }
  __device__ __forceinline__ float factor(int n, int e, float ref, bool first) const {
    const float old = first ? -INFINITY : word(n * kPer + D / 4 + e);
    return old == -INFINITY ? 0.f : ex2(old - ref);  // (NaN stays NaN times 0)
  }
};
template <int D, int NT>
constexpr size_t few_smem() {
  return kFewScan + few_ring<D, NT>();
}

// CTAs an SM holds: as many as their registers allow without spills to speak of.
template <int D, int NT, typename T>
constexpr int few_blocks() {
  return D == 256 || (D == 128 && NT == 2) ? 2 : D == 64 || sizeof(T) == 2 ? 4 - (NT - 1) : 3;
}

template <int D, int NT, typename T>
__global__ void __launch_bounds__(kFewThreads, few_blocks<D, NT, T>()) few_kernel(const AttendParams p) {
  constexpr bool kExact = sizeof(T) == 4;
  constexpr int NS = kExact ? 2 : 1, NP = NS;
  constexpr int kTiles = few_tiles<D>();
  constexpr int kChunkSlots = 16 * kTiles;
  extern __shared__ __align__(16) char raw_smem[];
  long long* scan = reinterpret_cast<long long*>(raw_smem);
  char* ring = raw_smem + kFewScan;
  float* rows_out = reinterpret_cast<float*>(ring);
  const TreeView tree(ring + few_ring<D, NT>(), ring, p.N);  // (if p.parent)
  const Fold<D, NT> fold{p.fold + (long long)blockIdx.x * (few_fold<D, NT, T>() / (int)sizeof(float)) +
                         threadIdx.x};
  pdl_wait();
  pdl_launch_dependents();
  const int cta = blockIdx.x, lane = lane_id(), warp = threadIdx.x / 32;
  const int g = lane / 4, t = lane % 4;
  const Share share = find_share<kFewThreads>(p, cta, gridDim.x, scan);
  if (threadIdx.x == 0) p.desc[4 * cta + 3] = 0;
  if (cta >= share.G) return;

  int b = share.b;
  long long at = share.at;             // in request b
  long long left = share.end - share.begin;
  bool first = true;
  Request r = request_of(p, b);
  while (left > 0) {
    while ((long long)r.chunks * r.tiles * p.cache.Hkv <= at) {  // (the next request with work)
      at = 0;
      r = request_of(p, ++b);
    }
    const int unit = (int)(at / r.chunks);
    const int c0 = (int)(at - (long long)unit * r.chunks);
    const int c1 = (int)min((long long)r.chunks, c0 + left);
    const int h = unit / r.tiles, tile = unit - h * r.tiles;
    const int rows = r.nq * p.group;  // of the request's head
    const int row0 = tile * 8 * NT;

    bool sees = r.ok && r.len > 0;
    if (p.parent && sees) sees = build_tree<kFewThreads>(p, b, r.nq, tree);

    Query<D, NT, NS> q;
    float unscale[NT][2];
    load_query<D, NT, NS, T>(p, b, h, row0, r.ok ? rows : 0, q, unscale);
    Rows<D, NT> acc;
    Where where[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        acc.ref[n][e] = -INFINITY;
        acc.l[n][e] = 0.f;
        const int row = min(row0 + 8 * n + 2 * t + e, max(rows - 1, 0));
        const int i = row / p.group;
        where[n].node[e] = i;
        where[n].pos[e] = r.base + (p.parent && sees ? tree.depth(i) : i);
        where[n].slope[e] = p.slopes ? p.slopes[h * p.group + row - i * p.group] * kLog2e : 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        acc.o[n][i][0] = acc.o[n][i][1] = acc.o[n][i][2] = acc.o[n][i][3] = 0.f;
    }

    if (sees) {
      const int from = r.lo / kChunkSlots;
      const int* table = p.cache.table + (long long)b * p.cache.M;
      const int mask = (1 << p.cache.shift) - 1;
      // scores before the cap, or in units of log2 where there is none
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) unscale[n][e] = score_factor(p, unscale[n][e]);
      // The warp's stages: chunk c's copies are queued kStages - 1 chunks ahead, its page ids
      // read one chunk before that.
      constexpr int kStageBytes = kTiles * Tile<D>::kBytes;
      char* stages = ring + warp * kStages * kStageBytes;
      const int block = page_bytes(1, D) << p.cache.shift;
      const char* head = p.cache.data + (long long)(2 * h) * block;
      const bool one_page = kTiles == 1 || p.cache.shift >= 5;  // a chunk lies in one page
      int next[kTiles] = {};
      auto queue = [&](int c, char* stage) {
        if (c < c1) {
          const int token = ((from + c) * kChunkSlots) & mask;
          if (one_page) {
            queue_tiles<D, kTiles>(p.cache, head, block, next[0], token, stage);
          } else {
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
              queue_tiles<D, 1>(p.cache, head, block, next[k], (token + 16 * k) & mask,
                                stage + k * Tile<D>::kBytes);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      auto fetch_ids = [&](int c) {
        const int slot = (from + c) * kChunkSlots;
        next[0] = c < c1 && slot < r.len ? table[slot >> p.cache.shift] : -1;
        if (!one_page)
#pragma unroll
          for (int k = 1; k < kTiles; ++k)
            next[k] = c < c1 && slot + 16 * k < r.len ? table[(slot + 16 * k) >> p.cache.shift] : -1;
      };
#pragma unroll
      for (int st = 0; st < kStages - 1; ++st) {
        fetch_ids(c0 + warp + st * kFewWarps);
        queue(c0 + warp + st * kFewWarps, stages + st * kStageBytes);
      }
      fetch_ids(c0 + warp + (kStages - 1) * kFewWarps);
      int now = 0, then = kStages - 1;
      for (int c = c0 + warp; c < c1; c += kFewWarps) {
        const int slot0 = (from + c) * kChunkSlots;
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();  // (every lane's copies are in, and its loads of the stage before done)
        queue(c + (kStages - 1) * kFewWarps, stages + then * kStageBytes);
        fetch_ids(c + kStages * kFewWarps);
        const char* stage = stages + now * kStageBytes;
        now = now + 1 == kStages ? 0 : now + 1;
        then = then + 1 == kStages ? 0 : then + 1;
        float s[kTiles][NT][4];
#pragma unroll
        for (int k = 0; k < kTiles; ++k)
          scores<D, NT, NS>(stage + k * Tile<D>::kBytes, q, s[k]);
        // a chunk before the step's tokens that every row sees whole needs no masks
        const bool edge = slot0 + kChunkSlots > r.base ||
                          (p.window > 0 && slot0 <= r.base + r.nq - 1 - p.window);
        const bool plain = !edge && p.softcap == 0.f && !p.slopes;
        if (!plain) {
          auto each = [&](auto f) {
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[k][n][e] = f(s[k][n][e] * unscale[n][e & 1]);
          };
          if (p.softcap > 0.f)
            cap_all<kExact>(p.softcap * kLog2e, each);
          else
            each([](float y) { return y; });
        }
        if (edge || p.slopes) {
#pragma unroll
          for (int k = 0; k < kTiles; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int slot = slot0 + 16 * k + 4 * (g >> 1) + (g & 1) + 2 * x;
              const int node = slot - r.base;
              const bool there = slot < r.len;
              int pos = slot;
              if (p.parent && node >= 0 && there) pos = r.base + tree.depth(node);
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int far = where[n].pos[e] - pos;
                  float& y = s[k][n][2 * x + e];
                  if (p.slopes) y = fmaf(-where[n].slope[e], (float)far, y);
                  if (edge) {
                    bool seen = there;
                    if (node >= 0 && there)
                      seen = p.parent ? tree.sees(where[n].node[e], node) : node <= where[n].node[e];
                    if (p.window > 0 && far >= p.window) seen = false;
                    if (!seen) y = -INFINITY;
                  }
                }
            }
        }
        uint32_t P[kTiles][NT][NP][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // each row's reference: 15 below its largest score, rounded up, so that no exponent is above 15. The
          // lanes of a column meet only where one of them found a larger score
          float f[2], top[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[e] = plain ? unscale[n][e] : 1.f;
            top[e] = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
            for (int k = 1; k < kTiles; ++k)
              top[e] = fmaxf(top[e], fmaxf(s[k][n][e], s[k][n][e + 2]));
            top[e] *= f[e];
          }
          // (and in every chunk of rows whose references are far from 0)
          if (__any_sync(kAll, top[0] - acc.ref[n][0] > kFewShift || top[1] - acc.ref[n][1] > kFewShift ||
                                   fabsf(acc.ref[n][0]) >= kFar || fabsf(acc.ref[n][1]) >= kFar)) {
            bool far = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float ref = fmaxf(__fadd_ru(top[e], -kFewShift), acc.ref[n][e]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) ref = fmaxf(ref, __shfl_xor_sync(kAll, ref, x));
              const float g1 = acc.ref[n][e] == -INFINITY ? 0.f : ex2(acc.ref[n][e] - ref);
              acc.ref[n][e] = ref;
              acc.l[n][e] *= g1;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                acc.o[n][i][e] *= g1;
                acc.o[n][i][e + 2] *= g1;
              }
              far |= fabsf(ref) >= kFar;
            }
            if (__any_sync(kAll, far)) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int k = 0; k < kTiles; ++k)
#pragma unroll
                  for (int x = 0; x < 4; x += 2) s[k][n][e + x] = __fmul_rn(s[k][n][e + x], f[e]);
                f[e] = 1.f;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float off = acc.ref[n][e] == -INFINITY ? 0.f : -acc.ref[n][e];
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
#pragma unroll
              for (int x = 0; x < 4; x += 2) {
                const float w = ex2(fmaf(s[k][n][e + x], f[e], off));
                s[k][n][e + x] = w;
                acc.l[n][e] += w;
              }
          }
#pragma unroll
          for (int k = 0; k < kTiles; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float w0 = s[k][n][2 * x], w1 = s[k][n][2 * x + 1];
#pragma unroll
              for (int part = 0; part < NP; ++part) {
                const uint32_t w = pack_f16(w0, w1);
                P[k][n][part][x] = transpose8(w);
                const float2 got = unpack_f16(w);
                w0 -= got.x;
                w1 -= got.y;
              }
            }
        }
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
          uint32_t dead = 0;
          if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int slot = slot0 + 16 * k + 4 * t + i;
              dead |= (slot < r.lo || slot >= r.len ? 1u : 0u) << i;
            }
          }
          values<D, NT, NP>(stage + k * Tile<D>::kBytes, P[k], dead, acc.o);
        }
        if (kExact) {
          const int done = (c - c0) / kFewWarps + 1;
          if (done % fold_chunks<D>() == 0) fold.add(acc, done == fold_chunks<D>());
        }
      }
      if (kExact && (c1 - c0 - warp + kFewWarps - 1) / kFewWarps >= fold_chunks<D>()) fold.take(acc);
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();  // (the stages are read)

    // join the warps: each leaves its rows in shared memory
    constexpr int kRows = 8 * NT, kStep = D + 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = acc.l[n][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(kAll, l, x);
        float* row = rows_out + (warp * kRows + 8 * n + 2 * t + e) * kStep;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(row + dim_of<D>(i)) =
              make_float2(acc.o[n][i][e], acc.o[n][i][e + 2]);
        if (g == 0) {
          row[D] = acc.ref[n][e];
          row[D + 1] = l;
        }
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == r.chunks;
    float* part = p.part + (long long)(2 * cta + (first ? 0 : 1)) * kRows * kStep;
    for (int x = threadIdx.x; x < kRows * (D / 4); x += kFewThreads) {
      const int row = x / (D / 4), d = x % (D / 4) * 4;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, rows_out[(w * kRows + row) * kStep + D]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float* src = rows_out + (w * kRows + row) * kStep;
        const float f = src[D] == -INFINITY ? (src[D + 1] == 0.f ? 0.f : 1.f) : ex2(src[D] - m);
        const float4 v = *reinterpret_cast<const float4*>(src + d);
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
        l = fmaf(src[D + 1], f, l);
      }
      if (whole) {
        const int global = row0 + row;
        if (global >= rows) continue;
        const int i = global / p.group, j = global - i * p.group;
        const long long to = ((long long)b * p.N + i) * p.Hq + h * p.group + j;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
        if (kExact)
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to * D + d) = o;
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to * D + d) =
              make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
        if (p.out_lse && d == 0) p.out_lse[to] = log_sum(m, l, 0.f);
      } else {
        float* dst = part + row * kStep;
        *reinterpret_cast<float4*>(dst + d) = o;
        if (d == 0) {
          dst[D] = m;
          dst[D + 1] = l;
        }
      }
    }
    if (!whole && c0 == 0 && threadIdx.x == 0) {  // the first piece of a split unit
      int* desc = p.desc + 4 * cta;
      desc[0] = b;
      desc[1] = h;
      desc[2] = tile | (first ? 0 : 1 << 30);
      desc[3] = pieces_of(share, cta, share.end - left + r.chunks);
    }
    __syncthreads();
    at += c1 - c0;
    left -= c1 - c0;
    first = false;
  }
}

// Joins the pieces of the unit that begins in CTA blockIdx.x's share and is
// split, and reports the requests' statuses.  One warp a row; or, where units are few and
// their pieces many (WIDE), a block of 8 warps a row, the pieces dealt to the warps: a call of a token
// over 16000 slots for 8 heads (76 pieces each) takes 26 instead of 36 us.  Below 16 pieces a
// unit one warp is as fast or faster (8.9 instead of 10.1 us at 128 slots).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

template <int D, typename T, bool WIDE>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  if (p.out_status && blockIdx.y == 0) {  // (a warp a request)
    const int lane = lane_id();
    bool late = false;  // (a wait that ran out is every request's, so seldom is it)
    if (p.late)
      for (int i = lane; i < (int)gridDim.x; i += 32) late |= p.late[i] != 0;
    const int ran_out = __any_sync(kAll, late) ? kTimeout : 0;
    for (int b = blockIdx.x * kJoinWarps + threadIdx.x / 32; b < p.B; b += gridDim.x * kJoinWarps) {
      const Request r = request_of(p, b);
      int st = r.ok ? page_status(p.cache, b, r.lo, r.len - r.lo) : kBadDraftLen;
      if (r.ok && p.parent) {
        const int* parent = p.parent + (long long)b * p.parent_stride;
        bool bad = false;
        for (int n = 1 + lane; n < r.nq; n += 32)
          bad |= (parent[n - 1] < 0) | (parent[n - 1] >= n);
        if (__any_sync(kAll, bad)) st |= kBadTree;
      }
      if (lane == 0) p.out_status[b] = st | ran_out;
    }
  }
  if (!p.desc) return;  // (a step of no tokens: statuses alone)
  const int cta = blockIdx.x;
  const int4 d4 = *reinterpret_cast<const int4*>(p.desc + 4 * cta);
  const int pieces = d4.w;
  if (pieces == 0) return;
  const int b = d4.x, h = d4.y, tile = d4.z & 0x3fffffff, second = d4.z >> 30;
  const Request r = request_of(p, b);
  constexpr int kStep = D + 4, kVec = D / 32;  // values a lane: D / 32
  const int lane = lane_id();
  const int n_rows = min(p.rows, r.nq * p.group - tile * p.rows);
  const int warp = threadIdx.x / 32;
  __shared__ float sums[WIDE ? kJoinWarps : 1][D + 1], maxes[kJoinWarps];
  for (int row = WIDE ? blockIdx.y : blockIdx.y * kJoinWarps + warp; row < n_rows;
       row += WIDE ? gridDim.y : gridDim.y * kJoinWarps) {
    auto src_of = [&](int k) {
      const int slot = k == 0 ? 2 * cta + second : 2 * (cta + k);
      return p.part + ((long long)slot * p.rows + row) * kStep;
    };
    const int k_first = WIDE ? warp : 0, k_step = WIDE ? kJoinWarps : 1;
    float m = -INFINITY;
    for (int k = k_first + lane * k_step; k < pieces; k += 32 * k_step) m = fmaxf(m, src_of(k)[D]);
    m = warp_max_nan(m);
    if (WIDE) {
      if (lane == 0) maxes[warp] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i) m = fmaxf(m, maxes[i]);
    }
    // 32 pieces at a time: a lane works out one's factor, then every lane adds its dimensions of them
    // all, whose loads wait for nothing
    float o[kVec] = {}, l = 0.f;
    for (int k0 = k_first; k0 < pieces; k0 += 32 * k_step) {
      float f = 0.f;
      if (k0 + lane * k_step < pieces) {
        const float2 ml = *reinterpret_cast<const float2*>(src_of(k0 + lane * k_step) + D);
        f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - m);
        l = fmaf(ml.y, f, l);
      }
      const int n = min(32, (pieces - k0 + k_step - 1) / k_step);
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float g = __shfl_sync(kAll, f, k);
        const float* src = src_of(k0 + k * k_step) + lane * kVec;
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          const float2 v = *reinterpret_cast<const float2*>(src + e);
          o[e] = fmaf(v.x, g, o[e]);
          o[e + 1] = fmaf(v.y, g, o[e + 1]);
        }
      }
    }
    l = warp_sum(l);
    if (WIDE) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) sums[warp][lane * kVec + e] = o[e];
      if (lane == 0) sums[warp][D] = l;
      __syncthreads();
      if (warp == 0) {
        l = 0.f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) o[e] = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) {
          l += sums[i][D];
#pragma unroll
          for (int e = 0; e < kVec; ++e) o[e] += sums[i][lane * kVec + e];
        }
      }
    }
    if (!WIDE || warp == 0) {
      const int global = tile * p.rows + row;
      const int i = global / p.group, j = global - i * p.group;
      const long long to = ((long long)b * p.N + i) * p.Hq + h * p.group + j;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        if (sizeof(T) == 4)
          *reinterpret_cast<float2*>(static_cast<float*>(p.out) + to * D + lane * kVec + e) =
              make_float2(o[e] * inv, o[e + 1] * inv);
        else
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + to * D + lane * kVec +
                                       e) = pack_bf16(o[e] * inv, o[e + 1] * inv);
      }
      if (p.out_lse && lane == 0) p.out_lse[to] = log_sum(m, l, p.shift);
    }
    if (WIDE) __syncthreads();
  }
}

// Resident CTAs of a kernel on the current device (with `smem`; `most` is what a launch may ask for).
template <class K>
cudaError_t resident(K fn, int threads, size_t smem, size_t most, std::atomic<int>* cache,
                     int* ctas) {
  DeviceInfo info;
  cudaError_t err = device_info(&info);
  if (err != cudaSuccess) return err;
  int dev = 0;
  if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
  int n = cache[dev].load(std::memory_order_relaxed);  // (device_info: dev < 64)
  if (!n) {
    err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (err != cudaSuccess) return err;
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem);
    if (err != cudaSuccess) return err;
    if (n < 1) return cudaErrorInvalidConfiguration;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  *ctas = n * info.sms;
  return cudaSuccess;
}

template <int D, int NT, typename T>
cudaError_t plan_one(AttendPlan* plan) {
  static std::atomic<int> cache[64];
  plan->rows = 8 * NT;
  plan->chunk = D == 256 ? 16 : 32;
  plan->least = kFewWarps;
  plan->shift = 0.f;  // (partial rows hold references)
  plan->fold = few_fold<D, NT, T>();
  return resident(few_kernel<D, NT, T>, kFewThreads, few_smem<D, NT>(),
                  few_smem<D, NT>() + tree_bytes(SV_MAX_STEP), cache, &plan->ctas);
}

}  // namespace

#define SV_FEW(CALL)                                                        \
  if (dtype == SV_F32) {                                                    \
    if (D == 64) return CALL(64, 1, float);                                 \
    if (D == 128) return CALL(128, 1, float);                               \
    if (D == 256) return CALL(256, 1, float);                               \
  } else if (rows <= 8) {                                                   \
    if (D == 64) return CALL(64, 1, __nv_bfloat16);                         \
    if (D == 128) return CALL(128, 1, __nv_bfloat16);                       \
    if (D == 256) return CALL(256, 1, __nv_bfloat16);                       \
  } else {                                                                  \
    if (D == 64) return CALL(64, 2, __nv_bfloat16);                         \
    if (D == 128) return CALL(128, 2, __nv_bfloat16);                       \
    if (D == 256) return CALL(256, 1, __nv_bfloat16);                       \
  }                                                                         \
  return cudaErrorInvalidValue;

cudaError_t plan_few(int D, int dtype, int rows, AttendPlan* plan) {
#define SV_PLAN(d, n, T) (plan_one<d, n, T>(plan))
  SV_FEW(SV_PLAN)
#undef SV_PLAN
}

cudaError_t launch_few(const AttendParams& p, int D, int dtype, const AttendPlan& plan,
                       cudaStream_t stream) {
  const int rows = plan.rows;
#define SV_LAUNCH(d, n, T) \
  (launch_early(few_kernel<d, n, T>, plan.ctas, kFewThreads, \
                few_smem<d, n>() + (p.parent ? tree_bytes(p.N) : 0), 1, stream, p))
  SV_FEW(SV_LAUNCH)
#undef SV_LAUNCH
}

cudaError_t launch_join(const AttendParams& p, int D, int dtype, int ctas, int units,
                        cudaStream_t stream) {
  // units in 16 pieces or more, or whole, and few rows (a block each for many takes longer to launch)
  const bool wide = p.rows <= 16 && units * 16 <= ctas;
  const dim3 grid(ctas, wide ? std::min(p.rows, p.N * p.group)
                             : p.rows > 16 ? (p.rows + kJoinWarps - 1) / kJoinWarps : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
#define SV_JOIN(d)                                                                          \
  if (D == d) {                                                                             \
    if (dtype == SV_F32)                                                                    \
      return wide ? cudaLaunchKernelEx(&cfg, join_kernel<d, float, true>, p)                \
                  : cudaLaunchKernelEx(&cfg, join_kernel<d, float, false>, p);              \
    return wide ? cudaLaunchKernelEx(&cfg, join_kernel<d, __nv_bfloat16, true>, p)          \
                : cudaLaunchKernelEx(&cfg, join_kernel<d, __nv_bfloat16, false>, p);        \
  }
  SV_JOIN(64) SV_JOIN(128) SV_JOIN(256)
#undef SV_JOIN
  return cudaErrorInvalidValue;
}

sv_status check_cache(CacheView* c, const void* cache, int64_t page_stride, const int32_t* table,
                      int pages, int page_size, int B, int M, int kv_heads, int head_dim);

namespace {

// The kernel and split of a call of `rows` query rows a key/value head.  Tensor memory's tiles of 32 or
// 48 rows against tiles of 16 whose codes are decoded again for each: 269 against 286 us at 24
// rows, 273 against 294 at 32, 304 against 419 at 40, 308 against 425 at 48 (64 requests of up to 8192
// slots, 8 heads of 128; 48 rows have come to 284 since), but 164 for the small tiles at 16 rows, which decode
// once.  Heads of
// 256 and fp32 (two fp16 parts of everything) have the small tiles only.
bool many_rows(sv_dtype dtype, int rows, int D) {
  return dtype == SV_BF16 && D <= 128 && rows > 16;
}
cudaError_t plan_of(sv_dtype dtype, int rows, int D, AttendPlan* plan) {
  return many_rows(dtype, rows, D) ? plan_many(rows, plan) : plan_few(D, dtype, rows, plan);
}

// The workspace: the split units, a flag for each CTA, the unfinished rows, second sums.
size_t flag_offset(const AttendPlan& plan) { return (size_t)plan.ctas * 16; }
size_t part_offset(const AttendPlan& plan) {
  return flag_offset(plan) + ((size_t)plan.ctas * 4 + 15) / 16 * 16;
}
size_t fold_offset(const AttendPlan& plan, int D) {
  return part_offset(plan) + (size_t)plan.ctas * 2 * plan.rows * (D + 4) * sizeof(float);
}
size_t workspace_bytes(const AttendPlan& plan, int D) {
  return fold_offset(plan, D) + (size_t)plan.ctas * plan.fold;
}

bool shape_ok(int N, int Hq, int Hkv, int D) {
  return N >= 0 && N <= SV_MAX_STEP && Hkv >= 1 && Hkv <= SV_MAX_HEADS && Hq >= 1 &&
         Hq <= SV_MAX_HEADS && Hq % Hkv == 0 && (D == 64 || D == 128 || D == 256);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_cache_attention_workspace_size(sv_dtype dtype, int N, int q_heads,
                                                      int kv_heads, int head_dim) {
  if ((dtype != SV_F32 && dtype != SV_BF16) || !shape_ok(N, q_heads, kv_heads, head_dim)) return 0;
  AttendPlan plan;
  if (plan_of(dtype, std::max(N, 1) * (q_heads / kv_heads), head_dim, &plan) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return workspace_bytes(plan, head_dim);
}

extern "C" sv_status spec_cache_attention(
    const void* q, const int64_t* q_strides, const void* cache, int64_t page_stride,
    const int32_t* table, const int32_t* lens, const int32_t* q_lens, const int32_t* tree_parent,
    int parent_stride, const float* slopes, float scale, float softcap, int window, void* out,
    float* out_lse, int32_t* out_status, sv_dtype dtype, int pages, int page_size, int B, int N,
    int M, int q_heads, int kv_heads, int head_dim, void* workspace, size_t ws_bytes,
    sv_stream_t stream) {
  AttendParams p;
  memset(&p, 0, sizeof p);
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (!shape_ok(N, q_heads, kv_heads, head_dim)) return SV_ERR_SHAPE;
  const sv_status rc = check_cache(&p.cache, cache, page_stride, table, pages, page_size, B, M,
                                   kv_heads, head_dim);
  if (rc != SV_OK) return rc;
  if (!(scale == scale) || scale - scale != 0.f || !(softcap >= 0.f && softcap <= 1e30f) || window < 0)
    return SV_ERR_SCORE;
  if (tree_parent && parent_stride != 0 && parent_stride != N - 1) return SV_ERR_TREE;
  if (B == 0 || (N == 0 && !out_status)) return SV_OK;
  if (N == 0) {  // no rows, but the requests' lengths and pages are looked at
    if (!lens) return SV_ERR_NULL;
    p.out_status = out_status;
    p.lens = lens;
    p.q_lens = q_lens;
    p.B = B;
    p.window = window;
    p.rows = p.chunk = p.group = 1;
    const int blocks = std::min((B + kJoinWarps - 1) / kJoinWarps, 1024);
    return launch_join(p, head_dim, dtype, blocks, blocks, (cudaStream_t)stream) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
  }
  if (!lens || !q || !q_strides || !out || ((uintptr_t)q & 15) || ((uintptr_t)out & 15))
    return SV_ERR_NULL;
  const int esize = dtype == SV_F32 ? 4 : 2;
  const int n[3] = {B, N, q_heads};
  long long st[3];
  for (int i = 0; i < 3; ++i) {
    st[i] = n[i] > 1 ? q_strides[i] : 0;
    if (st[i] < 0 || st[i] > (1LL << 60) / n[i]) return SV_ERR_SHAPE;
    if (st[i] % 16) return SV_ERR_NULL;
  }
  // (rows of other tiles are read while a tile's are written)
  const size_t row = (size_t)head_dim * esize;
  const char *q0 = static_cast<const char*>(q), *o0 = static_cast<const char*>(out);
  size_t q_bytes = row;
  for (int i = 0; i < 3; ++i) q_bytes += (size_t)(n[i] - 1) * st[i];
  if (q0 < o0 + (size_t)B * N * q_heads * row && o0 < q0 + q_bytes) return SV_ERR_ALIAS;
  p.q = q;
  p.qb = st[0] / esize;
  p.qn = st[1] / esize;
  p.qh = st[2] / esize;
  p.out = out;
  p.out_lse = out_lse;
  p.out_status = out_status;
  p.lens = lens;
  p.q_lens = q_lens;
  p.parent = tree_parent;
  p.parent_stride = parent_stride;
  p.slopes = slopes;
  p.B = B;
  p.N = N;
  p.Hq = q_heads;
  p.group = q_heads / kv_heads;
  p.window = window;
  p.scale = scale;
  p.softcap = softcap;
  AttendPlan plan;
  if (plan_of(dtype, N * p.group, head_dim, &plan) != cudaSuccess) return SV_ERR_CUDA;
  p.rows = plan.rows;
  p.chunk = plan.chunk;
  p.least = plan.least;
  if (!workspace || ((uintptr_t)workspace & 15) || ws_bytes < workspace_bytes(plan, head_dim))
    return SV_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const bool many = many_rows(dtype, N * p.group, head_dim);
  p.desc = reinterpret_cast<int*>(ws);
  p.late = many ? reinterpret_cast<int*>(ws + flag_offset(plan)) : nullptr;
  p.part = reinterpret_cast<float*>(ws + part_offset(plan));
  p.fold = reinterpret_cast<float*>(ws + fold_offset(plan, head_dim));
  p.shift = plan.shift;
  p.wait_ns = wait_limit_ns();
  const cudaStream_t s = (cudaStream_t)stream;
  if ((many ? launch_many(p, head_dim, plan, s) : launch_few(p, head_dim, dtype, plan, s)) !=
      cudaSuccess)
    return SV_ERR_CUDA;
  const long long units = (long long)B * kv_heads * ((N * p.group + p.rows - 1) / p.rows);
  const int some = (int)std::min(units, (long long)plan.ctas);
  return launch_join(p, head_dim, dtype, plan.ctas, some, s) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
