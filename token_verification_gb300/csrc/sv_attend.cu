// sv_attend.cu - attention of a step's tokens over the 4-bit cache
// (spec_cache_attention): the kernel for few query rows, the join of split
// units, and the entry point.
//
// Few rows (a token or a few drafts of a group of heads): bound by HBM, if the
// decoding of the codes keeps up.  So no code passes through shared memory: a
// warp's lanes load the cache's words straight into the registers of the tensor
// instruction's fragments (m16n8k16) and decode them there, 1.4 instructions a value.
//   S^T = K Q^T   A = 16 slots x 16 dimensions of keys in bf16, B = 8 query rows.
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
// fp16 for the rest, and take Q as three bf16 numbers, which is exact).
//
// Each of the four warps of a CTA walks its own chunks of 32 slots with its own
// running max and sum; the warps join at the end of a piece.
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

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
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
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NW words from an address aligned to them.
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

// A lane's words of 16 slots.  g = lane / 4, t = lane % 4; slots 4 (g / 2) + g % 2 and two on
// of the keys, slots 4 t .. 4 t + 3 of the values.
template <int D>
struct Raw {
  static constexpr int KW = D / 32, VW = D / 64;  // words of a slot
  static constexpr int KG = KW > 4 ? KW / 4 : 1;  // groups of the lane's keys
  uint32_t k[2][KW], v[4][VW], ks[KG], vs;
};

template <int D>
__device__ __forceinline__ void load_raw(const CacheView& c, int id, int token, int h, Raw<D>& r) {
  const int lane = lane_id(), g = lane / 4, t = lane % 4;
  if ((unsigned)id >= (unsigned)c.pages) {  // no such page: slots of NaN
#pragma unroll
    for (int w = 0; w < Raw<D>::KW; ++w) r.k[0][w] = r.k[1][w] = 0;
#pragma unroll
    for (int w = 0; w < Raw<D>::VW; ++w) r.v[0][w] = r.v[1][w] = r.v[2][w] = r.v[3][w] = 0;
#pragma unroll
    for (int i = 0; i < Raw<D>::KG; ++i) r.ks[i] = 0xffffffffu;
    r.vs = 0;
    return;
  }
  const char* kb = page_block<D>(c, id, h, 0);
  const char* vb = page_block<D>(c, id, h, 1);
  constexpr int kRow = D / 2;
  const int slot = token + 4 * (g >> 1) + (g & 1);
  load_words<Raw<D>::KW>(kb + slot * kRow + t * (kRow / 4), r.k[0]);
  load_words<Raw<D>::KW>(kb + (slot + 2) * kRow + t * (kRow / 4), r.k[1]);
#pragma unroll
  for (int i = 0; i < Raw<D>::KG; ++i) {
    const int group = t * (D / 4) / kGroup + i;
    r.ks[i] = *reinterpret_cast<const uint32_t*>(kb + scale_at<D>(c, token, group) + 4 * (g >> 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    load_words<Raw<D>::VW>(vb + (token + 4 * t + i) * kRow + g * (kRow / 8), r.v[i]);
  r.vs = *reinterpret_cast<const uint32_t*>(vb + scale_at<D>(c, token, g * (D / 8) / kGroup) + 4 * t);
}

// A key scale byte as a pair of bf16, and -136 times it.
__device__ __forceinline__ void key_scale(uint32_t byte, uint32_t& s, uint32_t& off) {
  uint32_t x = (byte + kScaleBias) << 4;
  if (byte == kNanScale) x = 0x7fff;
  s = x | x << 16;
  off = fma_bf16x2(s, 0xc308c308u, 0x80008000u);  // -136 s
}

template <int D, int NT, int NS>
struct Query {  // B fragments of NT tiles of 8 rows, NS bf16 parts each
  uint32_t b[NT][NS][D / 16][2];
};

// S^T of 16 slots: s[n] = {slot, row 2 t}, {slot, row 2 t + 1}, and the same two slots on.
template <int D, int NT, int NS>
__device__ __forceinline__ void scores(const Raw<D>& r, const Query<D, NT, NS>& q,
                                       float (&s)[NT][4]) {
  const int g = lane_id() / 4;
#pragma unroll
  for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
  uint32_t s0 = 0, o0 = 0, s1 = 0, o1 = 0;
#pragma unroll
  for (int w = 0; w < Raw<D>::KW; ++w) {
    if (w % 4 == 0) {
      const uint32_t pair = r.ks[w / 4] >> ((g & 1) * 8);
      key_scale(pair & 255, s0, o0);
      key_scale((pair >> 16) & 255, s1, o1);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t a[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int sh = 8 * half + 4 * j;
        a[2 * j] = fma_bf16x2(((r.k[0][w] >> sh) & 0x000f000fu) | 0x43004300u, s0, o0);
        a[2 * j + 1] = fma_bf16x2(((r.k[1][w] >> sh) & 0x000f000fu) | 0x43004300u, s1, o1);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < NS; ++i)
          mma_bf16(s[n], a, q.b[n][i][2 * w + half][0], q.b[n][i][2 * w + half][1]);
    }
  }
}

// O^T += V^T P^T of 16 slots; P: operand fragments, NP fp16 parts.  Slots whose bit of `dead` (of
// the lane's four) is set count as zeros whatever they hold.
template <int D, int NT, int NP>
__device__ __forceinline__ void values(const Raw<D>& r, const uint32_t (&P)[NT][NP][2],
                                       uint32_t dead, float (&o)[NT][D / 16][4]) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = scale_of((r.vs >> (8 * i)) & 255);
    if (dead >> i & 1) f[i] = 0.f;
  }
  const uint32_t sa = pack_f16(f[0], f[1]), sb = pack_f16(f[2], f[3]);
  const uint32_t oa = fma_f16x2(sa, 0xd480d480u, 0x80008000u);  // -72 s
  const uint32_t ob = fma_f16x2(sb, 0xd480d480u, 0x80008000u);
#pragma unroll
  for (int w = 0; w < Raw<D>::VW; ++w) {
    const uint32_t x[4] = {__byte_perm(r.v[0][w], r.v[1][w], 0x5410),
                           __byte_perm(r.v[0][w], r.v[1][w], 0x7632),
                           __byte_perm(r.v[2][w], r.v[3][w], 0x5410),
                           __byte_perm(r.v[2][w], r.v[3][w], 0x7632)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = i == 0 ? x[j] << 4 : x[j] >> (4 * i - 4);
        a[j] = fma_f16x2((y & 0x00f000f0u) | 0x54005400u, j < 2 ? sa : sb, j < 2 ? oa : ob);
      }
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

template <int D, int NT, int NS, typename T>
__device__ __forceinline__ void load_query(const AttendParams& p, int b, int h, int row0, int rows,
                                           Query<D, NT, NS>& q) {
  const int lane = lane_id(), g = lane / 4, t = lane % 4;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = row0 + 8 * n + g;
    const bool ok = row < rows;
    const int i = row / p.group, j = row - i * p.group;
    const T* src = static_cast<const T*>(p.q) + b * p.qb + i * p.qn +
                   (long long)(h * p.group + j) * p.qh + t * (D / 4);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 x = ok ? load2<T>(src + 4 * k + 2 * e) : make_float2(0.f, 0.f);
#pragma unroll
        for (int s = 0; s < NS; ++s) {  // the next 8 bits of what is left
          const uint32_t w = pack_bf16(x.x, x.y);
          q.b[n][s][k][e] = w;
          if (NS > 1) {
            // (infinity minus itself would leave NaN in the parts that follow)
            x.x = is_finite(x.x) ? x.x - bf16_lo(w) : 0.f;
            x.y = is_finite(x.y) ? x.y - bf16_hi(w) : 0.f;
          }
        }
      }
  }
}

// What the lanes of a warp keep of their rows (2 t and 2 t + 1 of each tile).
template <int D, int NT>
struct Rows {
  float m[NT][2], l[NT][2];  // running max (log2), the lane's part of the sum
  float o[NT][D / 16][4];
};

struct Where {  // of a tile's rows: the step's token and its position, a slope
  int node[2], pos[2];
  float slope[2];
};

template <int D>
struct FewSmem {
  long long scan[kFewWarps + 3];
  TreeView tree;
  alignas(16) float o[1];  // [warps][rows][D + 4]
};

template <int D, int NT>
constexpr size_t few_smem() {
  return offsetof(FewSmem<D>, o) + sizeof(float) * kFewWarps * 8 * NT * (D + 4);
}

template <int D, int NT, typename T>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const AttendParams p) {
  constexpr bool kExact = sizeof(T) == 4;
  constexpr int NS = kExact ? 3 : 1, NP = kExact ? 2 : 1;
  constexpr int kTiles = D == 256 ? 1 : 2;  // of 16 slots, a chunk
  constexpr int kChunkSlots = 16 * kTiles;
  extern __shared__ __align__(16) char raw_smem[];
  FewSmem<D>& sm = *reinterpret_cast<FewSmem<D>*>(raw_smem);
  pdl_wait();
  pdl_launch_dependents();
  const int cta = blockIdx.x, lane = lane_id(), warp = threadIdx.x / 32;
  const int g = lane / 4, t = lane % 4;
  const Share share = find_share<kFewThreads>(p, cta, gridDim.x, sm.scan);
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
    if (p.parent && sees) sees = build_tree<kFewThreads>(p, b, r.nq, sm.tree);

    Query<D, NT, NS> q;
    load_query<D, NT, NS, T>(p, b, h, row0, r.ok ? rows : 0, q);
    Rows<D, NT> acc;
    Where where[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        acc.m[n][e] = -INFINITY;
        acc.l[n][e] = 0.f;
        const int row = min(row0 + 8 * n + 2 * t + e, max(rows - 1, 0));
        const int i = row / p.group;
        where[n].node[e] = i;
        where[n].pos[e] = r.base + (p.parent && sees ? sm.tree.depth[i] : i);
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
      auto fetch_ids = [&](int c, int (&id)[kTiles]) {
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
          const int slot = (from + c) * kChunkSlots + 16 * k;
          id[k] = c < c1 && slot < r.len ? table[slot >> p.cache.shift] : -1;
        }
      };
      auto fetch = [&](int c, const int (&id)[kTiles], Raw<D> (&raw)[kTiles]) {
#pragma unroll
        for (int k = 0; k < kTiles; ++k)
          load_raw<D>(p.cache, id[k], ((from + c) * kChunkSlots + 16 * k) & mask, h, raw[k]);
      };
      int id[kTiles];
      Raw<D> next[kTiles];
      fetch_ids(c0 + warp, id);
      fetch(c0 + warp, id, next);
      fetch_ids(c0 + warp + kFewWarps, id);
      for (int c = c0 + warp; c < c1; c += kFewWarps) {
        Raw<D> now[kTiles];
#pragma unroll
        for (int k = 0; k < kTiles; ++k) now[k] = next[k];
        if (c + kFewWarps < c1) {
          fetch(c + kFewWarps, id, next);
          fetch_ids(c + 2 * kFewWarps, id);
        }
        float s[kTiles][NT][4];
#pragma unroll
        for (int k = 0; k < kTiles; ++k) scores<D, NT, NS>(now[k], q, s[k]);
        const int slot0 = (from + c) * kChunkSlots;
        // a chunk before the step's tokens that every row sees whole needs no masks
        const bool edge = slot0 + kChunkSlots > r.base || p.window > 0 || p.slopes;
#pragma unroll
        for (int k = 0; k < kTiles; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[k][n][e] = score_of<kExact>(p, s[k][n][e]);
        if (edge) {
#pragma unroll
          for (int k = 0; k < kTiles; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int slot = slot0 + 16 * k + 4 * (g >> 1) + (g & 1) + 2 * x;
              const int node = slot - r.base;
              const bool there = slot < r.len;
              int pos = slot;
              if (p.parent && node >= 0 && there) pos = r.base + sm.tree.depth[node];
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  bool seen = there;
                  if (node >= 0 && there)
                    seen = p.parent ? (sm.tree.seen[where[n].node[e]][node >> 5] >> (node & 31)) & 1
                                    : node <= where[n].node[e];
                  const int far = where[n].pos[e] - pos;
                  if (p.window > 0 && far >= p.window) seen = false;
                  float& y = s[k][n][2 * x + e];
                  y = seen ? fmaf(-where[n].slope[e], (float)far, y) : -INFINITY;
                }
            }
        }
        // the running max of each row, over the lanes of a column
        uint32_t P[kTiles][NT][NP][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
            for (int k = 1; k < kTiles; ++k) top = fmaxf(top, fmaxf(s[k][n][e], s[k][n][e + 2]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
            const float m = fmaxf(acc.m[n][e], top);
            if (__any_sync(kAll, m > acc.m[n][e])) {
              const float f = acc.m[n][e] == -INFINITY ? 0.f : ex2(acc.m[n][e] - m);
              acc.m[n][e] = m;
              acc.l[n][e] *= f;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                acc.o[n][i][e] *= f;
                acc.o[n][i][e + 2] *= f;
              }
            }
            const float off = m == -INFINITY ? 0.f : kShift - m;
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
#pragma unroll
              for (int x = 0; x < 4; x += 2) {
                const float w = ex2(s[k][n][e + x] + off);
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
                if (NP > 1) {
                  const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w));
                  w0 -= back.x;
                  w1 -= back.y;
                }
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
          values<D, NT, NP>(now[k], P[k], dead, acc.o);
        }
      }
    }

    // join the warps: each leaves its rows in shared memory
    constexpr int kRows = 8 * NT, kStep = D + 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = acc.l[n][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(kAll, l, x);
        float* row = sm.o + (warp * kRows + 8 * n + 2 * t + e) * kStep;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(row + dim_of<D>(i)) =
              make_float2(acc.o[n][i][e], acc.o[n][i][e + 2]);
        if (g == 0) {
          row[D] = acc.m[n][e];
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
      for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, sm.o[(w * kRows + row) * kStep + D]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float* src = sm.o + (w * kRows + row) * kStep;
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
        if (p.out_lse && d == 0)
          p.out_lse[to] = l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * 0.6931471805599453f;
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
// split, one warp a row, and reports the requests' statuses.
constexpr int kJoinThreads = 256;

template <int D, typename T>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  if (p.out_status && blockIdx.y == 0) {
    for (int b = blockIdx.x * kJoinThreads + threadIdx.x; b < p.B; b += gridDim.x * kJoinThreads) {
      const Request r = request_of(p, b);
      int st = r.ok ? page_status(p.cache, b, r.lo, r.len - r.lo) : kBadDraftLen;
      if (r.ok && p.parent) {
        const int* parent = p.parent + (long long)b * p.parent_stride;
        for (int n = 1; n < r.nq; ++n)
          if (parent[n - 1] < 0 || parent[n - 1] >= n) st |= kBadTree;
      }
      p.out_status[b] = st;
    }
  }
  const int cta = blockIdx.x;
  const int4 d4 = *reinterpret_cast<const int4*>(p.desc + 4 * cta);
  const int pieces = d4.w;
  if (pieces == 0) return;
  const int b = d4.x, h = d4.y, tile = d4.z & 0x3fffffff, second = d4.z >> 30;
  const Request r = request_of(p, b);
  constexpr int kStep = D + 4, kVec = D / 32;  // values a lane: D / 32
  const int lane = lane_id();
  const int n_rows = min(p.rows, r.nq * p.group - tile * p.rows);
  for (int row = blockIdx.y * (kJoinThreads / 32) + threadIdx.x / 32; row < n_rows;
       row += gridDim.y * (kJoinThreads / 32)) {
    auto src_of = [&](int k) {
      const int slot = k == 0 ? 2 * cta + second : 2 * (cta + k);
      return p.part + ((long long)slot * p.rows + row) * kStep;
    };
    float m = -INFINITY;
    for (int k = lane; k < pieces; k += 32) m = fmaxf(m, src_of(k)[D]);
    m = warp_max_nan(m);
    float o[kVec] = {}, l = 0.f;
#pragma unroll 4
    for (int k = 0; k < pieces; ++k) {
      const float* src = src_of(k);
      const float pm = src[D], pl = src[D + 1];
      const float f = pm == -INFINITY ? (pl == 0.f ? 0.f : 1.f) : ex2(pm - m);
      l = fmaf(pl, f, l);
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        const float2 v = *reinterpret_cast<const float2*>(src + lane * kVec + e);
        o[e] = fmaf(v.x, f, o[e]);
        o[e + 1] = fmaf(v.y, f, o[e + 1]);
      }
    }
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
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + to * D + lane * kVec + e) =
            pack_bf16(o[e] * inv, o[e + 1] * inv);
    }
    if (p.out_lse && lane == 0)
      p.out_lse[to] = l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * 0.6931471805599453f;
  }
}

// Resident CTAs of a kernel on the current device.
template <class K>
cudaError_t resident(K fn, int threads, size_t smem, std::atomic<int>* cache, int* ctas) {
  DeviceInfo info;
  cudaError_t err = device_info(&info);
  if (err != cudaSuccess) return err;
  int dev = 0;
  if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
  int n = cache[dev].load(std::memory_order_relaxed);  // (device_info: dev < 64)
  if (!n) {
    err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
  return resident(few_kernel<D, NT, T>, kFewThreads, few_smem<D, NT>(), cache, &plan->ctas);
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
  (launch_early(few_kernel<d, n, T>, plan.ctas, kFewThreads, few_smem<d, n>(), 1, stream, p))
  SV_FEW(SV_LAUNCH)
#undef SV_LAUNCH
}

cudaError_t launch_join(const AttendParams& p, int D, int dtype, int ctas, int units,
                        cudaStream_t stream) {
  // where units are few, each is in many pieces: a warp a row of every tile
  const dim3 grid(ctas, units * 4 <= ctas ? (p.rows + 7) / 8 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
#define SV_JOIN(d)                                                                   \
  if (D == d)                                                                        \
    return dtype == SV_F32 ? cudaLaunchKernelEx(&cfg, join_kernel<d, float>, p)      \
                           : cudaLaunchKernelEx(&cfg, join_kernel<d, __nv_bfloat16>, p);
  SV_JOIN(64) SV_JOIN(128) SV_JOIN(256)
#undef SV_JOIN
  return cudaErrorInvalidValue;
}

sv_status check_cache(CacheView* c, const void* cache, int64_t page_stride, const int32_t* table,
                      int pages, int page_size, int B, int M, int kv_heads, int head_dim);

namespace {

// The kernel and split of a call; 0 CTAs when nothing has to run.
cudaError_t plan_of(sv_dtype dtype, int rows, int head_dim, AttendPlan* plan) {
  return plan_few(head_dim, dtype, rows, plan);
}

size_t desc_bytes(const AttendPlan& plan) { return (size_t)plan.ctas * 16; }
size_t workspace_bytes(const AttendPlan& plan, int D) {
  return desc_bytes(plan) + (size_t)plan.ctas * 2 * plan.rows * (D + 4) * sizeof(float);
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
  if (!(scale == scale) || scale - scale != 0.f || !(softcap >= 0.f) || softcap - softcap != 0.f ||
      window < 0)
    return SV_ERR_SCORE;
  if (tree_parent && parent_stride != 0 && parent_stride != N - 1) return SV_ERR_TREE;
  if (B == 0 || N == 0) return SV_OK;
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
  p.desc = static_cast<int*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + desc_bytes(plan));
  const cudaStream_t s = (cudaStream_t)stream;
  if (launch_few(p, head_dim, dtype, plan, s) != cudaSuccess) return SV_ERR_CUDA;
  const long long units = (long long)B * kv_heads * ((N * p.group + p.rows - 1) / p.rows);
  const int many = (int)std::min(units, (long long)plan.ctas);
  return launch_join(p, head_dim, dtype, plan.ctas, many, s) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
