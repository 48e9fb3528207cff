// sv_top.cu - the k largest logits of each row with its log-sum-exp
// (spec_top_logits), and beam selection over beams and vocabulary
// (spec_beam_select): one kernel, a thread-block cluster per row or request.
//
// A row (of a request's W beams, or the one row of a record) is cut into
// `slices`; the (row, slice) items are dealt to the cluster's CTAs.  One pass
// over an item reads every logit once and keeps, per thread, a running
// softmax sum and max, and per 32 elements their max (rounded up to bf16, in
// shared memory).  The selection then follows from the thread maxes alone:
// if `units` disjoint parts of the data have maxes u_1.., the n-th largest of
// them is a bound that at least n elements reach, so every kept element is at
// or above it, and little else is: with n of 256 parts occupied, about
// 256 ln(256 / (256 - n)) elements (74 for n = 64).  Only the 32-element
// groups whose max reaches the bound are read again (from L2), their elements
// at or above it are listed, and the list is sorted by counting.
//
// A beam's candidates compare by score = offset + logit with offset =
// scores[w] - lse[w] in 64 bits; a record's offset is 0.  Bounds are in fp32
// rounded down, which can only lengthen the list.
//
// When the list does not fit (long rows of equal logits), the leader CTA
// selects each row by radix descent on whole-number keys, 8 bits a pass.
#include <string.h>

#include "../../include/spec_verify.h"
#include "sv_launch.h"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

#ifndef RING_BF16
#define RING_BF16 3
#define RING_F32 2
#define TOPB 3
#endif
constexpr int kTopThreads = 256;
constexpr int kTopWarps = kTopThreads / kWarp;
constexpr int kTopSpan = 8192;        // elements of a CTA's iteration: 32 a thread
constexpr int kMaxItems = 64;         // (row, slice) items per cluster
constexpr int kMaxUnits = 512;        // units per cluster
constexpr int kMaxCands = 1024;       // candidates of a cluster, 32-element groups of a CTA
constexpr int kMaxTables = 256;       // iterations of a CTA over its items: 512 bytes each
constexpr int kRankAll = 384;         // lists longer than this are cut to the bound first

struct TopParams {
  const void* logits;   // [B*P, V] (record) or [B*W, V] (beams)
  const int* lens;      // [B] or null (record)
  const float* scores;  // [B*W] (beams)
  int* out_ids;         // [B*P, k] / tokens [B, n]
  int* out_parents;     // beams: [B, n]
  float* out_values;    // [B*P, k] / scores [B, n]
  float* out_lse;       // record: [B*P]
  int* out_status;
  int P;                // record: rows per request
  int W;                // rows per cluster (record: 1)
  int V, n;
  int slices, slice;    // slices per row, elements per slice (a multiple of 256)
  int iters;            // iterations per item
  int upi;              // units per item (a power of two)
  int table_bytes;
  float cc;             // log2(e) / T
  float T;
  RowSpan span;
};

struct alignas(16) TopShared {
  float2 part[kMaxItems][kTopWarps];  // per item and warp: {max, sum of 2^((l - max) c)}
  float unit[kMaxUnits];              // unit maxes, item by item
  double off[SV_MAX_BEAMS];           // beams: score - lse of each row (-inf: no candidates)
  float off_down[SV_MAX_BEAMS];       // the same rounded down
  float thr[SV_MAX_BEAMS];            // the lowest logit a candidate of the row can have
  float lse;                          // record
  unsigned hist[256];
  int flag[2][kTopWarps];
  int n_hits, n_cands, overflow, bad, pick[4];
};

// The candidates, in the memory of the load stages once all are consumed.
struct alignas(16) Lists {
  unsigned long long key[kMaxCands];  // record: (ordered logit, ~index), a total order;
                                      // beams: the ordered score, idx = w * V + v
  int idx[kMaxCands];
  int rank[kMaxCands];                // until the list is sorted: the groups to read again
};

// Load stages: each warp streams 1024-element chunks through its own ring by
// asynchronous copies (a word more than a chunk, for rows off 16-byte
// boundaries); no barrier but the warp's own.
template <typename T>
struct Ring {
  static constexpr int kBytes = kChunk * (int)sizeof(T) + 16;
  static constexpr int kStages = sizeof(T) == 2 ? RING_BF16 : RING_F32;
  static constexpr int kWarpBytes = kBytes * kStages;
  static constexpr int kTotal = kWarpBytes * kTopWarps;
};

// The upper 16 bits of v rounded up: a bf16 value >= v (v itself for bf16).
__device__ __forceinline__ uint16_t up_bf16(float v) {
  const uint32_t b = __float_as_uint(v);
  return (uint16_t)((b & 0x80000000u) ? b >> 16 : (b + 0xffffu) >> 16);
}

// The n-th largest of the cluster's unit bounds to 16 bits (rounded down); -inf
// when fewer than n are finite.  A whole-CTA call: each warp holds all units
// as ordered keys, and every round tests one threshold per warp, so the range
// of keys shrinks ninefold (a bisection by one warp took 4000 cycles of a
// row's 87000; this takes a quarter).
template <int kPer>
__device__ float unit_bound(TopShared& s, int units, int n) {
  const int warp = threadIdx.x / kWarp;
  int k[kPer], hi = 0, lo = 0xffff;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = j * kWarp + lane_id();
    const float v = i < units ? s.unit[i] : -INFINITY;
    k[j] = v > -INFINITY ? (int)(ordered(v) >> 16) : 0;  // below every finite value's key
    hi = max(hi, k[j]);
    lo = min(lo, k[j]);
  }
  if (units < n) return -INFINITY;
  lo = __reduce_min_sync(0xffffffffu, lo);       // at least n units reach lo
  hi = __reduce_max_sync(0xffffffffu, hi) + 1;   // fewer than n reach hi
  for (int round = 0; hi - lo > 1; ++round) {
    const int step = (hi - lo + kTopWarps) / (kTopWarps + 1), at = lo + step * (warp + 1);
    unsigned c = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) c += k[j] >= at ? 1u : 0u;
    const bool ok = at < hi && (int)__reduce_add_sync(0xffffffffu, c) >= n;
    // the warps' answers are monotone; two sets of flags need one barrier a round
    if (lane_id() == 0) s.flag[round & 1][warp] = ok ? 1 : 0;
    __syncthreads();
    const unsigned yes = __ballot_sync(0xffffffffu, lane_id() < kTopWarps &&
                                                        s.flag[round & 1][lane_id() % kTopWarps]);
    const int up = __popc(yes);
    hi = min(hi, lo + step * (up + 1));
    lo += step * up;
  }
  return lo ? of_ordered((uint32_t)lo << 16) : -INFINITY;
}

template <bool kBeam>
__device__ __forceinline__ void set_candidate(Lists& s, int o, float l, double off, int idx) {
  s.key[o] = kBeam ? ordered(off + (double)l)
                   : ((unsigned long long)ordered(l) << 32) | (uint32_t)~idx;
  s.idx[o] = idx;
}

// One row's n largest finite elements by radix descent, appended to the list
// from `at` on (a whole-CTA call); returns how many.
template <typename T, bool kBeam>
__device__ int select_row_slow(TopShared& s, Lists& ls, const T* row, int V, int n, double off,
                               int base, int at) {
  const int t = threadIdx.x;
  auto key_of = [&](int j) {  // (logit in order, index from the end), 0 if not finite
    const float l = j < V ? load_logit(row, j) : -INFINITY;
    return l > -INFINITY
               ? ((unsigned long long)ordered(l) << 24) | (unsigned long long)(0xffffff - j)
               : 0ull;
  };
  unsigned long long cut = 0;
  int need = n;
  bool all = false;
  for (int shift = 48; shift >= 0; shift -= 8) {
    for (int i = t; i < 256; i += kTopThreads) s.hist[i] = 0;
    __syncthreads();
    for (int j0 = 0; j0 < V; j0 += kTopThreads) {
      const unsigned long long k = key_of(j0 + t);
      const bool in = k != 0 && ((k ^ cut) >> (shift + 8)) == 0;
      const unsigned digit = in ? (unsigned)(k >> shift) & 255u : 256u;
      const unsigned peers = __match_any_sync(0xffffffffu, digit);
      if (in && lane_id() == __ffs(peers) - 1) atomicAdd(&s.hist[digit], (unsigned)__popc(peers));
    }
    __syncthreads();
    if (t == 0) {
      int d = 255, above = 0;
      for (; d > 0 && above + (int)s.hist[d] < need; --d) above += (int)s.hist[d];
      s.pick[0] = d;
      s.pick[1] = above;
      s.pick[2] = (int)s.hist[d];
    }
    __syncthreads();
    const int above = s.pick[1], here = s.pick[2];
    cut |= (unsigned long long)s.pick[0] << shift;
    __syncthreads();
    if (above + here < need) {  // (first pass only) fewer than n finite elements: all of them
      all = true;
      break;
    }
    need -= above;
    if (here == need) break;  // every element of this prefix is kept
  }
  if (all) cut = 1;
  if (t == 0) s.pick[3] = at;
  __syncthreads();
  for (int j0 = 0; j0 < V; j0 += kTopThreads) {
    const unsigned long long k = key_of(j0 + t);
    if (k != 0 && k >= cut) {
      const int o = atomicAdd(&s.pick[3], 1);
      set_candidate<kBeam>(ls, o, load_logit(row, j0 + t), off, base + j0 + t);
    }
  }
  __syncthreads();
  return s.pick[3] - at;
}

// Whether entry j of the list comes before an entry of (key, idx).
template <bool kBeam>
__device__ __forceinline__ bool before(const Lists& s, int j, unsigned long long key, int idx) {
  const unsigned long long kj = s.key[j];
  return kj > key || (kBeam && kj == key && s.idx[j] < idx);
}

// rank[i] = the number of entries that come before entry i, i < count: the
// whole CTA, each entry's comparisons shared by as many threads as there are
// warps for all entries.
template <bool kBeam>
__device__ void rank_list(Lists& s, int count) {
  const int t = threadIdx.x;
  for (int i = t; i < count; i += kTopThreads) s.rank[i] = 0;
  __syncthreads();
  const int width = (count + kWarp - 1) / kWarp * kWarp;
  if (width <= kTopThreads / 2) {
    const int ways = kTopThreads / width, way = t / width, i = t - way * width;
    if (way < ways && i < count) {
      const unsigned long long key = s.key[i];
      const int idx = s.idx[i];
      int r = 0;
#pragma unroll 4
      for (int j = way; j < count; j += ways) r += before<kBeam>(s, j, key, idx) ? 1 : 0;
      atomicAdd(&s.rank[i], r);
    }
  } else {
    for (int i = t; i < count; i += kTopThreads) {
      const unsigned long long key = s.key[i];
      const int idx = s.idx[i];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < count; ++j) r += before<kBeam>(s, j, key, idx) ? 1 : 0;
      s.rank[i] = r;
    }
  }
  __syncthreads();
}

// Cuts the list to the entries at or above its n-th largest 32-bit key prefix.
__device__ int prune(TopShared& s, Lists& ls, int count, int n) {
  constexpr int kPer = kMaxCands / kTopThreads;
  unsigned long long k[kPer];
  int ix[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = q * kTopThreads + threadIdx.x;
    k[q] = i < count ? ls.key[i] : 0ull;
    ix[q] = i < count ? ls.idx[i] : 0;
  }
  uint32_t t = 0;
  for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
    const uint32_t at = t | bit;
    int c = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) c += (uint32_t)(k[q] >> 32) >= at ? 1 : 0;
    c = (int)__reduce_add_sync(0xffffffffu, (unsigned)c);
    if (threadIdx.x == 0) s.pick[0] = 0;
    __syncthreads();
    if (lane_id() == 0) atomicAdd(&s.pick[0], c);
    __syncthreads();
    if (s.pick[0] >= n) t = at;
    __syncthreads();
  }
  if (threadIdx.x == 0) s.pick[1] = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (q * kTopThreads + threadIdx.x < count && (uint32_t)(k[q] >> 32) >= t) {
      const int o = atomicAdd(&s.pick[1], 1);
      ls.key[o] = k[q];
      ls.idx[o] = ix[q];
    }
  __syncthreads();
  return s.pick[1];
}

template <bool kBeam>
__device__ __forceinline__ void write_slot(const TopParams& p, long long grp, int slot,
                                           unsigned long long key, int idx) {
  const long long o = grp * p.n + slot;
  const int w = kBeam && idx >= 0 ? idx / p.V : 0;
  p.out_ids[o] = idx < 0 ? -1 : idx - w * p.V;
  if (kBeam) p.out_parents[o] = idx < 0 ? -1 : w;
  p.out_values[o] = idx < 0 ? -INFINITY
                    : kBeam ? (float)of_ordered(key)
                            : of_ordered((uint32_t)(key >> 32));
}

template <typename T, bool kAligned, bool kBeam>
__global__ void __launch_bounds__(kTopThreads, TOPB) top_kernel(const TopParams p) {
  constexpr int VEC = Group<T>::VEC;
  constexpr int kGroups = kChunk / (kWarp * VEC);  // 16-byte groups of a lane: 32 elements
  using R = Ring<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  TopShared& s = *reinterpret_cast<TopShared*>(smem);
  // per iteration over this CTA's items, the thread's 32 elements' max
  uint16_t* table = reinterpret_cast<uint16_t*>(smem + sizeof(TopShared));
  unsigned char* rings = smem + sizeof(TopShared) + p.table_bytes;
  Lists& ls = *reinterpret_cast<Lists*>(rings);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long grp = blockIdx.x / C;
  const int t = threadIdx.x, lane = lane_id(), warp = t / kWarp;
  const int items = p.W * p.slices;
  const T* tag = nullptr;

  if (!kBeam && p.lens) {  // a record's row that is not needed (the whole cluster leaves)
    const int b = (int)(grp / p.P), i = (int)(grp - (long long)b * p.P);
    const int len = p.lens[b];
    const bool ok = len >= 0 && len <= p.P;
    if (!ok || i >= len) {
      if (rank == 0) {
        for (int j = t; j < p.n; j += kTopThreads) write_slot<kBeam>(p, grp, j, 0, -1);
        if (t == 0) {
          p.out_lse[grp] = -INFINITY;
          if (p.out_status) p.out_status[grp] = ok ? 0 : SV_REQ_BAD_DRAFT_LEN;
        }
      }
      return;
    }
  }
  if (t == 0) s.n_hits = s.n_cands = s.overflow = s.bad = 0;
  // no CTA writes into another's shared memory before that one has started
  if (C > 1) cluster_arrive();

  // One pass over each item.
  const int fold = kTopThreads / p.upi;
  for (int it = rank, mine = 0; it < items; it += C, ++mine) {
    const int w = it / p.slices, e0 = (it - w * p.slices) * p.slice;
    const int e1 = min(e0 + p.slice, p.V);
    const long long rowid = grp * p.W + w;
    const T* row = reinterpret_cast<const T*>(p.logits) + rowid * (long long)p.V;
    uint16_t* mine_table = table + mine * p.iters * kTopThreads + t;
    const bool live = !kBeam || p.scores[rowid] != -INFINITY;
    RunningSum r;
    if (live) {
      const int chunks = (e1 - e0 + kChunk - 1) / kChunk;
      const int todo = (chunks - warp + kTopWarps - 1) / kTopWarps;  // this warp's (may be <= 0)
      const uint32_t off = kAligned ? 0u : (uint32_t)(uintptr_t)row & 15u;
      const uint32_t ring = smem_u32(rings) + warp * R::kWarpBytes;
      auto issue = [&](int i) {  // iteration i's chunk into its stage
        if (i < todo) {
          const int j = e0 + (i * kTopWarps + warp) * kChunk;
          load_chunk_async<T, kAligned>(ring + i % R::kStages * R::kBytes, row, j, min(j + kChunk, e1),
                                        off, p.span);
        }
        copies_commit();
      };
#pragma unroll
      for (int i = 0; i < R::kStages - 1; ++i) issue(i);
      for (int i = 0; i < p.iters; ++i) {
        if (i >= todo) {
          mine_table[i * kTopThreads] = 0xff80u;
          continue;
        }
        copies_wait_but<R::kStages - 2>();
        __syncwarp();  // every lane's copies of this stage landed; the stage before is read
        uint4 g[kGroups];
        const uint32_t stage = ring + i % R::kStages * R::kBytes;
        const int j = e0 + (i * kTopWarps + warp) * kChunk;
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          const uint32_t at = stage + (u * kWarp + lane) * 16;
          g[u] = lds128(at);
          if (!kAligned && off) g[u] = shift_pair(g[u], lds128(at + 16), off);
        }
        if (j + kChunk > e1) clip_chunk<T>(g, j, e1);
        issue(i + R::kStages - 1);
        mine_table[i * kTopThreads] = up_bf16(r.add(g, p.cc, tag));
      }
      __syncwarp();  // (the next item refills the stages)
    } else {
      for (int i = 0; i < p.iters; ++i) mine_table[i * kTopThreads] = 0xff80u;
    }
    const float2 wr = warp_running(r, p.cc);
    float um = r.m;
    for (int o = 1; o < fold; o <<= 1) um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, o));
    if (C > 1 && mine == 0) cluster_wait();
    for (int c = 0; c < C; ++c) {
      TopShared* to = C > 1 ? cluster.map_shared_rank(&s, c) : &s;
      if (lane == 0) to->part[it][warp] = wr;
      if ((t & (fold - 1)) == 0) to->unit[it * p.upi + t / fold] = um;
    }
  }
  if (C > 1) {
    if (rank >= items) cluster_wait();
    cluster.sync();
  } else {
    __syncthreads();
  }

  // Each row's log-sum-exp and offset (every CTA for itself).
  const int parts = p.slices * kTopWarps;  // <= 64
  for (int w = warp; w < p.W; w += kTopWarps) {
    const float2* pt = &s.part[w * p.slices][0];
    const float2 a = lane < parts ? pt[lane] : make_float2(-INFINITY, 0.f);
    const float2 b = lane + kWarp < parts ? pt[lane + kWarp] : make_float2(-INFINITY, 0.f);
    const float m = warp_max_nan(max_nan(a.x, b.x));
    const float2 sum = warp_sum_pair(a.y * to_frame(a.x, m, p.cc) + b.y * to_frame(b.x, m, p.cc));
    if (lane == 0) {
      const float2 l = log_pair(sum);
      const float score = kBeam ? p.scores[grp * p.W + w] : 0.f;
      const bool dead = kBeam && score == -INFINITY;
      if (!dead && (m != m || m == INFINITY || score != score || score == INFINITY)) s.bad = 1;
      if (kBeam) {
        double off = -INFINITY;
        if (!dead && m != -INFINITY) off = ((double)score - (double)m) - ((double)l.x + (double)l.y);
        s.off[w] = off;
        s.off_down[w] = __double2float_rd(off);
      } else {
        s.lse = m == -INFINITY ? -INFINITY : m / p.T + (l.x + l.y);
      }
    }
  }
  __syncthreads();
  const bool bad = s.bad != 0;
  if (rank == 0 && t == 0) {
    if (!kBeam) p.out_lse[grp] = bad ? qnan() : s.lse;
    if (p.out_status) p.out_status[grp] = bad ? SV_REQ_BAD_LOGITS : 0;
  }
  if (bad) {  // the same in every CTA
    if (rank == 0)
      for (int j = t; j < p.n; j += kTopThreads) write_slot<kBeam>(p, grp, j, 0, -1);
    return;
  }

  // The bound that n elements reach, and each row's lowest candidate logit.
  const int units = items * p.upi;
  if (kBeam) {
    for (int u = t; u < units; u += kTopThreads) {
      const float l = s.unit[u], off = s.off_down[u / (p.upi * p.slices)];
      s.unit[u] = l == -INFINITY || off == -INFINITY ? -INFINITY : __fadd_rd(off, l);
    }
    __syncthreads();
  }
  const float bound = units <= 64    ? unit_bound<2>(s, units, p.n)
                      : units <= 256 ? unit_bound<8>(s, units, p.n)
                                     : unit_bound<16>(s, units, p.n);
  if (kBeam) {
    for (int w = t; w < p.W; w += kTopThreads) {
      const double off = s.off[w];
      // below it, off + l rounds below the bound (the slack covers the roundings); -inf never
      // passes: at least the lowest finite value
      s.thr[w] = off == -INFINITY ? INFINITY
                 : bound == -INFINITY
                     ? -FLT_MAX
                     : fmaxf(-FLT_MAX,
                             __double2float_rd(((double)bound - off) -
                                               1e-7 * (fabs((double)bound) + fabs(off))));
    }
    __syncthreads();
  }
  auto threshold = [&](int w) { return kBeam ? s.thr[w] : fmaxf(bound, -FLT_MAX); };

  // The groups that reach it, eight table entries a thread.
  for (int it = rank, mine = 0; it < items; it += C, ++mine) {
    const float thr = threshold(it / p.slices);
    const uint16_t* entries = table + mine * p.iters * kTopThreads;
    for (int v = t; v < p.iters * (kTopThreads / 8); v += kTopThreads) {
      const uint4 e = load128(entries + 8 * v);
      const uint32_t w[4] = {e.x, e.y, e.z, e.w};
      unsigned hits = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        hits |= (bf16_lo(w[q]) >= thr ? 1u << (2 * q) : 0u) |
                (bf16_hi(w[q]) >= thr ? 2u << (2 * q) : 0u);
      if (hits) {
        int h = atomicAdd(&s.n_hits, __popc(hits));
        for (; hits; hits &= hits - 1u, ++h)
          if (h < kMaxCands) ls.rank[h] = mine * p.iters * kTopThreads + 8 * v + __ffs(hits) - 1;
      }
    }
  }
  __syncthreads();
  TopShared* lead = C > 1 ? cluster.map_shared_rank(&s, 0) : &s;
  Lists* lead_ls = C > 1 ? cluster.map_shared_rank(&ls, 0) : &ls;
  const int hits = s.n_hits;
  if (hits > kMaxCands) {
    if (t == 0) lead->overflow = 1;
  } else {
    for (int q = t; q < hits * kGroups; q += kTopThreads) {
      const int at = ls.rank[q / kGroups], u = q % kGroups;
      const int mi = at / kTopThreads, ti = at % kTopThreads;
      const int mine = mi / p.iters, i = mi - mine * p.iters;
      const int it = rank + mine * C;
      const int w = it / p.slices, e0 = (it - w * p.slices) * p.slice;
      const int j = e0 + (i * kTopWarps + ti / kWarp) * kChunk + (u * kWarp + ti % kWarp) * VEC;
      if (j >= min(e0 + p.slice, p.V)) continue;
      const T* row = reinterpret_cast<const T*>(p.logits) + (grp * p.W + w) * (long long)p.V;
      const uint4 g = load_group<T, kAligned>(row, j, p.V, p.span);
      const float thr = threshold(w);
      unsigned in = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) in |= (Lane<T, VEC>::get(g, e) >= thr ? 1u : 0u) << e;
      if (in) {
        int o = atomicAdd(&lead->n_cands, __popc(in));
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (in >> e & 1u) {
            // the logit now, the key when the list is complete
            if (o < kMaxCands) {
              lead_ls->key[o] = __float_as_uint(Lane<T, VEC>::get(g, e));
              lead_ls->idx[o] = w * p.V + j + e;
            }
            ++o;
          }
      }
    }
  }
  if (C > 1) cluster.sync(); else __syncthreads();
  if (rank != 0) return;

  int count = s.n_cands;
  if (s.overflow || count > kMaxCands) {
    __syncthreads();
    count = 0;
    for (int w = 0; w < p.W; ++w) {
      const double off = kBeam ? s.off[w] : 0.0;
      if (off == -INFINITY) continue;
      const T* row = reinterpret_cast<const T*>(p.logits) + (grp * p.W + w) * (long long)p.V;
      const int got = select_row_slow<T, kBeam>(s, ls, row, p.V, p.n, off, w * p.V, count);
      // keep the n best of the rows so far (at most 2 n <= 256 entries, one a thread)
      const int total = count + got;
      rank_list<kBeam>(ls, total);
      const unsigned long long key = t < total ? ls.key[t] : 0;
      const int idx = t < total ? ls.idx[t] : 0, r = t < total ? ls.rank[t] : p.n;
      __syncthreads();
      if (r < p.n) {
        ls.key[r] = key;
        ls.idx[r] = idx;
      }
      count = min(total, p.n);
      __syncthreads();
    }
  } else {
    for (int i = t; i < count; i += kTopThreads) {
      const int idx = ls.idx[i];
      set_candidate<kBeam>(ls, i, __uint_as_float((uint32_t)ls.key[i]),
                           kBeam ? s.off[idx / p.V] : 0.0, idx);
    }
    __syncthreads();
    if (count > kRankAll) count = prune(s, ls, count, p.n);
  }
  rank_list<kBeam>(ls, count);
  for (int i = t; i < count; i += kTopThreads) {
    const int r = ls.rank[i];
    if (r < p.n) write_slot<kBeam>(p, grp, r, ls.key[i], ls.idx[i]);
  }
  for (int j = count + t; j < p.n; j += kTopThreads) write_slot<kBeam>(p, grp, j, 0, -1);
}

template <typename T>
constexpr int union_bytes() {
  return Ring<T>::kTotal > (int)sizeof(Lists) ? Ring<T>::kTotal : (int)sizeof(Lists);
}

template <typename T, bool kAligned, bool kBeam>
cudaError_t launch_top(const TopParams& p, long long groups, int C, cudaStream_t stream) {
  static PerDevice once;
  auto* fn = top_kernel<T, kAligned, kBeam>;
  const cudaError_t err = per_device(once, nullptr, [&](int&) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(TopShared) + kMaxTables * kTopThreads * 2 +
                                    union_bytes<T>());
  });
  if (err != cudaSuccess) return err;
  const size_t smem = sizeof(TopShared) + p.table_bytes + union_bytes<T>();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * C));
  cfg.blockDim = dim3(kTopThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <bool kBeam>
sv_status run_top(TopParams& p, sv_dtype dtype, long long groups, cudaStream_t stream) {
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return SV_ERR_CUDA;
  // The cluster: 8 CTAs while the rows do not fill the GPU by themselves (or
  // the row's group maxes need the shared memory of several), else one per row
  // (beams: one per beam, up to 8).
  int C = 1;
  while (C < 8 && C < p.W) C *= 2;
  while (C < 8 && (groups * C < 2LL * dev.sms ||
                   ((long long)p.W * ((p.V + kTopSpan - 1) / kTopSpan) + C - 1) / C > kMaxTables))
    C *= 2;
  p.slices = C > p.W ? C / p.W : 1;
  // no more slices than 256-element pieces
  const int pieces = (p.V + 255) / 256;
  p.slices = p.slices < pieces ? p.slices : pieces;
  p.slice = (pieces + p.slices - 1) / p.slices * 256;
  p.iters = (p.slice + kTopSpan - 1) / kTopSpan;
  const int items = p.W * p.slices;
  if (items > kMaxItems || (long long)((items + C - 1) / C) * p.iters > kMaxTables)
    return SV_ERR_SHAPE;
  // four units per kept candidate (or the finest there are), at least one a warp
  p.upi = kTopThreads;
  while (p.upi > kTopWarps && items * p.upi > kMaxUnits) p.upi /= 2;
  while (p.upi > kTopWarps && items * p.upi / 2 >= 4 * p.n) p.upi /= 2;
  p.table_bytes = (items + C - 1) / C * p.iters * kTopThreads * 2;
  const size_t esz = dtype == SV_BF16 ? 2 : 4;
  const char* first = static_cast<const char*>(p.logits);
  p.span.first = first;
  p.span.last = first + (size_t)groups * p.W * (size_t)p.V * esz;
  const bool aligned = ((uintptr_t)first & 15u) == 0 && ((size_t)p.V * esz) % 16 == 0;
  cudaError_t err;
  if (dtype == SV_BF16)
    err = aligned ? launch_top<uint16_t, true, kBeam>(p, groups, C, stream)
                  : launch_top<uint16_t, false, kBeam>(p, groups, C, stream);
  else
    err = aligned ? launch_top<float, true, kBeam>(p, groups, C, stream)
                  : launch_top<float, false, kBeam>(p, groups, C, stream);
  return err == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

sv_status spec_top_logits(const void* logits, int k, float temperature, const int32_t* lens,
                          int32_t* out_ids, float* out_logits, float* out_lse,
                          int32_t* out_status, sv_dtype dtype, int B, int P, int V,
                          sv_stream_t stream) {
  if (!(temperature > 0.f) || isinf(temperature)) return SV_ERR_TEMPERATURE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (B < 0 || B > SV_MAX_B || P < 1 || (long long)B * P > SV_MAX_ROWS || V < 1 || V > SV_MAX_V ||
      k < 1 || k > SV_MAX_TOP)
    return SV_ERR_SHAPE;
  if (B == 0) return SV_OK;
  if (!logits || !out_ids || !out_logits || !out_lse) return SV_ERR_NULL;
  if ((uintptr_t)logits & (dtype == SV_BF16 ? 1u : 3u)) return SV_ERR_NULL;
  TopParams p;
  memset(&p, 0, sizeof p);
  p.logits = logits;
  p.lens = lens;
  p.out_ids = out_ids;
  p.out_values = out_logits;
  p.out_lse = out_lse;
  p.out_status = out_status;
  p.P = P;
  p.W = 1;
  p.V = V;
  p.n = k;
  p.cc = exponent_scale(temperature);
  p.T = temperature;
  return run_top<false>(p, dtype, (long long)B * P, (cudaStream_t)stream);
}

sv_status spec_beam_select(const void* logits, const float* scores, int32_t* out_tokens,
                           int32_t* out_parents, float* out_scores, int32_t* out_status,
                           sv_dtype dtype, int B, int W, int V, int n, sv_stream_t stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (B < 0 || B > SV_MAX_B || W < 1 || W > SV_MAX_BEAMS || V < 1 || V > SV_MAX_V || n < 1 ||
      n > SV_MAX_TOP ||
      (long long)((W + 7) / 8) * ((V + kTopSpan - 1) / kTopSpan) > kMaxTables)
    return SV_ERR_SHAPE;
  if (B == 0) return SV_OK;
  if (!logits || !scores || !out_tokens || !out_parents || !out_scores) return SV_ERR_NULL;
  if ((uintptr_t)logits & (dtype == SV_BF16 ? 1u : 3u)) return SV_ERR_NULL;
  TopParams p;
  memset(&p, 0, sizeof p);
  p.logits = logits;
  p.scores = scores;
  p.out_ids = out_tokens;
  p.out_parents = out_parents;
  p.out_values = out_scores;
  p.out_status = out_status;
  p.P = 1;
  p.W = W;
  p.V = V;
  p.n = n;
  p.cc = 1.4426950408889634f;
  p.T = 1.f;
  return run_top<true>(p, dtype, B, (cudaStream_t)stream);
}

}  // extern "C"
