// sv_select.cuh - selection of the n largest values of streamed rows: the parts
// shared by the cluster kernel (sv_top.cu) and the row kernel (sv_toprows.cu).
//
// One pass over a row reads every logit once and keeps, per thread, a running
// softmax sum and max, and per 32 elements their max (rounded up to bf16, in
// shared memory).  The selection follows from the thread maxes alone: if
// `units` disjoint parts of the data have maxes u_1.., the n-th largest of
// them is a bound that at least n elements reach, so every kept element is at
// or above it, and little else is: with n of U parts occupied about
// U ln(U / (U - n)) elements (89 for n = 64 of 128).  Only the 32-element
// groups whose max reaches the bound are read again (from L2), their elements
// at or above it are listed, and the list is sorted by counting.  When large
// logits crowd at neighbouring tokens the list is longer (logits that fall with
// the token's id, 912 rows of 152064 bf16, k = 64: 54 us with a spread of 3 around
// the slope, 85 us with 1.5, against 51 us shuffled).  When the list does not fit
// (long rows of equal logits, sorted rows, steep slopes), each row is selected by
// radix descent on whole-number keys, 8 bits a pass, by one CTA: 1.3 ms a row of
// 152064 logits, 5.7 ms for 912.
#pragma once

#include <type_traits>

#include "../../include/spec_verify.h"
#include "sv_launch.h"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {

constexpr int kTopSpan = 8192;        // elements of a CTA's iteration: 32 a thread
constexpr int kMaxTables = 256;       // iterations of a CTA over its items: 512 bytes each
constexpr int kRowsSmem = 112 * 1024;  // shared memory of a CTA of the row kernel: two on an SM

struct TopParams {
  const void* logits;   // [B*P, V] (record) or [B*W, V] (beams)
  const int* lens;      // [B] or null (record)
  const float* scores;  // [B*W] (beams)
  int* out_ids;         // [rows, n] (record, row kernel), tokens [B, n] (beams)
  int* out_parents;     // beams: [B, n]
  float* out_values;    // logits [rows, n], scores [B, n]
  float* out_lse;       // record: [B*P]
  double* out_off;      // row kernel for beams: [B*W] offsets (-inf: no candidates, NaN: kOff*)
  float* out_max;       // and the rows' maxes
  int* out_status;
  int P;                // record: rows per request
  int W;                // rows per cluster (record: 1)
  int V, n;
  int slices, slice;    // slices per row, elements per slice (a multiple of 256)
  int iters;            // iterations per item
  int upi, fold;        // units per item (a multiple of 8), threads per unit
  int table_bytes;
  float cc;             // log2(e) / T
  float T;
  unsigned long long wait_ns;  // limit of the waits
  char* first;          // the logits' memory
  char* last;
};

// Whether rows of V logits fit the row kernel's shared memory.
bool top_rows_fit(int V);
// Rows one CTA each, as many CTAs as fit taking row after row (sv_toprows.cu).
cudaError_t launch_top_rows(sv_dtype dtype, bool aligned, TopParams p, long long rows,
                            cudaStream_t stream);
// The n best of each request's W row selections.
cudaError_t launch_beam_merge(const TopParams& p, const int* ids, const float* values,
                              const double* off, const float* row_max, int B,
                              cudaStream_t stream);

namespace {

constexpr int kTopThreads = 256;
constexpr int kTopWarps = kTopThreads / kWarp;
constexpr int kEntry = 32;            // elements of a table entry
// They are one piece of 32 consecutive elements (bf16) or two of 16 (fp32): a
// lane's 64 bytes of a 2 KB chunk, one chunk or two an entry.
template <typename T>
struct Piece {
  static constexpr int kPieces = (int)sizeof(T) / 2;
  static constexpr int kSize = kEntry / kPieces;
  static constexpr int kChunkSize = kSize * kWarp;  // elements of a chunk
  static constexpr int kWords = 4;                  // 16-byte words of a piece
};
// The element (of the slice) at which word q of an entry's kPieces * 4 starts;
// `threads` the streaming threads.
template <typename T>
__device__ __forceinline__ int entry_element(int entry, int q, int threads) {
  using P = Piece<T>;
  const int i = entry / threads, t = entry - i * threads;
  return ((i * P::kPieces + q / P::kWords) * threads + t) * P::kSize +
         q % P::kWords * Group<T>::VEC;
}
constexpr int kMaxUnits = 512;        // units per cluster
constexpr int kMaxCands = 1024;       // candidates of a cluster, 32-element groups of a CTA
constexpr int kRankAll = 384;         // lists longer than this are cut to the bound first

// A barrier of 256 threads: the whole CTA of the cluster kernel (barrier 0),
// the selecting part of the row kernel's. The form without .aligned: a warp
// may reach it in parts (after a branch of one lane), which the aligned form
// counts as a whole warp each.
template <int kBar>
__device__ __forceinline__ void group_sync() {
  if (kBar == 0) __syncthreads();
  else asm volatile("barrier.sync %0, 256;" ::"n"(kBar) : "memory");
}

// Scratch of a selection.
struct Select {
  unsigned hist[256];
  unsigned bound;  // ordered
  int n_hits, n_cands, overflow, bad, pick[4];
};

// The candidates.
struct alignas(16) Lists {
  unsigned long long key[kMaxCands + 4];  // record: (ordered logit, ~index), a total order;
                                      // beams: the ordered score, idx = w * V + v
  int idx[kMaxCands + 4];
  int rank[kMaxCands];                // until the list is sorted: the groups to read again
};
// Beams' also have their logits, in order: of a beam's tokens whose scores round to
// one 64-bit number (a score of -1e30, say) the larger logit is the better.
struct alignas(16) BeamLists : Lists {
  uint32_t logit[kMaxCands];
};
template <bool kBeam>
using ListOf = std::conditional_t<kBeam, BeamLists, Lists>;

// Load stages: each warp streams 2 KB chunks through its own ring by 16-byte
// asynchronous copies (a word more than a chunk, for rows off 16-byte
// boundaries); no barrier but the warp's own. 2 KB bulk copies into the same
// ring reached 5.2 TB/s where these reach 6.5 (912 and 2432 rows of 152064
// bf16 logits, the slope).
struct Ring {
  static constexpr int kBytes = 2048 + 16;
  static constexpr int kStages = 3;
  static constexpr int kWarpBytes = kBytes * kStages;
};

// Packed bf16 comparisons (1.0 where true) and additions.
__device__ __forceinline__ uint32_t gt_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The two halves of w that are >= those of thr, as bits 0 and 1.
__device__ __forceinline__ unsigned ge_bits_bf16x2(uint32_t w, uint32_t thr) {
  unsigned r;
  asm("{\n .reg .pred p, q;\n .reg .u32 h;\n setp.ge.bf16x2 p|q, %1, %2;\n"
      " selp.u32 %0, 1, 0, p;\n selp.u32 h, 2, 0, q;\n or.b32 %0, %0, h;\n}"
      : "=&r"(r)
      : "r"(w), "r"(thr));
  return r;
}

// The upper 16 bits of v rounded down: a bf16 value <= v (v itself for bf16).
__device__ __forceinline__ uint16_t down_bf16(float v) {
  const uint32_t b = __float_as_uint(v);
  return (uint16_t)((b & 0x80000000u) ? (b + 0xffffu) >> 16 : b >> 16);
}

// The upper 16 bits of v rounded up: a bf16 value >= v (v itself for bf16).
__device__ __forceinline__ uint16_t up_bf16(float v) {
  const uint32_t b = __float_as_uint(v);
  return (uint16_t)((b & 0x80000000u) ? b >> 16 : (b + 0xffffu) >> 16);
}

// The n-th largest of up to 512 units (bf16 values in unit[], rounded down);
// -inf when fewer than n are finite or there are fewer than n. A call of the
// group: each thread counts how many units are above its own, eight to a
// 16-byte word, two to an instruction (counts up to 256 are exact in bf16); the
// least unit with fewer than n above it is the bound.
template <int kBar>
__device__ float unit_bound(Select& s, const uint16_t* unit, int units, int n) {
  if (units < n) return -INFINITY;
  const int t = threadIdx.x % kTopThreads;
  if (t == 0) s.bound = 0xffffffffu;
  group_sync<kBar>();
  const uint4* words = reinterpret_cast<const uint4*>(unit);
  for (int i = t; i < units; i += kTopThreads) {
    const uint32_t mine = unit[i], both = mine | mine << 16;
    float above = 0.f;
    for (int w0 = 0; w0 < units / 8; w0 += 16) {  // units: a multiple of 8
      uint32_t a = 0, b = 0;                      // two bf16 counts each, up to 32
#pragma unroll 4
      for (int w = w0; w < min(w0 + 16, units / 8); ++w) {
        const uint4 v = words[w];
        a = add_bf16x2(a, add_bf16x2(gt_bf16x2(v.x, both), gt_bf16x2(v.y, both)));
        b = add_bf16x2(b, add_bf16x2(gt_bf16x2(v.z, both), gt_bf16x2(v.w, both)));
      }
      above += (bf16_lo(a) + bf16_hi(a)) + (bf16_lo(b) + bf16_hi(b));
    }
    if (above < (float)n) atomicMin(&s.bound, ordered(bf16_lo(mine)));
  }
  group_sync<kBar>();
  return of_ordered(s.bound);
}

// Offsets that are no number: a bad row or score, and a row whose wait ran out.
constexpr unsigned long long kOffBad = 0x7fffffffffffffffull, kOffLate = 0x7ff8000000000001ull;

// A beam's continuation scores offset + (l - m) in 64 bits, with m the row's max
// and offset = score - log of the row's sum in m's frame (as a pair): l - m
// first, so that rows of any magnitude keep their scores.
__device__ __forceinline__ double row_offset(float score, float2 log_sum) {
  return (double)score - ((double)log_sum.x + (double)log_sum.y);
}
__device__ __forceinline__ double beam_score(double off, float m, float l) {
  return off + ((double)l - (double)m);
}
__device__ __forceinline__ float beam_score_down(float off_down, float m, float l) {
  return __fadd_rd(off_down, __fadd_rd(l, -m));
}

constexpr int ring_bytes(int warps) { return Ring::kWarpBytes * warps; }

template <bool kBeam>
__device__ __forceinline__ void set_candidate(ListOf<kBeam>& s, int o, float l, double off,
                                              float m, int idx) {
  s.key[o] = kBeam ? ordered(beam_score(off, m, l))
                   : ((unsigned long long)ordered(l) << 32) | (uint32_t)~idx;
  s.idx[o] = idx;
  if constexpr (kBeam) s.logit[o] = ordered(l);
}

// One row's n largest finite elements by radix descent, appended to the list
// from `at` on (a call of the group); returns how many.
template <typename T, bool kBeam, int kBar>
__device__ int select_row_slow(Select& s, ListOf<kBeam>& ls, const T* row, int V, int n,
                               double off, float m, int base, int at) {
  const int t = threadIdx.x % kTopThreads;
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
    group_sync<kBar>();
    for (int j0 = 0; j0 < V; j0 += kTopThreads) {
      const unsigned long long k = key_of(j0 + t);
      const bool in = k != 0 && ((k ^ cut) >> (shift + 8)) == 0;
      const unsigned digit = in ? (unsigned)(k >> shift) & 255u : 256u;
      const unsigned peers = __match_any_sync(0xffffffffu, digit);
      if (in && lane_id() == __ffs(peers) - 1) atomicAdd(&s.hist[digit], (unsigned)__popc(peers));
    }
    group_sync<kBar>();
    if (t == 0) {
      int d = 255, above = 0;
      for (; d > 0 && above + (int)s.hist[d] < need; --d) above += (int)s.hist[d];
      s.pick[0] = d;
      s.pick[1] = above;
      s.pick[2] = (int)s.hist[d];
    }
    group_sync<kBar>();
    const int above = s.pick[1], here = s.pick[2];
    cut |= (unsigned long long)s.pick[0] << shift;
    group_sync<kBar>();
    if (above + here < need) {  // (first pass only) fewer than n finite elements: all of them
      all = true;
      break;
    }
    need -= above;
    if (here == need) break;  // every element of this prefix is kept
  }
  if (all) cut = 1;
  if (t == 0) s.pick[3] = at;
  group_sync<kBar>();
  for (int j0 = 0; j0 < V; j0 += kTopThreads) {
    const unsigned long long k = key_of(j0 + t);
    if (k != 0 && k >= cut) {
      const int o = atomicAdd(&s.pick[3], 1);
      set_candidate<kBeam>(ls, o, load_logit(row, j0 + t), off, m, base + j0 + t);
    }
  }
  group_sync<kBar>();
  return s.pick[3] - at;
}

// Whether entry j of a beam list comes before entry i of the same score: the
// earlier beam, in a beam the larger logit, of equal ones the lower token.
__device__ __forceinline__ bool tied_before(const BeamLists& s, int j, int i, int V) {
  const int a = s.idx[j], b = s.idx[i];
  const uint32_t x = s.logit[j], y = s.logit[i];
  return x == y || a / V != b / V ? a < b : x > y;
}

// rank[i] = the number of entries that come before entry i, i < count: the
// whole group, each entry's comparisons shared by 2^k neighbouring threads, four
// keys at a time (those past the list are 0: before none). The code runs once
// or a few times a launch: kept short, as its first run waits for instructions.
template <bool kBeam, int kBar>
__device__ void rank_list(ListOf<kBeam>& s, int count, int V) {
  const int t = threadIdx.x % kTopThreads;
  if (t < 4) s.key[count + t] = 0;
  group_sync<kBar>();
  const int k = min(5, max(0, __clz(count - 1) - 24)), way = t & ((1 << k) - 1);
  for (int i0 = 0; i0 < count; i0 += kTopThreads >> k) {
    const int i = i0 + (t >> k);
    const unsigned long long key = i < count ? s.key[i] : ~0ull;
    int r = 0;
#pragma unroll 1
    for (int j = 4 * way; j < count; j += 4 << k) {
      const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&s.key[j]);
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&s.key[j + 2]);
      r += (a.x > key) + (a.y > key) + (b.x > key) + (b.y > key);
      if constexpr (kBeam) {  // (seldom: scores equal to 64 bits)
        const int ties = (a.x == key) + (a.y == key) + (b.x == key) + (b.y == key);
        if (ties > ((unsigned)(i - j) < 4u ? 1 : 0)) {
#pragma unroll 1
          for (int q = j; q < j + 4; ++q)
            if (s.key[q] == key && tied_before(s, q, i, V)) ++r;
        }
      }
    }
    for (int o = 1; o < 1 << k; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (i < count && way == 0) s.rank[i] = r;
  }
  group_sync<kBar>();
}

// The n best of a list of at most 256 entries, to its front; returns how many.
template <bool kBeam, int kBar>
__device__ int keep_best(ListOf<kBeam>& ls, int total, int n, int V) {
  rank_list<kBeam, kBar>(ls, total, V);
  const int t = threadIdx.x % kTopThreads, r = t < total ? ls.rank[t] : n;
  const unsigned long long key = t < total ? ls.key[t] : 0;
  const int idx = t < total ? ls.idx[t] : 0;
  uint32_t logit = 0;
  if constexpr (kBeam) logit = t < total ? ls.logit[t] : 0;
  group_sync<kBar>();
  if (r < n) {
    ls.key[r] = key;
    ls.idx[r] = idx;
    if constexpr (kBeam) ls.logit[r] = logit;
  }
  group_sync<kBar>();
  return total < n ? total : n;
}

// Cuts the list to the entries at or above its n-th largest 32-bit key prefix.
template <bool kBeam, int kBar>
__device__ int prune(Select& s, ListOf<kBeam>& ls, int count, int n) {
  constexpr int kPer = kMaxCands / kTopThreads;
  const int tid = threadIdx.x % kTopThreads;
  unsigned long long k[kPer];
  int ix[kPer];
  uint32_t lx[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = q * kTopThreads + tid;
    k[q] = i < count ? ls.key[i] : 0ull;
    ix[q] = i < count ? ls.idx[i] : 0;
    if constexpr (kBeam) lx[q] = i < count ? ls.logit[i] : 0;
  }
  // Three counters in turn, one barrier a round. A round clears the counter of the next
  // one, last read before the barrier of the round before; the counter of the round
  // before may still be read by other warps.
  if (tid < 3) s.pick[tid] = 0;
  group_sync<kBar>();
  uint32_t t = 0;
  int now = 0;
  for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
    const uint32_t at = t | bit;
    unsigned c = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) c += (uint32_t)(k[q] >> 32) >= at ? 1u : 0u;
    c = __reduce_add_sync(0xffffffffu, c);
    const int next = now == 2 ? 0 : now + 1;
    if (lane_id() == 0) atomicAdd(&s.pick[now], (int)c);
    if (tid == 0) s.pick[next] = 0;
    group_sync<kBar>();
    if (s.pick[now] >= n) t = at;
    now = next;
  }
  group_sync<kBar>();
  if (tid == 0) s.pick[1] = 0;
  group_sync<kBar>();
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (q * kTopThreads + tid < count && (uint32_t)(k[q] >> 32) >= t) {
      const int o = atomicAdd(&s.pick[1], 1);
      ls.key[o] = k[q];
      ls.idx[o] = ix[q];
      if constexpr (kBeam) ls.logit[o] = lx[q];
    }
  group_sync<kBar>();
  return s.pick[1];
}

// One pass of kWarps warps over elements e0 .. e1 - 1 of a row: the thread's
// running sum, and at table[i * kWarps * 32] the max of its entry of iteration
// i (chunk c of the slice is warp c % kWarps').
template <typename T, bool kAligned, int kWarps>
__device__ __forceinline__ RunningSum stream_slice(uint32_t ring, int warp, const T* row, int e0,
                                                   int e1, int iters, float c, uint16_t* table,
                                                   const RowSpan& span) {
  constexpr int VEC = Group<T>::VEC;
  using P = Piece<T>;
  const int lane = lane_id();
  const T* tag = nullptr;
  const int chunks = (e1 - e0 + P::kChunkSize - 1) / P::kChunkSize;
  const int todo = (chunks - warp + kWarps - 1) / kWarps;  // this warp's (may be <= 0)
  const uint32_t off = kAligned ? 0u : (uint32_t)(uintptr_t)row & 15u;
  ring += warp * Ring::kWarpBytes;
  auto issue = [&](int i) {  // this warp's chunk i into its stage
    if (i < todo) {
      const int j = e0 + (i * kWarps + warp) * P::kChunkSize;
      load_chunk_async<T, kAligned>(ring + i % Ring::kStages * Ring::kBytes, row, j,
                                    min(j + P::kChunkSize, e1), off, span);
    }
    copies_commit();
  };
  RunningSum r;
  // the chunks, kShift words from where the row's misalignment puts them
  auto pass = [&](auto kShift) {
    float entry = -INFINITY;
    for (int i = 0; i < iters * P::kPieces; ++i) {
      float gm = -INFINITY;
      if (i < todo) {
        copies_wait_but<Ring::kStages - 2>();
        __syncwarp();  // every lane's copies of this stage landed; the stage before is read
        issue(i + Ring::kStages - 1);
        const uint32_t stage = ring + i % Ring::kStages * Ring::kBytes + lane * 64;
        const int j = e0 + (i * kWarps + warp) * P::kChunkSize + lane * P::kSize;
        uint4 g[P::kWords];
#pragma unroll
        for (int u = 0; u < P::kWords; ++u) {
          // the lane's words in an order that keeps a quarter warp off each other's banks
          const uint32_t at = stage + ((u + (lane >> 1)) & (P::kWords - 1)) * 16;
          g[u] = lds128(at);
          if (!kAligned && off) g[u] = shift_words<kShift.value>(g[u], lds128(at + 16), off * 8);
        }
        if (e0 + (i * kWarps + warp + 1) * P::kChunkSize > e1) {
#pragma unroll
          for (int u = 0; u < P::kWords; ++u)
            clip_group<T>(g[u], j + ((u + (lane >> 1)) & (P::kWords - 1)) * VEC, e1);
        }
        gm = r.add(g, c, tag);
      }
      if (P::kPieces == 1) {
        table[i * kWarps * kWarp] = up_bf16(gm);
      } else if ((i & 1) == 0) {
        entry = gm;
      } else {
        table[(i >> 1) * kWarps * kWarp] = up_bf16(max_nan(entry, gm));
      }
    }
  };
#pragma unroll
  for (int i = 0; i < Ring::kStages - 1; ++i) issue(i);
  // one copy of the loop a shift: the words then need no selection in registers
  if (kAligned || off < 4) pass(Shift<0>());
  else if (off < 8) pass(Shift<1>());
  else if (off < 12) pass(Shift<2>());
  else pass(Shift<3>());
  __syncwarp();  // (the next slice refills the stages)
  return r;
}

// The table entries at or above thr, eight a thread and step, as `base` plus
// their number in rank[] (at most kMaxCands; n_hits counts all).
__device__ __forceinline__ void scan_table(Select& s, Lists& ls, const uint16_t* table,
                                           int entries, float thr, int base) {
  const uint32_t up = up_bf16(thr), both = up | up << 16;  // entry >= thr: entry >= thr rounded up
  for (int v = threadIdx.x % kTopThreads; v < entries / 8; v += kTopThreads) {
    const uint4 e = load128(table + 8 * v);
    unsigned hits = ge_bits_bf16x2(e.x, both) | ge_bits_bf16x2(e.y, both) << 2 |
                    ge_bits_bf16x2(e.z, both) << 4 | ge_bits_bf16x2(e.w, both) << 6;
    if (hits) {
      int h = atomicAdd(&s.n_hits, __popc(hits));
      for (; hits; hits &= hits - 1u, ++h)
        if (h < kMaxCands) ls.rank[h] = base + 8 * v + __ffs(hits) - 1;
    }
  }
}

// The elements of a group at or above thr go to a list: a record's keys as they
// are, for beams the logit now and the key when the list is complete.
template <typename T, bool kBeam>
__device__ __forceinline__ void list_group(int* n_cands, Lists* to, const uint4& g, float thr,
                                           int idx) {
  constexpr int VEC = Group<T>::VEC;
  unsigned in = 0;
#pragma unroll
  for (int e = 0; e < VEC; ++e) in |= (Lane<T, VEC>::get(g, e) >= thr ? 1u : 0u) << e;
  if (!in) return;
  int o = atomicAdd(n_cands, __popc(in));
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    if (in >> e & 1u) {
      if (o < kMaxCands) {
        const float l = Lane<T, VEC>::get(g, e);
        to->key[o] = kBeam ? __float_as_uint(l)
                           : ((unsigned long long)ordered(l) << 32) | (uint32_t)~(idx + e);
        to->idx[o] = idx + e;
      }
      ++o;
    }
}

// A row's {max, sum as a pair} from its warps' parts (one warp, up to 64 parts).
__device__ __forceinline__ float row_sum(const float2* parts, int n, float c, float2& sum) {
  const int lane = lane_id();
  const float2 a = lane < n ? parts[lane] : make_float2(-INFINITY, 0.f);
  const float2 b = lane + kWarp < n ? parts[lane + kWarp] : make_float2(-INFINITY, 0.f);
  const float m = warp_max_nan(max_nan(a.x, b.x));
  sum = warp_sum_pair(a.y * to_frame(a.x, m, c) + b.y * to_frame(b.x, m, c));
  return m;
}

// Units of `fold` threads: two per kept candidate, counting only the threads
// that a slice gives anything (its 2 KB chunks go to the warps in turn); padded
// to a multiple of 8 per item (the idle threads' -inf), at most kMaxUnits in
// all (64 items of 8 fit).
inline void set_units(TopParams& p, sv_dtype dtype, int items, int slice, int threads) {
  const int chunk = dtype == SV_BF16 ? Piece<uint16_t>::kChunkSize : Piece<float>::kChunkSize;
  const int chunks = (slice + chunk - 1) / chunk;
  const int busy = chunks * kWarp < threads ? chunks * kWarp : threads;
  const auto units = [&](int fold) { return (busy + fold - 1) / fold; };
  const auto padded = [&](int fold) { return (units(fold) + 7) / 8 * 8; };
  p.fold = 1;
  while (p.fold < kWarp &&
         (items * padded(p.fold) > kMaxUnits || items * units(2 * p.fold) >= 2 * p.n))
    p.fold *= 2;
  p.upi = padded(p.fold);
}

}  // namespace
}  // namespace sv
