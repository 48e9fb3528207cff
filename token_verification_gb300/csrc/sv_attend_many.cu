// sv_attend_many.cu - attention over the 4-bit cache for many query rows
// (spec_cache_attention): tensor memory and tcgen05 instructions.
//
// A unit is a tile of 32 or 48 query rows of a key/value head (tokens of the step times the
// heads of the group), a chunk 128 slots, which takes
//   S^T = K Q^T    128 slots x rows x D, both operands in shared memory
//   O^T += V^T P^T  D x rows x 128 slots, values and weights P in shared memory
// in fp16 with 32-bit sums in tensor memory.  Slots and dimensions lie on the instruction's side of
// 128, so a tile of few rows costs what its rows cost (rows on that side would count as 128
// each time).  Decoded keys and values are exact in fp16; a row of Q is scaled by a power of two
// (exact), weights are rounded to 2^-11.  One CTA an SM works on two shares of the call side by
// side; of each
//   4 warps  do the softmax, a thread a slot: its scores of every row from tensor memory, weights
//            to shared memory;
//   4 warps  decode the chunk's keys, then its values, a chunk ahead in registers.  Both lie as
//            rows of a slot, 64 dimensions (128 bytes) a block, 128-byte swizzle: K-major for the
//            keys, MN-major for the values;
//   1 warp   issues the tensor instructions: S of the next chunk before O of this one;
//   1 warp   finds the pages of the chunks ahead and brings the pieces' Q.
// The keys of a chunk are decoded while the one before is in the softmax, its values while the
// tensor pipe and the softmax work on its scores; what is left of a share's waits the other fills.
// A row's weights are relative to a reference that follows its running max only when a
// score exceeds it by 2^8: the weights, at most 2^15 then, stay within fp16, and the
// threads, which hold one slot of every row, need to agree on a row's max (and to rescale O in
// tensor memory) a few times a piece instead of every chunk.
//
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/spec_verify.h"
#include "sv_attend.cuh"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

constexpr int kManyThreads = 640;
constexpr int kSides = 2;  // shares of a CTA
constexpr int kSlotsTile = 128;
constexpr float kManyShift = 7.f, kSlack = 8.f;
constexpr float kNoRef = 3e38f;  // in place of shift - max for a row without a score yet
constexpr int kTmemCols = 512;
constexpr int kSideCols = 256;
constexpr int kOCol = 128;  // O's columns; S: 0 and 64

// ---- tcgen05 -------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
               "n"(kTmemCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(kTmemCols));
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_loaded() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
// Waits as a warp: all lanes answer alike.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned long long limit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit));
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Shared-memory descriptors: 128-byte swizzle, version 1.  Keys and queries (K-major): 8 rows of 128
// bytes every 1024.  Values (MN-major): 64 dimensions a block, blocks 16384 bytes
// apart, 8 slots every 1024.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t kBlockBytes = 128 * 128;  // 128 rows or slots of 64 dimensions
// Instruction: fp32 results, fp16 operands, M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool mn_major) {
  return 1u << 4 | (mn_major ? 3u << 15 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}

// A chunk ahead: addresses of each 16 slots' key codes (0: no such page) and key scales, and
// which of its slots are seen by anybody (first <= slot in the chunk < last).
constexpr int kRefs = 4;
struct ChunkRef {
  unsigned long long codes[8], scales[8];
  int first, last;
};

template <int D, int NC>
struct Side {
  static constexpr int kTileBytes = D / 64 * (int)kBlockBytes;
  alignas(1024) char v[kTileBytes];  // (first: at D = 64 a descriptor reaches one tile on)
  alignas(1024) char k[kTileBytes];
  alignas(1024) char p[kBlockBytes];  // weights [slot][64 rows]; a finished piece's rows
  alignas(1024) char q[D / 64 * NC * 128];
  // the piece's rows, brought with Q: a score's factor, the step's token, its row of `out`
  // counted from the request's first, a slope
  float unscale[NC], slope[NC];
  int node[NC], out_row[NC];
  // {factor, factor, shift - reference, the same} of pairs of rows, the reference, the last
  // change of it, 1 / sum, positions; what the warps leave to be joined
  alignas(16) float4 fo[NC / 2];
  alignas(16) float m[NC], change[NC], inv[NC];
  int pos[NC];
  float part[4][NC];
  // completed by: k_full, v_full the decoding warps; qk_done, pv_done the tensor pipe (which then no
  // longer needs the keys, or the values and the weights); p_full the softmax (weights
  // in place); q_full and ref_full the last warp; q_empty the tensor pipe and the softmax
  alignas(8) unsigned long long k_full, v_full, qk_done[2], pv_done, p_full, q_full, q_empty, drained;
  unsigned long long ref_full[kRefs], ref_empty[kRefs];  // (empty: the decoding warps)
  ChunkRef refs[kRefs];
};
template <int D, int NC>
struct ManySmem {
  Side<D, NC> side[kSides];
  uint32_t tmem;
  int late;
  long long scan[kManyThreads / 32 + 2 * kSides];
};
template <int D, int NC>
constexpr size_t many_smem(bool tree) {
  // (more than half of an SM's: one CTA an SM, as tensor memory needs)
  return std::max((size_t)120 * 1024, 1024 + (sizeof(ManySmem<D, NC>) + 15) / 16 * 16) + (tree ? kSides * sizeof(TreeView) : 0);
}

// Barriers of the softmax warps.
__device__ __forceinline__ void meet(int barrier) {
  asm volatile("bar.sync %0, 128;" ::"r"(barrier) : "memory");
}
__device__ __forceinline__ bool any_of_them(bool x, int barrier) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(barrier)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_top(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// A decoding thread's part of a chunk: kU rows of one group of 32 values.
template <int D>
struct Part {
  static constexpr int kU = D / 32;
  uint4 w[kU];
  uint32_t scale[kU];  // bytes
  uint32_t off;        // bit i: row i counts as NaN (keys) or 0 (values), whatever its byte
};

// Loads that nothing waits for until their registers are used: where `ok`, else zeros.
__device__ __forceinline__ uint4 load16_if(const char* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n"
      " mov.u32 %2, 0;\n mov.u32 %3, 0;\n @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)ok));
  return v;
}
__device__ __forceinline__ uint32_t load_byte_if(const char* p, bool ok) {
  uint32_t v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.u32 %0, 0;\n"
      " @p ld.global.u8 %0, [%1];\n}"
      : "=&r"(v)
      : "l"(p), "r"((uint32_t)ok));
  return v;
}

// Row `row` of the head's `rows`: its values to row `at` of Q, and its constants.
template <int D, int NC>
__device__ __forceinline__ void bring_row(const AttendParams& p, const Walk& w, int row, int rows,
                                          int at, Side<D, NC>& sm) {
  const bool ok = row < rows && w.r.ok;
  const int clamped = min(row, max(rows - 1, 0));
  const int i = clamped / p.group, head = w.h * p.group + clamped - i * p.group;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                    w.b * p.qb + i * p.qn + (long long)head * p.qh);
  uint32_t top2 = 0;
#pragma unroll 4
  for (int x = 0; x < D / 8; ++x) {
    const uint4 v = ok ? src[x] : make_uint4(0, 0, 0, 0);
    // (magnitudes of bf16 order as whole numbers)
    top2 = __vmaxu2(__vmaxu2(top2, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
    top2 = __vmaxu2(__vmaxu2(top2, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
  }
  const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  const int e = min(max((int)(top >> 7) - 127, -98), 126);
  float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
  if (top >= 0x7f80u) up = qnan();  // (a row with NaN or infinity is NaN)
  if (p.scale < 0.f) up = -up;
  sm.unscale[at] = __uint_as_float((uint32_t)(127 + e - 14) << 23) * fabsf(p.scale) *
                   (p.softcap > 0.f ? 1.f / p.softcap : kLog2e);
  sm.slope[at] = p.slopes ? p.slopes[head] * kLog2e : 0.f;
  sm.node[at] = i;
  sm.out_row[at] = i * p.Hq + head;
#pragma unroll 4
  for (int x = 0; x < D / 8; ++x) {
    const uint4 v = ok ? src[x] : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(sm.q + (x / 8) * (NC * 128) + at * 128 +
                              (((x & 7) ^ (at & 7)) << 4)) =
        make_uint4(pack_f16(bf16_lo(v.x) * up, bf16_hi(v.x) * up),
                   pack_f16(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                   pack_f16(bf16_lo(v.z) * up, bf16_hi(v.z) * up),
                   pack_f16(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
  }
}

template <int D, int NC>
__global__ void __launch_bounds__(kManyThreads, 1) many_kernel(const AttendParams p) {
  extern __shared__ __align__(16) char many_raw[];
  ManySmem<D, NC>& all = *reinterpret_cast<ManySmem<D, NC>*>(
      many_raw + ((1024 - (smem_u32(many_raw) & 1023)) & 1023));
  constexpr int G = D / 32;  // groups of a row
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  // warps 0-7 softmax, 8-15 decoding (four a side), 16, 17 tensor pipe, 18, 19 the rest
  const int side = warp < 16 ? warp / 4 & 1 : warp & 1;
  Side<D, NC>& sm = all.side[side];
  TreeView& tree = reinterpret_cast<TreeView*>(reinterpret_cast<char*>(&all) +
                                               (sizeof(all) + 15) / 16 * 16)[side];  // (if p.parent)
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSides; ++i) {
      Side<D, NC>& x = all.side[i];
      mbar_init(smem_u32(&x.k_full), 4);
      mbar_init(smem_u32(&x.v_full), 4);
      mbar_init(smem_u32(&x.qk_done[0]), 1);
      mbar_init(smem_u32(&x.qk_done[1]), 1);
      mbar_init(smem_u32(&x.pv_done), 1);
      mbar_init(smem_u32(&x.p_full), 128);
      mbar_init(smem_u32(&x.q_full), 32);
      mbar_init(smem_u32(&x.q_empty), 1 + 128);
      mbar_init(smem_u32(&x.drained), 1);
      for (int k = 0; k < kRefs; ++k) {
        mbar_init(smem_u32(&x.ref_full[k]), 1);
        mbar_init(smem_u32(&x.ref_empty[k]), 4);
      }
    }
    fence_mbar_init();
    all.late = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  // (shares 0 .. gridDim.x - 1 first: few of them go to as many SMs)
  const int ctas[kSides] = {(int)blockIdx.x, (int)(blockIdx.x + gridDim.x)};
  const int cta = ctas[side];
  const Share share =
      find_share<kManyThreads>(p, ctas, side, kSides * (int)gridDim.x, all.scan);
  if (threadIdx.x < kSides) {
    p.desc[4 * ctas[threadIdx.x] + 3] = 0;
    if (ctas[0] >= share.G) p.late[ctas[threadIdx.x]] = 0;
  }
  if (ctas[0] >= share.G) return;
  if (warp == 16) tmem_alloc(smem_u32(&all.tmem));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = all.tmem + side * kSideCols;
  const unsigned long long limit = p.wait_ns;
  const bool has = cta < share.G;  // a share at all
  auto bar = [](unsigned long long& b) { return smem_u32(&b); };

  if (warp < 8) {
    // ---- softmax: thread = slot of the chunk, or dimension, = lane of tensor memory
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    const int tid = threadIdx.x & 127, quarter = warp & 3, barrier = 2 + side;
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16);
    Walk w(p, share, has);
    unsigned j = 0, piece = 0;  // chunks and pieces so far
    bool late = false;
    const float cap = p.softcap * kLog2e;
    while (w.left > 0) {
      const int b = w.b, h = w.h, c0 = w.c;
      const Request r = w.r;
      const int c1 = (int)min((long long)r.chunks, c0 + w.left);
      const int row0 = w.tile * NC, n_rows = min(NC, r.nq * p.group - row0);
      bool sees = r.ok && r.len > 0;
      if (p.parent && sees) sees = build_tree<128>(p, b, r.nq, tree, tid, barrier);
      late = late || !warp_wait(bar(sm.q_full), piece & 1, limit);
      ++piece;
      // the piece's rows
      if (tid < NC) {
        const float f = sm.unscale[tid];
        float* fo = reinterpret_cast<float*>(&sm.fo[tid / 2]);
        fo[tid & 1] = f;
        fo[2 + (tid & 1)] = kNoRef;
        sm.m[tid] = -INFINITY;
        const int node = sm.node[tid];
        sm.pos[tid] = r.base + (p.parent && sees ? tree.depth[node] : node);
      }
      f32x2 l[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l[i] = pack2(0.f, 0.f);
      meet(barrier);
      for (int c = c0; c < c1; ++c, ++j) {
        const uint32_t s_at = mine + (j & 1) * 64;
        late = late || !warp_wait(bar(sm.qk_done[j & 1]), j >> 1 & 1, limit);
        // (a wait that ran out leaves numbers without meaning, and the four warps in step)
        fence_after();
        const int slot0 = (r.lo / kSlotsTile + c) * kSlotsTile, slot = slot0 + tid;
        const bool edge = !sees || slot0 + kSlotsTile > r.base ||
                          (p.window > 0 && slot0 <= r.base + r.nq - 1 - p.window);
        const bool plain = !edge && p.softcap == 0.f && !p.slopes;
        // scores in units of log2, before the rows' factors where plain
        float s[NC];
        auto load_scores = [&] {
#pragma unroll
          for (int i = 0; i < NC / 16; ++i)
            tmem_load16(s_at + 16 * i, reinterpret_cast<uint32_t*>(s) + 16 * i);
          tmem_loaded();
          if (plain) return;
          const bool there = sees && slot < r.len;
          const int node = slot - r.base;
          int at = slot;
          if (p.parent && there && node >= 0) at = r.base + tree.depth[node];
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float y = s[i] * reinterpret_cast<const float*>(&sm.fo[i / 2])[i & 1];
            if (p.softcap > 0.f) y = cap_of<false>(cap, y);
            if (p.slopes) y = fmaf(-sm.slope[i], (float)(sm.pos[i] - at), y);
            s[i] = y;
          }
          if (!edge) return;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            bool seen = there;
            if (there && node >= 0) {
              const int mine_node = sm.node[i];
              seen = p.parent ? tree.seen[mine_node][node >> 5] >> (node & 31) & 1
                              : node <= mine_node;
            }
            if (p.window > 0 && sm.pos[i] - at >= p.window) seen = false;
            if (!seen) s[i] = -INFINITY;
          }
        };
        for (;;) {
          load_scores();
          // exponents of the weights; is one too large for its row's reference?
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) {
            const float4 fo = sm.fo[i];
            const f32x2 f = plain ? pack2(fo.x, fo.y) : pack2(1.f, 1.f);
            unpack2(fma2(pack2(s[2 * i], s[2 * i + 1]), f, pack2(fo.z, fo.w)), s[2 * i],
                    s[2 * i + 1]);
            top[i & 3] = max3(top[i & 3], s[2 * i], s[2 * i + 1]);
          }
          if (!any_of_them(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) >
                           kManyShift + kSlack, barrier))
            break;
          // each row's max over the chunk's slots
          load_scores();
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float y = s[i];
            if (plain) y *= reinterpret_cast<const float*>(&sm.fo[i / 2])[i & 1];
            y = warp_top(y);
            if (lane == (i & 31)) sm.part[quarter][i] = y;
          }
          meet(barrier);
          if (tid < NC) {
            const float old = sm.m[tid];
            const float m = fmaxf(fmaxf(old, sm.part[0][tid]),
                                  max3(sm.part[1][tid], sm.part[2][tid], sm.part[3][tid]));
            sm.m[tid] = m;
            sm.change[tid] = old == -INFINITY ? 0.f : ex2(old - m);
            reinterpret_cast<float*>(&sm.fo[tid / 2])[2 + (tid & 1)] =
                m == -INFINITY ? kNoRef : kManyShift - m;
          }
          meet(barrier);
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) {
            const float2 g = *reinterpret_cast<const float2*>(&sm.change[2 * i]);
            l[i] = fma2(l[i], pack2(g.x, g.y), pack2(0.f, 0.f));
          }
          if (c > c0) {  // O so far
            late = late || !warp_wait(bar(sm.pv_done), (j - 1) & 1, limit);
            fence_after();
#pragma unroll
            for (int i = 0; i < NC / 16; ++i) {
              uint32_t o[16];
              tmem_load16(mine + kOCol + 16 * i, o);
              tmem_loaded();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * sm.change[16 * i + e]);
              tmem_store16(mine + kOCol + 16 * i, o);
            }
            tmem_stored();
          }
        }
        if (j > 0) late = late || !warp_wait(bar(sm.pv_done), (j - 1) & 1, limit);
        char* to = sm.p + tid * 128;
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w0 = ex2(s[8 * i + 2 * e]), w1 = ex2(s[8 * i + 2 * e + 1]);
            l[4 * i + e] = add2(l[4 * i + e], pack2(w0, w1));
            x[e] = pack_f16(w0, w1);
          }
          *reinterpret_cast<uint4*>(to + ((i ^ (tid & 7)) << 4)) =
              make_uint4(x[0], x[1], x[2], x[3]);
        }
        fence_proxy_async();
        fence_before();
        bar_arrive(bar(sm.p_full));
      }
      const bool whole = c0 == 0 && c1 == r.chunks;
      const bool first = w.left == share.end - share.begin;
      float* part = p.part + (long long)(2 * cta + (first ? 0 : 1)) * NC * (D + 4);
      const long long out0 = (long long)b * p.N * p.Hq;
      late = late || !warp_wait(bar(sm.pv_done), (j - 1) & 1, limit);
      fence_after();
      // the rows' sums over the slots, by way of the weights' place
      float* sums = reinterpret_cast<float*>(sm.p);
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) {
        float x, y;
        unpack2(l[i], x, y);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (lane < 16) *reinterpret_cast<float2*>(&sums[(quarter * 16 + lane) * NC + 2 * i]) = make_float2(x, y);
      }
      if (any_of_them(late, barrier)) late = true;
      if (tid < 2 * NC) {
        float sum = 0.f;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) sum += sums[(tid / NC * 32 + i) * NC + tid % NC];
        sm.part[tid / NC][tid % NC] = sum;
      }
      meet(barrier);
      if (tid < NC) {
        float sum = sm.part[0][tid] + sm.part[1][tid];
        if (late) sum = qnan();
        sm.inv[tid] = sum == 0.f ? 0.f : 1.f / sum;
        if (tid < n_rows) {
          if (!whole) {
            part[tid * (D + 4) + D] = sm.m[tid];
            part[tid * (D + 4) + D + 1] = sum;
          } else if (p.out_lse) {
            p.out_lse[out0 + sm.out_row[tid]] =
                sum == 0.f ? -INFINITY : (sm.m[tid] - kManyShift + log2f(sum)) * 0.6931471805599453f;
          }
        }
      }
      meet(barrier);
      uint16_t* rows_out = reinterpret_cast<uint16_t*>(sm.p);  // [row][D], as bf16
      if (D == 128 || quarter < 2) {
#pragma unroll
        for (int i = 0; i < NC / 16; ++i) {
          uint32_t o[16];
          tmem_load16(mine + kOCol + 16 * i, o);
          tmem_loaded();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int row = 16 * i + e;
            float x = late ? qnan() : __uint_as_float(o[e]);
            if (!whole) {
              if (row < n_rows) part[row * (D + 4) + tid] = x;
            } else {
              const float inv = sm.inv[row];
              x = inv == 0.f ? 0.f : x * inv;
              rows_out[row * D + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
            }
          }
        }
      }
      if (whole) {
        meet(barrier);
        constexpr int kPer = D / 8;  // 16-byte units of a row
        for (int i = tid; i < n_rows * kPer; i += 128)
          reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                   (out0 + sm.out_row[i / kPer]) * D)[i % kPer] =
              reinterpret_cast<const uint4*>(rows_out)[i];
      }
      fence_before();
      bar_arrive(bar(sm.q_empty));
      if (!whole && c0 == 0 && tid == 0) {
        int* desc = p.desc + 4 * cta;
        desc[0] = b;
        desc[1] = h;
        desc[2] = w.tile | (first ? 0 : 1 << 30);
        desc[3] = pieces_of(share, cta, share.end - w.left + r.chunks);
      }
      meet(barrier);  // (the rows' constants are read)
      // (pieces behind a wait that ran out are written as NaN)
      w.left -= c1 - c0;
      w.c = c1;
      if (c1 == r.chunks) w.next_unit(p);
    }
    if (late) all.late = 1;
  } else if (warp < 16) {
    // ---- decoding.  A thread takes kU rows of one group of 32 values, of keys and values alike.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    constexpr int kU = G;
    const int u = threadIdx.x & 127, r8 = u & 7, g = (u >> 3) % G, blk = (u >> 3) / G;
    const int block = page_bytes(1, D) << p.cache.shift;
    const int code_at = r8 * (D / 2) + g * 16, scale_off = g * 16 + r8;
    const unsigned n = (unsigned)(share.end - share.begin);
    bool late = false;
    auto load = [&](unsigned j, bool values, Part<D>& x) {  // of chunk j
      const ChunkRef& ref = sm.refs[j % kRefs];
      const int more = values ? block : 0, first = ref.first, last = ref.last;
      x.off = 0;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int b8 = blk + 16 / G * i;  // the row's 8 slots
        const char* codes = reinterpret_cast<const char*>(ref.codes[b8 >> 1]);
        const char* bytes = reinterpret_cast<const char*>(ref.scales[b8 >> 1]);
        const bool ok = codes != nullptr;
        const int slot = 8 * b8 + r8;
        x.w[i] = load16_if(codes + (more + code_at + (b8 & 1) * 4 * D), ok);
        x.scale[i] = load_byte_if(bytes + (more + scale_off + (b8 & 1) * 8), ok);
        x.off |= (!ok || (values && (slot < first || slot >= last)) ? 1u : 0u) << i;
      }
    };
    auto put = [&](const Part<D>& x, bool values) {
      char* tile = (values ? sm.v : sm.k) + (g >> 1) * kBlockBytes;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        Scale2 sc;
        const uint32_t half = x.off >> i & 1 ? (values ? 0u : 0x7fffu) : x.scale[i] * 128u + 0x400u;
        sc.set(half * 0x10001u);
        char* row = tile + (8 * (blk + 16 / G * i) + r8) * 128;
        const uint32_t words[4] = {x.w[i].x, x.w[i].y, x.w[i].z, x.w[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t d[4];
          decode_word(words[q], sc, d);
          *reinterpret_cast<uint4*>(row + ((((g & 1) * 4 + q) ^ r8) << 4)) =
              make_uint4(d[0], d[1], d[2], d[3]);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) bar_arrive(bar(values ? sm.v_full : sm.k_full));
    };
    Part<D> keys, vals;
    if (n > 0) late = !warp_wait(bar(sm.ref_full[0]), 0, limit);
    if (n > 0 && !late) {
      load(0, false, keys);
      load(0, true, vals);
    }
    for (unsigned j = 0; j < n && !late; ++j) {
      if (j > 0) late = !warp_wait(bar(sm.qk_done[(j - 1) & 1]), (j - 1) >> 1 & 1, limit);
      if (late) break;
      put(keys, false);
      const bool more = j + 1 < n;
      if (more) {
        late = !warp_wait(bar(sm.ref_full[(j + 1) % kRefs]), (j + 1) / kRefs & 1, limit);
        if (late) break;
        load(j + 1, false, keys);
      }
      if (j > 0) late = !warp_wait(bar(sm.pv_done), (j - 1) & 1, limit);
      if (late) break;
      put(vals, true);
      if (more) {
        load(j + 1, true, vals);
        __syncwarp();
        if (lane == 0) bar_arrive(bar(sm.ref_empty[(j + 1) % kRefs]));
      }
      if (j == 0 && lane == 0) bar_arrive(bar(sm.ref_empty[0]));
    }
    if (late) all.late = 1;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp < 18) {
      // ---- the tensor pipe.  The warp walks together, so that addresses and descriptors are
      // uniform; one elected lane issues.
      Walk w(p, share, has);
      const long long n = w.left;
      unsigned piece = 0;
      bool late = false;
      const uint64_t q = smem_desc(smem_u32(sm.q), 16), k = smem_desc(smem_u32(sm.k), 16);
      const uint64_t v = smem_desc(smem_u32(sm.v), kBlockBytes);
      const uint64_t pw = smem_desc(smem_u32(sm.p), kBlockBytes);
      auto score = [&](unsigned j) {  // S of the chunk that `w` stands at; w steps on
        if (j == 0 || w.c == 0) {     // a piece starts
          if (j > 0) ++piece;
          late = late || !warp_wait(bar(sm.q_full), piece & 1, limit);
        }
        late = late || !warp_wait(bar(sm.k_full), j & 1, limit);
        if (late) return;
        fence_after();
        w.step(p);
        const bool ends = w.left == 0 || w.c == 0;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_ss(tmem + (j & 1) * 64, k + ((i / 4) * kBlockBytes + (i % 4) * 32 >> 4),
                   q + ((i / 4) * (NC * 128) + (i % 4) * 32 >> 4), idesc(NC, false), i > 0);
          mma_commit(bar(sm.qk_done[j & 1]));
          if (ends) mma_commit(bar(sm.q_empty));
        }
        __syncwarp();
      };
      bool starts = true;  // chunk j is its piece's first
      if (n > 0) score(0);
      for (unsigned j = 0; j < n && !late; ++j) {
        // (the next piece's Q comes when this one's rows are out, behind its last O)
        const bool next_starts = w.c == 0;
        if (j + 1 < n && !next_starts) score(j + 1);
        late = late || !warp_wait(bar(sm.p_full), j & 1, limit);
        late = late || !warp_wait(bar(sm.v_full), j & 1, limit);
        if (late) break;
        fence_after();
        // (at D = 64 the second block of dimensions is the next tile, and nothing reads its rows)
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kSlotsTile / 16; ++i)
            mma_ss(tmem + kOCol, v + (i * 2048 >> 4), pw + (i * 2048 >> 4), idesc(NC, true),
                   !starts || i > 0);
          mma_commit(bar(sm.pv_done));
        }
        __syncwarp();
        if (j + 1 < n && next_starts) score(j + 1);
        starts = next_starts;
      }
      // nothing is in flight when tensor memory is freed
      if (elect_one()) mma_commit(bar(sm.drained));
      __syncwarp();
      mbar_wait(bar(sm.drained), 0);
      if (late) all.late = 1;
      __syncwarp();
    } else {
      // ---- pages of the chunks ahead (lane k < 8 the k-th 16 slots' codes, lane k + 8 their
      // scales), and at a piece's first chunk its Q, a lane a row
      Walk w(p, share, has);
      bool late = false;
      const int block = page_bytes(1, D) << p.cache.shift;
      const int mask = (1 << p.cache.shift) - 1;
      unsigned piece = 0;
      for (unsigned j = 0; w.left > 0; ++j) {
        const int slot0 = (w.r.lo / kSlotsTile + w.c) * kSlotsTile, slot = slot0 + 16 * (lane & 7);
        int id = -1;
        if (slot < w.r.len)
          id = p.cache.table[(long long)w.b * p.cache.M + (slot >> p.cache.shift)];
        unsigned long long at = 0;
        if ((unsigned)id < (unsigned)p.cache.pages) {
          const int token = slot & mask;
          at = reinterpret_cast<unsigned long long>(p.cache.data) +
               (unsigned long long)(unsigned)id * p.cache.page_stride +
               (long long)(2 * w.h) * block +
               (lane & 8 ? ((D / 2) << p.cache.shift) + token * (D / kGroup) : token * (D / 2));
        }
        if (j >= kRefs)
          late = !warp_wait(bar(sm.ref_empty[j % kRefs]), (j / kRefs - 1) & 1, limit);
        if (late) break;
        ChunkRef& ref = sm.refs[j % kRefs];
        if (lane < 8) ref.codes[lane] = at;
        if (lane >= 8 && lane < 16) ref.scales[lane - 8] = at;
        if (lane == 0) {
          ref.first = max(0, w.r.lo - slot0);
          ref.last = min(kSlotsTile, w.r.len - slot0);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(bar(sm.ref_full[j % kRefs]));
        if (j == 0 || w.c == 0) {
          if (piece > 0) late = !warp_wait(bar(sm.q_empty), (piece - 1) & 1, limit);
          if (late) break;
          ++piece;
          const int rows = w.r.nq * p.group;
          for (int at_row = lane; at_row < NC; at_row += 32)
            bring_row<D, NC>(p, w, w.tile * NC + at_row, rows, at_row, sm);
          fence_proxy_async();
          bar_arrive(bar(sm.q_full));
        }
        w.step(p);
      }
      if (late) all.late = 1;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x < kSides) p.late[ctas[threadIdx.x]] = all.late;
  if (warp == 16) tmem_free(all.tmem);
}

template <int D, int NC>
cudaError_t launch_one(const AttendParams& p, const AttendPlan& plan, cudaStream_t stream) {
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    err = cudaFuncSetAttribute(many_kernel<D, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)many_smem<D, NC>(true));
    if (err != cudaSuccess) return err;
    ready[dev].store(1, std::memory_order_relaxed);
  }
  return launch_early(many_kernel<D, NC>, plan.ctas / kSides, kManyThreads,
                      many_smem<D, NC>(p.parent != nullptr), 1, stream, p);
}

}  // namespace

cudaError_t plan_many(int rows, AttendPlan* plan) {
  DeviceInfo info;
  const cudaError_t err = device_info(&info);
  if (err != cudaSuccess) return err;
  // the tile that leaves fewer rows empty
  plan->rows = (rows + 31) / 32 * 32 < (rows + 47) / 48 * 48 ? 32 : 48;
  plan->chunk = kSlotsTile;
  plan->least = 1;
  plan->shift = kManyShift;
  plan->ctas = kSides * info.sms;  // (shares)
  return cudaSuccess;
}

cudaError_t launch_many(const AttendParams& p, int D, const AttendPlan& plan, cudaStream_t stream) {
#define SV_MANY(d, n) \
  if (D == d && plan.rows == n) return launch_one<d, n>(p, plan, stream);
  SV_MANY(64, 32) SV_MANY(64, 48) SV_MANY(128, 32) SV_MANY(128, 48)
#undef SV_MANY
  return cudaErrorInvalidValue;
}

}  // namespace sv
