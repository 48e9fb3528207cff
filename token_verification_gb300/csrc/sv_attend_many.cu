// sv_attend_many.cu - attention over the 4-bit cache for many query rows
// (spec_cache_attention): tensor memory and tcgen05 instructions.
//
// A unit is a tile of 32, 48 or 64 query rows of a key/value head (tokens of the step times the
// heads of the group), a chunk 128 slots.  One CTA an SM; a chunk takes
//   S^T = K Q^T    128 slots x rows x D, both operands in shared memory
//   O^T += V^T P^T  D x rows x 128 slots, values and weights P in shared memory
// in fp16 with 32-bit sums in tensor memory.  Slots and dimensions lie on the instruction's side of
// 128, so a tile of few rows costs what its rows cost (rows on that side would count as 128
// each time).  Decoded keys and values are exact in fp16; a row of Q is scaled by a power of two
// (exact), weights are rounded to 2^-11.  The warps:
//   0-3    the softmax, a thread a slot: its scores of every row from tensor memory, weights to
//          shared memory;
//   4-7, 8-11  decode the chunk's keys and values, two chunks ahead in registers, into two stages
//          of shared memory each.  Both lie as rows of a slot, 64 dimensions (128 bytes)
//          a block, 128-byte swizzle: K-major for the keys, MN-major for the values;
//   12     issues the tensor instructions: S of the next chunk before O of this one, so that the
//          tensor pipe works while the softmax does;
//   13     brings the next piece's Q and its rows' constants.
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

constexpr int kManyThreads = 512;
constexpr int kSlotsTile = 128;
constexpr float kManyShift = 7.f, kSlack = 8.f;
constexpr float kNoRef = 3e38f;  // in place of shift - max for a row without a score yet
constexpr int kTmemCols = 256;
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

template <int D, int NC>
struct ManySmem {
  static constexpr int kTileBytes = D / 64 * (int)kBlockBytes;
  alignas(1024) char q[2][D / 64 * NC * 128];
  alignas(1024) char p[2][kBlockBytes];  // weights [slot][64 rows]
  alignas(1024) char v[2][kTileBytes];  // (not last: at D = 64 a descriptor reaches one tile on)
  alignas(1024) char k[2][kTileBytes];
  // rows: of two pieces, brought with Q (a score's factor, the step's token, its row of `out`
  // counted from the request's first, a slope) ...
  float unscale[2][NC], slope[2][NC];
  int node[2][NC], out_row[2][NC];
  // ... and of the current piece: {factor, factor, shift - reference, the same} of pairs of rows,
  // the reference, the last change of it, positions; what the warps leave to be joined
  alignas(16) float4 fo[NC / 2];
  alignas(16) float m[NC], change[NC], inv[NC];
  int pos[NC];
  float part[4][NC];
  // completed by: k_full, v_full the decoding warps; qk_done, pv_done the tensor pipe (which then no
  // longer needs the keys, or the values and the weights); p_full the softmax (weights
  // in place); q_full warp 13; q_empty the tensor pipe and the softmax
  alignas(8) unsigned long long k_full[2], v_full[2], qk_done[2], pv_done[2], p_full[2], q_full[2],
      q_empty[2], drained;
  uint32_t tmem;
  int late;
  long long scan[kManyThreads / 32 + 3];
  TreeView tree;
};
template <int D, int NC>
constexpr size_t many_smem() {  // (more than half of an SM's: one CTA an SM)
  return std::max(sizeof(ManySmem<D, NC>) + 1024, (size_t)120 * 1024);
}

// Barriers of the softmax warps.
__device__ __forceinline__ void meet() { asm volatile("bar.sync 2, 128;" ::: "memory"); }
__device__ __forceinline__ bool any_of_them(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_top(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// A chunk of a unit as the decoding threads need it.
struct ChunkRef {
  const int* table;
  int h, slot0, lo, len;
};
__device__ __forceinline__ ChunkRef chunk_ref(const AttendParams& p, const Walk& w) {
  return {p.cache.table + (long long)w.b * p.cache.M, w.h,
          (w.r.lo / kSlotsTile + w.c) * kSlotsTile, w.r.lo, w.r.len};
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

template <int D, int NC>
__global__ void __launch_bounds__(kManyThreads, 1) many_kernel(const AttendParams p) {
  extern __shared__ __align__(16) char many_raw[];
  ManySmem<D, NC>& sm = *reinterpret_cast<ManySmem<D, NC>*>(
      many_raw + ((1024 - (smem_u32(many_raw) & 1023)) & 1023));
  constexpr int kTileBytes = ManySmem<D, NC>::kTileBytes;
  constexpr int G = D / 32;  // groups of a row
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int cta = blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), 4);
      mbar_init(smem_u32(&sm.v_full[i]), 4);
      mbar_init(smem_u32(&sm.qk_done[i]), 1);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), 128);
      mbar_init(smem_u32(&sm.q_full[i]), 32);
      mbar_init(smem_u32(&sm.q_empty[i]), 1 + 128);
    }
    mbar_init(smem_u32(&sm.drained), 1);
    fence_mbar_init();
    sm.late = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  const Share share = find_share<kManyThreads>(p, cta, gridDim.x, sm.scan);
  if (tid == 0) {
    p.desc[4 * cta + 3] = 0;
    if (cta >= share.G) p.late[cta] = 0;
  }
  if (cta >= share.G) return;
  if (warp == 12) tmem_alloc(smem_u32(&sm.tmem));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  const unsigned long long limit = p.wait_ns;
  auto bar = [](unsigned long long& b) { return smem_u32(&b); };

  if (warp < 4) {
    // ---- softmax: thread = slot of the chunk, or dimension, = lane of tensor memory
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
    Walk w(p, share);
    unsigned j = 0, piece = 0;  // chunks and pieces so far
    bool late = false;
    const float cap = p.softcap * kLog2e;
    while (w.left > 0) {
      const int b = w.b, h = w.h, c0 = w.c;
      const Request r = w.r;
      const int c1 = (int)min((long long)r.chunks, c0 + w.left);
      const int row0 = w.tile * NC, n_rows = min(NC, r.nq * p.group - row0);
      const int buf = piece & 1;
      bool sees = r.ok && r.len > 0;
      if (p.parent && sees) sees = build_tree<128>(p, b, r.nq, sm.tree);
      late = late || !warp_wait(bar(sm.q_full[buf]), piece >> 1 & 1, limit);
      ++piece;
      // the piece's rows
      if (tid < NC) {
        const float f = sm.unscale[buf][tid];
        float* fo = reinterpret_cast<float*>(&sm.fo[tid / 2]);
        fo[tid & 1] = f;
        fo[2 + (tid & 1)] = kNoRef;
        sm.m[tid] = -INFINITY;
        const int node = sm.node[buf][tid];
        sm.pos[tid] = r.base + (p.parent && sees ? sm.tree.depth[node] : node);
      }
      f32x2 l[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) l[i] = pack2(0.f, 0.f);
      meet();
      for (int c = c0; c < c1; ++c, ++j) {
        const uint32_t s_at = mine + (j & 1) * 64;
        late = late || !warp_wait(bar(sm.qk_done[j & 1]), j >> 1 & 1, limit);
        if (j >= 2) late = late || !warp_wait(bar(sm.pv_done[j & 1]), (j >> 1 & 1) ^ 1, limit);
        // (the four warps meet below: they leave together)
        if (any_of_them(late)) late = true;
        if (late) break;
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
          if (p.parent && there && node >= 0) at = r.base + sm.tree.depth[node];
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float y = s[i] * reinterpret_cast<const float*>(&sm.fo[i / 2])[i & 1];
            if (p.softcap > 0.f) y = cap_of<false>(cap, y);
            if (p.slopes) y = fmaf(-sm.slope[buf][i], (float)(sm.pos[i] - at), y);
            s[i] = y;
          }
          if (!edge) return;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            bool seen = there;
            if (there && node >= 0) {
              const int mine_node = sm.node[buf][i];
              seen = p.parent ? sm.tree.seen[mine_node][node >> 5] >> (node & 31) & 1
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
                           kManyShift + kSlack))
            break;
          // each row's max over the chunk's slots
          load_scores();
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float y = s[i];
            if (plain) y *= reinterpret_cast<const float*>(&sm.fo[i / 2])[i & 1];
            y = warp_top(y);
            if (lane == (i & 31)) sm.part[warp][i] = y;
          }
          meet();
          if (tid < NC) {
            const float old = sm.m[tid];
            const float m = fmaxf(fmaxf(old, sm.part[0][tid]),
                                  max3(sm.part[1][tid], sm.part[2][tid], sm.part[3][tid]));
            sm.m[tid] = m;
            sm.change[tid] = old == -INFINITY ? 0.f : ex2(old - m);
            reinterpret_cast<float*>(&sm.fo[tid / 2])[2 + (tid & 1)] =
                m == -INFINITY ? kNoRef : kManyShift - m;
          }
          meet();
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) {
            const float2 g = *reinterpret_cast<const float2*>(&sm.change[2 * i]);
            l[i] = fma2(l[i], pack2(g.x, g.y), pack2(0.f, 0.f));
          }
          if (c > c0) {  // O so far
            late = late || !warp_wait(bar(sm.pv_done[(j - 1) & 1]), (j - 1) >> 1 & 1, limit);
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
        char* to = sm.p[j & 1] + tid * 128;
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
        bar_arrive(bar(sm.p_full[j & 1]));
      }
      // the rows' sums over the slots: each warp's by halves (lane k ends with rows k, k + 32), then
      // over the warps
      {
        float v[NC];
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) unpack2(l[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const float sum = warp_sum(v[i]);
          if (lane == (i & 31)) sm.part[warp][i] = sum;
        }
      }
      meet();
      const bool whole = c0 == 0 && c1 == r.chunks;
      const bool first = w.left == share.end - share.begin;
      float* part = p.part + (long long)(2 * cta + (first ? 0 : 1)) * NC * (D + 4);
      const long long out0 = (long long)b * p.N * p.Hq;
      if (!late) late = !warp_wait(bar(sm.pv_done[(j - 1) & 1]), (j - 1) >> 1 & 1, limit);
      if (any_of_them(late)) late = true;
      fence_after();
      if (tid < NC) {
        float sum = (sm.part[0][tid] + sm.part[1][tid]) + (sm.part[2][tid] + sm.part[3][tid]);
        if (late) sum = qnan();
        sm.inv[tid] = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        if (tid < n_rows) {
          if (!whole) {
            part[tid * (D + 4) + D] = sm.m[tid];
            part[tid * (D + 4) + D + 1] = sum;
          } else if (p.out_lse) {
            p.out_lse[out0 + sm.out_row[buf][tid]] =
                sum == 0.f ? -INFINITY : (sm.m[tid] - kManyShift + log2f(sum)) * 0.6931471805599453f;
          }
        }
      }
      meet();
      if (D == 128 || warp < 2) {
#pragma unroll
        for (int i = 0; i < NC / 16; ++i) {
          uint32_t o[16];
          tmem_load16(mine + kOCol + 16 * i, o);
          tmem_loaded();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int row = 16 * i + e;
            if (row >= n_rows) continue;
            const float inv = sm.inv[row];
            const float x = late ? qnan() : inv == 0.f ? 0.f : __uint_as_float(o[e]) * inv;
            if (!whole)
              part[row * (D + 4) + tid] = x;
            else
              static_cast<__nv_bfloat16*>(p.out)[(out0 + sm.out_row[buf][row]) * D + tid] =
                  __float2bfloat16_rn(x);
          }
        }
      }
      fence_before();
      bar_arrive(bar(sm.q_empty[buf]));
      if (!whole && c0 == 0 && tid == 0) {
        int* desc = p.desc + 4 * cta;
        desc[0] = b;
        desc[1] = h;
        desc[2] = w.tile | (first ? 0 : 1 << 30);
        desc[3] = pieces_of(share, cta, share.end - w.left + r.chunks);
      }
      meet();  // (the rows' constants are read)
      // (pieces behind a wait that ran out are written as NaN)
      w.left -= c1 - c0;
      w.c = c1;
      if (c1 == r.chunks) w.next_unit(p);
    }
    if (late) sm.late = 1;
  } else if (warp < 12) {
    // ---- decoding: warps 4-7 keys, 8-11 values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    constexpr int kU = Part<D>::kU;
    const bool values = warp >= 8;
    const int u = tid & 127, r8 = u & 7, g = (u >> 3) % G, blk = (u >> 3) / G;
    const int block = page_bytes(1, D) << p.cache.shift;
    const int mask = (1 << p.cache.shift) - 1;
    Walk w(p, share);
    ChunkRef ref = chunk_ref(p, w);
    int ids[kU];
    // page ids of the chunk that `w` stands at, into ids; then w steps on
    auto fetch_ids = [&] {
      if (w.left <= 0) return;
      ref = chunk_ref(p, w);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int slot = ref.slot0 + 8 * (blk + 16 / G * i);
        ids[i] = slot < ref.len ? ref.table[slot >> p.cache.shift] : -1;
      }
      w.step(p);
    };
    auto load = [&](Part<D>& x) {  // of ref
      x.off = 0;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int slot = ref.slot0 + 8 * (blk + 16 / G * i) + r8;
        const bool ok = (unsigned)ids[i] < (unsigned)p.cache.pages;
        const char* base = p.cache.data + (unsigned long long)(unsigned)ids[i] * p.cache.page_stride +
                           (long long)(2 * ref.h + values) * block;
        const int token = slot & mask;
        x.w[i] = load16_if(base + token * (D / 2) + g * 16, ok);
        x.scale[i] = load_byte_if(base + scale_at<D>(p.cache, token, g) + (token & 15), ok);
        x.off |= (!ok || (values && (slot < ref.lo || slot >= ref.len)) ? 1u : 0u) << i;
      }
    };
    const long long n = w.left;
    char* tiles = values ? sm.v[0] : sm.k[0];
    unsigned long long* full = values ? sm.v_full : sm.k_full;
    unsigned long long* done = values ? sm.pv_done : sm.qk_done;
    bool late = false;
    auto put = [&](unsigned j, Part<D>& x) {
      const int st = j & 1;
      if (j >= 2) late = late || !warp_wait(bar(done[st]), (j >> 1 & 1) ^ 1, limit);
      if (late) return;
      char* tile = tiles + st * kTileBytes + (g >> 1) * kBlockBytes;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        Scale2 sc;
        const uint32_t half = x.off >> i & 1 ? (values ? 0u : 0x7fffu) : x.scale[i] * 128u + 0x400u;
        sc.set(half * 0x10001u);
        const int slot = 8 * (blk + 16 / G * i) + r8;
        const uint32_t words[4] = {x.w[i].x, x.w[i].y, x.w[i].z, x.w[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t d[4];
          decode_word(words[q], sc, d);
          *reinterpret_cast<uint4*>(tile + slot * 128 + ((((g & 1) * 4 + q) ^ r8) << 4)) =
              make_uint4(d[0], d[1], d[2], d[3]);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) bar_arrive(bar(full[st]));
    };
    Part<D> a, c;
    fetch_ids();
    load(a);
    if (n > 1) {
      fetch_ids();
      load(c);
    }
    fetch_ids();
    for (unsigned j = 0; j < n && !late; j += 2) {
      put(j, a);
      if (j + 2 < n) {
        load(a);
        fetch_ids();
      }
      if (j + 1 < n) {
        put(j + 1, c);
        if (j + 3 < n) {
          load(c);
          fetch_ids();
        }
      }
    }
    if (late) sm.late = 1;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 12) {
      // ---- the tensor pipe
      if (lane == 0) {
        Walk w(p, share);
        const long long n = w.left;
        unsigned piece = 0;
        bool late = false;
        auto score = [&](unsigned j) {  // S of the chunk that `w` stands at; w steps on
          const bool starts = j == 0 || w.c == 0;
          if (starts) {
            if (j > 0) ++piece;
            late = late || !mbar_wait(bar(sm.q_full[piece & 1]), piece >> 1 & 1, limit);
          }
          late = late || !mbar_wait(bar(sm.k_full[j & 1]), j >> 1 & 1, limit);
          if (late) return;
          fence_after();
          const uint32_t q = smem_u32(sm.q[piece & 1]), k = smem_u32(sm.k[j & 1]);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            mma_ss(tmem + (j & 1) * 64,
                   smem_desc(k + (i / 4) * kBlockBytes + (i % 4) * 32, 16),
                   smem_desc(q + (i / 4) * (NC * 128) + (i % 4) * 32, 16), idesc(NC, false), i > 0);
          }
          mma_commit(bar(sm.qk_done[j & 1]));
          w.step(p);
          if (w.left == 0 || w.c == 0) mma_commit(bar(sm.q_empty[piece & 1]));
        };
        bool starts = true;  // chunk j is its piece's first
        score(0);
        for (unsigned j = 0; j < n && !late; ++j) {
          const bool next_starts = w.c == 0;
          if (j + 1 < n) score(j + 1);
          late = late || !mbar_wait(bar(sm.p_full[j & 1]), j >> 1 & 1, limit);
          late = late || !mbar_wait(bar(sm.v_full[j & 1]), j >> 1 & 1, limit);
          if (late) break;
          fence_after();
          // (at D = 64 the second block of dimensions is the next tile, and nothing reads its rows)
          const uint32_t v = smem_u32(sm.v[j & 1]), pw = smem_u32(sm.p[j & 1]);
#pragma unroll
          for (int i = 0; i < kSlotsTile / 16; ++i)
            mma_ss(tmem + kOCol, smem_desc(v + i * 2048, kBlockBytes),
                   smem_desc(pw + i * 2048, kBlockBytes), idesc(NC, true), !starts || i > 0);
          mma_commit(bar(sm.pv_done[j & 1]));
          starts = next_starts;
        }
        // nothing is in flight when tensor memory is freed
        mma_commit(bar(sm.drained));
        mbar_wait(bar(sm.drained), 0);
        if (late) sm.late = 1;
      }
      __syncwarp();
    } else if (warp == 13) {
      // ---- Q: a lane takes four rows of each piece
      Walk w(p, share);
      bool late = false;
      for (unsigned piece = 0; w.left > 0 && !late; ++piece) {
        const int buf = piece & 1;
        if (piece >= 2) late = !warp_wait(bar(sm.q_empty[buf]), (piece >> 1 & 1) ^ 1, limit);
        if (late) break;
        const int rows = w.r.nq * p.group;
        for (int at = lane; at < NC; at += 32) {
          const int row = w.tile * NC + at;
          const bool ok = row < rows && w.r.ok;
          const int clamped = min(row, max(rows - 1, 0));
          const int i = clamped / p.group, head = w.h * p.group + clamped - i * p.group;
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(p.q) + w.b * p.qb + i * p.qn +
              (long long)head * p.qh);
          uint32_t top2 = 0;
          for (int x = 0; x < D / 8; ++x) {
            const uint4 v = ok ? src[x] : make_uint4(0, 0, 0, 0);
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)  // (magnitudes of bf16 order as whole numbers)
              top2 = __vmaxu2(top2, words[e] & 0x7fff7fffu);
          }
          const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
          const int e = min(max((int)(top >> 7) - 127, -98), 126);
          float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          if (top >= 0x7f80u) up = qnan();  // (a row with NaN or infinity is NaN)
          if (p.scale < 0.f) up = -up;
          sm.unscale[buf][at] = __uint_as_float((uint32_t)(127 + e - 14) << 23) * fabsf(p.scale) *
                                (p.softcap > 0.f ? 1.f / p.softcap : kLog2e);
          sm.slope[buf][at] = p.slopes ? p.slopes[head] * kLog2e : 0.f;
          sm.node[buf][at] = i;
          sm.out_row[buf][at] = i * p.Hq + head;
          for (int x = 0; x < D / 8; ++x) {
            const uint4 v = ok ? src[x] : make_uint4(0, 0, 0, 0);
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
            uint32_t d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              d[q] = pack_f16(bf16_lo(words[q]) * up, bf16_hi(words[q]) * up);
            *reinterpret_cast<uint4*>(sm.q[buf] + (x / 8) * (NC * 128) + at * 128 +
                                      (((x & 7) ^ (at & 7)) << 4)) =
                make_uint4(d[0], d[1], d[2], d[3]);
          }
        }
        fence_proxy_async();
        bar_arrive(bar(sm.q_full[buf]));
        const int take = (int)min((long long)w.r.chunks - w.c, w.left);
        w.left -= take;
        w.next_unit(p);
      }
      if (late) sm.late = 1;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (tid == 0) p.late[cta] = sm.late;
  if (warp == 12) tmem_free(tmem);
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
                               (int)many_smem<D, NC>());
    if (err != cudaSuccess) return err;
    ready[dev].store(1, std::memory_order_relaxed);
  }
  return launch_early(many_kernel<D, NC>, plan.ctas, kManyThreads, many_smem<D, NC>(), 1, stream, p);
}

}  // namespace

cudaError_t plan_many(int rows, AttendPlan* plan) {
  DeviceInfo info;
  const cudaError_t err = device_info(&info);
  if (err != cudaSuccess) return err;
  plan->rows = rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
  plan->chunk = kSlotsTile;
  plan->least = 1;
  plan->shift = kManyShift;
  plan->ctas = info.sms;
  return cudaSuccess;
}

cudaError_t launch_many(const AttendParams& p, int D, const AttendPlan& plan, cudaStream_t stream) {
#define SV_MANY(d, n) \
  if (D == d && plan.rows == n) return launch_one<d, n>(p, plan, stream);
  SV_MANY(64, 32) SV_MANY(64, 48) SV_MANY(64, 64)
  SV_MANY(128, 32) SV_MANY(128, 48) SV_MANY(128, 64)
#undef SV_MANY
  return cudaErrorInvalidValue;
}

}  // namespace sv
