// sv_attend_many.cu - attention over the 4-bit cache for many query rows
// (spec_cache_attention): tensor memory and tcgen05 instructions.
//
// A unit is 128 query rows of a key/value head (tokens of the step times the heads
// of the group), a chunk 128 slots.  One CTA an SM; a chunk takes
//   S = Q K^T   128 x 128 x D, both operands in shared memory, S in tensor memory
//   O += P V    128 x D x 128, the weights P in tensor memory (over S), V in shared memory
// in fp16 with 32-bit sums.  Decoded keys and values are exact in fp16; a row of Q is
// scaled by a power of two (exact), weights are rounded to 2^-11.  Its
// warps:
//   0-3    the softmax, a thread a row: scores from tensor memory, weights back;
//   4-7, 8-11  decode the chunk's keys and values, two chunks ahead in registers, into two stages
//          of shared memory each.  Both lie as rows of a slot, 64 dimensions (128 bytes)
//          a block, 128-byte swizzle: K-major for K^T, MN-major for V;
//   12     issues the tensor instructions: S of the next chunk before O of this one, so that the
//          tensor pipe works while the softmax does;
//   13     brings the next piece's Q.
// The running max follows a row's scores only when they exceed it by 2^8: the
// weights, at most 2^15 then, stay within fp16, and O is rescaled in tensor memory a few
// times a piece.
//
// What bounds it: a chunk is 4 x 128 x 128 x D / 2 products on the tensor pipe (1024 cycles at D =
// 128, whatever the number of rows), 17408 bytes of HBM (800 cycles of an SM's share), and
// about as many issue slots for the decoding and the softmax.
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
constexpr int kRowsTile = 128, kSlotsTile = 128;
constexpr float kManyShift = 7.f, kSlack = 8.f;
constexpr int kTmemCols = 512;
constexpr int kOCol = 256;  // O's columns; S and P: 0 and 128

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
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
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
#define SV_R8(a, i) \
  a[i], a[i + 1], a[i + 2], a[i + 3], a[i + 4], a[i + 5], a[i + 6], a[i + 7]
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_loaded() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
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
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn_major) {
  return 1u << 4 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}

template <int D>
struct ManySmem {
  static constexpr int kTileBytes = D / 64 * (int)kBlockBytes;
  alignas(1024) char q[2][kTileBytes];
  alignas(1024) char k[2][kTileBytes];
  alignas(1024) char v[2][kTileBytes];
  float unscale[2][kRowsTile];
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
template <int D>
constexpr size_t many_smem() {  // (more than half of an SM's: one CTA an SM, as tensor memory needs)
  return std::max(sizeof(ManySmem<D>) + 1024, (size_t)120 * 1024);
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
  uint32_t scale[kU];  // a pair of 64 s
};

template <int D>
__global__ void __launch_bounds__(kManyThreads, 1) many_kernel(const AttendParams p) {
  extern __shared__ __align__(16) char many_raw[];
  ManySmem<D>& sm = *reinterpret_cast<ManySmem<D>*>(
      many_raw + ((1024 - (smem_u32(many_raw) & 1023)) & 1023));
  constexpr int kTileBytes = ManySmem<D>::kTileBytes;
  constexpr int G = D / 32;  // groups of a row
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int cta = blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), 4);
      mbar_init(smem_u32(&sm.v_full[i]), 4);
      mbar_init(smem_u32(&sm.qk_done[i]), 1);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
      mbar_init(smem_u32(&sm.p_full[i]), kRowsTile);
      mbar_init(smem_u32(&sm.q_full[i]), 32);
      mbar_init(smem_u32(&sm.q_empty[i]), 1 + kRowsTile);
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
    // ---- softmax: thread = row = lane of tensor memory
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
    Walk w(p, share);
    unsigned j = 0, piece = 0;  // chunks and pieces so far
    bool late = false;
    while (w.left > 0) {
      const int b = w.b, h = w.h, c0 = w.c;
      const Request r = w.r;
      const int c1 = (int)min((long long)r.chunks, c0 + w.left);
      const int rows = r.nq * p.group, row = w.tile * kRowsTile + tid;
      const bool warp_has = w.tile * kRowsTile + warp * 32 < rows;
      bool sees = r.ok && r.len > 0;
      if (p.parent && sees) sees = build_tree<kRowsTile>(p, b, r.nq, sm.tree);
      const int node_of = min(row, max(rows - 1, 0)) / p.group;
      const int head = h * p.group + min(row, max(rows - 1, 0)) - node_of * p.group;
      const int pos = r.base + (p.parent && sees ? sm.tree.depth[node_of] : node_of);
      const float slope = p.slopes ? p.slopes[head] * kLog2e : 0.f;
      late = late || !warp_wait(bar(sm.q_full[piece & 1]), piece >> 1 & 1, limit);
      const float unscale = sm.unscale[piece & 1][tid] * fabsf(p.scale) *
                            (p.softcap > 0.f ? 1.f / p.softcap : kLog2e);
      bar_arrive(bar(sm.q_empty[piece & 1]));
      ++piece;
      float m = -INFINITY, l = 0.f;
      for (int c = c0; c < c1; ++c, ++j) {
        const uint32_t s_at = mine + (j & 1) * 128;
        late = late || !warp_wait(bar(sm.qk_done[j & 1]), j >> 1 & 1, limit);
        if (late) break;
        if (warp_has) {
          fence_after();
          uint32_t s[kSlotsTile];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_load32(s_at + 32 * i, s + 32 * i);
          tmem_loaded();
          const int slot0 = (r.lo / kSlotsTile + c) * kSlotsTile;
          const bool edge = !sees || slot0 + kSlotsTile > r.base || p.slopes ||
                            (p.window > 0 && slot0 <= r.base + r.nq - 1 - p.window);
          const bool plain = !edge && p.softcap == 0.f;
          if (!plain) {
#pragma unroll
            for (int i = 0; i < kSlotsTile; ++i) {
              float y = __uint_as_float(s[i]) * unscale;
              if (p.softcap > 0.f) y = cap_of<false>(p.softcap * kLog2e, y);
              s[i] = __float_as_uint(y);
            }
          }
          if (edge) {
#pragma unroll
            for (int i = 0; i < kSlotsTile; ++i) {
              const int slot = slot0 + i, node = slot - r.base;
              bool seen = sees && slot < r.len;
              int at = slot;
              if (seen && node >= 0) {
                if (p.parent) {
                  seen = (sm.tree.seen[node_of][node >> 5] >> (node & 31)) & 1;
                  at = r.base + sm.tree.depth[node];
                } else {
                  seen = node <= node_of;
                }
              }
              const int far = pos - at;
              if (p.window > 0 && far >= p.window) seen = false;
              s[i] = __float_as_uint(
                  seen ? fmaf(-slope, (float)far, __uint_as_float(s[i])) : -INFINITY);
            }
          }
          const float f = plain ? unscale : 1.f;
          float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kSlotsTile; ++i) top4[i & 3] = fmaxf(top4[i & 3], __uint_as_float(s[i]));
          const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * f;
          if (__any_sync(0xffffffffu, top > m + kSlack)) {  // (m = -inf: the first scores seen)
            const float up = fmaxf(m, top);
            const float g = m == -INFINITY ? 0.f : ex2(m - up);
            m = up;
            l *= g;
            if (c > c0) {  // O so far
              late = late || !warp_wait(bar(sm.pv_done[(j - 1) & 1]), (j - 1) >> 1 & 1, limit);
              fence_after();
#pragma unroll
              for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                tmem_load32(mine + kOCol + 32 * i, o);
                tmem_loaded();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * g);
                tmem_store32(mine + kOCol + 32 * i, o);
              }
            }
          }
          const float off = m == -INFINITY ? 0.f : kManyShift - m;
          const f32x2 f2 = pack2(f, f), off2 = pack2(off, off);
          f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w2[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int at = 64 * half + 2 * i;
              float x, y;
              unpack2(fma2(pack2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), f2, off2), x,
                      y);
              x = ex2(x);
              y = ex2(y);
              sum[i & 1] = add2(sum[i & 1], pack2(x, y));
              w2[i] = pack_f16(x, y);
            }
            tmem_store32(s_at + 32 * half, w2);
          }
          float a0, a1, b0, b1;
          unpack2(sum[0], a0, a1);
          unpack2(sum[1], b0, b1);
          l += (a0 + a1) + (b0 + b1);
          tmem_stored();
          fence_before();
        }
        bar_arrive(bar(sm.p_full[j & 1]));
      }
      // the piece's rows
      const bool whole = c0 == 0 && c1 == r.chunks;
      const bool first = w.left == share.end - share.begin;
      if (!late) late = !warp_wait(bar(sm.pv_done[(j - 1) & 1]), (j - 1) >> 1 & 1, limit);
      fence_after();
      if (late) l = qnan();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float* part = p.part + ((long long)(2 * cta + (first ? 0 : 1)) * kRowsTile + tid) * (D + 4);
      const long long to = ((long long)b * p.N + node_of) * p.Hq + head;
      if (warp_has) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          if (!late) {
            tmem_load32(mine + kOCol + 32 * i, o);
            tmem_loaded();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          // (a row that saw nothing has weights of 0, and what O holds may be anything)
          if (l == 0.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + 32 * i + e) =
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else if (row < rows) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + to * D + 32 * i;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = pack_bf16(__uint_as_float(o[e + 2 * k]) * inv,
                                 __uint_as_float(o[e + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>(dst + e) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
        }
        if (!whole) {
          part[D] = m;
          part[D + 1] = l;
        } else if (row < rows && p.out_lse) {
          p.out_lse[to] =
              l == 0.f ? -INFINITY : (m - kManyShift + log2f(l)) * 0.6931471805599453f;
        }
      }
      fence_before();
      if (!whole && c0 == 0 && tid == 0) {
        int* desc = p.desc + 4 * cta;
        desc[0] = b;
        desc[1] = h;
        desc[2] = w.tile | (first ? 0 : 1 << 30);
        desc[3] = pieces_of(share, cta, share.end - w.left + r.chunks);
      }
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
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int slot = ref.slot0 + 8 * (blk + 16 / G * i) + r8;
        x.w[i] = make_uint4(0, 0, 0, 0);
        x.scale[i] = values ? 0xf8u : kNanScale;  // (-8: a scale of 0)
        if ((unsigned)ids[i] < (unsigned)p.cache.pages) {
          const char* base = p.cache.data + (unsigned long long)(unsigned)ids[i] * p.cache.page_stride +
                             (long long)(2 * ref.h + values) * block;
          const int token = slot & mask;
          x.w[i] = *reinterpret_cast<const uint4*>(base + token * (D / 2) + g * 16);
          const uint32_t byte = *reinterpret_cast<const unsigned char*>(
              base + scale_at<D>(p.cache, token, g) + (token & 15));
          x.scale[i] = values && (slot < ref.lo || slot >= ref.len) ? 0xf8u : byte;
        }
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
        sc.set(((x.scale[i] + 8) << 7 & 0x7fffu) * 0x10001u);
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
            const uint32_t at = (i / 4) * kBlockBytes + (i % 4) * 32;
            mma_ss(tmem + (j & 1) * 128, smem_desc(q + at, 16), smem_desc(k + at, 16),
                   idesc(kSlotsTile, false), i > 0);
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
          const uint32_t v = smem_u32(sm.v[j & 1]);
#pragma unroll
          for (int i = 0; i < kSlotsTile / 16; ++i)
            mma_ts(tmem + kOCol, tmem + (j & 1) * 128 + 8 * i,
                   smem_desc(v + i * 2048, kBlockBytes), idesc(D, true), !starts || i > 0);
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
        const int rows = w.r.ok ? w.r.nq * p.group : 0;
        for (int k = 0; k < 4; ++k) {
          const int at = 32 * k + lane, row = w.tile * kRowsTile + at;
          const bool ok = row < rows;
          const int i = row / p.group;
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(p.q) + w.b * p.qb + i * p.qn +
              (long long)(w.h * p.group + row - i * p.group) * p.qh);
          uint32_t top2 = 0;
          for (int x = 0; x < D / 8; ++x) {
            const uint4 v = ok ? src[x] : make_uint4(0, 0, 0, 0);
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // magnitudes of bf16 order as whole numbers
              const uint32_t mag = words[e] & 0x7fff7fffu;
              top2 = __vmaxu2(top2, mag);
            }
          }
          const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
          const int e = min(max((int)(top >> 7) - 127, -98), 126);
          float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          if (top >= 0x7f80u) up = qnan();  // (a row with NaN or infinity is NaN)
          if (p.scale < 0.f) up = -up;
          sm.unscale[buf][at] = __uint_as_float((uint32_t)(127 + e - 14) << 23);
          for (int x = 0; x < D / 8; ++x) {
            const uint4 v = ok ? src[x] : make_uint4(0, 0, 0, 0);
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
            uint32_t d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              d[q] = pack_f16(bf16_lo(words[q]) * up, bf16_hi(words[q]) * up);
            *reinterpret_cast<uint4*>(sm.q[buf] + (x / 8) * kBlockBytes + at * 128 +
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

}  // namespace

cudaError_t plan_many(int D, AttendPlan* plan) {
  DeviceInfo info;
  const cudaError_t err = device_info(&info);
  if (err != cudaSuccess) return err;
  plan->rows = kRowsTile;
  plan->chunk = kSlotsTile;
  plan->least = 1;
  plan->shift = kManyShift;
  plan->ctas = info.sms;
  return cudaSuccess;
}

cudaError_t launch_many(const AttendParams& p, int D, const AttendPlan& plan, cudaStream_t stream) {
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (!ready[dev & 63].load(std::memory_order_relaxed)) {
    err = cudaFuncSetAttribute(many_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)many_smem<64>());
    if (err == cudaSuccess)
      err = cudaFuncSetAttribute(many_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)many_smem<128>());
    if (err != cudaSuccess) return err;
    ready[dev & 63].store(1, std::memory_order_relaxed);
  }
  if (D == 64)
    return launch_early(many_kernel<64>, plan.ctas, kManyThreads, many_smem<64>(), 1, stream, p);
  if (D == 128)
    return launch_early(many_kernel<128>, plan.ctas, kManyThreads, many_smem<128>(), 1, stream, p);
  return cudaErrorInvalidValue;
}

}  // namespace sv
