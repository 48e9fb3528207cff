// sv_attend_many.cu - attention over the 4-bit cache for many query rows
// (spec_cache_attention): tensor memory and tcgen05 instructions.
//
// A unit is a tile of 32 or 48 query rows, all that a key/value head has (tokens of the step times the
// heads of the group; for more see sv_attend_rows.cu), a chunk 128 slots, which takes
//   S^T = K Q^T    128 slots x rows x D, both operands in shared memory
//   O^T += V^T P^T  D x rows x 128 slots, values and weights P in shared memory
// in fp16 with 32-bit sums in tensor memory.  Slots and dimensions lie on the instruction's side of
// 128, so a tile of few rows costs what its rows cost (rows on that side would count as 128
// each time).  Decoded keys and values are exact in fp16; a row of Q is scaled by a power of two
// (exact), weights are rounded to 2^-11.
//
// Two CTAs an SM, whose 8 warps all do the same: decode keys and values (rows of a slot, 64
// dimensions or 128 bytes a block, 128-byte swizzle: K-major for the keys, MN-major for the
// values), and between them the softmax, a thread a slot and half of the rows: scores from
// tensor memory, weights to shared memory.  One thread issues the products: S of the next chunk once its
// keys are in, while this one's weights are worked out (S has two places), and O of this chunk
// while the next one's keys are decoded.
// Bound by latencies between 16 warps an SM (issue slots 46 % used, tensor pipe 45 %, shared memory 47 %),
// not by HBM; of about 690 instructions a warp and chunk 300 decode and 60 are exponentials.  Measured:
// 285 us for 6 tokens each of 64 requests of up to 8192 slots (8 heads a group, 8 groups of 128; 1.6 TB/s).
// In an earlier form, on six tiles of 48 rows of 32 trees (470 us here), one CTA an SM took 732 us, and
// warps of one task each (softmax, decoding, issuing) 757: each of their instructions waited
// to be fetched.  Issuing S and O together at the chunk's end: 487.
// A row's weights are relative to a reference that follows its running max only when a
// score exceeds it by 2^8: the weights, at most 2^15 then, stay within fp16, and the
// threads, which hold one slot of every row, need to agree on a row's max (and to rescale O in
// tensor memory) a few times a piece instead of every chunk. Sums in tensor memory are cut off, by 2^-23.3 of them
// a product of 16 slots: a bf16 result's rounding outweighs that up to some 2^18 slots of one CTA.
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/spec_verify.h"
#include "sv_attend_tc.cuh"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

constexpr int kManyThreads = 256;
constexpr int kTmemCols = 256;
constexpr int kSCol = 64, kOCol = 128;  // columns: S of chunk j at kSCol (j mod 2), O

template <int D, int NC>
struct ManySmem {
  static constexpr int kTileBytes = D / 64 * (int)kBlockBytes;
  alignas(1024) char v[kTileBytes];  // (first: at D = 64 a descriptor reaches one tile on)
  alignas(1024) char k[kTileBytes];
  // weights [slot][64 rows]; at other times a finished piece's rows (or their sums), behind them
  // what the warps leave to be joined, or a tree's parents
  alignas(1024) char p[kBlockBytes];
  static_assert(64 * NC * 4 + 16 * NC <= (int)kBlockBytes && NC * D * 2 <= 64 * NC * 4, "");
  alignas(1024) char q[D / 64 * NC * 128];
  uint4 raw[2][D / 64][kManyThreads];  // the codes of keys and values on their way
  // the piece's rows: {factor of scores, the same, shift - reference, the same} of pairs of rows,
  // the reference, the last change of it, 1 / sum, a slope, the position, the step's
  // token, the row of `out` counted from the request's first
  alignas(16) float4 fo[NC / 2];
  alignas(16) float m[NC], change[NC], inv[NC], slope[NC];
  int pos[NC], node[NC], out_row[NC];
  alignas(8) unsigned long long qk_done, pv_done, drained;  // completed by the tensor pipe
  ChunkRef refs[4];  // of chunk j in j mod 4
  uint32_t tmem;
  long long scan[kManyThreads / 32 + 2];
  static __host__ __device__ constexpr int used() {
    return (int)(offsetof(ManySmem, scan) + sizeof(scan));
  }
};
// Where the members end (the struct's size is a whole number of 1024), and with what aligns them.
template <int D, int NC>
__host__ __device__ constexpr int many_used() {
  return ManySmem<D, NC>::used();
}
template <int D, int NC>
constexpr size_t many_smem() {
  return 1024 + many_used<D, NC>();
}

__device__ __forceinline__ float warp_top(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// N columns of tensor memory from `addr` on.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&x)[N]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  if constexpr (N == 16) {
    tmem_load16(addr, r);
  } else {
    static_assert(N == 24, "");
    tmem_load16(addr, r);
    tmem_load8(addr + 16, r + 16);
  }
  tmem_loaded();
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const float (&x)[N]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
  if constexpr (N == 16) {
    tmem_store16(addr, r);
  } else {
    static_assert(N == 24, "");
    tmem_store16(addr, r);
    tmem_store8(addr + 16, r + 16);
  }
  tmem_stored();
}

template <int D, int NC>
__global__ void __launch_bounds__(kManyThreads, 2) many_kernel(const AttendParams p) {
  extern __shared__ __align__(16) char many_raw[];
  ManySmem<D, NC>& sm = *reinterpret_cast<ManySmem<D, NC>*>(
      many_raw + ((1024 - (smem_u32(many_raw) & 1023)) & 1023));
  const TreeView tree(reinterpret_cast<char*>(&sm) + many_used<D, NC>(), sm.p, p.N);  // (if p.parent)
  float(&joined)[4][NC] = *reinterpret_cast<float(*)[4][NC]>(sm.p + 64 * NC * sizeof(float));
  constexpr int G = D / 32;     // groups of a row
  constexpr int kU = Part<D>::kU;
  constexpr int NH = NC / 2;    // rows of a thread
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int cta = blockIdx.x;
  if (tid == 0) {
    mbar_init(smem_u32(&sm.qk_done), 1);
    mbar_init(smem_u32(&sm.pv_done), 1);
    mbar_init(smem_u32(&sm.drained), 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  const Share share = find_share<kManyThreads>(p, cta, gridDim.x, sm.scan);
  if (tid == 0) {
    p.desc[4 * cta + 3] = 0;
    p.late[cta] = 0;
  }
  if (cta >= share.G) return;
  if (warp == 0) tmem_alloc<kTmemCols>(smem_u32(&sm.tmem));
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  const unsigned long long limit = p.wait_ns;
  const uint32_t qk_bar = smem_u32(&sm.qk_done), pv_bar = smem_u32(&sm.pv_done);

  // decoding: rows `slot` and (D = 128) 8 behind it, in one 16 slots' page, of the chunk's; group g
  const int r8 = tid & 7, g = (tid >> 3) % G, my_slot = (tid >> 3) / G * (8 * kU) + r8;
  const int block = page_bytes(1, D) << p.cache.shift;
  Part<D> keys, vals;
  Finder<D, false> finder;  // (warp 7)
  auto find = [&] {
    if (warp == 7) finder.find(p, sm.refs);
  };
  const int code_at = (my_slot & 15) * (D / 2) + g * 16;  // from the 16 slots' first codes
  const int scale_off = (my_slot & 15) + g * 16;          // and from their scales
  const uint32_t raw_at = smem_u32(&sm.raw[0][0][tid]);
  auto load = [&](const ChunkRef& ref, Part<D>& x, bool values) {
    x.off = 0;
    if (ref.valid) {  // (the cache has a page at all)
      const int more = values ? block : 0;
      const unsigned long long codes = ref.codes[my_slot >> 4] + (code_at + more);
      const unsigned long long scales = ref.scales[my_slot >> 4] + (scale_off + more);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        copy16(raw_at + ((values ? kU : 0) + i) * kManyThreads * 16, codes + i * 4 * D);
        x.scale[i] = load_byte(scales + i * 8);
      }
    }
    if (!ref.whole) {
      const bool there = ref.valid >> (my_slot >> 4) & 1;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int slot = my_slot + 8 * i;
        if (!there || (values && (slot < ref.first || slot >= ref.last))) x.off |= 1u << i;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // where the thread's four words of a row go (the rows of a tile's next blocks follow at a stride)
  uint32_t row_to[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    row_to[q] = smem_u32(sm.v) + (g >> 1) * kBlockBytes + my_slot * 128 +
                ((((g & 1) * 4 + q) ^ r8) << 4);
  // `tile`: bytes from the values' tile on; `nothing`: the scale of a row that has none (the codes are in)
  auto put = [&](const Part<D>& x, int tile, uint32_t nothing) {
    uint4 w4[kU];  // (all loads before the stores, behind which the compiler leaves them)
#pragma unroll
    for (int i = 0; i < kU; ++i) w4[i] = sm.raw[tile == 0][i][tid];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      Scale2 sc;
      sc.set((x.off >> i & 1 ? nothing : x.scale[i] * 128u + 0x400u) * 0x10001u);
      const uint32_t words[4] = {w4[i].x, w4[i].y, w4[i].z, w4[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t d[4];
        decode_word(words[q], sc, d);
        store16(row_to[q] + tile + 8 * i * 128, d);
      }
    }
  };
  constexpr int kKeyTile = D / 64 * (int)kBlockBytes;  // (behind the values')

  // Q and the constants of the rows of the piece that `w` stands at: D / 8 threads a row
  auto bring_rows = [&](const Walk& w, bool sees) {
    constexpr int kPer = D / 8;
    const int rows = w.r.nq * p.group, x = tid % kPer;
    for (int at = tid / kPer; at < NC; at += kManyThreads / kPer) {
      const int row = w.tile * NC + at;
      const int clamped = min(row, max(rows - 1, 0));
      const int i = clamped / p.group, head = w.h * p.group + clamped - i * p.group;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < rows && w.r.ok)
        v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + w.b * p.qb +
                                           i * p.qn + (long long)head * p.qh)[x];
      float down;
      *reinterpret_cast<uint4*>(sm.q + (x / 8) * (NC * 128) + at * 128 + (((x & 7) ^ (at & 7)) << 4)) =
          scaled_query<kPer>(v, p.scale < 0.f, &down);
      if (x == 0) {
        float* fo = reinterpret_cast<float*>(&sm.fo[at / 2]) + (at & 1);
        fo[0] = score_factor(p, down);
        fo[2] = kNoRef;
        sm.m[at] = -INFINITY;
        sm.slope[at] = p.slopes ? p.slopes[head] * kLog2e : 0.f;
        sm.node[at] = i;
        sm.pos[at] = w.r.base + (p.parent && sees ? tree.depth(i) : i);
        sm.out_row[at] = i * p.Hq + head;
      }
    }
  };

  const uint64_t q_desc = smem_desc(smem_u32(sm.q), 16), k_desc = smem_desc(smem_u32(sm.k), 16);
  const uint64_t v_desc = smem_desc(smem_u32(sm.v), kBlockBytes);
  const uint64_t p_desc = smem_desc(smem_u32(sm.p), kBlockBytes);
  auto issue_scores = [&](unsigned j) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      mma_ss(tmem + (j & 1) * kSCol, k_desc + (((i / 4) * kBlockBytes + (i % 4) * 32) >> 4),
             q_desc + (((i / 4) * (NC * 128) + (i % 4) * 32) >> 4), idesc(NC, false, false), i > 0);
    mma_commit(qk_bar);
  };
  // (at D = 64 the second block of dimensions is the next tile, and nothing reads its rows)
  auto issue_out = [&](bool add) {
#pragma unroll
    for (int i = 0; i < kSlotsTile / 16; ++i)
      mma_ss(tmem + kOCol, v_desc + (i * 2048 >> 4), p_desc + (i * 2048 >> 4), idesc(NC, true, true),
             add || i > 0);
    mma_commit(pv_bar);
  };

  // softmax: this thread's slot of the chunk (or dimension of O), its half of the rows
  const int quarter = warp & 3, row_at = (warp >> 2) * NH, slot_at = quarter * 32 + lane;
  const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + row_at;
  const float cap = p.softcap * kLog2e;

  Walk w(p, share);
  finder.start(p, share, nullptr);
  find();
  find();
  find();
  __syncthreads();
  load(sm.refs[0], keys, false);
  load(sm.refs[0], vals, true);
  // (a chunk's worth of work lies between a load and the use of it)
  const unsigned n = (unsigned)w.left;
  // (copies of keys and of values are queued in turn, so one group behind the wanted one may be in
  // flight: the other's.  Not behind a piece's second keys, which come right after the first, nor
  // behind its last values, before which no keys are put.)
  auto put_keys = [&](unsigned i, bool second) {  // of chunk i, then the next one's are on their way
    if (second)
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    put(keys, kKeyTile, 0x7fffu);
    if (i + 1 < n)
      load(sm.refs[(i + 1) & 3], keys, false);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto put_values = [&](unsigned i, bool last) {
    if (last)
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    put(vals, 0, 0u);
    if (i + 1 < n)
      load(sm.refs[(i + 1) & 3], vals, true);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
  };
  unsigned j = 0;       // chunks so far
  bool late = false;    // a wait ran out (the same in every thread)
  while (w.left > 0) {
    const int b = w.b, h = w.h, tile = w.tile, c0 = w.c;
    const Request r = w.r;
    const long long left0 = w.left;
    const int c1 = (int)min((long long)r.chunks, c0 + left0);
    const int row0 = tile * NC, n_rows = min(NC, r.nq * p.group - row0);
    bool sees = r.ok && r.len > 0;
    if (p.parent && sees) sees = build_tree<kManyThreads>(p, b, r.nq, tree);
    bring_rows(w, sees);
    put_keys(j, false);
    fence_proxy_async();
    fence_before();
    __syncthreads();
    if (warp == 0 && !late && elect_one()) {
      fence_after();
      issue_scores(j);
    }
    __syncwarp();
    f32x2 l[NH / 2];
#pragma unroll
    for (int i = 0; i < NH / 2; ++i) l[i] = pack2(0.f, 0.f);
    bool far = false;  // a row's max is (the same in every thread)
    for (int c = c0; c < c1 && !late; ++c, ++j) {
      bool out_of_time = !sleep_wait(qk_bar, j & 1, limit);
      // the next chunk's keys, whose product runs while this chunk's weights are worked out
      if (c + 1 < c1) put_keys(j + 1, c == c0);
      fence_proxy_async();
      fence_after();
      const int slot0 = (r.lo / kSlotsTile + c) * kSlotsTile, slot = slot0 + slot_at;
      const bool edge = !sees || slot0 + kSlotsTile > r.base ||
                        (p.window > 0 && slot0 <= r.base + r.nq - 1 - p.window);
      const bool plain = !edge && p.softcap == 0.f && !p.slopes;
      float s[NH];
      // scores in units of log2, before the rows' factors where plain
      auto load_scores = [&] {
        tmem_load(mine + (j & 1) * kSCol, s);
        if (plain) return;
        const bool there = sees && slot < r.len;
        const int node = slot - r.base;
        int at = slot;
        if (p.parent && there && node >= 0) at = r.base + tree.depth(node);
        auto each = [&](auto f) {
#pragma unroll
          for (int i = 0; i < NH; ++i)
            s[i] = f(s[i] * reinterpret_cast<const float*>(&sm.fo[(row_at + i) / 2])[i & 1]);
        };
        if (p.softcap > 0.f)
          cap_all<false>(cap, each);
        else
          each([](float y) { return y; });
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          const int row = row_at + i;
          float y = s[i];
          if (p.slopes) y = fmaf(-sm.slope[row], (float)(sm.pos[row] - at), y);
          bool seen = there;
          if (edge && there && node >= 0) {
            const int other = sm.node[row];
            seen = p.parent ? tree.sees(other, node) : node <= other;
          }
          if (edge && p.window > 0 && sm.pos[row] - at >= p.window) seen = false;
          s[i] = seen ? y : -INFINITY;
        }
      };
      for (bool moved = false;;) {
        load_scores();
        // exponents of the weights; is one too large for its row's reference?
        float top[2] = {-INFINITY, -INFINITY};
        if (far) {
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const int row = row_at + i;
            const float f = plain ? reinterpret_cast<const float*>(&sm.fo[row / 2])[row & 1] : 1.f;
            s[i] = far_exponent(s[i], f, sm.m[row], kManyShift);
          }
        } else if (plain) {
#pragma unroll
          for (int i = 0; i < NH / 2; ++i) {
            const float4 fo = sm.fo[row_at / 2 + i];
            unpack2(fma2(pack2(s[2 * i], s[2 * i + 1]), pack2(fo.x, fo.y), pack2(fo.z, fo.w)),
                    s[2 * i], s[2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NH / 2; ++i) {
            const float4 fo = sm.fo[row_at / 2 + i];
            s[2 * i] += fo.z;
            s[2 * i + 1] += fo.w;
          }
        }
        if (moved) break;
#pragma unroll
        for (int i = 0; i < NH / 2; ++i) top[i & 1] = max3(top[i & 1], s[2 * i], s[2 * i + 1]);
        fence_before();
        moved = __syncthreads_or(fmaxf(top[0], top[1]) > kManyShift + kSlack);
        if (warp == 0 && !late && c + 1 < c1 && elect_one()) {
          fence_after();
          issue_scores(j + 1);
        }
        __syncwarp();
        if (!moved) break;
        // each row's max over the chunk's slots (`joined` lies in the last chunk's weights)
        if (c > c0) out_of_time |= !sleep_wait(pv_bar, (j - 1) & 1, limit);
        fence_after();
        load_scores();
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          float y = s[i];
          if (plain) y *= reinterpret_cast<const float*>(&sm.fo[(row_at + i) / 2])[i & 1];
          y = warp_top(y);
          if (lane == i) joined[quarter][row_at + i] = y;
        }
        __syncthreads();
        bool mine_far = false;
        if (tid < NC) {
          const float old = sm.m[tid];
          const float m = fmaxf(fmaxf(old, joined[0][tid]),
                                max3(joined[1][tid], joined[2][tid], joined[3][tid]));
          sm.m[tid] = m;
          sm.change[tid] = old == -INFINITY ? 0.f : ex2(old - m);
          reinterpret_cast<float*>(&sm.fo[tid / 2])[2 + (tid & 1)] =
              m == -INFINITY ? kNoRef : kManyShift - m;
          mine_far = is_far(m);
        }
        far = __syncthreads_or(mine_far) != 0;
        if (c > c0) {  // the sums and O so far
          float o[NH];
          tmem_load(mine + kOCol, o);
#pragma unroll
          for (int i = 0; i < NH / 2; ++i) {
            const float2 x = *reinterpret_cast<const float2*>(&sm.change[row_at + 2 * i]);
            l[i] = fma2(l[i], pack2(x.x, x.y), pack2(0.f, 0.f));
            o[2 * i] *= x.x;
            o[2 * i + 1] *= x.y;
          }
          tmem_store(mine + kOCol, o);
        }
      }
      find();  // (in the place of the chunk before this one)
      uint32_t x[NH / 2];
#pragma unroll
      for (int i = 0; i < NH / 2; ++i) {
        const float w0 = ex2(s[2 * i]), w1 = ex2(s[2 * i + 1]);
        l[i] = add2(l[i], pack2(w0, w1));
        x[i] = pack_f16(w0, w1);
      }
      // weights and values in the place of the last chunk's, whose product had the time since
      if (c > c0) out_of_time |= !sleep_wait(pv_bar, (j - 1) & 1, limit);
      const uint32_t to = smem_u32(sm.p) + slot_at * 128;
#pragma unroll
      for (int i = 0; i < NH / 8; ++i)
        store16(to + (((row_at / 8 + i) ^ (slot_at & 7)) << 4),
                {x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]});
      put_values(j, c + 1 == c1);
      fence_proxy_async();
      fence_before();
      late = __syncthreads_or(out_of_time);
      if (warp == 0 && !late && elect_one()) {
        fence_after();
        issue_out(c > c0);
      }
      __syncwarp();
    }

    w.skip(p, c1 - c0);  // (stands at the next piece from here on)

    // the piece's rows: their sums over the slots, by way of the weights' place
    if (!late) late = __syncthreads_or(!mbar_wait(pv_bar, (j - 1) & 1, limit));
    fence_after();
    const bool whole = c0 == 0 && c1 == r.chunks;
    float* part = p.part + (long long)(2 * cta + (left0 == share.end - share.begin ? 0 : 1)) * NC * (D + 4);
    const long long out0 = (long long)b * p.N * p.Hq;
    float* sums = reinterpret_cast<float*>(sm.p);
#pragma unroll
    for (int i = 0; i < NH / 2; ++i) {
      float x, y;
      unpack2(l[i], x, y);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      y += __shfl_xor_sync(0xffffffffu, y, 16);
      if (lane < 16)
        *reinterpret_cast<float2*>(&sums[(quarter * 16 + lane) * NC + row_at + 2 * i]) =
            make_float2(x, y);
    }
    __syncthreads();
    if (tid < 4 * NC) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += sums[(tid / NC * 16 + i) * NC + tid % NC];
      joined[tid / NC][tid % NC] = sum;
    }
    __syncthreads();
    if (tid < NC) {
      float sum = (joined[0][tid] + joined[1][tid]) + (joined[2][tid] + joined[3][tid]);
      if (late) sum = qnan();
      sm.inv[tid] = sum == 0.f ? 0.f : 1.f / sum;
      if (tid < n_rows) {
        if (!whole) {
          part[tid * (D + 4) + D] = sm.m[tid];
          part[tid * (D + 4) + D + 1] = sum;
        } else if (p.out_lse) {
          p.out_lse[out0 + sm.out_row[tid]] = log_sum(sm.m[tid], sum, kManyShift);
        }
      }
    }
    __syncthreads();
    uint16_t* rows_out = reinterpret_cast<uint16_t*>(sm.p);  // [row][D], as bf16
    if (D == 128 || quarter < 2) {
      float o[NH];
      tmem_load(mine + kOCol, o);
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const int row = row_at + i;
        float x = late ? qnan() : o[i];
        if (!whole) {
          if (row < n_rows) part[row * (D + 4) + slot_at] = x;
        } else {
          const float inv = sm.inv[row];
          x = inv == 0.f ? 0.f : x * inv;
          rows_out[row * D + slot_at] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        }
      }
    }
    __syncthreads();
    if (whole) {
      constexpr int kPer = D / 8;  // 16-byte units of a row
      for (int i = tid; i < n_rows * kPer; i += kManyThreads)
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                 (out0 + sm.out_row[i / kPer]) * D)[i % kPer] =
            reinterpret_cast<const uint4*>(rows_out)[i];
    } else if (c0 == 0 && tid == 0) {
      int* desc = p.desc + 4 * cta;
      desc[0] = b;
      desc[1] = h;
      desc[2] = tile | (left0 == share.end - share.begin ? 0 : 1 << 30);
      desc[3] = pieces_of(share, cta, share.end - left0 + r.chunks);
    }
    fence_before();
    __syncthreads();  // (the rows' constants are read)
  }
  if (late && tid == 0) p.late[cta] = 1;
  // nothing is in flight when tensor memory is freed
  if (warp == 0) {
    if (elect_one()) mma_commit(smem_u32(&sm.drained));
    __syncwarp();
    mbar_wait(smem_u32(&sm.drained), 0);
    __syncwarp();
    tmem_free<kTmemCols>(tmem);
  }
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
                               (int)(many_smem<D, NC>() + tree_bytes(SV_MAX_STEP)));
    if (err != cudaSuccess) return err;
    ready[dev].store(1, std::memory_order_relaxed);
  }
  return launch_early(many_kernel<D, NC>, plan.ctas, kManyThreads,
                      many_smem<D, NC>() + (p.parent ? tree_bytes(p.N) : 0), 1, stream, p);
}

}  // namespace

cudaError_t plan_many(int rows, AttendPlan* plan) {
  DeviceInfo info;
  const cudaError_t err = device_info(&info);
  if (err != cudaSuccess) return err;
  // One tile of 32 or 48 rows, or tiles of 128 (sv_attend_rows.cu): of 32 requests of up to 4096 slots, 8 heads of
  // 128, 32 rows take 92 against 106 us, 48 rows 112 against 111 (but 288 against 302 of 64 requests of up to
  // 8192); two tiles of 32 take 154 against 115, two of 48 183 against 122, 252 against 200 at 144 rows.  (For
  // one request of 64 or 96 rows the small tiles would be faster, 28 against 35 us and 32 against
  // 38, for one of 244 slower, 48 against 42.)
  plan->rows = rows <= 32 ? 32 : rows <= 48 ? 48 : 128;
  plan->chunk = kSlotsTile;
  plan->least = 1;
  plan->shift = kManyShift;
  plan->ctas = 2 * info.sms;
  plan->fold = 0;
  return cudaSuccess;
}

cudaError_t launch_many(const AttendParams& p, int D, const AttendPlan& plan, cudaStream_t stream) {
  if (plan.rows == 128) return launch_rows(p, D, plan, stream);
#define SV_MANY(d, n) \
  if (D == d && plan.rows == n) return launch_one<d, n>(p, plan, stream);
  SV_MANY(64, 32) SV_MANY(64, 48) SV_MANY(128, 32) SV_MANY(128, 48)
#undef SV_MANY
  return cudaErrorInvalidValue;
}

}  // namespace sv
