// sv_attend_rows.cu - attention over the 4-bit cache for very many query rows
// (spec_cache_attention): tensor memory, 128 rows a tile.
//
// A unit is a tile of 128 query rows of a key/value head, a chunk 128 slots:
//   S = Q K^T    128 rows x 128 slots x D, both operands in shared memory
//   O += P V     128 rows x D x 128 slots, the weights P in tensor memory over S
// in fp16 with 32-bit sums.  What the kernel for tiles of 32 or 48 rows (sv_attend_many.cu) spends on
// decoding a chunk serves 128 rows here.  A thread has a row and half of the chunk's slots, so
// that a row's factors, max and sum are its own; scores are read from tensor memory twice, once for the
// largest and once for the weights, 16 at a time (32: spilled registers, 294 instead of 230 us below).
// Two CTAs an SM, whose 8 warps all do the same; the next chunk's keys take the place of this one's as
// soon as S is out, the values' codes wait in registers.
// The tensor pipe counts as busy in 87 % of the cycles, issue slots are 45 % used; a chunk of a tile takes some 4800
// cycles of an SM where its products at the measured peak rate would take 1300, and whether the products themselves or
// what they wait for makes the difference has not been measured apart.  Measured: 222 us for trees of 61 nodes over 32 requests
// of up to 4096 slots (4 heads a group, 8 groups of 128), 450 TFLOP/s of the trees' own products.
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/spec_verify.h"
#include "sv_attend_tc.cuh"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

constexpr int kRowsThreads = 256;
constexpr int kTileRows = 128;
constexpr int kTmemCols = 256;
constexpr int kOCol = 128;  // O's columns; S and P: 0

template <int D>
struct RowsSmem {
  static constexpr int kTileBytes = D / 64 * (int)kBlockBytes;
  alignas(1024) char v[kTileBytes];  // (while a piece begins: a tree's parents)
  alignas(1024) char k[kTileBytes];
  alignas(1024) char q[kTileBytes];
  uint4 raw[D / 64][kRowsThreads];  // the codes of keys on their way
  float joined[2][kTileRows];       // of a row's two threads
  // the piece's rows: factor of scores, a slope, the position, the step's token, the row of `out` counted
  // from the request's first
  float fo[kTileRows], slope[kTileRows];
  int pos[kTileRows], node[kTileRows], out_row[kTileRows];
  alignas(8) unsigned long long qk_done, pv_done, drained;  // completed by the tensor pipe
  ChunkRef refs[4];  // of chunk j in j mod 4
  FinderState finder;
  uint32_t tmem;
  long long scan[kRowsThreads / 32 + 2];
  static __host__ __device__ constexpr int used() {
    return (int)(offsetof(RowsSmem, scan) + sizeof(scan));
  }
};
template <int D>
__host__ __device__ constexpr int rows_used() {
  return RowsSmem<D>::used();
}
template <int D>
constexpr size_t rows_smem() {
  return 1024 + rows_used<D>();
}

__device__ __forceinline__ uint4 load16(unsigned long long src) {
  uint4 x;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(src)
               : "memory");
  return x;
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads, 2) rows_kernel(const AttendParams p) {
  extern __shared__ __align__(16) char rows_raw[];
  RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>(
      rows_raw + ((1024 - (smem_u32(rows_raw) & 1023)) & 1023));
  const TreeView tree(reinterpret_cast<char*>(&sm) + rows_used<D>(), sm.v, p.N);  // (if p.parent)
  constexpr int G = D / 32, kU = Part<D>::kU;  // groups of a row; rows of keys or values a thread decodes
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
  const Share share = find_share<kRowsThreads>(p, cta, gridDim.x, sm.scan);
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

  // decoding: rows `my_slot` and (D = 128) 8 behind it, in one 16 slots' page, of the chunk's; group g
  const int r8 = tid & 7, g = (tid >> 3) % G, my_slot = (tid >> 3) / G * (8 * kU) + r8;
  const int block = page_bytes(1, D) << p.cache.shift;
  Part<D> keys, vals;
  uint4 codes[kU];        // of the values
  Finder<D, true> finder;  // (warp 7)
  const int code_at = (my_slot & 15) * (D / 2) + g * 16;  // from the 16 slots' first codes
  const int scale_off = (my_slot & 15) + g * 16;          // and from their scales
  const uint32_t raw_at = smem_u32(&sm.raw[0][tid]);
  auto load_keys = [&](const ChunkRef& ref) {
    keys.off = 0;
    if (ref.valid) {  // (the cache has a page at all)
      const unsigned long long from = ref.codes[my_slot >> 4] + code_at;
      const unsigned long long scales = ref.scales[my_slot >> 4] + scale_off;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        copy16(raw_at + i * kRowsThreads * 16, from + i * 4 * D);
        keys.scale[i] = load_byte(scales + i * 8);
      }
    }
    if (!(ref.valid >> (my_slot >> 4) & 1)) keys.off = (1u << kU) - 1;
  };
  auto load_values = [&](const ChunkRef& ref) {
    vals.off = 0;
    if (ref.valid) {
      const unsigned long long from = ref.codes[my_slot >> 4] + (code_at + block);
      const unsigned long long scales = ref.scales[my_slot >> 4] + (scale_off + block);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        codes[i] = load16(from + i * 4 * D);
        vals.scale[i] = load_byte(scales + i * 8);
      }
    }
    if (!ref.whole) {
      const bool there = ref.valid >> (my_slot >> 4) & 1;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int slot = my_slot + 8 * i;
        if (!there || slot < ref.first || slot >= ref.last) vals.off |= 1u << i;
      }
    }
  };
  // where the thread's four words of a row go (the second row follows at a stride)
  uint32_t row_to[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    row_to[q] = smem_u32(sm.v) + (g >> 1) * kBlockBytes + my_slot * 128 +
                ((((g & 1) * 4 + q) ^ r8) << 4);
  // `tile`: bytes from the values' tile on; `nothing`: the scale of a row that has none
  auto put = [&](const Part<D>& x, const uint4 (&w4)[kU], int tile, uint32_t nothing) {
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
  const unsigned n = (unsigned)(share.end - share.begin);
  auto put_keys = [&](unsigned i) {  // of chunk i, then the next one's are on their way
    asm volatile("cp.async.wait_all;" ::: "memory");
    uint4 w4[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) w4[u] = sm.raw[u][tid];
    put(keys, w4, D / 64 * (int)kBlockBytes, 0x7fffu);
    if (i + 1 < n) load_keys(sm.refs[(i + 1) & 3]);
  };
  auto put_values = [&](unsigned i) {
    put(vals, codes, 0, 0u);
    if (i + 1 < n) load_values(sm.refs[(i + 1) & 3]);
  };

  // Q and the constants of the rows of the piece that `w` stands at: D / 8 threads a row
  auto bring_rows = [&](const Walk& w, bool sees) {
    constexpr int kPer = D / 8;
    const int rows = w.r.nq * p.group, x = tid % kPer;
    for (int at = tid / kPer; at < kTileRows; at += kRowsThreads / kPer) {
      const int row = w.tile * kTileRows + at;
      const int clamped = min(row, max(rows - 1, 0));
      const int i = clamped / p.group, head = w.h * p.group + clamped - i * p.group;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row < rows && w.r.ok)
        v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + w.b * p.qb +
                                           i * p.qn + (long long)head * p.qh)[x];
      float down;
      *reinterpret_cast<uint4*>(sm.q + (x / 8) * kBlockBytes + at * 128 + (((x & 7) ^ (at & 7)) << 4)) =
          scaled_query<kPer>(v, p.scale < 0.f, &down);
      if (x == 0) {
        sm.fo[at] = score_factor(p, down);
        sm.slope[at] = p.slopes ? p.slopes[head] * kLog2e : 0.f;
        sm.node[at] = i;
        sm.pos[at] = w.r.base + (p.parent && sees ? tree.depth(i) : i);
        sm.out_row[at] = i * p.Hq + head;
      }
    }
  };

  const uint64_t q_desc = smem_desc(smem_u32(sm.q), 16), k_desc = smem_desc(smem_u32(sm.k), 16);
  const uint64_t v_desc = smem_desc(smem_u32(sm.v), kBlockBytes);
  auto issue_scores = [&] {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint64_t at = ((i / 4) * kBlockBytes + (i % 4) * 32) >> 4;
      mma_ss(tmem, q_desc + at, k_desc + at, idesc(kSlotsTile, false, false), i > 0);
    }
    mma_commit(qk_bar);
  };
  auto issue_out = [&](bool add) {  // (weights of 64 slots lie in the first 32 columns of their scores')
#pragma unroll
    for (int i = 0; i < kSlotsTile / 16; ++i)
      mma_ts(tmem + kOCol, tmem + i / 4 * 64 + i % 4 * 8, v_desc + (i * 2048 >> 4),
             idesc(D, false, true), add || i > 0);
    mma_commit(pv_bar);
  };

  // softmax: this thread's row, its half of the chunk's slots and of O's dimensions
  const int row = (warp & 3) * 32 + lane, half = warp >> 2;
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), mine = lanes + half * 64;
  const float cap = p.softcap * kLog2e;

  Walk w(p, share);
  if (warp == 7) {
    finder.start(p, share, &sm.finder);
    for (int i = 0; i < 3; ++i) finder.find(p, sm.refs);
  }
  __syncthreads();
  load_keys(sm.refs[0]);
  load_values(sm.refs[0]);
  unsigned j = 0;       // chunks so far
  bool late = false;    // a wait ran out (the same in every thread)
  while (w.left > 0) {
    const int b = w.b, h = w.h, tile = w.tile, c0 = w.c;
    const Request r = w.r;
    const long long left0 = w.left;
    const int c1 = (int)min((long long)r.chunks, c0 + left0);
    const int n_rows = min(kTileRows, r.nq * p.group - tile * kTileRows);
    bool sees = r.ok && r.len > 0;
    if (p.parent && sees) sees = build_tree<kRowsThreads>(p, b, r.nq, tree);
    bring_rows(w, sees);
    put_keys(j);
    fence_proxy_async();
    fence_before();
    __syncthreads();
    if (warp == 0 && !late && elect_one()) {
      fence_after();
      issue_scores();
    }
    __syncwarp();
    const float f = sm.fo[row];
    float m = -INFINITY;
    f32x2 l = pack2(0.f, 0.f);
    for (int c = c0; c < c1 && !late; ++c, ++j) {
      bool out_of_time = false;
      if (c > c0) {  // the last chunk's product is out: its weights' and values' places are free
        out_of_time = !sleep_wait(pv_bar, (j - 1) & 1, limit);
        __syncwarp();
        fence_after();
        if (warp == 0 && !__any_sync(0xffffffffu, out_of_time) && elect_one()) issue_scores();
        __syncwarp();
      }
      put_values(j);
      out_of_time = !sleep_wait(qk_bar, j & 1, out_of_time ? 0 : limit) || out_of_time;
      __syncwarp();
      fence_after();
      const int slot0 = (r.lo / kSlotsTile + c) * kSlotsTile;
      const bool edge = !sees || slot0 + kSlotsTile > r.base ||
                        (p.window > 0 && slot0 <= r.base + r.nq - 1 - p.window);
      const bool plain = !edge && p.softcap == 0.f && !p.slopes;
      // scores of 16 slots in units of log2, before the row's factor where plain
      auto load_scores = [&](int part, float (&s)[16]) {
        tmem_load16(mine + 16 * part, reinterpret_cast<uint32_t*>(s));
        tmem_loaded();
        if (plain) return;
        auto each = [&](auto fn) {
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = fn(s[i] * f);
        };
        if (p.softcap > 0.f)
          cap_all<false>(cap, each);
        else
          each([](float y) { return y; });
        if (!edge && !p.slopes) return;
        const int first = slot0 + 64 * half + 16 * part, other = sm.node[row], pos = sm.pos[row];
        const float slope = sm.slope[row];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int slot = first + i, node = slot - r.base;
          bool seen = sees && slot < r.len;
          int at = slot;
          if (node >= 0 && seen) {
            if (p.parent) at = r.base + tree.depth(node);
            seen = p.parent ? tree.sees(other, node) : node <= other;
          }
          if (p.slopes) s[i] = fmaf(-slope, (float)(pos - at), s[i]);
          if (p.window > 0 && pos - at >= p.window) seen = false;
          if (!seen) s[i] = -INFINITY;
        }
      };
      const float fe = plain ? f : 1.f;
      float top = -INFINITY;
#pragma unroll 1
      for (int part = 0; part < 4; ++part) {
        float s[16], t[2] = {-INFINITY, -INFINITY};
        load_scores(part, s);
#pragma unroll
        for (int i = 0; i < 16; i += 2) t[i / 2 & 1] = max3(t[i / 2 & 1], s[i], s[i + 1]);
        top = max3(top, t[0], t[1]);
      }
      top *= fe;  // (factors are not negative)
      if (__syncthreads_or(top - m > kSlack)) {
        // each row's max over the chunk's slots
        sm.joined[half][row] = top;
        __syncthreads();
        const float now = max3(m, top, sm.joined[half ^ 1][row]);
        const float change = m == -INFINITY ? 0.f : ex2(m - now);
        m = now;
        l = fma2(l, pack2(change, change), pack2(0.f, 0.f));
        if (c > c0) {
#pragma unroll 1
          for (int part = 0; part < D / 64; ++part) {
            float o[32];
            const uint32_t at = lanes + kOCol + half * (D / 2) + 32 * part;
            tmem_load32(at, o);
            tmem_loaded();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= change;
            tmem_store16(at, reinterpret_cast<const uint32_t*>(o));
            tmem_store16(at + 16, reinterpret_cast<const uint32_t*>(o + 16));
          }
          tmem_stored();
        }
      }
      if (warp == 7) finder.find(p, sm.refs);  // (in the place of the chunk before this one)
      const float off = m == -INFINITY ? kNoRef : kManyShift - m;
      auto weights = [&](auto exponents) {
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {
          float s[16];
          uint32_t x[8];
          load_scores(part, s);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float w0, w1;
            unpack2(exponents(s[2 * i], s[2 * i + 1]), w0, w1);
            w0 = ex2(w0);
            w1 = ex2(w1);
            l = add2(l, pack2(w0, w1));
            x[i] = pack_f16(w0, w1);
          }
          tmem_store8(mine + 8 * part, x);
        }
      };
      if (!__any_sync(0xffffffffu, is_far(m)))
        weights([&](float y0, float y1) {
          return fma2(pack2(y0, y1), pack2(fe, fe), pack2(off, off));
        });
      else
        weights([&](float y0, float y1) {
          return pack2(far_exponent(y0, fe, m, kManyShift), far_exponent(y1, fe, m, kManyShift));
        });
      tmem_stored();
      // the next chunk's keys (their place is free: this chunk's scores are out)
      if (c + 1 < c1) put_keys(j + 1);
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
    if (!late) late = __syncthreads_or(!mbar_wait(pv_bar, (j - 1) & 1, limit));
    __syncwarp();
    fence_after();
    const bool whole = c0 == 0 && c1 == r.chunks;
    const bool first = left0 == share.end - share.begin;
    float l0, l1;
    unpack2(l, l0, l1);
    sm.joined[half][row] = l0 + l1;
    __syncthreads();
    float sum = sm.joined[0][row] + sm.joined[1][row];
    if (late) sum = qnan();
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float* part = p.part + ((long long)(2 * cta + (first ? 0 : 1)) * kTileRows + row) * (D + 4);
    const long long to = (long long)b * p.N * p.Hq + sm.out_row[row];
    if (half == 0 && row < n_rows) {
      if (!whole) {
        part[D] = m;
        part[D + 1] = sum;
      } else if (p.out_lse) {
        p.out_lse[to] = log_sum(m, sum, kManyShift);
      }
    }
#pragma unroll 1
    for (int at = half * (D / 2); at < (half + 1) * (D / 2); at += 32) {
      float o[32];
      tmem_load32(lanes + kOCol + at, o);
      tmem_loaded();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (late) o[i] = qnan();
        if (whole) o[i] = inv == 0.f ? 0.f : o[i] * inv;
      }
      if (row >= n_rows) {
      } else if (!whole) {
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(part + at + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to * D + at + i) =
              make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]),
                         pack_bf16(o[i + 4], o[i + 5]), pack_bf16(o[i + 6], o[i + 7]));
      }
      __syncwarp();
    }
    if (!whole && c0 == 0 && tid == 0) {
      int* desc = p.desc + 4 * cta;
      desc[0] = b;
      desc[1] = h;
      desc[2] = tile | (first ? 0 : 1 << 30);
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

template <int D>
cudaError_t launch_one(const AttendParams& p, const AttendPlan& plan, cudaStream_t stream) {
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    err = cudaFuncSetAttribute(rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)(rows_smem<D>() + tree_bytes(SV_MAX_STEP)));
    if (err != cudaSuccess) return err;
    ready[dev].store(1, std::memory_order_relaxed);
  }
  return launch_early(rows_kernel<D>, plan.ctas, kRowsThreads,
                      rows_smem<D>() + (p.parent ? tree_bytes(p.N) : 0), 1, stream, p);
}

}  // namespace

cudaError_t launch_rows(const AttendParams& p, int D, const AttendPlan& plan, cudaStream_t stream) {
  return D == 64 ? launch_one<64>(p, plan, stream) : launch_one<128>(p, plan, stream);
}

}  // namespace sv
