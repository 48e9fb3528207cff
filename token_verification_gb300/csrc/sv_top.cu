// sv_top.cu - the k largest logits of each row with its log-sum-exp
// (spec_top_logits), and beam selection over beams and vocabulary
// (spec_beam_select): the entry points, and the kernel for few rows, a
// thread-block cluster per row or request.
//
// A row (of a request's W beams, or the one row of a record) is cut into
// `slices`; the (row, slice) items are dealt to the cluster's CTAs, which
// stream them and select as sv_select.cuh describes.  Each CTA sends its items'
// sums and units to all others (asynchronous remote stores counted by the
// receiver's mbarrier) and works out offsets and bound for itself; the
// candidates go to the leader CTA's list, before a cluster barrier.
//
// It is bound by the chain of its steps - launch, stream, exchange, bound, reload,
// sort -, not by bytes: 1 to 8 rows of 64000 to 128256 bf16 logits take 6.0 to 6.4
// us (k = 32, calls of a captured graph), four beams of 32000 7.8 us. Ordering
// cluster barriers in place of the counted stores cost 0.7 us.
//
// A beam's candidates compare by their scores in 64 bits (tied_before: and then), a
// record's by their logits.  Bounds are in fp32 rounded down, which can only lengthen the list.
#include <string.h>

#include <algorithm>

#include "sv_select.cuh"

namespace sv {
namespace {

constexpr int kMaxItems = 64;         // (row, slice) items per cluster

struct alignas(16) TopShared {
  alignas(16) float2 part[kMaxItems][kTopWarps];  // per item and warp: {max, sum of 2^((l - max) c)}
  alignas(16) uint16_t unit[kMaxUnits];  // unit maxes, item by item: bf16 rounded down
  double off[SV_MAX_BEAMS];           // beams: each row's offset (-inf: no candidates)
  float max[SV_MAX_BEAMS];            // and its max
  float off_down[SV_MAX_BEAMS];       // the same rounded down
  float thr[SV_MAX_BEAMS];            // the lowest logit a candidate of the row can have
  unsigned long long part_bar;        // the other CTAs' items have come
  Select sel;
};

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
__global__ void __launch_bounds__(kTopThreads, 3) top_kernel(const TopParams p) {
  constexpr int VEC = Group<T>::VEC;
  constexpr int kWords = kEntry / VEC;  // 16-byte words of a table entry
  extern __shared__ __align__(16) unsigned char smem[];
  TopShared& s = *reinterpret_cast<TopShared*>(smem);
  // per iteration over this CTA's items, the thread's 32 elements' max
  uint16_t* table = reinterpret_cast<uint16_t*>(smem + sizeof(TopShared));
  unsigned char* rings = smem + sizeof(TopShared) + p.table_bytes;
  ListOf<kBeam>& ls = *reinterpret_cast<ListOf<kBeam>*>(rings);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long grp = blockIdx.x / C;
  const int t = threadIdx.x, lane = lane_id(), warp = t / kWarp;
  const int items = p.W * p.slices;
  const RowSpan span = {p.first, p.last};

  pdl_wait();
  pdl_launch_dependents();
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
  const int own = rank < items ? (items - rank + C - 1) / C : 0;
  const int sent = 64 + 2 * p.upi;  // bytes of an item's parts and units
  if (t == 0) {
    s.sel.n_hits = s.sel.n_cands = s.sel.overflow = s.sel.bad = 0;
    if (C > 1) {
      mbar_init(smem_u32(&s.part_bar), 1);
      fence_mbar_init();
      mbar_arrive_expect_tx(smem_u32(&s.part_bar), (uint32_t)((items - own) * sent));
    }
  }
  // no CTA writes into another's shared memory before that one has started
  if (C > 1) cluster_arrive();

  // One pass over each item.
  const int fold = p.fold;
  for (int it = rank, mine = 0; it < items; it += C, ++mine) {
    const int w = it / p.slices, e0 = (it - w * p.slices) * p.slice;
    const int e1 = min(e0 + p.slice, p.V);
    const long long rowid = grp * p.W + w;
    const T* row = reinterpret_cast<const T*>(p.logits) + rowid * (long long)p.V;
    uint16_t* mine_table = table + mine * p.iters * kTopThreads + t;
    const bool live = !kBeam || p.scores[rowid] != -INFINITY;
    RunningSum r;
    if (live) {
      r = stream_slice<T, kAligned, kTopWarps>(smem_u32(rings), warp, row, e0, e1, p.iters, p.cc,
                                               mine_table, span);
    } else {
      for (int i = 0; i < p.iters; ++i) mine_table[i * kTopThreads] = 0xff80u;
    }
    const float2 wr = warp_running(r, p.cc);
    float um = r.m;
    for (int o = 1; o < fold; o <<= 1) um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, o));
    if (lane == 0) s.part[it][warp] = wr;
    if ((t & (fold - 1)) == 0 && t / fold < p.upi) s.unit[it * p.upi + t / fold] = down_bf16(um);
  }
  __syncthreads();
  if (C > 1) {  // this CTA's items to the others, theirs to come
    cluster_wait();
    const int pieces = sent / 16;
    for (int q = t; q < own * pieces * C; q += kTopThreads) {
      const int c = q % C, it = rank + q / C / pieces * C, piece = q / C % pieces;
      const void* from = piece < 4 ? reinterpret_cast<const char*>(s.part[it]) + 16 * piece
                                   : reinterpret_cast<const char*>(s.unit + it * p.upi) +
                                         16 * (piece - 4);
      if (c != rank)
        send16(in_cta(smem_u32(from), c), in_cta(smem_u32(&s.part_bar), c),
               *reinterpret_cast<const float4*>(from));
    }
    if (warp == 0 && !mbar_wait_cluster(smem_u32(&s.part_bar), 0, p.wait_ns)) {
      s.sel.bad = SV_REQ_TIMEOUT;
      cluster.map_shared_rank(&s, 0)->sel.overflow = 1;  // the leader reads all rows itself
      // what was sent lands before the CTA leaves; a peer that has not sent by then has failed
      mbar_wait_cluster(smem_u32(&s.part_bar), 0, kWaitLimitNs);
    }
    __syncthreads();
  }

  // Beams: each row's offset (every CTA for itself). A record's log-sum-exp is for
  // the leader to write when it has loads to wait for; here every warp sees by the
  // max whether there is anything to select.
  const int parts = p.slices * kTopWarps;  // <= 64
  int bad = 0;
  float m = -INFINITY;
  if (kBeam) {
    for (int w = warp; w < p.W; w += kTopWarps) {
      float2 sum;
      const float mw = row_sum(&s.part[w * p.slices][0], parts, p.cc, sum);
      if (lane == 0) {
        const float2 l = log_pair(sum);
        const float score = p.scores[grp * p.W + w];
        const bool dead = score == -INFINITY;
        if (!dead && (mw != mw || mw == INFINITY || score != score || score == INFINITY))
          atomicOr(&s.sel.bad, SV_REQ_BAD_LOGITS);
        double off = -INFINITY;
        if (!dead && mw != -INFINITY) off = row_offset(score, l);
        s.off[w] = off;
        s.max[w] = mw;
        s.off_down[w] = __double2float_rd(off);
      }
    }
    __syncthreads();
    bad = s.sel.bad;
  } else {
    m = warp_max_nan(max_nan(lane < parts ? (&s.part[0][0])[lane].x : -INFINITY,
                             lane + kWarp < parts ? (&s.part[0][0])[lane + kWarp].x : -INFINITY));
    bad = s.sel.bad | (m != m || m == INFINITY ? SV_REQ_BAD_LOGITS : 0);
  }
  if (rank == 0 && t == 0) {
    if (!kBeam && bad) p.out_lse[grp] = qnan();
    if (p.out_status) p.out_status[grp] = bad;
  }
  if (bad) {  // (the same in every CTA, or some did not get their parts)
    if (C > 1) cluster.sync();
    if (rank == 0)
      for (int j = t; j < p.n; j += kTopThreads) write_slot<kBeam>(p, grp, j, 0, -1);
    return;
  }

  // The bound that n elements reach, and each row's lowest candidate logit.
  const int units = items * p.upi;
  if (kBeam) {  // the units' scores, rounded down
    for (int u = t; u < units; u += kTopThreads) {
      const int w = u / (p.upi * p.slices);
      const float l = bf16_lo(s.unit[u]), off = s.off_down[w];
      s.unit[u] = l == -INFINITY || off == -INFINITY
                      ? 0xff80u
                      : down_bf16(beam_score_down(off, s.max[w], l));
    }
  }
  const float bound = unit_bound<0>(s.sel, s.unit, units, p.n);
  if (kBeam) {
    for (int w = t; w < p.W; w += kTopThreads) {
      const double off = s.off[w];
      // below it, the score rounds below the bound (the slack covers the roundings); -inf
      // never passes: at least the lowest finite value
      s.thr[w] = off == -INFINITY ? INFINITY
                 : bound == -INFINITY
                     ? -FLT_MAX
                     : fmaxf(-FLT_MAX,
                             __double2float_rd((((double)bound - off) -
                                                1e-7 * (fabs((double)bound) + fabs(off))) +
                                               (double)s.max[w]));
    }
    __syncthreads();
  }
  auto threshold = [&](int w) { return kBeam ? s.thr[w] : fmaxf(bound, -FLT_MAX); };

  // The groups that reach it, eight table entries a thread.
  for (int it = rank, mine = 0; it < items; it += C, ++mine) {
    scan_table(s.sel, ls, table + mine * p.iters * kTopThreads, p.iters * kTopThreads,
               threshold(it / p.slices), mine * p.iters * kTopThreads);
  }
  __syncthreads();
  TopShared* lead = C > 1 ? cluster.map_shared_rank(&s, 0) : &s;
  ListOf<kBeam>* lead_ls = C > 1 ? cluster.map_shared_rank(&ls, 0) : &ls;
  const int hits = s.sel.n_hits;
  if (hits > kMaxCands) {
    if (t == 0) lead->sel.overflow = 1;
  } else {
    for (int q = t; q < hits * kWords; q += kTopThreads) {
      const int at = ls.rank[q / kWords];
      const int mine = at / (p.iters * kTopThreads), it = rank + mine * C;
      const int w = it / p.slices, e0 = (it - w * p.slices) * p.slice;
      const int j =
          e0 + entry_element<T>(at - mine * p.iters * kTopThreads, q % kWords, kTopThreads);
      if (j >= min(e0 + p.slice, p.V)) continue;
      const T* row = reinterpret_cast<const T*>(p.logits) + (grp * p.W + w) * (long long)p.V;
      list_group<T, kBeam>(&lead->sel.n_cands, lead_ls, load_group<T, kAligned>(row, j, p.V, span),
                    threshold(w), w * p.V + j);
    }
  }
  if (!kBeam && rank == 0 && warp == kTopWarps - 1) {  // the warp with the least to load
    float2 sum;
    row_sum(&s.part[0][0], parts, p.cc, sum);
    const float2 l = log_pair(sum);
    if (lane == 0) p.out_lse[grp] = m == -INFINITY ? -INFINITY : m / p.T + (l.x + l.y);
  }
  if (C > 1) cluster.sync(); else __syncthreads();
  if (rank != 0) return;

  int count = s.sel.n_cands;
  if (s.sel.overflow || count > kMaxCands) {
    __syncthreads();
    count = 0;
    for (int w = 0; w < p.W; ++w) {
      const double off = kBeam ? s.off[w] : 0.0;
      if (off == -INFINITY) continue;
      const T* row = reinterpret_cast<const T*>(p.logits) + (grp * p.W + w) * (long long)p.V;
      const int got = select_row_slow<T, kBeam, 0>(s.sel, ls, row, p.V, p.n, off,
                                                   kBeam ? s.max[w] : 0.f, w * p.V, count);
      // keep the n best of the rows so far (at most 2 n <= 256 entries, one a thread)
      count = keep_best<kBeam, 0>(ls, count + got, p.n, p.V);
    }
  } else {
    if (kBeam) {
      for (int i = t; i < count; i += kTopThreads) {
        const int idx = ls.idx[i];
        const int w = idx / p.V;
        set_candidate<kBeam>(ls, i, __uint_as_float((uint32_t)ls.key[i]), s.off[w], s.max[w], idx);
      }
      __syncthreads();
    }
    if (count > kRankAll) count = prune<kBeam, 0>(s.sel, ls, count, p.n);
  }
  rank_list<kBeam, 0>(ls, count, p.V);
  for (int i = t; i < count; i += kTopThreads) {
    const int r = ls.rank[i];
    if (r < p.n) write_slot<kBeam>(p, grp, r, ls.key[i], ls.idx[i]);
  }
  for (int j = count + t; j < p.n; j += kTopThreads) write_slot<kBeam>(p, grp, j, 0, -1);
}

// The candidates lie in the memory of the load stages, which are consumed by then.
constexpr int kUnionBytes = ring_bytes(kTopWarps) > (int)sizeof(BeamLists)
                                ? ring_bytes(kTopWarps)
                                : (int)sizeof(BeamLists);

template <typename T, bool kAligned, bool kBeam>
cudaError_t launch_top(const TopParams& p, long long groups, int C, cudaStream_t stream) {
  static PerDevice once;
  auto* fn = top_kernel<T, kAligned, kBeam>;
  const cudaError_t err = per_device(once, nullptr, [&](int&) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(TopShared) + kMaxTables * kTopThreads * 2 +
                                    kUnionBytes);
  });
  if (err != cudaSuccess) return err;
  const size_t smem = sizeof(TopShared) + p.table_bytes + kUnionBytes;
  return launch_early(fn, (unsigned)(groups * C), kTopThreads, smem, C, stream, p);
}

// The logits' memory, and whether all rows start on a 16-byte boundary.
bool set_span(TopParams& p, sv_dtype dtype, long long rows) {
  const size_t esz = dtype == SV_BF16 ? 2 : 4;
  p.first = static_cast<char*>(const_cast<void*>(p.logits));
  p.last = p.first + (size_t)rows * (size_t)p.V * esz;
  return ((uintptr_t)p.first & 15u) == 0 && ((size_t)p.V * esz) % 16 == 0;
}

// Which kernel. The row kernel streams at HBM's rate but gives a row to one
// CTA; the cluster kernel spreads a row over four or eight and ends sooner when
// there are few and long ones. Records (us, cluster / row kernel, k = 32): 32
// rows of 128256 bf16 8.2 / 11.0, 96 rows 10.7 / 11.3, 128 rows 13.9 / 11.4; 96
// rows of 50001 fp32 10.1 / 11.1; of 32000 bf16 (64 KB) 6.9 / 6.6 at 32 rows and
// 7.5 / 6.6 at 96.
bool record_by_rows(sv_dtype dtype, long long rows, int V) {
  const long long bytes = (long long)V * (dtype == SV_BF16 ? 2 : 4);
  return (rows > 96 || bytes < 128000) && top_rows_fit(V);
}
// Beams go through the row kernel in two launches. (us, cluster / rows, n = 16,
// bf16: 1 x 4 of 32000 8.1 / 9.9; 100 x 4 of 32000 (26 MB) 12.1 / 16.9; 16 x 8 of
// 128256 (33 MB) 17.8 / 15.1.  Past 8 beams a cluster's CTAs have two or more
// each, at any V: one request of 9, 16, 32, 64 beams of 1000 tokens 10.0 / 9.8,
// 10.5 / 9.9, 15.9 / 10.1, 27.3 / 10.1; of 32000 11.8 / 10.5, 12.3 / 10.8, 19.1 /
// 11.0, 33.6 / 11.0; eight requests of 9 and 64 beams of 8000 10.1 / 9.8 and
// 29.3 / 14.3.)
bool beams_by_rows(sv_dtype dtype, int B, int W, int V) {
  const long long bytes = (long long)B * W * V * (dtype == SV_BF16 ? 2 : 4);
  return (W > 8 || bytes > (28ll << 20)) && top_rows_fit(V);
}

template <bool kBeam>
sv_status run_top(TopParams& p, sv_dtype dtype, long long groups, cudaStream_t stream) {
  const bool aligned = set_span(p, dtype, groups * p.W);
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return SV_ERR_CUDA;
  // The cluster: one CTA per row (beams: per beam, up to 8), more while twice
  // as many still come to at most 2.8 an SM (64 rows of 128256 bf16: 10.5 us with
  // clusters of 4, 14.5 with 8), or while the rows' tables need the shared memory
  // of several.
  int C = 1;
  while (C < 8 && C < p.W) C *= 2;
  while (C < 8 && (5LL * groups * C <= 7LL * dev.sms ||
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
  set_units(p, dtype, items, std::min(p.slice, p.V), kTopThreads);
  p.table_bytes = (items + C - 1) / C * p.iters * kTopThreads * 2;
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
  p.wait_ns = wait_limit_ns();
  const long long rows = (long long)B * P;
  if (record_by_rows(dtype, rows, V)) {
    const bool aligned = set_span(p, dtype, rows);
    return launch_top_rows(dtype, aligned, p, rows, (cudaStream_t)stream) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
  }
  return run_top<false>(p, dtype, rows, (cudaStream_t)stream);
}

size_t spec_beam_workspace_size(sv_dtype dtype, int B, int W, int V, int n) {
  if ((dtype != SV_F32 && dtype != SV_BF16) || B < 0 || B > SV_MAX_B || W < 1 ||
      W > SV_MAX_BEAMS || V < 1 || V > SV_MAX_V || n < 1 || n > SV_MAX_TOP)
    return 0;
  const size_t rows = (size_t)B * W;
  // each row's offset and max, then its n best logits and their tokens
  return beams_by_rows(dtype, B, W, V) ? rows * (16 + 8 * (size_t)n) : 0;
}

sv_status spec_beam_select(const void* logits, const float* scores, int32_t* out_tokens,
                           int32_t* out_parents, float* out_scores, int32_t* out_status,
                           sv_dtype dtype, int B, int W, int V, int n, void* workspace,
                           size_t ws_bytes, sv_stream_t stream) {
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (B < 0 || B > SV_MAX_B || W < 1 || W > SV_MAX_BEAMS || V < 1 || V > SV_MAX_V || n < 1 ||
      n > SV_MAX_TOP ||
      (long long)((W + 7) / 8) * ((V + kTopSpan - 1) / kTopSpan) > kMaxTables)
    return SV_ERR_SHAPE;
  if (B == 0) return SV_OK;
  if (!logits || !scores || !out_tokens || !out_parents || !out_scores) return SV_ERR_NULL;
  if ((uintptr_t)logits & (dtype == SV_BF16 ? 1u : 3u)) return SV_ERR_NULL;
  const size_t need = spec_beam_workspace_size(dtype, B, W, V, n);
  if (need && (!workspace || ((uintptr_t)workspace & 15u) || ws_bytes < need))
    return SV_ERR_WORKSPACE;
  TopParams p;
  memset(&p, 0, sizeof p);
  p.logits = logits;
  p.scores = scores;
  p.P = 1;
  p.V = V;
  p.n = n;
  p.cc = 1.4426950408889634f;
  p.T = 1.f;
  p.wait_ns = wait_limit_ns();
  const cudaStream_t st = (cudaStream_t)stream;
  if (need) {  // each beam's n best, then the requests'
    const long long rows = (long long)B * W;
    double* off = static_cast<double*>(workspace);
    float* row_max = reinterpret_cast<float*>(off + rows);
    float* values = row_max + 2 * rows;
    int* ids = reinterpret_cast<int*>(values + rows * n);
    TopParams q = p;
    q.W = 1;
    q.out_ids = ids;
    q.out_values = values;
    q.out_off = off;
    q.out_max = row_max;
    const bool aligned = set_span(q, dtype, rows);
    if (launch_top_rows(dtype, aligned, q, rows, st) != cudaSuccess) return SV_ERR_CUDA;
    p.W = W;
    p.out_ids = out_tokens;
    p.out_parents = out_parents;
    p.out_values = out_scores;
    p.out_status = out_status;
    return launch_beam_merge(p, ids, values, off, row_max, B, st) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  }
  p.out_ids = out_tokens;
  p.out_parents = out_parents;
  p.out_values = out_scores;
  p.out_status = out_status;
  p.W = W;
  return run_top<true>(p, dtype, B, st);
}

}  // extern "C"
