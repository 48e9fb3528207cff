// sv_toprows.cu - the k largest logits of each of many rows with its
// log-sum-exp, and the merge of a request's row selections (beams).
//
// With a CTA per row (sv_top.cu) all resident CTAs stream at the same pace and
// then select at the same time, and HBM idles meanwhile: a quarter of the
// call. Here each CTA has two halves of eight warps: one streams row after
// row, the other selects from the row before, over two sets of tables and
// sums, handed over through named barriers. Rows come from the launch's own
// queue (cluster launch control: a CTA cancels a CTA of the grid that has not
// started and takes its row), so the last rows spread evenly without a
// counter in memory; the selecting half asks for them while the other streams,
// and deals with rows that need no work by itself.
//
// What it measured (bf16, k = 64): 912 rows of 152064 logits 51.9 us, 2432 rows
// 120.4 us: 45 ns a row (6.7 TB/s) and 11 us beside them, half of it the last
// rows' selection. Shorter rows are bound by the selecting half: 2400 rows of
// 50000 61 us (25 ns a row, 3.9 TB/s).
#include "sv_select.cuh"

namespace sv {
namespace {

constexpr int kStreamWarps = 8;
constexpr int kRowStreamers = kStreamWarps * kWarp;
constexpr int kRowThreads = kRowStreamers + kTopThreads;
constexpr int kRowSpan = kRowStreamers * kEntry;  // elements of an iteration
// named barriers, two each but the first
enum : int { kBarSelect = 1, kBarFull = 2, kBarEmpty = 4, kBarNext = 6 };

struct alignas(16) RowShared {
  uint4 answer;                 // the queue's answer
  unsigned long long bar;       // its arrival
  long long next[2];            // the row to stream next, by parity (-1: none)
  struct Slot {
    float2 part[kStreamWarps];  // the row's sums by warp
    alignas(16) uint16_t unit[kRowStreamers];  // its unit maxes, bf16 rounded down
  } slot[2];
  Select sel;
  int late;                     // the queue did not answer in time: this CTA's rows from there on
                                // are marked SV_REQ_TIMEOUT
  int lost;                     // nor within the waits' default limit
};
constexpr int kLive = -1;

__device__ __forceinline__ void bar_sync(int bar, int threads) {
  asm volatile("barrier.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int bar, int threads) {
  asm volatile("barrier.arrive %0, %1;" ::"r"(bar), "r"(threads) : "memory");
}

// Asks for a CTA of this grid that has not started; the answer (16 bytes)
// completes on mbarrier `bar`.
__device__ __forceinline__ void ask_for_cta(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(answer),
      "r"(bar)
      : "memory");
}
// The CTA taken over (its index in a grid of one dimension), or -1.
__device__ __forceinline__ long long taken_cta(uint32_t answer) {
  uint32_t got, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 a;\n ld.shared.b128 a, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n"
      " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n}"
      : "=r"(got), "=r"(x)
      : "r"(answer)
      : "memory");
  return got ? (long long)x : -1;
}

// kLive, or the status of a row that is not read.
__device__ __forceinline__ int row_state(const TopParams& p, long long row) {
  if (p.scores) return p.scores[row] == -INFINITY ? 0 : kLive;
  if (!p.lens) return kLive;
  const int b = (int)(row / p.P), i = (int)(row - (long long)b * p.P), len = p.lens[b];
  if (len < 0 || len > p.P) return SV_REQ_BAD_DRAFT_LEN;
  return i < len ? kLive : 0;
}

__device__ __forceinline__ void fill_slots(const TopParams& p, long long row, int from) {
  for (int j = from + threadIdx.x % kTopThreads; j < p.n; j += kTopThreads) {
    p.out_ids[row * p.n + j] = -1;
    p.out_values[row * p.n + j] = -INFINITY;
  }
}

// The outputs of a row that is not selected from (a call of the selecting half).
__device__ __forceinline__ void leave_row(const TopParams& p, long long row, int status) {
  fill_slots(p, row, 0);
  if (threadIdx.x % kTopThreads == 0) {
    const bool late = status == SV_REQ_TIMEOUT;
    if (p.out_off) p.out_off[row] = late ? __longlong_as_double((long long)kOffLate) : -INFINITY;
    else p.out_lse[row] = late ? qnan() : -INFINITY;
    if (p.out_status) p.out_status[row] = status;
  }
}

// The next row that needs work, -1 when the queue is empty; the outputs of the
// others on the way (a call of the selecting half).  `row`: a row taken already,
// or -1 to ask.
__device__ long long next_live(RowShared& s, const TopParams& p, long long row, int& asked) {
  const int t = threadIdx.x % kTopThreads;
  for (;;) {
    if (row < 0) {
      group_sync<kBarSelect>();  // the last answer is read by all
      if (t == 0) {
        fence_proxy_async();
        mbar_arrive_expect_tx(smem_u32(&s.bar), 16);
        ask_for_cta(smem_u32(&s.answer), smem_u32(&s.bar));
      }
      // (the limit twice: see mbar_wait_cluster)
      const uint32_t bar = smem_u32(&s.bar), phase = asked & 1;
      if (!mbar_wait(bar, phase, p.wait_ns) && !mbar_wait(bar, phase, p.wait_ns)) {
        s.late = 1;
        // the answer lands before the next question or the CTA's end
        if (!mbar_wait(bar, phase) && !mbar_wait(bar, phase)) s.lost = 1;
      }
      ++asked;
      group_sync<kBarSelect>();
      if (s.lost) return -1;
      row = taken_cta(smem_u32(&s.answer));
      if (row < 0) return -1;
    }
    const int state = row_state(p, row);
    if (state == kLive && !s.late) return row;
    leave_row(p, row, state == kLive ? SV_REQ_TIMEOUT : state);
    row = -1;
  }
}

// The selecting half: one row from its table, sums and units.
template <typename T, bool kAligned>
__device__ void select_row(RowShared& s, Lists& ls, const RowShared::Slot& slot, long long row,
                           const uint16_t* table, const TopParams& p, const RowSpan& span) {
  constexpr int VEC = Group<T>::VEC;
  constexpr int kWords = kEntry / VEC;
  const int t = threadIdx.x % kTopThreads;
  if (t == 0) s.sel.n_hits = s.sel.n_cands = 0;
  // every warp for itself: the max decides whether there is anything to select
  const float m = warp_max_nan(lane_id() < kStreamWarps ? slot.part[lane_id()].x : -INFINITY);
  const float score = p.scores ? p.scores[row] : 0.f;
  const bool bad = m != m || m == INFINITY || score != score || score == INFINITY;
  auto row_outputs = [&]() {  // one warp: the log-sum-exp, or the beam's offset
    float2 sum;
    row_sum(slot.part, kStreamWarps, p.cc, sum);
    if (lane_id() != 0) return;
    const float2 l = log_pair(sum);
    if (p.out_off) {
      p.out_off[row] = bad              ? __longlong_as_double((long long)kOffBad)
                       : m == -INFINITY ? -INFINITY
                                        : row_offset(score, l);
      p.out_max[row] = m;
    } else {
      p.out_lse[row] = bad ? qnan() : m == -INFINITY ? -INFINITY : m / p.T + (l.x + l.y);
      if (p.out_status) p.out_status[row] = bad ? SV_REQ_BAD_LOGITS : 0;
    }
  };
  if (bad || m == -INFINITY) {
    if (t < kWarp) row_outputs();
    fill_slots(p, row, 0);
    return;
  }
  const float thr = fmaxf(unit_bound<kBarSelect>(s.sel, slot.unit, p.upi, p.n), -FLT_MAX);
  if (p.upi < p.n) group_sync<kBarSelect>();  // (the bound's barriers were not passed)
  scan_table(s.sel, ls, table, p.iters * kRowStreamers, thr, 0);
  group_sync<kBarSelect>();
  const T* data = reinterpret_cast<const T*>(p.logits) + row * (long long)p.V;
  const int hits = s.sel.n_hits;
  if (hits <= kMaxCands) {
    // two loads in flight a thread: the usual list is one round
    for (int q = t; q < hits * kWords; q += 2 * kTopThreads) {
      const int q2 = q + kTopThreads;
      const int j = entry_element<T>(ls.rank[q / kWords], q % kWords, kRowStreamers);
      const int j2 = q2 < hits * kWords
                         ? entry_element<T>(ls.rank[q2 / kWords], q2 % kWords, kRowStreamers)
                         : p.V;
      uint4 g = Lane<T, VEC>::pad(), g2 = g;
      if (j < p.V) g = load_group<T, kAligned>(data, j, p.V, span);
      if (j2 < p.V) g2 = load_group<T, kAligned>(data, j2, p.V, span);
      list_group<T, false>(&s.sel.n_cands, &ls, g, thr, j);
      list_group<T, false>(&s.sel.n_cands, &ls, g2, thr, j2);
    }
  }
  if (t >= kTopThreads - kWarp) row_outputs();  // the warp with the least to load
  group_sync<kBarSelect>();
  int count = s.sel.n_cands;
  if (hits > kMaxCands || count > kMaxCands) {
    group_sync<kBarSelect>();
    count = select_row_slow<T, false, kBarSelect>(s.sel, ls, data, p.V, p.n, 0.0, 0.f, 0, 0);
  } else if (count > kRankAll) {
    count = prune<false, kBarSelect>(s.sel, ls, count, p.n);
  }
  rank_list<false, kBarSelect>(ls, count, p.V);
  for (int i = t; i < count; i += kTopThreads) {
    const int r = ls.rank[i];
    if (r < p.n) {
      p.out_ids[row * p.n + r] = ls.idx[i];
      p.out_values[row * p.n + r] = of_ordered((uint32_t)(ls.key[i] >> 32));
    }
  }
  fill_slots(p, row, count);
  group_sync<kBarSelect>();  // the lists are read
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kRowThreads, 2) top_rows_kernel(const TopParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  RowShared& s = *reinterpret_cast<RowShared*>(smem);
  Lists& ls = *reinterpret_cast<Lists*>(smem + sizeof(RowShared));
  uint16_t* tables = reinterpret_cast<uint16_t*>(smem + sizeof(RowShared) + sizeof(Lists));
  const int table = p.iters * kRowStreamers;
  unsigned char* rings = smem + sizeof(RowShared) + sizeof(Lists) + 2 * 2 * table;
  const bool streams = threadIdx.x < kRowStreamers;
  const int t = streams ? threadIdx.x : threadIdx.x - kRowStreamers;
  const int lane = lane_id(), warp = t / kWarp;
  const RowSpan span = {p.first, p.last};
  if (threadIdx.x == 0) {
    s.late = s.lost = 0;
    mbar_init(smem_u32(&s.bar), 1);
    fence_mbar_init();
  }
  pdl_wait();
  __syncthreads();
  const bool first_live = row_state(p, blockIdx.x) == kLive;

  if (!streams) {  // the selecting half
    int asked = 0;
    long long row = next_live(s, p, blockIdx.x, asked);
    if (!first_live) {
      if (t == 0) s.next[0] = row;
      bar_arrive(kBarNext, kRowThreads);
    }
    for (int k = 0; row >= 0; ++k) {
      const int b = k & 1;
      const long long next = next_live(s, p, -1, asked);
      if (t == 0) s.next[b ^ 1] = next;
      bar_arrive(kBarNext + (b ^ 1), kRowThreads);
      bar_sync(kBarFull + b, kRowThreads);
      if (s.late) leave_row(p, row, SV_REQ_TIMEOUT);
      else select_row<T, kAligned>(s, ls, s.slot[b], row, tables + b * table, p, span);
      bar_arrive(kBarEmpty + b, kRowThreads);
      row = next;
    }
    return;
  }

  // The streaming half.
  const int fold = p.fold;
  long long row = blockIdx.x;
  if (!first_live) {
    bar_sync(kBarNext, kRowThreads);
    row = s.next[0];
  }
  int k = 0;
  for (; row >= 0; ++k) {
    const int b = k & 1;
    RowShared::Slot& slot = s.slot[b];
    if (k >= 2) bar_sync(kBarEmpty + b, kRowThreads);  // row k - 2 is selected
    const T* data = reinterpret_cast<const T*>(p.logits) + row * (long long)p.V;
    const RunningSum r = stream_slice<T, kAligned, kStreamWarps>(
        smem_u32(rings), warp, data, 0, p.V, p.iters, p.cc, tables + b * table + t, span);
    const float2 wr = warp_running(r, p.cc);
    float um = r.m;
    for (int o = 1; o < fold; o <<= 1) um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, o));
    if (lane == 0) slot.part[warp] = wr;
    if ((t & (fold - 1)) == 0 && t / fold < p.upi) slot.unit[t / fold] = down_bf16(um);
    bar_arrive(kBarFull + b, kRowThreads);
    bar_sync(kBarNext + (b ^ 1), kRowThreads);
    row = s.next[b ^ 1];
  }
  // (sooner, the kernel after this one would take the place of CTAs yet to start)
  pdl_launch_dependents();
  // every arrival is waited for before the CTA ends
  if (k >= 2) bar_sync(kBarEmpty + (k & 1), kRowThreads);
  if (k >= 1) bar_sync(kBarEmpty + ((k - 1) & 1), kRowThreads);
}

template <typename T, bool kAligned>
cudaError_t launch_rows(TopParams p, long long rows, cudaStream_t stream) {
  static PerDevice once;
  auto* fn = top_rows_kernel<T, kAligned>;
  const size_t fixed = sizeof(RowShared) + sizeof(Lists) + ring_bytes(kStreamWarps);
  const cudaError_t err = per_device(once, nullptr, [&](int&) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
  });
  if (err != cudaSuccess) return err;
  return launch_early(fn, (unsigned)rows, kRowThreads,
                      fixed + 4 * (size_t)p.iters * kRowStreamers, 1, stream, p);
}

// The n best of a request's W selections.  Four threads to each of 256 units,
// whose elements (up to 32) lie at different places of different rows; the
// bound of the unit maxes leaves a list that fits (or, with many equal scores,
// the rows go in one after the other).  Bound by the latency of its steps, so a
// request has 1024 threads: 24 x 32 beams of 50001 fp32 logits, n = 64, both
// launches, 36.2 us (with 256 threads that worked through eight elements each,
// 11 us more).
constexpr int kMergeThreads = 1024;
constexpr int kMergePer = SV_MAX_BEAMS * SV_MAX_TOP / kMergeThreads;  // elements a thread

__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(
    const TopParams p, const FastDiv div_n, const FastDiv div_w, const int* __restrict__ ids,
    const float* __restrict__ values, const double* __restrict__ off,
    const float* __restrict__ row_max) {
  __shared__ BeamLists ls;
  __shared__ Select sel;
  __shared__ __align__(16) uint16_t unit[kTopThreads];
  __shared__ double s_off[SV_MAX_BEAMS];
  __shared__ float off_down[SV_MAX_BEAMS], s_max[SV_MAX_BEAMS];
  pdl_wait();
  pdl_launch_dependents();
  const long long b = blockIdx.x;
  const int t = threadIdx.x, all = p.W * p.n;
  ids += b * all;
  values += b * all;
  // Each row's are in descending order: place r of row w is taken for r + w n / W
  // (mod n), so that a unit's elements, 256 apart, are of all ranks.
  int row[kMergePer];    // -1: none
  int place[kMergePer];  // in all rows
  float v[kMergePer];
#pragma unroll
  for (int q = 0; q < kMergePer; ++q) {
    const uint32_t i = (uint32_t)(4 * q + t % 4) * kTopThreads + t / 4;
    row[q] = -1;
    if (i < (uint32_t)all) {
      const uint32_t w = fast_div(i, div_n);
      uint32_t r = i - w * p.n + fast_div(w * p.n, div_w);
      if (r >= (uint32_t)p.n) r -= p.n;
      row[q] = (int)w;
      place[q] = (int)(w * p.n + r);
      v[q] = values[place[q]];
    }
  }
  const double o = t < p.W ? off[b * p.W + t] : 0.0;
  const float m = t < p.W ? row_max[b * p.W + t] : 0.f;
  if (t == 0) sel.n_cands = sel.bad = 0;
  __syncthreads();
  if (t < p.W) {
    s_off[t] = o;
    off_down[t] = __double2float_rd(o);
    s_max[t] = o == -INFINITY ? 0.f : m;  // (a row not read has none)
    if (o != o)
      atomicOr(&sel.bad, (unsigned long long)__double_as_longlong(o) == kOffLate
                             ? SV_REQ_TIMEOUT
                             : SV_REQ_BAD_LOGITS);
  }
  __syncthreads();
  const int bad = sel.bad;
  if (t == 0 && p.out_status) p.out_status[b] = bad;
  auto write = [&](int slot, unsigned long long key, int idx) {
    const long long o = b * p.n + slot;
    const int w = idx < 0 ? -1 : idx / p.V;
    p.out_ids[o] = idx < 0 ? -1 : idx - w * p.V;
    p.out_parents[o] = w;
    p.out_values[o] = idx < 0 ? -INFINITY : (float)of_ordered(key);
  };
  int count = 0;
  if (!bad) {
    // the scores in fp32, rounded down to -FLT_MAX at least (-inf for an empty slot)
    float score[kMergePer], um = -INFINITY;
#pragma unroll
    for (int q = 0; q < kMergePer; ++q) {
      score[q] = -INFINITY;
      if (row[q] >= 0 && v[q] > -INFINITY)
        score[q] = fmaxf(beam_score_down(off_down[row[q]], s_max[row[q]], v[q]), -FLT_MAX);
      um = fmaxf(um, score[q]);
    }
    um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 1));
    um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 2));
    if (t % 4 == 0) unit[t / 4] = down_bf16(um);
    __syncthreads();
    if (t < kTopThreads) unit_bound<kBarSelect>(sel, unit, kTopThreads, p.n);
    __syncthreads();
    const float bound = of_ordered(sel.bound);
#pragma unroll
    for (int q = 0; q < kMergePer; ++q) {
      const float f = score[q];
      // what stays below the bound with its roundings given back - of the offset, of
      // l - m, at most |score| + |offset|, and of their sum - is below n others
      if (f > -INFINITY && fmaf(fabsf(f) + fabsf(off_down[row[q]]), 1e-6f, f) >= bound) {
        const int at = atomicAdd(&sel.n_cands, 1);
        if (at < kMaxCands) {
          set_candidate<true>(ls, at, v[q], s_off[row[q]], s_max[row[q]],
                              row[q] * p.V + ids[place[q]]);
        }
      }
    }
    __syncthreads();
    if (t >= kTopThreads) return;  // the list is the first 256 threads' from here on
    count = sel.n_cands;
    if (count > kMaxCands) {
      __syncthreads();
      count = 0;
      for (int w = 0; w < p.W; ++w) {
        if (s_off[w] == -INFINITY) continue;
        int got = 0;  // (the finite ones come first)
        if (t < p.n && values[w * p.n + t] > -INFINITY) {
          set_candidate<true>(ls, count + t, values[w * p.n + t], s_off[w], s_max[w],
                              w * p.V + ids[w * p.n + t]);
          got = 1;
        }
        got = __syncthreads_count(got);
        count = keep_best<true, 0>(ls, count + got, p.n, p.V);
      }
    } else if (count > kRankAll) {
      count = prune<true, 0>(sel, ls, count, p.n);
    }
    rank_list<true, 0>(ls, count, p.V);
    for (int i = t; i < count; i += kTopThreads) {
      const int r = ls.rank[i];
      if (r < p.n) write(r, ls.key[i], ls.idx[i]);
    }
  }
  if (t < kTopThreads)
    for (int j = count + t; j < p.n; j += kTopThreads) write(j, 0, -1);
}

}  // namespace

bool top_rows_fit(int V) {
  const size_t tables = 4 * (size_t)((V + kRowSpan - 1) / kRowSpan) * kRowStreamers;
  return sizeof(RowShared) + sizeof(Lists) + ring_bytes(kStreamWarps) + tables <=
         (size_t)kRowsSmem;
}

cudaError_t launch_top_rows(sv_dtype dtype, bool aligned, TopParams p, long long rows,
                            cudaStream_t stream) {
  p.slices = 1;
  p.slice = (p.V + 255) / 256 * 256;
  p.iters = (p.V + kRowSpan - 1) / kRowSpan;
  set_units(p, dtype, 1, p.V, kRowStreamers);
  if (dtype == SV_BF16)
    return aligned ? launch_rows<uint16_t, true>(p, rows, stream)
                   : launch_rows<uint16_t, false>(p, rows, stream);
  return aligned ? launch_rows<float, true>(p, rows, stream)
                 : launch_rows<float, false>(p, rows, stream);
}

cudaError_t launch_beam_merge(const TopParams& p, const int* ids, const float* values,
                              const double* off, const float* row_max, int B,
                              cudaStream_t stream) {
  return launch_early(beam_merge_kernel, (unsigned)B, kMergeThreads, 0, 1, stream, p,
                      make_fastdiv((uint32_t)p.n), make_fastdiv((uint32_t)p.W), ids, values, off,
                      row_max);
}

}  // namespace sv
