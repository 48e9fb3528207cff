// sv_reorder.cu - reordering of per-beam states (spec_beam_reorder).
//
// A gather of byte runs: out[g, b, w, h, l] = state[g, b, parents[b, w], h, l].
// When the l entries of a (g, b, w, h) lie back to back in both tensors they
// form one run of lens[b] * row_bytes bytes, else each entry is a run of its
// own.  The runs (at their full length) are laid end to end and cut into
// units of the widest type every address allows (16 bytes as a rule); a CTA
// takes kUnits * 256 of them, each thread every 256th, all its loads in
// flight before the first store.  Pure HBM traffic: 1.6 GB of valid bytes moved
// along random parents of 8 beams in 394 us, 2.7 GB of distinct bytes at the
// copy rate (6.8 TB/s).
#include <string.h>

#include <algorithm>

#include "../../include/spec_verify.h"
#include "sv_launch.h"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

constexpr int kReorderThreads = 256;
constexpr int kUnits = 8;  // units per thread

struct ReorderParams {
  const char* state;
  char* out;
  const int* parents;  // [B, Wo]
  const int* lens;     // [B] or null
  int* out_status;     // [B] or null
  long long ss[5], os[5];  // byte strides of g, b, w, h, l
  int B, W, Wo, L;
  int runs_l;          // runs per (g, b, w, h): 1 (contiguous) or L
  long long row_units; // units per entry
  uint32_t run_units;  // units per run
  unsigned long long total;  // units in all
  FastDiv div_l, div_h, div_w, div_b;
};

template <typename U>
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const ReorderParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x;
  if (p.out_status) {
    const long long b = (long long)blockIdx.x * kReorderThreads + t;
    if (b < p.B) {
      int st = 0;
      for (int w = 0; w < p.Wo; ++w) {
        const int pa = p.parents[b * p.Wo + w];
        if (pa < -1 || pa >= p.W) st |= SV_REQ_BAD_TREE;
      }
      if (p.lens && (p.lens[b] < 0 || p.lens[b] > p.L)) st |= SV_REQ_BAD_DRAFT_LEN;
      p.out_status[b] = st;
    }
  }
  const unsigned long long first = (unsigned long long)blockIdx.x * (kReorderThreads * kUnits);
  if (first >= p.total) return;
  uint32_t run = (uint32_t)(first / p.run_units);
  unsigned long long at = first - (unsigned long long)run * p.run_units + t;  // unit in the run
  const char* src = nullptr;
  char* dst = nullptr;
  long long valid = -1;  // units of the run that are moved; -1: run not looked up yet
  const U* from[kUnits];
  U* to[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const unsigned long long here = first + (unsigned long long)u * kReorderThreads + t;
    if (at >= p.run_units) {
      const uint32_t skip = at >> 32 ? (uint32_t)(at / p.run_units)
                                     : (uint32_t)at / p.run_units;
      run += skip;
      at -= (unsigned long long)skip * p.run_units;
      valid = -1;
    }
    from[u] = nullptr;
    if (here < p.total) {
      if (valid < 0) {
        uint32_t q = fast_div(run, p.div_l);
        const int l = (int)(run - q * p.div_l.d);
        uint32_t r = fast_div(q, p.div_h);
        const int h = (int)(q - r * p.div_h.d);
        q = fast_div(r, p.div_w);
        const int w = (int)(r - q * p.div_w.d);
        const uint32_t g = fast_div(q, p.div_b);
        const int b = (int)(q - g * p.div_b.d);
        const int pa = p.parents[(long long)b * p.Wo + w];
        int len = p.lens ? p.lens[b] : p.L;
        if (len < 0 || len > p.L) len = 0;
        valid = 0;
        if (pa >= 0 && pa < p.W) {
          valid = p.runs_l == 1 ? (long long)len * p.row_units
                                : (l < len ? p.row_units : 0);
          src = p.state + g * p.ss[0] + b * p.ss[1] + pa * p.ss[2] + h * p.ss[3] + l * p.ss[4];
          dst = p.out + g * p.os[0] + b * p.os[1] + w * p.os[2] + h * p.os[3] + l * p.os[4];
        }
      }
      if ((long long)at < valid) {
        from[u] = reinterpret_cast<const U*>(src) + at;
        to[u] = reinterpret_cast<U*>(dst) + at;
      }
    }
    at += kReorderThreads;
  }
  U v[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
    if (from[u]) v[u] = *from[u];
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
    if (from[u]) *to[u] = v[u];
}

template <typename U>
cudaError_t launch_reorder(const ReorderParams& p, unsigned blocks, cudaStream_t stream) {
  return launch_early(reorder_kernel<U>, blocks, kReorderThreads, 0, 1, stream, p);
}

// Whether an entry of one tensor shares a byte with an entry of another: whether
//   at + sum_k c_k stride_k,  lo_k <= c_k <= hi_k,
// (the distance of two entries, one term a dimension of each tensor, one for
// both where their strides agree) comes closer to 0 than row_bytes. Terms by
// falling stride, each tried only where the rest can still reach 0: a handful
// of nodes for the views of a dense cache. A search that grows past kMeetNodes
// (strides that interleave in other ways) says yes.
constexpr int kMeetNodes = 4096;
typedef __int128 Wide;  // (sums of ten extents of up to 2^60)
struct Term {
  long long stride, lo, hi;
};
struct Meet {
  Term term[10];
  Wide low[11], high[11];  // the sums of term k on, at least and at most
  int n = 0, nodes = 0;
  long long row_bytes;
  static Wide div_down(Wide a, long long b) { return a >= 0 ? a / b : -((-a + b - 1) / b); }
  bool from(int k, Wide at) {
    if (++nodes > kMeetNodes) return true;
    if (k == n) return at > -row_bytes && at < row_bytes;
    const Term& t = term[k];
    const Wide first = -div_down(-(-(Wide)row_bytes + 1 - high[k + 1] - at), t.stride);
    const Wide last = div_down((Wide)row_bytes - 1 - low[k + 1] - at, t.stride);
    for (Wide c = std::max(first, (Wide)t.lo); c <= std::min(last, (Wide)t.hi); ++c)
      if (from(k + 1, at + c * t.stride)) return true;
    return false;
  }
};
bool entries_meet(long long at, const int64_t* in, const long long* n_in, const int64_t* out,
                  const long long* n_out, long long row_bytes) {
  Meet m;
  m.row_bytes = row_bytes;
  for (int i = 0; i < 5; ++i) {
    if (in[i] == out[i]) {
      if (in[i] > 0) m.term[m.n++] = {in[i], 1 - n_out[i], n_in[i] - 1};
    } else {
      if (in[i] > 0 && n_in[i] > 1) m.term[m.n++] = {in[i], 0, n_in[i] - 1};
      if (out[i] > 0 && n_out[i] > 1) m.term[m.n++] = {out[i], 1 - n_out[i], 0};
    }
  }
  std::sort(m.term, m.term + m.n, [](const Term& a, const Term& b) { return a.stride > b.stride; });
  m.low[m.n] = m.high[m.n] = 0;
  for (int k = m.n - 1; k >= 0; --k) {
    m.low[k] = m.low[k + 1] + (Wide)m.term[k].lo * m.term[k].stride;
    m.high[k] = m.high[k + 1] + (Wide)m.term[k].hi * m.term[k].stride;
  }
  return m.from(0, at);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status spec_beam_reorder(const void* state, const int64_t* state_strides,
                                       const int32_t* parents, const int32_t* lens, void* out,
                                       const int64_t* out_strides, int32_t* out_status, int G,
                                       int B, int W, int W_out, int H, int L, int row_bytes,
                                       sv_stream_t stream) {
  if (G < 0 || B < 0 || B > SV_MAX_B || W < 0 || W > 65535 || W_out < 0 || W_out > 65535 || H < 0 ||
      L < 0 || row_bytes < 1)
    return SV_ERR_SHAPE;
  if (B == 0) return SV_OK;
  if (!state_strides || !out_strides || (W_out > 0 && !parents)) return SV_ERR_NULL;
  const long long n_out[5] = {G, B, W_out, H, L}, n_in[5] = {G, B, W, H, L};
  bool empty = false;
  for (int i = 0; i < 5; ++i) {
    if (state_strides[i] < 0 || out_strides[i] < 0) return SV_ERR_SHAPE;
    empty = empty || n_out[i] == 0 || n_in[i] == 0;
  }
  if (!empty && (!state || !out)) return SV_ERR_NULL;
  ReorderParams p;
  memset(&p, 0, sizeof p);
  p.parents = parents;
  p.lens = lens;
  p.out_status = out_status;
  p.B = B;
  p.W = W;
  p.Wo = W_out;
  p.L = L;
  unsigned long long align = 0;  // the OR of every address step
  if (!empty) {
    // memory spanned by each tensor; `out` must not fold onto itself
    long long ext_in = row_bytes, ext_out = row_bytes;
    int order[5] = {0, 1, 2, 3, 4};
    std::sort(order, order + 5, [&](int a, int b) { return out_strides[a] < out_strides[b]; });
    for (int i : order)
      if (n_out[i] > 1) {
        if (out_strides[i] < ext_out) return SV_ERR_ALIAS;
        if (out_strides[i] > (1LL << 60) / n_out[i]) return SV_ERR_SHAPE;
        ext_out += (n_out[i] - 1) * out_strides[i];
      }
    for (int i = 0; i < 5; ++i)
      if (n_in[i] > 1) {
        if (state_strides[i] > (1LL << 60) / n_in[i]) return SV_ERR_SHAPE;
        ext_in += (n_in[i] - 1) * state_strides[i];
      }
    const uintptr_t a = (uintptr_t)state, b = (uintptr_t)out;
    if (a < b + (uintptr_t)ext_out && b < a + (uintptr_t)ext_in &&
        entries_meet((long long)(a - b), state_strides, n_in, out_strides, n_out, row_bytes))
      return SV_ERR_ALIAS;
    p.state = static_cast<const char*>(state);
    p.out = static_cast<char*>(out);
    align = (unsigned long long)a | b | (unsigned long long)row_bytes;
    for (int i = 0; i < 5; ++i) {
      p.ss[i] = n_in[i] > 1 ? state_strides[i] : 0;
      p.os[i] = n_out[i] > 1 ? out_strides[i] : 0;
      align |= (unsigned long long)(p.ss[i] | p.os[i]);
    }
    p.runs_l = L == 1 || (p.ss[4] == row_bytes && p.os[4] == row_bytes) ? 1 : L;
  }
  int width = 16;
  while (align & (unsigned)(width - 1)) width /= 2;
  if (!empty) {
    const long long run_bytes = (long long)row_bytes * (p.runs_l == 1 ? L : 1);
    const unsigned long long runs =
        (unsigned long long)G * B * W_out;  // < 2^63; the rest is checked stepwise
    if (runs >= (1ull << 32) || runs * H >= (1ull << 32) || runs * H * p.runs_l >= (1ull << 32) ||
        run_bytes / width >= (1LL << 32))
      return SV_ERR_SHAPE;
    p.row_units = row_bytes / width;
    p.run_units = (uint32_t)(run_bytes / width);
    p.total = runs * H * p.runs_l * (unsigned long long)p.run_units;
    p.div_l = make_fastdiv((uint32_t)p.runs_l);
    p.div_h = make_fastdiv((uint32_t)H);
    p.div_w = make_fastdiv((uint32_t)W_out);
    p.div_b = make_fastdiv((uint32_t)B);
  }
  const unsigned long long per = kReorderThreads * kUnits;
  unsigned long long blocks = (p.total + per - 1) / per;
  if (out_status)
    blocks = std::max(blocks, (unsigned long long)(B + kReorderThreads - 1) / kReorderThreads);
  if (blocks == 0) return SV_OK;
  if (blocks >= (1ull << 31)) return SV_ERR_SHAPE;
  cudaError_t err;
  const cudaStream_t st = (cudaStream_t)stream;
  switch (width) {
    case 16: err = launch_reorder<uint4>(p, (unsigned)blocks, st); break;
    case 8: err = launch_reorder<uint2>(p, (unsigned)blocks, st); break;
    case 4: err = launch_reorder<uint32_t>(p, (unsigned)blocks, st); break;
    case 2: err = launch_reorder<uint16_t>(p, (unsigned)blocks, st); break;
    default: err = launch_reorder<uint8_t>(p, (unsigned)blocks, st); break;
  }
  return err == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
