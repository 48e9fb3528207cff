// sv_distill.cu - distillation from a teacher's top logits: the loss of each
// row, its gradient by the student's logits, or both from one read of them.
//
// A thread-block cluster takes a row; each CTA keeps its slice of the row in
// shared memory, so the row is read from HBM once even when the gradient is
// written too (a whole row of a 152064-token vocabulary is 304 KB, more than
// one SM holds).  The recorded tokens are taken out of the slice first and
// handled apart, in the k-sized part of the work: the sum over the rest of
// the row then never subtracts (1 - sum of the recorded q would lose the
// digits of a small remainder), and a small remainder keeps its own frame.
//
// With m and S the max and the sum of 2^((s_i - m) c) over the tokens outside
// the record (c = log2(e) / T), the gradient outside the record is
//   2^((s_i - m) c) * beta * grad_loss / T,   beta = (P q_rest - p_rest) / S,
// and on a recorded token (P 2^((s_j - M) c) / Z - p_j) * grad_loss / T with M
// and Z the max and sum over all tokens and P = sum p_j + p_rest the teacher's
// mass.  {m, beta, M, 1/Z} are the row's statistics.
//
// What it measured (1024 rows of 152064 bf16 logits, k = 64): loss and gradient
// 111 us (5.6 TB/s), the loss alone 56 us (5.6 TB/s), the gradient alone 91 us
// (6.8 TB/s, the copy rate). What bounds the first two is the shared memory of
// slices that wait: 38 KB a CTA, five CTAs an SM, each from its copy's issue to
// its last store. Slices of 76 KB in clusters of four took 141 us, of 25 KB in
// eight (a 50001-token fp32 row) the same as of 50 KB in four.
#include <float.h>
#include <string.h>

#include "../../include/spec_verify.h"
#include "sv_launch.h"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

constexpr int kDistillThreads = 256;
constexpr int kDistillWarps = kDistillThreads / kWarp;
constexpr int kMaxCluster = 8;
enum DistillMode : int { kLoss = 0, kLossGrad = 1, kGradOnly = 2 };

struct DistillParams {
  const void* student;      // [B*P, V]
  const int* top_ids;       // [B*P, k]
  const float* top_logits;  // [B*P, k]
  const float* top_lse;     // [B*P] or null
  const int* lens;          // [B] or null
  const float* grad_loss;   // [B*P] (gradient modes)
  const float4* stats;      // [B*P] (kGradOnly)
  float* out_loss;          // [B*P]
  float4* out_stats;        // [B*P] or null
  void* out_grad;           // [B*P, V]
  int* out_status;          // [B*P] or null
  int P, V, k;
  int slice;                // 16-byte words per CTA
  float cc;                 // log2(e) / T
  float T, inv_t;           // T and 1 / T
  unsigned long long wait_ns;  // limit of the wait for the slice
};

struct alignas(16) DistillShared {
  float4 part[kMaxCluster];      // each CTA's {max, sum, status bits, -} of its slice without the record
  float2 warp_part[kDistillWarps];
  unsigned long long bar;        // the slice's arrival
  unsigned long long part_bar;   // the cluster's parts' arrival
  int id[SV_MAX_TOP];            // the record (-1: unused)
  float t[SV_MAX_TOP];           // its logits (-inf: unused)
  float p[SV_MAX_TOP];           // its teacher probabilities
  float sv[SV_MAX_TOP];          // the student's logits at its tokens
  int bad, late, twice;
  int used;                      // bit 0: an entry is used, bit 1: with a finite logit
  float t_max;                   // the record's largest finite logit (0: none)
  float norm, norm_lo;           // the teacher's log-sum-exp - t_max / T:
                                 // log p_j = (t_j - t_max) / T - norm
  float p_sum, p_rest;           // the record's mass and 1 - it
  float p_slack;                 // what rounding can make of a p_rest of 0
  float mass;                    // the teacher's: 1, or a record's whose mass does not fit its log-sum-exp
  float top_m;                   // the student's max on the record (NaN: unusable)
  float2 top_z;                  // and its sum there in that frame (hi, lo)
  struct Sums {                  // the student's sums:
    float m, M;                  // max outside the record, and over all
    float2 S, Z;                 // the sums in their frames
    float beta, inv_z, q_top;    // q_top: the student's mass on the record
    int status;
  } sums;
};

__device__ __forceinline__ uint16_t to_bf16(float v) {  // round to nearest even
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void store_value(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void store_value(float* p, float v) { *p = v; }

__device__ __forceinline__ void store_bits(uint16_t* p, uint32_t v) { *p = (uint16_t)v; }
__device__ __forceinline__ void store_bits(float* p, uint32_t v) { *p = __uint_as_float(v); }
__device__ __forceinline__ uint32_t load_bits(const uint16_t* p) { return *p; }
__device__ __forceinline__ uint32_t load_bits(const float* p) { return __float_as_uint(*p); }

// Writes the 32-bit pattern v (equal halves) over `bytes` bytes at `dst` (2-byte
// aligned).
__device__ void fill_bytes(char* dst, int bytes, uint32_t v = 0) {
  const int t = threadIdx.x;
  const int head = min(bytes, (int)((16u - ((uint32_t)(uintptr_t)dst & 15u)) & 15u));
  for (int i = 2 * t; i < head; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = (uint16_t)v;
  const int vecs = (bytes - head) / 16;
  for (int i = t; i < vecs; i += kDistillThreads)
    *reinterpret_cast<uint4*>(dst + head + 16 * i) = make_uint4(v, v, v, v);
  for (int i = head + 16 * vecs + 2 * t; i < bytes; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = (uint16_t)v;
}

// `bytes` bytes from shared memory go to global `dst` (both 2-byte aligned;
// the aligned 16-byte words around the source are readable).
__device__ void store_slice(char* dst, const unsigned char* src, int bytes) {
  const int t = threadIdx.x;
  const int head = min(bytes, (int)((16u - ((uint32_t)(uintptr_t)dst & 15u)) & 15u));
  for (int i = 2 * t; i < head; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
  const int vecs = (bytes - head) / 16;
  const uint32_t r = (uint32_t)(uintptr_t)(src + head) & 15u;
  const unsigned char* words = src + head - r;
  for (int i = t; i < vecs; i += kDistillThreads) {
    const uint4 a = load128(words + 16 * i);
    *reinterpret_cast<uint4*>(dst + head + 16 * i) =
        r == 0 ? a : shift_pair(a, load128(words + 16 * i + 16), r);
  }
  for (int i = head + 16 * vecs + 2 * t; i < bytes; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
}

// 2^((l - m) c) * scale of each element of a group, in packed pairs.
__device__ __forceinline__ f32x2 scaled_pair(float a, float b, f32x2 nm2, f32x2 c2, f32x2 s2) {
  float x, y;
  unpack2(mul2(add2(pack2(a, b), nm2), c2), x, y);
  return mul2(pack2(ex2(x), ex2(y)), s2);
}
__device__ __forceinline__ uint4 scaled_group(const uint4& g, float c, float m, float scale,
                                              const uint16_t*) {
  const f32x2 nm2 = pack2(-m, -m), c2 = pack2(c, c), s2 = pack2(scale, scale);
  const uint32_t w[4] = {g.x, g.y, g.z, g.w};
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x, y;
    unpack2(scaled_pair(bf16_lo(w[q]), bf16_hi(w[q]), nm2, c2, s2), x, y);
    o[q] = to_bf16x2(x, y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 scaled_group(const uint4& g, float c, float m, float scale,
                                              const float*) {
  const f32x2 nm2 = pack2(-m, -m), c2 = pack2(c, c), s2 = pack2(scale, scale);
  float x0, x1, x2, x3;
  unpack2(scaled_pair(__uint_as_float(g.x), __uint_as_float(g.y), nm2, c2, s2), x0, x1);
  unpack2(scaled_pair(__uint_as_float(g.z), __uint_as_float(g.w), nm2, c2, s2), x2, x3);
  return make_uint4(__float_as_uint(x0), __float_as_uint(x1), __float_as_uint(x2),
                    __float_as_uint(x3));
}

// x / T as hi + lo.
__device__ __forceinline__ void add_ratio(Pair& a, float x, const DistillParams& p, float sign) {
  const float q = x / p.T;
  a.add(sign * q);
  a.add(sign * (fmaf(-q, p.T, x) * p.inv_t));
}

// The k-sized part of a row: its record, the teacher's probabilities, and (kStats)
// the student's logits at the recorded tokens with their max and sum, read
// straight from the row so that all of it overlaps the slice's copy.  Sets s.bad for
// a token out of range, for a NaN or +inf logit, and for a
// log-sum-exp that is not finite beside a used entry.  A whole-CTA call.
template <typename T, int kMode>
__device__ void load_record(DistillShared& s, const DistillParams& p, long long row,
                            const T* src, int rank) {
  constexpr bool kStats = kMode != kGradOnly;
  // for the loss alone the leader CTA has the teacher's part to itself, the
  // others need the tokens
  const bool full = kMode != kLoss || rank == 0;
  const int t = threadIdx.x;
  const float lse = p.top_lse ? p.top_lse[row] : 0.f;
  if (t < p.k) {
    const int id = p.top_ids[row * p.k + t];
    const float v = p.top_logits[row * p.k + t];
    const bool in = id >= 0 && id < p.V;
    if (kStats && full) s.sv[t] = in ? widen(src[id]) : -INFINITY;
    s.id[t] = id;
    s.t[t] = id < 0 ? -INFINITY : v;
    int bad = 0;
    if (id >= 0 ? !in : id != -1) bad |= SV_REQ_BAD_TOKEN;
    if (id >= 0) {
      if (v != v || v == INFINITY) bad |= SV_REQ_BAD_LOGITS;
      if (p.top_lse && !is_finite(lse)) bad |= SV_REQ_BAD_LOGITS;
      atomicOr(&s.used, v > -INFINITY ? 3 : 1);
    }
    if (bad) atomicOr(&s.bad, bad);
  }
  __syncthreads();
  if (!full) return;
  if (kStats && t >= kWarp && t < 2 * kWarp) {
    constexpr int kPer = SV_MAX_TOP / kWarp;
    float x[kPer], m = -INFINITY;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int j = q * kWarp + lane_id();
      x[q] = j < p.k ? s.sv[j] : -INFINITY;
      m = max_nan(m, x[q]);
    }
    m = warp_max_nan(m);
    float z = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) z += ex2((x[q] - frame_of(m)) * p.cc);
    const float2 sum = warp_sum_pair(z);
    if (lane_id() == 0) {
      s.top_m = m == INFINITY ? qnan() : m;
      s.top_z = sum;
    }
  }
  if (t < kWarp) {
    constexpr int kPer = SV_MAX_TOP / kWarp;
    float v[kPer], m = -INFINITY;
    int used = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int j = q * kWarp + t;
      v[q] = j < p.k ? s.t[j] : -INFINITY;
      used += j < p.k && s.id[j] >= 0 ? 1 : 0;
      m = fmaxf(m, v[q]);
    }
    m = frame_of(warp_max(m));
    Pair norm;
    if (p.top_lse) {
      norm.add(lse);
      if (is_finite(m / p.T)) add_ratio(norm, m, p, -1.f);
      else norm.hi = m > 0.f ? -INFINITY : INFINITY;
    } else {  // the record's own
      float z = 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) z += expf((v[q] - m) * p.inv_t);
      const float2 l = log_pair(warp_sum_pair(z));
      norm.add(l.x);
      norm.add(l.y);
    }
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int j = q * kWarp + t;
      const float pj =
          v[q] == -INFINITY ? 0.f : expf(fmaf(v[q] - m, p.inv_t, -norm.hi) - norm.lo);
      if (j < p.k) s.p[j] = pj;
      sum += pj;
    }
    const float2 total = warp_sum_pair(sum);
    used = (int)__reduce_add_sync(0xffffffffu, (unsigned)used);
    if (t == 0) {
      s.t_max = m;
      s.norm = norm.hi;
      s.norm_lo = norm.lo;
      s.p_sum = total.x + total.y;
      s.p_rest = p.top_lse && used < p.V ? fmaxf(0.f, (1.f - total.x) - total.y) : 0.f;
      s.mass = p.top_lse && s.p_rest == 0.f ? s.p_sum : 1.f;
      // log-sum-exp: half a step of it, and as much in a sum it was rounded from; the p_j: 2^-20
      s.p_slack = 0x1p-20f + 0x1p-23f * fabsf(lse);
    }
  }
}

using Sums = DistillShared::Sums;

// From the record's and the cluster's parts; a call of one warp.
__device__ Sums row_sums(const DistillShared& s, int C, float c) {
  const int lane = lane_id();
  const float4 v = lane < C ? s.part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
  Sums r;
  r.m = warp_max_nan(v.x);
  r.S = warp_sum_pair<kMaxCluster>(v.y * to_frame(v.x, r.m, c));
  r.M = max_nan(r.m, s.top_m);
  r.status = (int)__reduce_or_sync(0xffffffffu, lane < C ? __float_as_uint(v.z) : 0u);
  // (a teacher mass past the range: a log-sum-exp far below its record)
  if (!(is_finite(r.M) && is_finite(s.p_sum)) && !(r.status & SV_REQ_TIMEOUT))
    r.status |= SV_REQ_BAD_LOGITS;
  const float up = to_frame(s.top_m, r.M, c), down = to_frame(r.m, r.M, c);
  const float rest = r.S.x * down, top = s.top_z.x * up;
  Pair Z;
  Z.add(top);
  Z.add(rest);
  Z.add(fmaf(s.top_z.x, up, -top) + s.top_z.y * up);
  Z.add(fmaf(r.S.x, down, -rest) + r.S.y * down);
  r.Z = make_float2(Z.hi, Z.lo);
  r.inv_z = r.status ? qnan() : 1.f / Z.value();
  r.q_top = top * r.inv_z;
  // q_rest - p_rest, of the two masses outside the record or of the two on it, whichever
  // are smaller: the roundings of two masses near 1 would be most of a small difference
  const float out = s.p_rest > 0.f && s.p_sum + r.q_top < 1.f ? s.p_sum - r.q_top
                                                              : s.mass * (rest * r.inv_z) - s.p_rest;
  r.beta = r.m == -INFINITY ? 0.f : out / r.S.x;
  return r;
}

// The loss of a row, by one warp:
//   sum_j p_j (((t_j - t_max) - (s_j - M)) / T - K) + p_rest (log p_rest - log q_rest)
// with K = norm - log Z.  The differences are taken before anything is rounded
// to their terms' size: where student and teacher agree the loss is far below
// its terms, and neither need be near zero.
__device__ float row_loss(const DistillShared& s, const DistillParams& p, const Sums& r) {
  const int lane = lane_id();
  const bool rest = r.m != -INFINITY;
  // lane 0: log Z, lane 1: log S
  const float2 mine = log_pair(lane == 1 && rest ? r.S : r.Z);
  const float2 lz = make_float2(__shfl_sync(0xffffffffu, mine.x, 0),
                                __shfl_sync(0xffffffffu, mine.y, 0));
  const float2 ls = make_float2(__shfl_sync(0xffffffffu, mine.x, 1),
                                __shfl_sync(0xffffffffu, mine.y, 1));
  Pair K;
  K.add(s.norm);
  K.add(-lz.x);
  K.add(-lz.y);
  K.add(s.norm_lo);
  const float k = K.value();
  float loss = 0.f;
  for (int j = lane; j < p.k; j += kWarp)
    if (s.p[j] > 0.f) {
      const float d = (s.t[j] - s.t_max) - (s.sv[j] - r.M), x = d * p.inv_t;
      // (a masked token of the type's lowest value may pass the range before p_j counts)
      // (and one of no student mass is +inf, where p_j / T may be 0)
      loss = is_finite(x)      ? fmaf(s.p[j], x - k, loss)
             : d == INFINITY ? INFINITY
                             : fmaf(s.p[j] * p.inv_t, d, loss);
    }
  loss = warp_sum(loss);
  if (s.p_rest > 0.f) {
    if (!rest) return s.p_rest > s.p_slack ? INFINITY : loss;
    if (!is_finite((r.M - r.m) / p.T)) return fmaf(s.p_rest * p.inv_t, r.M - r.m, loss);
    // a remainder that is most of the mass: its logarithm from what is left of it
    const float lp = s.p_sum < 0.5f ? log1pf(-s.p_sum) : logf(s.p_rest);
    Pair d;  // else log q_rest = log S + (m - M) / T - log Z, whatever underflowed
    d.add(lp);
    if (r.q_top < 0.5f) {
      d.add(-log1pf(-r.q_top));
    } else {
      add_ratio(d, r.m - r.M, p, -1.f);
      d.add(lz.x - ls.x);
      d.add(lz.y);
      d.add(-ls.y);
    }
    loss += s.p_rest * d.value();
  }
  return loss;
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kDistillThreads, 5) distill_kernel(const DistillParams p) {
  constexpr int VEC = Group<T>::VEC, kSize = (int)sizeof(T);
  constexpr int UN = 4;
  extern __shared__ __align__(16) unsigned char smem[];
  DistillShared& s = *reinterpret_cast<DistillShared*>(smem);
  unsigned char* words = smem + sizeof(DistillShared);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long row = blockIdx.x / C;
  const int t = threadIdx.x, lane = lane_id(), warp = t / kWarp;
  const T* tag = nullptr;

  // The row in aligned 16-byte words: byte x of the row is byte x + r of word
  // 0 on, r its misalignment.  This CTA has words w0 .. w1 - 1, row bytes
  // x0 .. x1 - 1.
  const int nb = p.V * kSize;
  const char* src = static_cast<const char*>(p.student) + row * (long long)nb;
  const int r = (int)((uintptr_t)src & 15u);
  const int all = (r + nb + 15) / 16;
  const int w0 = min(rank * p.slice, all), w1 = min(w0 + p.slice, all), nw = w1 - w0;
  const int x0 = min(nb, max(0, 16 * w0 - r)), x1 = max(x0, min(nb, 16 * w1 - r));
  char* grad = kMode == kLoss ? nullptr : static_cast<char*>(p.out_grad) + row * (long long)nb;

  // A row without loss or gradient (not needed, or a data error seen by
  // every CTA of the cluster alike).
  auto leave = [&](float loss, int status) {
    if (kMode != kLoss) fill_bytes(grad + x0, x1 - x0);
    if (kMode != kGradOnly && rank == 0 && t == 0) {
      p.out_loss[row] = loss;
      // 1/Z NaN: a later backward pass writes zeros
      if (p.out_stats) p.out_stats[row] = make_float4(0.f, 0.f, 0.f, qnan());
      if (p.out_status) p.out_status[row] = status;
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  if (p.lens) {
    const int b = (int)(row / p.P), i = (int)(row - (long long)b * p.P);
    const int len = p.lens[b];
    const bool ok = len >= 0 && len <= p.P;
    if (!ok || i >= len) {
      leave(ok ? 0.f : qnan(), ok ? 0 : SV_REQ_BAD_DRAFT_LEN);
      return;
    }
  }
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);  // {m, beta, M, 1/Z}
  if (kMode == kGradOnly) {
    st = p.stats[row];
    if (st.w != st.w) {
      leave(0.f, 0);
      return;
    }
  }

  // The slice on its way into shared memory: the words inside the row as one
  // bulk copy, the row's first and last word by element, -inf around them.
  const int lo = nw > 0 && 16 * w0 - r < 0 ? 1 : 0;
  const int hi = max(lo, nw > 0 && 16 * w1 - r > nb ? nw - 1 : nw);
  if (t == 0) {
    s.bad = s.used = s.late = s.twice = 0;
    mbar_init(smem_u32(&s.bar), 1);
    if (kMode != kGradOnly && C > 1) mbar_init(smem_u32(&s.part_bar), 1);
    fence_mbar_init();
    if (kMode != kGradOnly && C > 1)
      mbar_arrive_expect_tx(smem_u32(&s.part_bar), 16u * (uint32_t)(C - 1));
    const uint32_t bytes = 16u * (uint32_t)(hi - lo);
    mbar_arrive_expect_tx(smem_u32(&s.bar), bytes);
    if (bytes)
      bulk_copy(smem_u32(words + 16 * lo), src + (16 * (w0 + lo) - r), bytes, smem_u32(&s.bar));
  }
  if (t == kWarp || t == kWarp + 1) {
    const int i = t == kWarp ? (lo > 0 ? 0 : -1) : (hi < nw ? hi : -1);
    if (i >= 0) {
      const int x = 16 * (w0 + i) - r;
      uint4 v = Lane<T, VEC>::pad();
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int y = x + e * kSize;
        if (y >= 0 && y < nb) put(v, e, *reinterpret_cast<const T*>(src + y));
      }
      *reinterpret_cast<uint4*>(words + 16 * i) = v;
    }
  }
  // (no CTA writes into another's shared memory before that one has started)
  if (kMode != kGradOnly && C > 1) cluster_arrive();
  __syncthreads();
  load_record<T, kMode>(s, p, row, reinterpret_cast<const T*>(src), rank);
  // one warp waits for the copy, the others at the barrier
  if (warp == kDistillWarps - 1 && !mbar_wait(smem_u32(&s.bar), 0, p.wait_ns)) {
    s.late = 1;
    mbar_wait(smem_u32(&s.bar), 0);  // the copy lands before the memory is left
  }
  __syncthreads();
  const bool late = s.late != 0;
  const int used = s.used;
  // (without a log-sum-exp the record has to hold some mass)
  const int bad_record = s.bad | (!p.top_lse && used == 1 ? SV_REQ_BAD_LOGITS : 0);
  if (bad_record || used == 0) {
    if (kMode != kGradOnly && C > 1) cluster_wait();
    leave(bad_record ? qnan() : 0.f, bad_record);
    return;
  }

  if (kMode == kGradOnly && late) {  // no status to say so: NaN (all bits set)
    fill_bytes(grad + x0, x1 - x0, 0xffffffffu);
    return;
  }

  // The student's logits at the recorded tokens leave the slice.
  const int my_id = t < p.k ? s.id[t] : -1;
  const int my_x = my_id * kSize;  // < 2^21
  const bool mine = my_id >= 0 && my_x >= x0 && my_x < x1;
  T* my_at = reinterpret_cast<T*>(words + (my_x + r - 16 * w0));
  float my_v = 0.f;
  if (mine) my_v = widen(*my_at);
  if (kMode != kGradOnly) {
    // a token given twice: of the entries that write their number there, one
    // does not find its own
    if (mine) store_bits(my_at, (uint32_t)t);
    __syncthreads();
    if (mine && load_bits(my_at) != (uint32_t)t) s.twice = 1;
  }
  if (mine) store_value(my_at, -INFINITY);
  __syncthreads();

  if (kMode != kGradOnly) {
    RunningSum run;
    int i = t;
    for (; i + (UN - 1) * kDistillThreads < nw; i += kDistillThreads * UN) {
      uint4 g[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) g[u] = load128(words + 16 * (i + u * kDistillThreads));
      run.add(g, p.cc, tag);
    }
    for (; i < nw; i += kDistillThreads) {
      const uint4 g[1] = {load128(words + 16 * i)};
      run.add(g, p.cc, tag);
    }
    const float2 wr = warp_running(run, p.cc);
    if (lane == 0) s.warp_part[warp] = wr;
    if (C > 1) cluster_wait();  // every CTA has started
    __syncthreads();
    if (warp == 0) {
      const float2 v = lane < kDistillWarps ? s.warp_part[lane] : make_float2(-INFINITY, 0.f);
      const float m = warp_max_nan(v.x);
      const float sum = warp_sum_pair<kDistillWarps>(v.y * to_frame(v.x, m, p.cc)).x;
      const int status = (late ? SV_REQ_TIMEOUT : 0) | (s.twice ? SV_REQ_BAD_TOKEN : 0);
      const float4 part = make_float4(m, sum, __uint_as_float((uint32_t)status), 0.f);
      bool came = true;
      if (lane == 0) s.part[rank] = part;
      __syncwarp();
      if (C > 1) {
        // to all others, or for the loss alone to the leader
        if (lane != rank && lane < (kMode == kLoss ? 1 : C))
          send16(in_cta(smem_u32(&s.part[rank]), lane), in_cta(smem_u32(&s.part_bar), lane), part);
        if (kMode == kLoss && rank != 0) return;
        // (a peer that does not send has failed; the limit is the waits' default)
        came = mbar_wait_cluster(smem_u32(&s.part_bar), 0, kWaitLimitNs);
      }
      Sums sums = row_sums(s, C, p.cc);
      if (!__all_sync(0xffffffffu, came)) {
        sums.status = SV_REQ_TIMEOUT;
        sums.inv_z = qnan();
      }
      if (lane == 0) {
        s.sums = sums;
        if (rank == 0) {
          const bool wrong = sums.status != 0;
          if (p.out_stats)
            p.out_stats[row] =
                wrong ? make_float4(0.f, 0.f, 0.f, qnan())
                      : make_float4(frame_of(sums.m), sums.beta, sums.M, sums.inv_z);
          if (p.out_status) p.out_status[row] = sums.status;
          if (wrong) p.out_loss[row] = qnan();
        }
      }
    }
    if (kMode == kLoss) {
      if (rank == 0 && warp == 0) {
        __syncwarp();
        if (s.sums.status == 0) {
          const float loss = row_loss(s, p, s.sums);
          if (lane == 0) p.out_loss[row] = loss;
        }
      }
      // (the parts sent here have arrived before the CTA's memory goes: warp 0 saw them)
      return;
    }
    __syncthreads();
    st = make_float4(frame_of(s.sums.m), s.sums.beta, s.sums.M, s.sums.inv_z);
  }

  // The gradient.
  if (st.w != st.w) {
    fill_bytes(grad + x0, x1 - x0);
    return;
  }
  // (past the range at the smallest temperatures: 0 gradients stay 0)
  const float g = p.grad_loss[row];
  const float scale = is_finite(g) ? fminf(fmaxf(g / p.T, -FLT_MAX), FLT_MAX) : g / p.T;
  const float beta = st.y * scale;
  const float my_q = ex2((my_v - st.z) * p.cc) * st.w;
  const float my_grad = (s.mass * my_q - (t < p.k ? s.p[t] : 0.f)) * scale;
  if (((uintptr_t)grad & 15u) == (uint32_t)r) {
    // word for word as the student's row; the recorded tokens after the words they lie in
    for (int i = t; i < nw; i += kDistillThreads) {
      const uint4 g = scaled_group(load128(words + 16 * i), p.cc, st.x, beta, tag);
      const int x = 16 * (w0 + i) - r;
      if (x >= 0 && x + 16 <= nb) {
        *reinterpret_cast<uint4*>(grad + x) = g;
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int y = x + e * kSize;
          if (y >= 0 && y < nb) store_value(reinterpret_cast<T*>(grad + y), Lane<T, VEC>::get(g, e));
        }
      }
    }
    __syncthreads();
    if (mine) store_value(reinterpret_cast<T*>(grad + my_x), my_grad);
  } else {  // in place, then shifted out
    for (int i = t; i < nw; i += kDistillThreads) {
      uint4* at = reinterpret_cast<uint4*>(words + 16 * i);
      *at = scaled_group(*at, p.cc, st.x, beta, tag);
    }
    __syncthreads();
    if (mine) store_value(my_at, my_grad);
    __syncthreads();
    store_slice(grad + x0, words + (x0 + r - 16 * w0), x1 - x0);
  }
  if (kMode == kLossGrad && rank == 0 && warp == 0) {  // nothing waits for the loss here
    const float loss = row_loss(s, p, s.sums);
    if (lane == 0) p.out_loss[row] = loss;
  }
}

constexpr int kMaxSliceBytes = SV_MAX_DISTILL_ROW / kMaxCluster + 64;

template <typename T, int kMode>
cudaError_t launch_distill(const DistillParams& p, long long rows, int C, cudaStream_t stream) {
  static PerDevice once;
  auto* fn = distill_kernel<T, kMode>;
  cudaError_t err = per_device(once, nullptr, [&](int&) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(DistillShared) + kMaxSliceBytes);
  });
  if (err != cudaSuccess) return err;
  // a word past the slice: the last shifted store reads it
  const size_t smem = sizeof(DistillShared) + 16 * ((size_t)p.slice + 1);
  return launch_early(fn, (unsigned)(rows * C), kDistillThreads, smem, C, stream, p);
}

template <int kMode>
sv_status run_distill(DistillParams& p, sv_dtype dtype, long long rows, cudaStream_t stream) {
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return SV_ERR_CUDA;
  const int esz = dtype == SV_BF16 ? 2 : 4;
  // A slice of at most 40 KB leaves five CTAs on an SM; few rows are spread
  // over more CTAs while a slice still gives every thread two words.
  int C = 1;
  while (C < kMaxCluster && ((long long)p.V * esz > 40960LL * C ||
                             (rows * C < 2LL * dev.sms && (long long)p.V * esz > 8192LL * C)))
    C *= 2;
  // words of a row at the worst alignment
  const bool aligned = ((uintptr_t)p.student & 15u) == 0 && (long long)p.V * esz % 16 == 0;
  const int all = (int)(((long long)p.V * esz + (aligned ? 0 : 16 - esz) + 15) / 16);
  p.slice = (all + C - 1) / C;
  const cudaError_t err = dtype == SV_BF16 ? launch_distill<uint16_t, kMode>(p, rows, C, stream)
                                           : launch_distill<float, kMode>(p, rows, C, stream);
  return err == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

sv_status check_distill(float temperature, sv_dtype dtype, int B, int P, int V, int k) {
  if (!(temperature > 0.f) || isinf(temperature)) return SV_ERR_TEMPERATURE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (B < 0 || B > SV_MAX_B || P < 1 || (long long)B * P > SV_MAX_ROWS || V < 1 ||
      (long long)V * (dtype == SV_BF16 ? 2 : 4) > SV_MAX_DISTILL_ROW || k < 1 || k > SV_MAX_TOP)
    return SV_ERR_SHAPE;
  return SV_OK;
}

// Whether two pieces of memory overlap (b may be null: no).
bool meet(const void* a, long long a_bytes, const void* b, long long b_bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// out_grad may be the student's logits themselves, or lie apart from them.
bool grad_overlaps(const void* student, const void* grad, size_t bytes) {
  return student != grad && meet(student, (long long)bytes, grad, (long long)bytes);
}

DistillParams distill_params(const void* student, const int32_t* ids, const float* logits,
                             const float* lse, const int32_t* lens, float temperature, int P,
                             int V, int k) {
  DistillParams p;
  memset(&p, 0, sizeof p);
  p.student = student;
  p.top_ids = ids;
  p.top_logits = logits;
  p.top_lse = lse;
  p.lens = lens;
  p.P = P;
  p.V = V;
  p.k = k;
  p.cc = exponent_scale(temperature);
  p.T = temperature;
  p.wait_ns = wait_limit_ns();
  const double inv = 1.0 / (double)temperature;
  p.inv_t = inv < (double)FLT_MAX ? (float)inv : FLT_MAX;
  return p;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

sv_status spec_distill(const void* student_logits, const int32_t* top_ids,
                       const float* top_logits, const float* top_lse, const int32_t* lens,
                       const float* grad_loss, float temperature, float* out_loss,
                       float* out_stats, void* out_grad, int32_t* out_status, sv_dtype dtype,
                       int B, int P, int V, int k, sv_stream_t stream) {
  const sv_status ok = check_distill(temperature, dtype, B, P, V, k);
  if (ok != SV_OK) return ok;
  if (B == 0) return SV_OK;
  const uintptr_t mask = dtype == SV_BF16 ? 1u : 3u;
  if (!student_logits || !top_ids || !top_logits || !out_loss || (grad_loss && !out_grad))
    return SV_ERR_NULL;
  if (((uintptr_t)student_logits & mask) || ((uintptr_t)out_stats & 15u)) return SV_ERR_NULL;
  DistillParams p = distill_params(student_logits, top_ids, top_logits, top_lse, lens,
                                   temperature, P, V, k);
  p.out_loss = out_loss;
  p.out_stats = reinterpret_cast<float4*>(out_stats);
  p.out_status = out_status;
  const long long rows = (long long)B * P;
  if (!grad_loss) return run_distill<kLoss>(p, dtype, rows, (cudaStream_t)stream);
  if ((uintptr_t)out_grad & mask) return SV_ERR_NULL;
  // (a row's CTAs read its weight until the end, after the leader wrote the row's loss)
  if (grad_overlaps(student_logits, out_grad, (size_t)rows * V * (dtype == SV_BF16 ? 2 : 4)) ||
      meet(grad_loss, 4 * rows, out_loss, 4 * rows) ||
      meet(grad_loss, 4 * rows, out_stats, 16 * rows) ||
      meet(grad_loss, 4 * rows, out_status, 4 * rows))
    return SV_ERR_ALIAS;
  p.grad_loss = grad_loss;
  p.out_grad = out_grad;
  return run_distill<kLossGrad>(p, dtype, rows, (cudaStream_t)stream);
}

sv_status spec_distill_grad(const void* student_logits, const int32_t* top_ids,
                            const float* top_logits, const float* top_lse, const int32_t* lens,
                            const float* stats, const float* grad_loss, float temperature,
                            void* out_grad, sv_dtype dtype, int B, int P, int V, int k,
                            sv_stream_t stream) {
  const sv_status ok = check_distill(temperature, dtype, B, P, V, k);
  if (ok != SV_OK) return ok;
  if (B == 0) return SV_OK;
  const uintptr_t mask = dtype == SV_BF16 ? 1u : 3u;
  if (!student_logits || !top_ids || !top_logits || !stats || !grad_loss || !out_grad)
    return SV_ERR_NULL;
  if (((uintptr_t)student_logits & mask) || ((uintptr_t)out_grad & mask) ||
      ((uintptr_t)stats & 15u))
    return SV_ERR_NULL;
  const long long rows = (long long)B * P;
  if (grad_overlaps(student_logits, out_grad, (size_t)rows * V * (dtype == SV_BF16 ? 2 : 4)))
    return SV_ERR_ALIAS;
  DistillParams p = distill_params(student_logits, top_ids, top_logits, top_lse, lens,
                                   temperature, P, V, k);
  p.stats = reinterpret_cast<const float4*>(stats);
  p.grad_loss = grad_loss;
  p.out_grad = out_grad;
  return run_distill<kGradOnly>(p, dtype, rows, (cudaStream_t)stream);
}

}  // extern "C"
