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
//   2^((s_i - m) c) * beta * grad_loss / T,   beta = (q_rest - p_rest) / S,
// and on a recorded token (2^((s_j - M) c) / Z - p_j) * grad_loss / T with M
// and Z the max and sum over all tokens.  {m, beta, M, 1/Z} are the row's
// statistics.
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
constexpr float kLn2 = 0.6931471805599453f;

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
  int slice;                // elements per CTA (a multiple of VEC)
  float cc;                 // log2(e) / T
  double inv_t;             // 1 / T
  RowSpan span;
};

struct DistillShared {
  float4 part[kMaxCluster];      // each CTA's {max, sum, -, -} over its slice without the record
  float2 warp_part[kDistillWarps];
  int id[SV_MAX_TOP];            // the record (-1: unused)
  float t[SV_MAX_TOP];           // its logits (-inf: unused)
  float p[SV_MAX_TOP];           // its teacher probabilities
  float sv[SV_MAX_TOP];          // the student's logits at its tokens
  int bad, used;
  double norm;                   // the teacher's log-sum-exp: log p_j = t_j / T - norm
  double p_rest;
  float m, M;                    // the student's max outside the record, and over all
  double S, Z;                   // its sums there, in the frames of m and M
  float4 stat;                   // {m, beta, M, 1/Z}
};

// Writes `bytes` bytes of zeros at `dst` (2-byte aligned).
__device__ void zero_bytes(char* dst, long long bytes) {
  const int t = threadIdx.x;
  const long long head = min(bytes, (long long)((16u - ((uint32_t)(uintptr_t)dst & 15u)) & 15u));
  for (long long i = 2 * t; i < head; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = 0;
  const long long vecs = (bytes - head) / 16;
  for (long long i = t; i < vecs; i += kDistillThreads)
    *reinterpret_cast<uint4*>(dst + head + 16 * i) = make_uint4(0, 0, 0, 0);
  for (long long i = head + 16 * vecs + 2 * t; i < bytes; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = 0;
}

// The slice of `bytes` bytes at shared address `src` (16-byte aligned) goes to
// global `dst` (2-byte aligned).
__device__ void store_slice(char* dst, const unsigned char* src, int bytes) {
  const int t = threadIdx.x;
  const int head = min(bytes, (int)((16u - ((uint32_t)(uintptr_t)dst & 15u)) & 15u));
  for (int i = 2 * t; i < head; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
  const int vecs = (bytes - head) / 16;
  if (head == 0) {
    for (int i = t; i < vecs; i += kDistillThreads)
      *reinterpret_cast<uint4*>(dst + 16 * i) = *reinterpret_cast<const uint4*>(src + 16 * i);
  } else {  // the 16 bytes from src + head + 16 i span two shared words
    for (int i = t; i < vecs; i += kDistillThreads) {
      const uint4* a = reinterpret_cast<const uint4*>(src + 16 * i);
      *reinterpret_cast<uint4*>(dst + head + 16 * i) = shift_pair(a[0], a[1], (uint32_t)head);
    }
  }
  for (int i = head + 16 * vecs + 2 * t; i < bytes; i += 2 * kDistillThreads)
    *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
}

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

// 2^((l - m) c) * scale of each element of a group.
__device__ __forceinline__ uint4 scaled_group(const uint4& g, float c, float m, float scale,
                                              const uint16_t*) {
  const uint32_t w[4] = {g.x, g.y, g.z, g.w};
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = to_bf16x2(ex2((bf16_lo(w[q]) - m) * c) * scale,
                     ex2((bf16_hi(w[q]) - m) * c) * scale);
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 scaled_group(const uint4& g, float c, float m, float scale,
                                              const float*) {
  auto f = [&](uint32_t w) {
    return __float_as_uint(ex2((__uint_as_float(w) - m) * c) * scale);
  };
  return make_uint4(f(g.x), f(g.y), f(g.z), f(g.w));
}

// The teacher's side of a row: its record and probabilities.  Sets s.bad for
// a token out of range or given twice, for a NaN or +inf logit, and for a
// log-sum-exp that is not finite beside a used entry.  By the
// first warps; the caller synchronises around it.
__device__ void load_record(DistillShared& s, const DistillParams& p, long long row) {
  const int t = threadIdx.x;
  const float lse = p.top_lse ? p.top_lse[row] : 0.f;
  if (t < p.k) {
    const int id = p.top_ids[row * p.k + t];
    const float v = p.top_logits[row * p.k + t];
    s.id[t] = id;
    s.t[t] = id < 0 ? -INFINITY : v;
    if (id < -1 || id >= p.V) atomicOr(&s.bad, SV_REQ_BAD_TOKEN);
    if (id >= 0) {
      atomicAdd(&s.used, 1);
      if (v != v || v == INFINITY) atomicOr(&s.bad, SV_REQ_BAD_LOGITS);
    }
  }
  __syncthreads();
  if (t == 0 && s.used > 0 && p.top_lse && !is_finite(lse)) atomicOr(&s.bad, SV_REQ_BAD_LOGITS);
  if (t < p.k && s.id[t] >= 0)
    for (int j = 0; j < t; ++j)
      if (s.id[j] == s.id[t]) atomicOr(&s.bad, SV_REQ_BAD_TOKEN);
  if (t < kWarp) {
    constexpr int kPer = SV_MAX_TOP / kWarp;
    double x[kPer];
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int j = q * kWarp + t;
      const float v = j < p.k ? s.t[j] : -INFINITY;
      x[q] = (double)v * p.inv_t;
      m = fmaxf(m, v);
    }
    double norm = (double)lse;
    if (!p.top_lse) {
      m = warp_max(m);
      const double mt = m == -INFINITY ? 0.0 : (double)m * p.inv_t;
      double z = 0.0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) z += (double)expf((float)(x[q] - mt));
      norm = mt + log(warp_sum(z));
    }
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int j = q * kWarp + t;
      const float pj = x[q] == -INFINITY ? 0.f : expf((float)(x[q] - norm));
      if (j < p.k) s.p[j] = pj;
      sum += (double)pj;
    }
    sum = warp_sum(sum);
    if (t == 0) {
      s.norm = norm;
      s.p_rest = p.top_lse && s.used < p.V ? fmax(0.0, 1.0 - sum) : 0.0;
    }
  }
}

// The loss of a row, by one warp.  The logarithms' differences are taken in 64
// bits: where student and teacher agree the loss is far below its terms.
__device__ double row_loss(const DistillShared& s, const DistillParams& p) {
  const int lane = lane_id();
  const double mine = log(lane == 0 ? s.Z : lane == 1 ? s.S : s.p_rest > 0.0 ? s.p_rest : 1.0);
  const double lz = __shfl_sync(0xffffffffu, mine, 0), ls = __shfl_sync(0xffffffffu, mine, 1),
               lr = __shfl_sync(0xffffffffu, mine, 2);
  double loss = 0.0;
  for (int j = lane; j < p.k; j += kWarp)
    if (s.p[j] > 0.f) {
      const double log_q = ((double)s.sv[j] - (double)s.M) * p.inv_t - lz;
      loss += (double)s.p[j] * (((double)s.t[j] * p.inv_t - s.norm) - log_q);
    }
  loss = warp_sum(loss);
  if (s.p_rest > 0.0)
    loss += s.m == -INFINITY
                ? INFINITY
                : s.p_rest * (lr - (ls + ((double)s.m - (double)s.M) * p.inv_t - lz));
  return loss;
}

template <typename T, bool kAligned, int kMode>
__global__ void __launch_bounds__(kDistillThreads, 4) distill_kernel(const DistillParams p) {
  constexpr int VEC = Group<T>::VEC;
  constexpr int UN = 4;
  extern __shared__ __align__(16) unsigned char smem[];
  DistillShared& s = *reinterpret_cast<DistillShared*>(smem);
  unsigned char* slice = smem + (sizeof(DistillShared) + 15) / 16 * 16;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long row = blockIdx.x / C;
  const int t = threadIdx.x, lane = lane_id(), warp = t / kWarp;
  const int e0 = min(rank * p.slice, p.V), e1 = min(e0 + p.slice, p.V);
  const T* tag = nullptr;
  char* grad = kMode == kLoss ? nullptr
                              : static_cast<char*>(p.out_grad) +
                                    (row * (long long)p.V + e0) * (long long)sizeof(T);
  const int bytes = (e1 - e0) * (int)sizeof(T);

  // A row without loss or gradient (not needed, or a data error seen by
  // every CTA of the cluster alike).
  auto leave = [&](float loss, int status) {
    if (kMode != kLoss) zero_bytes(grad, bytes);
    if (kMode != kGradOnly && rank == 0 && t == 0) {
      p.out_loss[row] = loss;
      // beta 0 and 1/Z NaN: a later backward pass writes zeros
      if (p.out_stats) p.out_stats[row] = make_float4(0.f, 0.f, 0.f, qnan());
      if (p.out_status) p.out_status[row] = status;
    }
  };
  if (p.lens) {
    const int b = (int)(row / p.P), i = (int)(row - (long long)b * p.P);
    const int len = p.lens[b];
    const bool ok = len >= 0 && len <= p.P;
    if (!ok || i >= len) {
      leave(ok ? 0.f : qnan(), ok ? 0 : SV_REQ_BAD_DRAFT_LEN);
      return;
    }
  }
  if (kMode == kGradOnly) {
    const float4 st = p.stats[row];
    if (st.w != st.w) {
      leave(0.f, 0);
      return;
    }
    if (t == 0) s.stat = st;
  }

  // The slice, and the record while it is under way.
  const T* src = reinterpret_cast<const T*>(p.student) + row * (long long)p.V;
  for (int j0 = e0; j0 < e1; j0 += kDistillThreads * VEC * UN) {
    uint4 g[UN];
    load_groups<T, kAligned>(g, src, j0 + t * VEC, kDistillThreads * VEC, e1, p.V, p.span);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int j = j0 + (u * kDistillThreads + t) * VEC;
      if (j < e1) *reinterpret_cast<uint4*>(slice + (size_t)(j - e0) * sizeof(T)) = g[u];
    }
  }
  if (t == 0) s.bad = s.used = 0;
  __syncthreads();
  load_record(s, p, row);
  __syncthreads();
  const int bad_record = s.bad, used = s.used;
  if (bad_record || used == 0) {
    leave(bad_record ? qnan() : 0.f, bad_record);
    return;
  }
  if (kMode != kGradOnly && C > 1) cluster.sync();  // every CTA has started

  // The student's logits at the recorded tokens leave the slice.
  if (t < p.k) {
    const int id = s.id[t];
    if (id >= e0 && id < e1) {
      T* at = reinterpret_cast<T*>(slice) + (id - e0);
      const float v = widen(*at);
      if (kMode != kGradOnly && C > 1) {
        for (int c = 0; c < C; ++c) cluster.map_shared_rank(&s, c)->sv[t] = v;
      } else {
        s.sv[t] = v;
      }
      store_value(at, -INFINITY);
    }
  }
  __syncthreads();

  if (kMode != kGradOnly) {
    RunningSum r;
    for (int j0 = 0; j0 < e1 - e0; j0 += kDistillThreads * VEC * UN) {
      uint4 g[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int j = j0 + (u * kDistillThreads + t) * VEC;
        g[u] = j < e1 - e0 ? load128(slice + (size_t)j * sizeof(T)) : Lane<T, VEC>::pad();
      }
      r.add(g, p.cc, tag);
    }
    const float2 wr = warp_running(r, p.cc);
    if (lane == 0) s.warp_part[warp] = wr;
    __syncthreads();
    if (warp == 0) {
      const float2 v = lane < kDistillWarps ? s.warp_part[lane] : make_float2(-INFINITY, 0.f);
      const float m = warp_max_nan(v.x);
      const float sum = warp_sum(v.y * to_frame(v.x, m, p.cc));
      if (lane < C) {
        DistillShared* to = C > 1 ? cluster.map_shared_rank(&s, lane) : &s;
        to->part[rank] = make_float4(m, sum, 0.f, 0.f);
      }
    }
    if (C > 1) cluster.sync(); else __syncthreads();

    if (warp == 0) {
      // the rest: its max m and sum S over the cluster's slices
      const float4 v = lane < C ? s.part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      const float m = warp_max_nan(v.x);
      const double S = warp_sum((double)(v.y * to_frame(v.x, m, p.cc)));
      // the record, and both together in the frame of M
      constexpr int kPer = SV_MAX_TOP / kWarp;
      float x[kPer], M = -INFINITY;
      bool wrong = m != m || m == INFINITY;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int j = q * kWarp + lane;
        x[q] = j < p.k && s.id[j] >= 0 ? s.sv[j] : -INFINITY;
        wrong = wrong || x[q] != x[q] || x[q] == INFINITY;
        M = fmaxf(M, x[q]);
      }
      M = fmaxf(warp_max(M), m);
      wrong = __any_sync(0xffffffffu, wrong) || M == -INFINITY;
      double z = 0.0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) z += (double)ex2((x[q] - M) * p.cc);
      const double rest = m == -INFINITY ? 0.0 : S * (double)ex2((m - M) * p.cc);
      const double Z = warp_sum(z) + rest;
      if (lane == 0) {
        const float beta = m == -INFINITY ? 0.f : (float)((rest / Z - s.p_rest) / S);
        s.m = m;
        s.M = M;
        s.S = m == -INFINITY ? 1.0 : S;
        s.Z = Z;
        s.stat = make_float4(frame_of(m), beta, M, wrong ? qnan() : (float)(1.0 / Z));
        if (rank == 0) {
          if (p.out_stats) p.out_stats[row] = wrong ? make_float4(0.f, 0.f, 0.f, qnan()) : s.stat;
          if (p.out_status) p.out_status[row] = wrong ? SV_REQ_BAD_LOGITS : 0;
          if (wrong) p.out_loss[row] = qnan();
        }
      }
    }
    if (kMode == kLoss) {
      if (rank == 0 && warp == 0) {
        __syncwarp();
        if (s.stat.w == s.stat.w) {
          const double loss = row_loss(s, p);
          if (lane == 0) p.out_loss[row] = (float)loss;
        }
      }
      return;
    }
    __syncthreads();
  }

  // The gradient: the slice in place, then the recorded tokens, then out.
  const float4 st = s.stat;
  if (st.w != st.w) {
    zero_bytes(grad, bytes);
    return;
  }
  const float scale = (float)((double)p.grad_loss[row] * p.inv_t);
  const float beta = st.y * scale;
  for (int j = t * VEC; j < e1 - e0; j += kDistillThreads * VEC) {
    uint4* at = reinterpret_cast<uint4*>(slice + (size_t)j * sizeof(T));
    *at = scaled_group(*at, p.cc, st.x, beta, tag);
  }
  __syncthreads();
  if (t < p.k) {
    const int id = s.id[t];
    if (id >= e0 && id < e1)
      store_value(reinterpret_cast<T*>(slice) + (id - e0),
                  (ex2((s.sv[t] - st.z) * p.cc) * st.w - s.p[t]) * scale);
  }
  __syncthreads();
  store_slice(grad, slice, bytes);
  if (kMode == kLossGrad && rank == 0 && warp == 0) {  // nothing waits for the loss here
    const double loss = row_loss(s, p);
    if (lane == 0) p.out_loss[row] = (float)loss;
  }
}

constexpr int kSharedHead = (int)(sizeof(DistillShared) + 15) / 16 * 16;
constexpr int kMaxSliceBytes = SV_MAX_DISTILL_ROW / kMaxCluster + 256;

template <typename T, bool kAligned, int kMode>
cudaError_t launch_distill(const DistillParams& p, long long rows, int C, cudaStream_t stream) {
  static PerDevice once;
  auto* fn = distill_kernel<T, kAligned, kMode>;
  cudaError_t err = per_device(once, nullptr, [&](int&) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSharedHead + kMaxSliceBytes);
  });
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kDistillThreads);
  // 16 bytes past the slice: the last shifted store reads the word after it
  cfg.dynamicSmemBytes = kSharedHead + (size_t)p.slice * sizeof(T) + 16;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <int kMode>
sv_status run_distill(DistillParams& p, sv_dtype dtype, long long rows, cudaStream_t stream) {
  DeviceInfo dev;
  if (device_info(&dev) != cudaSuccess) return SV_ERR_CUDA;
  const int esz = dtype == SV_BF16 ? 2 : 4;
  // A slice of at most 40 KB leaves five CTAs on an SM; few rows are spread
  // over more CTAs while a slice still gives every thread a group.
  int C = 1;
  while (C < kMaxCluster && ((long long)p.V * esz > 40960LL * C ||
                             (rows * C < 2LL * dev.sms && (long long)p.V * esz > 8192LL * C)))
    C *= 2;
  const int vec = 16 / esz;
  p.slice = ((p.V + C - 1) / C + vec - 1) / vec * vec;
  const char* first = static_cast<const char*>(p.student);
  const size_t bytes = (size_t)rows * (size_t)p.V * esz;
  p.span.first = first;
  p.span.last = first + bytes;
  const bool aligned = ((uintptr_t)first & 15u) == 0 && ((size_t)p.V * esz) % 16 == 0;
  cudaError_t err;
  if (dtype == SV_BF16)
    err = aligned ? launch_distill<uint16_t, true, kMode>(p, rows, C, stream)
                  : launch_distill<uint16_t, false, kMode>(p, rows, C, stream);
  else
    err = aligned ? launch_distill<float, true, kMode>(p, rows, C, stream)
                  : launch_distill<float, false, kMode>(p, rows, C, stream);
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

// out_grad may be the student's logits themselves, or lie apart from them.
bool grad_overlaps(const void* student, const void* grad, size_t bytes) {
  const uintptr_t a = (uintptr_t)student, b = (uintptr_t)grad;
  return a != b && a < b + bytes && b < a + bytes;
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
  p.inv_t = 1.0 / (double)temperature;
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
  if (grad_overlaps(student_logits, out_grad, (size_t)rows * V * (dtype == SV_BF16 ? 2 : 4)))
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
