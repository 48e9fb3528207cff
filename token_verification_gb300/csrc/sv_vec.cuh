// sv_vec.cuh - rows of any alignment in 16-byte groups, ordered keys, and
// cluster-wide shared memory: helpers of the top-logits, beam-selection and
// distillation kernels.
//
// Those kernels cut a row by element index - group i holds elements i*VEC ..
// i*VEC + VEC - 1 whatever the row's address - so that the order of every sum
// follows from the row's contents alone: equal rows give equal sums, and equal
// candidates of different beams stay equal.  A row that does not start on a
// 16-byte boundary (odd vocabularies) is read as the two aligned 16-byte
// words around each group, shifted together in registers.
#pragma once

#include <cooperative_groups.h>

#include "sv_common.cuh"

namespace sv {
namespace {

namespace cg = cooperative_groups;

// Bytes r .. r + 15 of the 32 bytes a, b (0 <= r < 16, r even).
__device__ __forceinline__ uint4 shift_pair(const uint4& a, const uint4& b, uint32_t r) {
  uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x;
  if (r & 8u) {
    w0 = a.z; w1 = a.w; w2 = b.x; w3 = b.y; w4 = b.z;
  }
  if (r & 4u) {
    const uint32_t w5 = (r & 8u) ? b.w : b.y;
    w0 = w1; w1 = w2; w2 = w3; w3 = w4; w4 = w5;
  }
  if (r & 2u) {
    w0 = __funnelshift_r(w0, w1, 16);
    w1 = __funnelshift_r(w1, w2, 16);
    w2 = __funnelshift_r(w2, w3, 16);
    w3 = __funnelshift_r(w3, w4, 16);
  }
  return make_uint4(w0, w1, w2, w3);
}

// The same with the shift in words known at compile time (4 * kWords + 0 or 2
// bytes; `bits` is the whole shift times 8).
template <int kWords>
struct Shift {
  static constexpr int value = kWords;
};
template <int kWords>
__device__ __forceinline__ uint4 shift_words(const uint4& a, const uint4& b, uint32_t bits) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const uint32_t half = bits & 16u;  // (a funnel shift by 0 is its first word)
  return make_uint4(__funnelshift_r(w[kWords], w[kWords + 1], half),
                    __funnelshift_r(w[kWords + 1], w[kWords + 2], half),
                    __funnelshift_r(w[kWords + 2], w[kWords + 3], half),
                    __funnelshift_r(w[kWords + 3], w[kWords + 4], half));
}

// A tensor of logit rows: [first, last) is its memory, read nowhere else.
struct RowSpan {
  const char* first;
  const char* last;
};

template <typename T>
struct Group {
  static constexpr int VEC = 16 / (int)sizeof(T);
};

__device__ __forceinline__ void put(uint4& v, int e, uint16_t x) {
  uint32_t* w = e < 2 ? &v.x : e < 4 ? &v.y : e < 6 ? &v.z : &v.w;
  *w = (e & 1) ? (*w & 0x0000ffffu) | ((uint32_t)x << 16) : (*w & 0xffff0000u) | x;
}
__device__ __forceinline__ void put(uint4& v, int e, float x) {
  uint32_t* w = e == 0 ? &v.x : e == 1 ? &v.y : e == 2 ? &v.z : &v.w;
  *w = __float_as_uint(x);
}

__device__ __forceinline__ uint4 load128(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// Elements j .. j + VEC - 1 of a row of V elements, -inf past its end.
// kAligned: every row of the tensor starts on a 16-byte boundary.
template <typename T, bool kAligned>
__device__ __forceinline__ uint4 load_group(const T* row, int j, int V, const RowSpan& span) {
  constexpr int VEC = Group<T>::VEC;
  if (j + VEC <= V) {
    const char* p = reinterpret_cast<const char*>(row + j);
    if (kAligned) return load128(p);
    const uint32_t r = (uint32_t)(uintptr_t)p & 15u;
    if (r == 0) return load128(p);
    const char* a = p - r;
    if (a >= span.first && a + 32 <= span.last) return shift_pair(load128(a), load128(a + 16), r);
  }
  uint4 v = Lane<T, VEC>::pad();
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    if (j + e < V) put(v, e, row[j + e]);
  return v;
}

// Unsigned keys in the order of the values (-0.0 counts as +0.0).
__device__ __forceinline__ uint32_t ordered(float v) {
  uint32_t b = __float_as_uint(v);
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_ordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ unsigned long long ordered(double v) {
  unsigned long long b = (unsigned long long)__double_as_longlong(v);
  if (b == 0x8000000000000000ull) b = 0ull;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ double of_ordered(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// Weights are 2^((l - m) c) in the frame of a max m: the difference first, so
// that rows of any magnitude (masks of the type's lowest value included) keep
// their precision; fma(l, c, -m c) would carry the rounding of m c into every
// exponent.  The frame of a part without a finite element is 0 (its weights
// are 2^-inf = 0).
__device__ __forceinline__ float frame_of(float m) { return m == -INFINITY ? 0.f : m; }

// c = log2(e) / T (a denormal T must not make it infinite: 0 * inf).
inline float exponent_scale(float T) {
  const double c = 1.4426950408889634 / (double)T;
  return c < (double)FLT_MAX ? (float)c : FLT_MAX;
}

// Moves a sum from the frame of a to that of b >= a (an empty part has sum 0).
__device__ __forceinline__ float to_frame(float a, float b, float c) {
  return ex2(fminf(frame_of(a) - frame_of(b), 0.f) * c);
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// NaN-propagating max of N groups.
template <int N>
__device__ __forceinline__ float groups_max(const uint4 (&g)[N], const uint16_t*) {
  uint32_t m[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    m[k] = bf16x2_max_nan(bf16x2_max_nan(g[k].x, g[k].y), bf16x2_max_nan(g[k].z, g[k].w));
#pragma unroll
  for (int o = N / 2; o > 0; o /= 2)
#pragma unroll
    for (int k = 0; k < o; ++k) m[k] = bf16x2_max_nan(m[k], m[k + o]);
  return max_nan(bf16_lo(m[0]), bf16_hi(m[0]));
}
template <int N>
__device__ __forceinline__ float groups_max(const uint4 (&g)[N], const float*) {
  float m[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    m[k] = max_nan(max_nan(__uint_as_float(g[k].x), __uint_as_float(g[k].y)),
                   max_nan(__uint_as_float(g[k].z), __uint_as_float(g[k].w)));
#pragma unroll
  for (int o = N / 2; o > 0; o /= 2)
#pragma unroll
    for (int k = 0; k < o; ++k) m[k] = max_nan(m[k], m[k + o]);
  return m[0];
}

// Sum of 2^((l - m) c) over N groups, in packed pairs.
template <int N>
__device__ __forceinline__ float groups_sum(const uint4 (&g)[N], float c, float m,
                                            const uint16_t*) {
  const f32x2 c2 = pack2(c, c), nm2 = pack2(-m, -m);
  f32x2 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = pack2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t w[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float a0, a1;
      unpack2(mul2(add2(pack2(bf16_lo(w[q]), bf16_hi(w[q])), nm2), c2), a0, a1);
      acc[q] = add2(acc[q], pack2(ex2(a0), ex2(a1)));
    }
  }
  float s0, s1, s2, s3;
  unpack2(add2(acc[0], acc[1]), s0, s1);
  unpack2(add2(acc[2], acc[3]), s2, s3);
  return (s0 + s1) + (s2 + s3);
}
template <int N>
__device__ __forceinline__ float groups_sum(const uint4 (&g)[N], float c, float m,
                                            const float*) {
  const f32x2 c2 = pack2(c, c), nm2 = pack2(-m, -m);
  f32x2 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = pack2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float a0, a1, a2, a3;
    unpack2(mul2(add2(pack2(__uint_as_float(g[k].x), __uint_as_float(g[k].y)), nm2), c2), a0,
            a1);
    unpack2(mul2(add2(pack2(__uint_as_float(g[k].z), __uint_as_float(g[k].w)), nm2), c2), a2,
            a3);
    acc[(2 * k) & 3] = add2(acc[(2 * k) & 3], pack2(ex2(a0), ex2(a1)));
    acc[(2 * k + 1) & 3] = add2(acc[(2 * k + 1) & 3], pack2(ex2(a2), ex2(a3)));
  }
  float s0, s1, s2, s3;
  unpack2(add2(acc[0], acc[1]), s0, s1);
  unpack2(add2(acc[2], acc[3]), s2, s3);
  return (s0 + s1) + (s2 + s3);
}

// A running softmax sum: s = sum of 2^((l - m) c) over the elements so far,
// m their max (NaN once a NaN was seen).
struct RunningSum {
  float m = -INFINITY, s = 0.f;
  template <int N, typename T>
  __device__ __forceinline__ float add(const uint4 (&g)[N], float c, const T* tag) {
    const float gm = groups_max(g, tag);
    const float mn = max_nan(m, gm);
    s = s * to_frame(m, mn, c) + groups_sum(g, c, frame_of(mn), tag);
    m = mn;
    return gm;
  }
};

// The warp's running sums as one (the lanes' frames moved to the warp max's).
__device__ __forceinline__ float2 warp_running(const RunningSum& r, float c) {
  const float wm = warp_max_nan(r.m);
  return make_float2(wm, warp_sum(r.s * to_frame(r.m, wm, c)));
}

// 16 bytes from global into shared memory, asynchronously, in groups.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>  // waits for all but this thread's last N groups
__device__ __forceinline__ void copies_wait_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's copies of elements j .. end - 1 (at most 2 KB) of a row into the
// stage at `dst`: the aligned words around them, `off` the misalignment of
// element j. A word that is not all inside the tensor goes by element.
template <typename T, bool kAligned>
__device__ __forceinline__ void load_chunk_async(uint32_t dst, const T* row, int j, int end,
                                                 uint32_t off, const RowSpan& span) {
  const char* a = reinterpret_cast<const char*>(row + j) - off;
  const int words = ((end - j) * (int)sizeof(T) + (int)off + 15) / 16;
  constexpr int kFull = 2048 / 16;
  if (words >= kFull && a >= span.first && a + 16 * (kFull + 1) <= span.last) {
#pragma unroll
    for (int q = 0; q < kFull / kWarp; ++q) {
      const int w = q * kWarp + lane_id();
      copy16_async(dst + 16 * w, a + 16 * w);
    }
    if (!kAligned && words > kFull && lane_id() == 0) copy16_async(dst + 16 * kFull, a + 16 * kFull);
    return;
  }
  for (int w = lane_id(); w < words; w += kWarp) {
    const char* p = a + 16 * w;
    if (p >= span.first && p + 16 <= span.last) {
      copy16_async(dst + 16 * w, p);
    } else {
      uint4 v = Lane<T, Group<T>::VEC>::pad();
#pragma unroll
      for (int e = 0; e < Group<T>::VEC; ++e) {
        const char* x = p + e * (int)sizeof(T);
        if (x >= span.first && x < span.last) put(v, e, *reinterpret_cast<const T*>(x));
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 16 * w), "r"(v.x),
                   "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    }
  }
}

// Elements from `end` on of the group at element j become -inf.
template <typename T>
__device__ __forceinline__ void clip_group(uint4& g, int j, int end) {
  constexpr int VEC = Group<T>::VEC;
  if (j >= end) {
    g = Lane<T, VEC>::pad();
  } else if (j + VEC > end) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (j + e >= end) Lane<T, VEC>::kill(g, e);
  }
}

// Launch with programmatic dependent launch, in clusters of C CTAs when C > 1:
// the launch itself overlaps the kernel before on the stream, and the kernel
// waits for that one's results first thing (pdl_wait).
template <class... P, class... A>
cudaError_t launch_early(void (*fn)(P...), unsigned grid, unsigned block, size_t smem, int C,
                         cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// The two halves of a cluster barrier without memory ordering (the ordering
// forms drain every access of the warp first): each CTA of the cluster has
// started, and has initialised its mbarriers before it arrived
// (fence_mbar_init).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The address in CTA `rank` of the cluster of a shared address of this CTA.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 16 bytes into another CTA's shared memory, their arrival counted by that
// CTA's mbarrier: nothing to flush or wait for on this side.
__device__ __forceinline__ void send16(uint32_t addr, uint32_t bar, const float4& v) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::
          "r"(addr),
      "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)),
      "r"(__float_as_uint(v.w)), "r"(bar)
      : "memory");
}
// mbar_wait for what other CTAs sent (a limit of 0 gives up without polling here too),
// with the limit twice: of a context that was switched out as a whole, the clock alone
// goes on.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity,
                                                  unsigned long long limit_ns) {
  auto arrived = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (limit_ns == 0) return false;
  if (arrived()) return true;
  for (int turn = 0; turn < 2; ++turn) {
    const unsigned long long t0 = global_ns();
    do {
      for (int i = 0; i < 64; ++i)
        if (arrived()) return true;
    } while (global_ns() - t0 <= limit_ns);
  }
  return false;
}

// hi + lo, |lo| about half a step of hi: sums of a few fp32 values without
// their roundings (Dekker 1971; Knuth's two-sum).  64-bit arithmetic is two
// orders slower than fp32 on this GPU: a logarithm in it takes a microsecond.
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fadd_rn(s, -hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -b)), __fadd_rn(x, -b)));
    hi = s;
  }
  __device__ __forceinline__ float value() const { return hi + lo; }
};

// A warp's sum as hi + lo, the additions' roundings kept in lo; of its first
// kLanes lanes (a power of two) when the others hold 0, in every lane.
template <int kLanes = kWarp>
__device__ __forceinline__ float2 warp_sum_pair(float x) {
  float hi = kLanes < kWarp ? __shfl_sync(0xffffffffu, x, lane_id() & (kLanes - 1)) : x, lo = 0.f;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, hi, o), yl = __shfl_xor_sync(0xffffffffu, lo, o);
    const float sum = __fadd_rn(hi, y);
    // both lanes of a pair take the larger first: the same rounding in each
    const float a = fmaxf(hi, y), b = fminf(hi, y);
    lo = __fadd_rn(__fadd_rn(lo, yl), __fadd_rn(b, -__fadd_rn(sum, -a)));
    hi = sum;
  }
  return make_float2(hi, lo);
}

// log(hi + lo) as an exact multiple of the leading bits of ln 2 (Cody and Waite
// 1980) plus a float below 0.36 in size: good to about 5e-8 without 64-bit logarithms, which
// cost microseconds here.  1 <= hi < 2^31.
__device__ __forceinline__ float2 log_pair(float2 s) {
  const uint32_t b = __float_as_uint(s.x);
  int e = (int)(b >> 23) - 127;
  float f = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);  // [1, 2)
  if (f > 1.41421356f) {
    f *= 0.5f;
    e += 1;
  }
  const float scale = __uint_as_float((uint32_t)(127 - e) << 23);
  // ln 2 = 0.693145751953125 (15 bits) + 1.42860682030941723e-6
  const float hi = (float)e * 0.693145751953125f;
  return make_float2(hi, logf(f) + fmaf((float)e, 1.42860682e-6f, s.y * scale / f));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

}  // namespace
}  // namespace sv
