// sv_cache.cu - writing the 4-bit cache, reading it back, and keeping a
// tree's path in it (spec_cache_write, spec_cache_read, spec_cache_keep).
//
// All three move bytes.  In the first two a thread takes the same 8 values of four neighbouring
// slots of a head, keys and values both: of each token a 16-byte load of bf16 and a 4-byte store of
// codes (or the reverse), of all four the scale bytes of a group as one word where all four are
// touched.  The D / 8 threads of a token lie side by side, consecutive slots in consecutive
// threads, so that a page's code rows are read and written whole.
// Measured for 8 prompts of up to 8192 tokens (8 heads of 128, bf16): write 44 us, 193 MB at 4.4 TB/s,
// bound by its instructions (issue slots 74 % used, 16 instructions a value); read
// 45 us, 308 MB with the zeros behind the prompts at 6.8 TB/s, bound by HBM.  A step's few tokens are bound
// by the launches.
#include <string.h>

#include <algorithm>

#include "../../include/spec_verify.h"
#include "sv_cache.cuh"
#include "sv_launch.h"
#include "sv_rows.cuh"
#include "sv_vec.cuh"

namespace sv {
namespace {

constexpr int kCacheThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

struct DenseView {  // dense keys or values: [B, N, Hkv, D] at element strides
  void* data;
  long long sb, sn, sh;
};

struct CacheParams {
  CacheView cache;
  DenseView k, v;
  const int* start;  // [B] or null (0)
  const int* lens;   // [B] or null (N)
  int* out_status;   // [B] or null
  int B, N;
  FastDiv div_n, div_h;      // four slots of a request, heads
  unsigned long long units;  // B * Hkv * four slots
  int fill;                  // rows that are not read become 0
};

// Request b's first slot and count of tokens; count -1 when they do not fit.
__device__ __forceinline__ int2 request_slots(const CacheParams& p, long long b) {
  const int first = p.start ? p.start[b] : 0, n = p.lens ? p.lens[b] : p.N;
  const long long room = (long long)p.cache.M << p.cache.shift;
  if (first < 0 || n < 0 || n > p.N || first + (long long)n > room) return make_int2(0, -1);
  return make_int2(first, n);
}

// (a warp a request)
__device__ __forceinline__ void write_status(const CacheParams& p) {
  if (!p.out_status) return;
  for (long long b = (long long)blockIdx.x * (kCacheThreads / 32) + threadIdx.x / 32; b < p.B;
       b += (long long)gridDim.x * (kCacheThreads / 32)) {
    const int2 s = request_slots(p, b);
    const int st = s.y < 0 ? kBadDraftLen : page_status(p.cache, b, s.x, s.y);
    if (lane_id() == 0) p.out_status[b] = st;
  }
}

constexpr int kSlots = 4;  // neighbouring slots of a thread

// A thread's place: request, head, its first slot's token (may lie before the request's first or
// behind its last), and where that slot is.
template <int D>
struct Place {
  long long b;
  int h, lane, first, n, token;  // token: of the thread's first slot
  int slot;                      // that slot in its page
  char *k, *v;                   // blocks of the page, null where there is none
  bool in;                       // a place at all
};

template <int D>
__device__ __forceinline__ Place<D> place_of(const CacheParams& p) {
  constexpr int kLanes = D / 8;
  Place<D> x;
  const unsigned long long unit =
      (unsigned long long)blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
  x.lane = threadIdx.x % kLanes;
  x.in = unit < p.units;
  x.k = x.v = nullptr;
  x.first = x.n = x.token = x.slot = 0;
  x.b = x.h = 0;
  if (!x.in) return x;
  const uint32_t bh = fast_div((uint32_t)unit, p.div_n);
  const int i = (int)((uint32_t)unit - bh * p.div_n.d);
  x.b = fast_div(bh, p.div_h);
  x.h = (int)(bh - (uint32_t)x.b * p.div_h.d);
  const int2 s = request_slots(p, x.b);
  x.first = s.x;
  x.n = s.y;
  const int slot = (s.x & ~(kSlots - 1)) + kSlots * i;
  x.token = slot - s.x;
  if (x.token < s.y) {  // (then some of its slots are the request's)
    const int id = p.cache.table[x.b * p.cache.M + (slot >> p.cache.shift)];
    if ((unsigned)id < (unsigned)p.cache.pages) {
      x.slot = slot & ((1 << p.cache.shift) - 1);
      x.k = page_block<D>(p.cache, id, x.h, 0);
      x.v = page_block<D>(p.cache, id, x.h, 1);
    }
  }
  return x;
}

// 8 values as fp32 bit patterns' source: bf16 pairs, or fp32.  cut(): magnitudes above 6272 = 7 * 896
// become that.
constexpr uint32_t kMost = 0x45c40000u;  // 6272
struct Eight16 {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void cut() {
    auto two = [](uint32_t u) {
      return __vminu2(u & 0x7fff7fffu, kMost | kMost >> 16) | (u & 0x80008000u);
    };
    w = make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
  }
  // the largest magnitude's bits (an fp32 number; NaN above infinity)
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t u = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
    return i & 1 ? bf16_hi(u) : bf16_lo(u);
  }
};
struct Eight32 {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void cut() {
    float* x[8] = {&a.x, &a.y, &a.z, &a.w, &b.x, &b.y, &b.z, &b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) *x[i] = fminf(fmaxf(*x[i], -6272.f), 6272.f);
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(get(i)) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ float get(int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w
         : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
};
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> : Eight16 {};
template <>
struct Eight<float> : Eight32 {};

// Codes of 8 values of at most 7 s at scale s (r = 1 / s to nearest).  The
// quotient's first value x r, corrected by its exact remainder, is x / s to nearest (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), so it
// is a half only where x / s is: a half h has 4 bits and s has 4, so an fp32 x beside h s
// gives a quotient beside h.  Adding 1.5 * 2^23 + 8 leaves the whole number (ties to even) plus 8 in
// the low bits, and the codes meet in one word by multiplications.
template <typename T>
__device__ __forceinline__ uint32_t encode8(const Eight<T>& x, float s, float r) {
  uint32_t w = -0x4b400000u * 0x11111111u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = x.get(i);
    const float t = v * r;
    const float q = fmaf(fmaf(-t, s, v), r, t);
    const int at = 4 * (i / 2 + 4 * (i % 2));
    w += __float_as_uint(q + 12582920.f) * (1u << at);
  }
  return w;
}

// 1 / s to nearest: an approximate one, off by a last place or two, and a Newton step, off by the
// square of that before it is rounded, 2^-44.  No 1 / s of a 4-bit s lies that near to the middle between
// two numbers.
__device__ __forceinline__ float inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.f), r, r);
}

template <int D, typename T>
__global__ void __launch_bounds__(kCacheThreads) write_kernel(const CacheParams p) {
  pdl_wait();
  pdl_launch_dependents();
  write_status(p);
  constexpr int kLanes = D / 8;  // threads of a token
  const Place<D> x = place_of<D>(p);
  if (!__any_sync(kAll, x.k != nullptr)) return;  // (of ragged prompts every other warp)
  Eight<T> k[kSlots], v[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const int i = x.token + j;
    if (x.k && i >= 0 && i < x.n) {
      k[j].load(static_cast<const T*>(p.k.data) + x.b * p.k.sb + i * p.k.sn + x.h * p.k.sh + x.lane * 8);
      v[j].load(static_cast<const T*>(p.v.data) + x.b * p.v.sb + i * p.v.sn + x.h * p.v.sh + x.lane * 8);
    } else {
      k[j].clear();
      v[j].clear();
    }
  }
  uint32_t tk[kSlots], tv[kSlots], top = 0;  // the slots' largest magnitudes, and that of all
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    tk[j] = k[j].top();
    tv[j] = v[j].top();
    top = max(top, max(tk[j], tv[j]));
  }
  // a token of which anything is not finite: values of 0 under the scale that says so
  unsigned bad = 0;
  if (__any_sync(kAll, top > kMost)) {  // (seldom)
    const unsigned mine = kLanes == 32 ? kAll
                                       : ((1u << (kLanes % 32)) - 1) << (lane_id() / kLanes * kLanes);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      if (__ballot_sync(kAll, max(tk[j], tv[j]) >= 0x7f800000u) & mine) {
        bad |= 1u << j;
        tk[j] = tv[j] = 0;
        k[j].clear();
        v[j].clear();
      }
      k[j].cut();
      v[j].cut();
    }
  }
  // the four lanes of a group work out one slot's scales each
  const int t4 = lane_id() & 3;
  auto spread = [&](const uint32_t (&x)[kSlots]) {  // the group's max of slot t4
    uint32_t a[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      a[i] = max(t4 & 2 ? x[2 + i] : x[i], __shfl_xor_sync(kAll, t4 & 2 ? x[i] : x[2 + i], 2));
    return max(t4 & 1 ? a[1] : a[0], __shfl_xor_sync(kAll, t4 & 1 ? a[0] : a[1], 1));
  };
  const uint32_t both = (uint32_t)scale_byte(__uint_as_float(spread(tk))) |
                        (uint32_t)scale_byte(__uint_as_float(spread(tv))) << 8;
  uint32_t kbytes = 0, vbytes = 0;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const uint32_t mine = __shfl_sync(kAll, both, j, 4), bk = mine & 255, bv = mine >> 8;
    const float sk = scale_of(bk), sv = scale_of(bv);
    const int i = x.token + j;
    const uint32_t wk = encode8<T>(k[j], sk, inverse(sk)), wv = encode8<T>(v[j], sv, inverse(sv));
    if (x.k && i >= 0 && i < x.n) {
      reinterpret_cast<uint32_t*>(x.k + (x.slot + j) * (D / 2))[x.lane] = wk;
      reinterpret_cast<uint32_t*>(x.v + (x.slot + j) * (D / 2))[x.lane] = wv;
    }
    kbytes |= (bad >> j & 1 ? (uint32_t)kNanScale : bk) << (8 * j);
    vbytes |= bv << (8 * j);
  }
  if (x.k && x.lane % 4 == 0) {
    const int at = scale_at<D>(p.cache, x.slot, x.lane / 4) + (x.slot & 15);
    if (x.token >= 0 && x.token + kSlots <= x.n) {
      *reinterpret_cast<uint32_t*>(x.k + at) = kbytes;
      *reinterpret_cast<uint32_t*>(x.v + at) = vbytes;
    } else {
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (x.token + j >= 0 && x.token + j < x.n) {
          x.k[at + j] = (char)(kbytes >> (8 * j));
          x.v[at + j] = (char)(vbytes >> (8 * j));
        }
    }
  }
}

// The 8 values of a word of codes in bf16, times the scale byte's scale: 128 + c is a bf16 number
// whose low bits are the code, and (128 + c) s - 136 s is exact (136 s has 8 bits).
__device__ __forceinline__ uint4 decode8(uint32_t w, uint32_t byte) {
  uint32_t s = byte * 16 + (kScaleBias << 4);
  if (byte == kNanScale) s = 0x7fff;
  s *= 0x10001u;
  uint32_t off, d[4];
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(off) : "r"(s), "r"(0xc308c308u));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d[i]) : "r"(c), "r"(s), "r"(off));
  }
  return make_uint4(d[0], d[1], d[2], d[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint4& x) {
  __stcs(reinterpret_cast<uint4*>(p), x);
}
__device__ __forceinline__ void store8(float* p, const uint4& x) {
  __stcs(reinterpret_cast<float4*>(p),
         make_float4(bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y)));
  __stcs(reinterpret_cast<float4*>(p) + 1,
         make_float4(bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)));
}

template <int D, typename T>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const CacheParams p) {
  pdl_wait();
  pdl_launch_dependents();
  write_status(p);
  const Place<D> x = place_of<D>(p);
  if (!x.in) return;
  uint32_t kw[kSlots], vw[kSlots], kbytes = 0, vbytes = 0;
  if (x.k) {
    // (all four slots lie in the page, whichever of them are wanted)
    const int at = scale_at<D>(p.cache, x.slot, x.lane / 4) + (x.slot & 15);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      kw[j] = reinterpret_cast<const uint32_t*>(x.k + (x.slot + j) * (D / 2))[x.lane];
      vw[j] = reinterpret_cast<const uint32_t*>(x.v + (x.slot + j) * (D / 2))[x.lane];
    }
    kbytes = *reinterpret_cast<const uint32_t*>(x.k + at);
    vbytes = *reinterpret_cast<const uint32_t*>(x.v + at);
  }
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const int i = x.token + j;
    if (i < 0 || i >= p.N) continue;
    const bool there = x.k && i < x.n;
    if (!there && !p.fill) continue;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (there) {
      const uint32_t bk = kbytes >> (8 * j) & 255, bv = vbytes >> (8 * j) & 255;
      k = decode8(kw[j], bk);
      v = decode8(vw[j], bk == kNanScale ? bk : bv);
    }
    store8(static_cast<T*>(p.k.data) + x.b * p.k.sb + i * p.k.sn + x.h * p.k.sh + x.lane * 8, k);
    store8(static_cast<T*>(p.v.data) + x.b * p.v.sb + i * p.v.sn + x.h * p.v.sh + x.lane * 8, v);
  }
}

struct KeepParams {
  CacheView cache;
  const int* start;  // [B]
  const int* path;   // [B, P]
  int* out_status;
  int B, P;
  FastDiv div_h;
  unsigned units;  // B * Hkv
};

// Request b's kept nodes (before the first -1), -1 when the path does not ascend, -2 when
// its slots do not lie inside the table.
__device__ __forceinline__ int path_length(const KeepParams& p, long long b) {
  const int* path = p.path + b * p.P;
  const int first = p.start[b];
  const long long room = (long long)p.cache.M << p.cache.shift;
  int last = -1, n = 0;
  for (; n < p.P; ++n) {
    const int x = path[n];
    if (x == -1) break;
    if (x <= last) return -1;
    last = x;
  }
  if (n > 0 && (first < 0 || first + (long long)last >= room)) return -2;
  return n;
}

// One warp moves a request's head.  Slot start + path[i] goes to start + i.
// The path ascends from 0 or above, so i <= path[i] < path[j] for i < j: no
// store lands on a slot that a later load reads, and a thread that moves
// the same bytes of every token may load a batch of them before it stores.  The launch
// and that chain of path, table, codes and store are what a call takes: writing a tree of 61 nodes, keeping 6 and
// reading them back is 11.8 us in three launches.
constexpr int kKeepBatch = 8;

template <int D>
__global__ void __launch_bounds__(kCacheThreads) keep_kernel(const KeepParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const CacheView& c = p.cache;
  const unsigned unit = blockIdx.x * (kCacheThreads / 32) + threadIdx.x / 32;
  if (unit >= p.units) return;
  const long long b = fast_div(unit, p.div_h);
  const int h = (int)(unit - (unsigned)b * p.div_h.d);
  const int n = path_length(p, b);
  const int* path = p.path + b * p.P;
  const int* table = c.table + b * c.M;
  const int start = p.start[b];
  if (p.out_status && h == 0) {
    bool bad = false;
    for (int i = lane_id(); i < n; i += 32)
      bad |= ((unsigned)table[(start + i) >> c.shift] >= (unsigned)c.pages) |
             ((unsigned)table[(start + path[i]) >> c.shift] >= (unsigned)c.pages);
    bad = __any_sync(kAll, bad);
    if (lane_id() == 0)
      p.out_status[b] = n == -1 ? kBadTree : n == -2 ? kBadDraftLen : bad ? kBadPage : 0;
  }
  if (n <= 0) return;
  const int mask = (1 << c.shift) - 1;
  // units of a token: words of 16 code bytes, and scale bytes, of keys and of values
  constexpr int kCodes = D / 32, kPer = kCodes + D / kGroup;
  for (int u = lane_id(); u < 2 * kPer; u += 32) {
    const int kv = u / kPer, w = u % kPer;
    for (int i0 = 0; i0 < n; i0 += kKeepBatch) {
      uint4 word[kKeepBatch];
      char* to[kKeepBatch];
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j) {
        to[j] = nullptr;
        if (i0 + j >= n) continue;
        const int s = start + path[i0 + j], d = start + i0 + j;
        if (s == d) continue;
        const int ps = table[s >> c.shift], pd = table[d >> c.shift];
        if ((unsigned)ps >= (unsigned)c.pages || (unsigned)pd >= (unsigned)c.pages) continue;
        const int ts = s & mask, td = d & mask;
        const char* from = page_block<D>(c, ps, h, kv);
        to[j] = page_block<D>(c, pd, h, kv);
        if (w < kCodes) {
          word[j] = *reinterpret_cast<const uint4*>(from + ts * (D / 2) + w * 16);
          to[j] += td * (D / 2) + w * 16;
        } else {
          word[j].x = (unsigned char)from[scale_at<D>(c, ts, w - kCodes) + (ts & 15)];
          to[j] += scale_at<D>(c, td, w - kCodes) + (td & 15);
        }
      }
#pragma unroll
      for (int j = 0; j < kKeepBatch; ++j) {
        if (!to[j]) continue;
        if (w < kCodes)
          *reinterpret_cast<uint4*>(to[j]) = word[j];
        else
          *to[j] = (char)word[j].x;
      }
    }
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

// The cache's arguments, shared by every entry point.
sv_status check_cache(CacheView* c, const void* cache, int64_t page_stride, const int32_t* table,
                      int pages, int page_size, int B, int M, int kv_heads, int head_dim) {
  const size_t bytes = spec_cache_page_bytes(page_size, head_dim);
  if (!bytes || pages < 0 || B < 0 || B > SV_MAX_B || M < 0 || kv_heads < 1 ||
      kv_heads > SV_MAX_HEADS || (long long)M * page_size > SV_MAX_SLOTS)
    return SV_ERR_SHAPE;
  if (pages <= 1) page_stride = 0;
  if (page_stride % 16 || page_stride < 0 || page_stride > UINT32_MAX ||
      (pages > 1 && page_stride < (int64_t)(2 * bytes * kv_heads)))
    return SV_ERR_SHAPE;
  if (B > 0 && ((pages > 0 && !cache) || (M > 0 && !table) || !aligned16(cache))) return SV_ERR_NULL;
  c->data = static_cast<char*>(const_cast<void*>(cache));
  c->page_stride = (uint32_t)page_stride;
  c->table = table;
  c->M = M;
  c->pages = pages;
  c->shift = 0;
  while ((1 << c->shift) < page_size) ++c->shift;
  c->Hkv = kv_heads;
  return SV_OK;
}

namespace {

// Dense keys or values: byte strides of b, n, h, every row 16-byte aligned.
sv_status check_dense(DenseView* d, const void* data, const int64_t* strides, int esize, int B,
                      int N, int H) {
  const int n[3] = {B, N, H};
  long long st[3];
  for (int i = 0; i < 3; ++i) {
    st[i] = n[i] > 1 ? strides[i] : 0;
    if (st[i] < 0 || st[i] > (1LL << 60) / n[i]) return SV_ERR_SHAPE;
    if (st[i] % 16) return SV_ERR_NULL;
  }
  if (!data || !aligned16(data)) return SV_ERR_NULL;
  *d = {const_cast<void*>(data), st[0] / esize, st[1] / esize, st[2] / esize};
  return SV_OK;
}

// Rows of an output must not share bytes: by ascending stride each steps over all before.
bool folds(const int64_t* strides, int B, int N, int H, int row) {
  const long long n[3] = {B, N, H};
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return strides[a] < strides[b]; });
  long long ext = row;
  for (int i : order)
    if (n[i] > 1) {
      if (strides[i] < ext) return true;
      ext += (n[i] - 1) * strides[i];
    }
  return false;
}

struct Dense {
  const void *k, *v;
  const int64_t *ks, *vs;
};

sv_status move(bool write, const void* cache, int64_t page_stride, const Dense& t,
               const int32_t* table, const int32_t* start, const int32_t* lens,
               int32_t* out_status, int fill, sv_dtype dtype, int pages, int page_size, int B,
               int N, int M, int kv_heads, int head_dim, sv_stream_t stream) {
  CacheParams p;
  memset(&p, 0, sizeof p);
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  // (a slot of place_of: up to 2 SV_MAX_SLOTS and a few, in 32 bits)
  if (N < 0 || N > SV_MAX_SLOTS) return SV_ERR_SHAPE;
  sv_status rc = check_cache(&p.cache, cache, page_stride, table, pages, page_size, B, M, kv_heads,
                             head_dim);
  if (rc != SV_OK) return rc;
  if (B == 0) return SV_OK;
  if ((unsigned long long)B * kv_heads * N >= 1ull << 31) return SV_ERR_SHAPE;
  // the most aligned fours that N slots can touch
  const unsigned fours = N == 0 ? 0 : ((unsigned)N + 2 * (kSlots - 1)) / kSlots;
  const unsigned long long units = (unsigned long long)B * kv_heads * fours;
  if (units >= 1ull << 32) return SV_ERR_SHAPE;
  const int esize = dtype == SV_F32 ? 4 : 2;
  if (units > 0) {
    if (!t.ks || !t.vs) return SV_ERR_NULL;
    if ((rc = check_dense(&p.k, t.k, t.ks, esize, B, N, kv_heads)) != SV_OK) return rc;
    if ((rc = check_dense(&p.v, t.v, t.vs, esize, B, N, kv_heads)) != SV_OK) return rc;
    if (!write && (folds(t.ks, B, N, kv_heads, head_dim * esize) ||
                   folds(t.vs, B, N, kv_heads, head_dim * esize)))
      return SV_ERR_ALIAS;
  }
  p.start = start;
  p.lens = lens;
  p.out_status = out_status;
  p.B = B;
  p.N = N;
  p.units = units;
  p.fill = fill;
  p.div_n = make_fastdiv(std::max(fours, 1u));
  p.div_h = make_fastdiv((uint32_t)kv_heads);
  const unsigned per = kCacheThreads / (head_dim / 8);
  unsigned blocks = (unsigned)((units + per - 1) / per);
  if (out_status) blocks = std::max(blocks, 1u);
  if (!blocks) return SV_OK;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t err = cudaErrorInvalidValue;
#define SV_MOVE(D)                                                                              \
  if (head_dim == D) {                                                                          \
    if (write)                                                                                  \
      err = dtype == SV_F32                                                                     \
                ? launch_early(write_kernel<D, float>, blocks, kCacheThreads, 0, 1, st, p)      \
                : launch_early(write_kernel<D, __nv_bfloat16>, blocks, kCacheThreads, 0, 1, st, p); \
    else                                                                                        \
      err = dtype == SV_F32                                                                     \
                ? launch_early(read_kernel<D, float>, blocks, kCacheThreads, 0, 1, st, p)       \
                : launch_early(read_kernel<D, __nv_bfloat16>, blocks, kCacheThreads, 0, 1, st, p); \
  }
  SV_MOVE(64) SV_MOVE(128) SV_MOVE(256)
#undef SV_MOVE
  return err == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_cache_page_bytes(int page_size, int head_dim) {
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return (size_t)page_bytes(page_size, head_dim);
}

extern "C" sv_status spec_cache_write(void* cache, int64_t page_stride, const void* k,
                                      const int64_t* k_strides, const void* v,
                                      const int64_t* v_strides, const int32_t* table,
                                      const int32_t* start, const int32_t* lens,
                                      int32_t* out_status, sv_dtype dtype, int pages,
                                      int page_size, int B, int N, int M, int kv_heads,
                                      int head_dim, sv_stream_t stream) {
  if (B > 0 && !start) return SV_ERR_NULL;
  return move(true, cache, page_stride, {k, v, k_strides, v_strides}, table, start, lens,
              out_status, 0, dtype, pages, page_size, B, N, M, kv_heads, head_dim, stream);
}

extern "C" sv_status spec_cache_read(const void* cache, int64_t page_stride, void* k,
                                     const int64_t* k_strides, void* v, const int64_t* v_strides,
                                     const int32_t* table, const int32_t* start,
                                     const int32_t* lens, int fill, int32_t* out_status,
                                     sv_dtype dtype, int pages, int page_size, int B, int N, int M,
                                     int kv_heads, int head_dim, sv_stream_t stream) {
  return move(false, cache, page_stride, {k, v, k_strides, v_strides}, table, start, lens,
              out_status, fill, dtype, pages, page_size, B, N, M, kv_heads, head_dim, stream);
}

extern "C" sv_status spec_cache_keep(void* cache, int64_t page_stride, const int32_t* table,
                                     const int32_t* start, const int32_t* path,
                                     int32_t* out_status, int pages, int page_size, int B, int P,
                                     int M, int kv_heads, int head_dim, sv_stream_t stream) {
  KeepParams p;
  memset(&p, 0, sizeof p);
  if (P < 0 || P > SV_MAX_STEP) return SV_ERR_SHAPE;
  const sv_status rc = check_cache(&p.cache, cache, page_stride, table, pages, page_size, B, M,
                                   kv_heads, head_dim);
  if (rc != SV_OK) return rc;
  if (B == 0) return SV_OK;
  if (!start || (P > 0 && !path)) return SV_ERR_NULL;
  p.start = start;
  p.path = path;
  p.out_status = out_status;
  p.B = B;
  p.P = P;
  p.div_h = make_fastdiv((uint32_t)kv_heads);
  p.units = (unsigned)B * (unsigned)kv_heads;
  const unsigned blocks = (p.units + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t err = cudaErrorInvalidValue;
  if (head_dim == 64) err = launch_early(keep_kernel<64>, blocks, kCacheThreads, 0, 1, st, p);
  if (head_dim == 128) err = launch_early(keep_kernel<128>, blocks, kCacheThreads, 0, 1, st, p);
  if (head_dim == 256) err = launch_early(keep_kernel<256>, blocks, kCacheThreads, 0, 1, st, p);
  return err == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
