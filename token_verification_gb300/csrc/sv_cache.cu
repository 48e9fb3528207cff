// sv_cache.cu - writing the 4-bit cache, reading it back, and keeping a
// tree's path in it (spec_cache_write, spec_cache_read, spec_cache_keep).
//
// All three move bytes and are bound by HBM (or by the launch for a step's few
// tokens).  A thread takes 8 values of a token's head, keys and values both:
// a 16-byte load of bf16 and a 4-byte store of codes (or the reverse) each, the
// D / 8 threads of a token side by side.  Consecutive tokens of a head go to
// consecutive threads, so that a page's code rows are read and written whole.
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
  FastDiv div_n, div_h;
  unsigned long long units;  // B * Hkv * N
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

// 8 values at a 16-byte (bf16) or 32-byte (fp32) step.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(u[i]);
    x[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)),
               b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // (exact: 7 significant bits)
    u[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

// Codes and scale byte of 8 values, with the three other threads of their group.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], int* byte) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
  top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
  top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
  const int b = scale_byte(top);
  const float s = scale_of(b);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // the quotient rounded to fp32 lies at or beside a half exactly when x / s does:
    // a half h has 4 bits and s 4, so x nearest to h s differs from it by 2^-24 of it
    const float q = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.f), 7.f);
    w |= (uint32_t)((int)q + 8) << (4 * (i / 2 + 4 * (i % 2)));
  }
  *byte = b;
  return w;
}

template <int D, typename T>
__global__ void __launch_bounds__(kCacheThreads) write_kernel(const CacheParams p) {
  pdl_wait();
  pdl_launch_dependents();
  write_status(p);
  constexpr int kLanes = D / 8;  // threads of a token
  const unsigned long long unit =
      (unsigned long long)blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  const CacheView& c = p.cache;
  float k[8] = {}, v[8] = {};
  char *kb = nullptr, *vb = nullptr;
  int token = 0;
  if (unit < p.units) {
    const uint32_t bh = fast_div((uint32_t)unit, p.div_n);
    const int i = (int)((uint32_t)unit - bh * p.div_n.d);
    const long long b = fast_div(bh, p.div_h);
    const int h = (int)(bh - (uint32_t)b * p.div_h.d);
    const int2 s = request_slots(p, b);
    if (i < s.y) {
      const int slot = s.x + i;
      const int id = c.table[b * c.M + (slot >> c.shift)];
      if ((unsigned)id < (unsigned)c.pages) {
        token = slot & ((1 << c.shift) - 1);
        kb = page_block<D>(c, id, h, 0);
        vb = page_block<D>(c, id, h, 1);
        load8(static_cast<const T*>(p.k.data) + b * p.k.sb + i * p.k.sn + h * p.k.sh + lane * 8, k);
        load8(static_cast<const T*>(p.v.data) + b * p.v.sb + i * p.v.sn + h * p.v.sh + lane * 8, v);
      }
    }
  }
  bool ok = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) ok = ok && is_finite(k[j]) && is_finite(v[j]);
  const unsigned mine = kLanes == 32 ? kAll
                                     : ((1u << (kLanes % 32)) - 1) << (lane_id() / kLanes * kLanes);
  const bool bad = (__ballot_sync(kAll, !ok) & mine) != 0;
  if (bad) {
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = v[j] = 0.f;
  }
  int kbyte, vbyte;
  const uint32_t kw = encode8(k, &kbyte), vw = encode8(v, &vbyte);
  if (kb) {
    reinterpret_cast<uint32_t*>(kb + token * (D / 2))[lane] = kw;
    reinterpret_cast<uint32_t*>(vb + token * (D / 2))[lane] = vw;
    if (lane % 4 == 0) {
      const int at = scale_at<D>(c, token, lane / 4) + (token & 15);
      kb[at] = (char)(bad ? kNanScale : kbyte);
      vb[at] = (char)vbyte;
    }
  }
}

// 8 values of a word of codes.
__device__ __forceinline__ void decode8(uint32_t w, float s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)((int)((w >> (4 * (i / 2 + 4 * (i % 2)))) & 15) - 8) * s;
}

template <int D, typename T>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const CacheParams p) {
  pdl_wait();
  pdl_launch_dependents();
  write_status(p);
  constexpr int kLanes = D / 8;
  const unsigned long long unit =
      (unsigned long long)blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  const CacheView& c = p.cache;
  if (unit >= p.units) return;
  const uint32_t bh = fast_div((uint32_t)unit, p.div_n);
  const int i = (int)((uint32_t)unit - bh * p.div_n.d);
  const long long b = fast_div(bh, p.div_h);
  const int h = (int)(bh - (uint32_t)b * p.div_h.d);
  const int2 s = request_slots(p, b);
  if (i >= s.y) return;
  const int slot = s.x + i;
  const int id = c.table[b * c.M + (slot >> c.shift)];
  if ((unsigned)id >= (unsigned)c.pages) return;
  const int token = slot & ((1 << c.shift) - 1);
  const char *kb = page_block<D>(c, id, h, 0), *vb = page_block<D>(c, id, h, 1);
  const int at = scale_at<D>(c, token, lane / 4) + (token & 15);
  const uint32_t kw = reinterpret_cast<const uint32_t*>(kb + token * (D / 2))[lane];
  const uint32_t vw = reinterpret_cast<const uint32_t*>(vb + token * (D / 2))[lane];
  const int kbyte = (unsigned char)kb[at], vbyte = (unsigned char)vb[at];
  float k[8], v[8];
  decode8(kw, kbyte == kNanScale ? qnan() : scale_of(kbyte), k);
  decode8(vw, kbyte == kNanScale ? qnan() : scale_of(vbyte), v);
  store8(static_cast<T*>(p.k.data) + b * p.k.sb + i * p.k.sn + h * p.k.sh + lane * 8, k);
  store8(static_cast<T*>(p.v.data) + b * p.v.sb + i * p.v.sn + h * p.v.sh + lane * 8, v);
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
// the same bytes of every token may load a batch of them before it stores.
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
      bad = bad || (unsigned)table[(start + i) >> c.shift] >= (unsigned)c.pages ||
            (unsigned)table[(start + path[i]) >> c.shift] >= (unsigned)c.pages;
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
               int32_t* out_status, sv_dtype dtype, int pages, int page_size, int B, int N, int M,
               int kv_heads, int head_dim, sv_stream_t stream) {
  CacheParams p;
  memset(&p, 0, sizeof p);
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (N < 0) return SV_ERR_SHAPE;
  sv_status rc = check_cache(&p.cache, cache, page_stride, table, pages, page_size, B, M, kv_heads,
                             head_dim);
  if (rc != SV_OK) return rc;
  if (B == 0) return SV_OK;
  const unsigned long long units = (unsigned long long)B * kv_heads * N;
  if (units >= 1ull << 31) return SV_ERR_SHAPE;
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
  p.div_n = make_fastdiv((uint32_t)std::max(N, 1));
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
              out_status, dtype, pages, page_size, B, N, M, kv_heads, head_dim, stream);
}

extern "C" sv_status spec_cache_read(const void* cache, int64_t page_stride, void* k,
                                     const int64_t* k_strides, void* v, const int64_t* v_strides,
                                     const int32_t* table, const int32_t* start,
                                     const int32_t* lens, int32_t* out_status, sv_dtype dtype,
                                     int pages, int page_size, int B, int N, int M, int kv_heads,
                                     int head_dim, sv_stream_t stream) {
  return move(false, cache, page_stride, {k, v, k_strides, v_strides}, table, start, lens,
              out_status, dtype, pages, page_size, B, N, M, kv_heads, head_dim, stream);
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
