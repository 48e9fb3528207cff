// sv_cache.cuh - the 4-bit key/value cache: format, and what a request's
// arguments say about its slots; internal.
//
// A page holds `page` tokens of each head: keys, then values, each as page
// rows of D / 2 code bytes followed by scale bytes [page / 16][D / 32][16]
// (tokens last, so that four tokens' scales of one group are one word).  A word
// of codes holds 8 values, value i in nibble i / 2 + 4 (i % 2): masking a word
// shifted by 4 p leaves values 2 p and 2 p + 1 in its two halves, as the low
// bits of two 16-bit floats.
//
// A code c stands for (c - 8) s.  s has 4 significant bits and lies in
// [2^-20, 896], so (c - 8) s has 7 and is exact in bf16 and in fp16 (the least,
// 2^-23, is a multiple of fp16's 2^-24).  64 s is an fp16 number whose bits are
// (byte + 8) << 7, and so is 72 s (at most 64512): codes in the low mantissa
// bits of an fp16 number near 16 or 1 stand for (c - 8) / 64 after a subtraction, or
// one fused multiply-add turns them into the exact value.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_common.cuh"

namespace sv {

constexpr int kGroup = 32;       // values of a token under one scale
constexpr int kTopScale = 238;   // the largest scale byte: 896
constexpr int kScaleBias = 856;  // byte + kScaleBias = the scale's fp32 bits >> 20
constexpr int kNanScale = 247;   // keys of a token that held NaN or infinity: 64 s would be NaN
constexpr int kBadPage = 32;     // SV_REQ_BAD_PAGE

__host__ __device__ constexpr int page_bytes(int page, int D) {
  return page * (D / 2 + D / kGroup);
}

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float((byte + kScaleBias) << 20);
}

// The least scale byte whose scale s has 7 s >= top (finite, >= 0).  7 s is exact in
// fp32.  top times 1 / 7, off by 2^-23 of it at most and cut to 4 bits, is that scale or at most
// two below it.
__device__ __forceinline__ int scale_byte(float top) {
  int b = (int)(__float_as_uint(top * 0.142857142857f) >> 20) - kScaleBias;
  b = min(max(b, 0), kTopScale);
  b += 7.f * scale_of(b) < top;
  b += 7.f * scale_of(b) < top;
  return min(b, kTopScale);
}

// Where tokens of a cache lie.
struct CacheView {
  char* data;
  uint32_t page_stride;   // bytes from one page to the next
  const int* table;       // [B, M] page ids
  int M;                  // pages a request can hold
  int pages;              // pages of the cache
  int shift;              // log2(tokens per page)
  int Hkv;
};

// The block of page `id` for head h, keys (0) or values (1).
template <int D>
__device__ __forceinline__ char* page_block(const CacheView& c, int id, int h, int kv) {
  return c.data + (unsigned long long)(unsigned)id * c.page_stride +
         (long long)((h * 2 + kv) * page_bytes(1, D)) * (1 << c.shift);
}

// Offset of the 16 scale bytes (16 tokens) of a group in a block, `token` = slot in the page.
template <int D>
__device__ __forceinline__ int scale_at(const CacheView& c, int token, int group) {
  return (D / 2 << c.shift) + ((token >> 4) * (D / kGroup) + group) * 16;
}

// Request b's bits for the pages that hold slots [first, first + count), found by a warp: the
// caller has checked that they lie inside the table.
__device__ __forceinline__ int page_status(const CacheView& c, long long b, int first, int count) {
  bool bad = false;
  if (count > 0)
    for (int i = (first >> c.shift) + lane_id(); i <= (first + count - 1) >> c.shift; i += 32)
      bad |= (unsigned)c.table[b * c.M + i] >= (unsigned)c.pages;  // (loads that wait for none)
  return __any_sync(0xffffffffu, bad) ? kBadPage : 0;
}

}  // namespace sv
