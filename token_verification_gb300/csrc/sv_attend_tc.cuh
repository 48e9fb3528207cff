// sv_attend_tc.cuh - attention over the 4-bit cache in tensor memory: the instructions, and what
// the kernels for many rows share of finding and decoding a chunk of slots; internal.
#pragma once

#include "sv_attend.cuh"
#include "sv_vec.cuh"

namespace sv {

constexpr int kSlotsTile = 128;  // slots of a chunk
constexpr float kManyShift = 7.f, kSlack = 8.f;  // of the weights' exponents
constexpr float kNoRef = -kLeast;  // in place of shift - max for a row without a score yet

// ---- tcgen05 -------------------------------------------------------------

template <int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
               "n"(COLS)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS>
__device__ __forceinline__ void tmem_free(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS));
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {  // A in tensor memory
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&x)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_loaded() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
// mbar_wait for waits that are long as a rule: the warp sleeps (for 20 us at a time) instead of asking
// again, which would take issue slots from the others.
__device__ __forceinline__ bool sleep_wait(uint32_t bar, uint32_t parity, unsigned long long limit) {
  if (limit == 0) return false;
  auto ask = [&] {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
  };
  if (ask()) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
    if (ask()) return true;
    if (global_ns() - t0 > limit) return false;
  }
}
__device__ __forceinline__ void store16(uint32_t addr, const uint32_t (&x)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3])
               : "memory");
}

// Shared-memory descriptors: 128-byte swizzle, version 1.  Keys and queries (K-major): 8 rows of 128
// bytes every 1024.  Values (MN-major): 64 dimensions a block, blocks 16384 bytes
// apart, 8 slots every 1024.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t kBlockBytes = 128 * 128;  // 128 rows or slots of 64 dimensions
// Instruction: fp32 results, fp16 operands, M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool a_mn_major, bool b_mn_major) {
  return 1u << 4 | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
         (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}

// A chunk ahead: addresses of each 16 slots' key codes and key scales (of some page where there is
// none), which of them are pages (bits), and which slots are seen by anybody (first <= slot in the chunk
// < last); whole: every slot is.
struct ChunkRef {
  unsigned long long codes[8], scales[8];
  uint32_t valid;
  int first, last, whole;
};

// A thread's part of a chunk's keys or values: kU rows of one group of 32 values.
template <int D>
struct Part {
  static constexpr int kU = D / 64;
  uint32_t scale[kU];  // bytes
  uint32_t off;        // bit i: row i counts as NaN (keys) or 0 (values), whatever its byte
};
__device__ __forceinline__ void copy16(uint32_t dst, unsigned long long src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// (volatile: where it stands, not where its result is used)
__device__ __forceinline__ uint32_t load_byte(unsigned long long src) {
  uint32_t x;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(x) : "l"(src) : "memory");
  return x;
}

// 8 values of a row of Q in fp16; PER threads that lie side by side have the row.  It is scaled by a power of
// two that takes its largest value to [2^14, 2^15) (*down: back); NaN or infinity in it: all NaN.
template <int PER>
__device__ __forceinline__ uint4 scaled_query(const uint4& v, bool negative, float* down) {
  // (magnitudes of bf16 order as whole numbers)
  uint32_t top2 = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                           __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
#pragma unroll
  for (int o = PER / 2; o > 0; o >>= 1) top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, o));
  const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  const int e = min(max((int)(top >> 7) - 127, -98), 127);
  float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
  if (top >= 0x7f80u) up = qnan();
  if (negative) up = -up;
  *down = __uint_as_float((uint32_t)(127 + e - 14) << 23);
  return make_uint4(pack_f16(bf16_lo(v.x) * up, bf16_hi(v.x) * up),
                    pack_f16(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                    pack_f16(bf16_lo(v.z) * up, bf16_hi(v.z) * up),
                    pack_f16(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
}

// Finds the addresses of a share's chunks in turn (one warp; lane k < 8 those of the k-th 16 slots' codes,
// lane k + 8 of their scales), from page ids that it read a chunk before that.  Where it stands is
// held in registers (of the whole block: the other warps' are idle), or with SHARED in shared memory: tiles of
// 128 rows have no registers left (attend: 230 -> 220 us), those of 48 are faster with (288, 296).
struct FinderState {
  Walk ahead;
  unsigned j;  // the chunk that is next
};
template <int D, bool SHARED>
struct Finder {
  FinderState *state, own;
  int id;
  __device__ __forceinline__ void keep(const Walk& ahead, unsigned j) {
    if (!SHARED) {
      own.ahead = ahead;
      own.j = j;
    } else {
      if (lane_id() == 0) {
        state->ahead = ahead;
        state->j = j;
      }
      __syncwarp();
    }
  }
  __device__ __forceinline__ void start(const AttendParams& p, const Share& s, FinderState* at) {
    state = at;
    const Walk ahead(p, s);
    keep(ahead, 0);
    fetch(p, ahead);
  }
  __device__ __forceinline__ void fetch(const AttendParams& p, const Walk& ahead) {
    const int slot =
        (ahead.r.lo / kSlotsTile + ahead.c) * kSlotsTile + 16 * ((int)lane_id() & 7);
    id = ahead.left > 0 && slot < ahead.r.len
             ? p.cache.table[(long long)ahead.b * p.cache.M + (slot >> p.cache.shift)]
             : -1;
  }
  __device__ __forceinline__ void find(const AttendParams& p, ChunkRef (&refs)[4]) {
    Walk ahead = SHARED ? state->ahead : own.ahead;
    const unsigned j = SHARED ? state->j : own.j;
    if (SHARED) __syncwarp();
    if (ahead.left <= 0) return;
    const int lane = lane_id();
    const int slot0 = (ahead.r.lo / kSlotsTile + ahead.c) * kSlotsTile;
    const int block = page_bytes(1, D) << p.cache.shift;
    const bool ok = (unsigned)id < (unsigned)p.cache.pages;
    const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xffu;
    const int token = (slot0 + 16 * (lane & 7)) & ((1 << p.cache.shift) - 1);
    const unsigned long long at =
        reinterpret_cast<unsigned long long>(p.cache.data) +
        (unsigned long long)(ok ? (unsigned)id : 0u) * p.cache.page_stride +
        (long long)(2 * ahead.h) * block +
        (lane & 8 ? ((D / 2) << p.cache.shift) + token * (D / kGroup) : token * (D / 2));
    ChunkRef& ref = refs[j & 3];
    if (lane < 8) ref.codes[lane] = at;
    if (lane >= 8 && lane < 16) ref.scales[lane - 8] = at;
    if (lane == 0) {
      ref.valid = valid;
      ref.first = max(0, ahead.r.lo - slot0);
      ref.last = min(kSlotsTile, ahead.r.len - slot0);
      ref.whole = valid == 0xffu && slot0 >= ahead.r.lo && slot0 + kSlotsTile <= ahead.r.len;
    }
    ahead.skip(p, 1);
    keep(ahead, j + 1);
    fetch(p, ahead);
  }
};

}  // namespace sv
