// Shared by the serving kernels (q4tp product, 4-bit key/value cache): the
// two 16-bit element types and the 4-bit codes as numbers of those types.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace gq {

// kMagic16 with a code c in the top four mantissa bits is the number 16 + c;
// shift(i) puts nibble i of each 16-bit half there.
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  using T2 = __nv_bfloat162;
  static constexpr uint32_t kMagic16 = 0x41804180u, kMask16 = 0x00780078u;
  static constexpr int kPos = 3;  // lowest of the top four mantissa bits
  static constexpr uint32_t kExp = 0x7F80u;
  static __device__ __forceinline__ T2 make2(float a, float b) { return __floats2bfloat162_rn(a, b); }
  static __device__ __forceinline__ float2 to2(T2 v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float a) { return __float2bfloat16_rn(a); }
  static __device__ __forceinline__ float to(__nv_bfloat16 a) { return __bfloat162float(a); }
};
template <>
struct Elem<__half> {
  using T2 = __half2;
  static constexpr uint32_t kMagic16 = 0x4C004C00u, kMask16 = 0x03C003C0u;
  static constexpr int kPos = 6;
  static constexpr uint32_t kExp = 0x7C00u;
  static __device__ __forceinline__ T2 make2(float a, float b) { return __floats2half2_rn(a, b); }
  static __device__ __forceinline__ float2 to2(T2 v) { return __half22float2(v); }
  static __device__ __forceinline__ __half from(float a) { return __float2half_rn(a); }
  static __device__ __forceinline__ float to(__half a) { return __half2float(a); }
};

template <class T2>
__device__ __forceinline__ uint32_t bits2(T2 v) {
  return *reinterpret_cast<uint32_t*>(&v);
}
template <class T2>
__device__ __forceinline__ T2 from_bits2(uint32_t v) {
  return *reinterpret_cast<T2*>(&v);
}

// (x & MASK) | magic as the one instruction it is (from the C expression the
// compiler makes two, and the ALUs bound the kernels that decode).
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "n"(MASK), "r"(magic));
  return r;
}

// (16 + nibble i of the low half, 16 + nibble i of the high half) as T2.
template <class T>
__device__ __forceinline__ typename Elem<T>::T2 code16(uint32_t w, int i) {
  constexpr int kPos = Elem<T>::kPos;
  const int sh = 4 * i - kPos;
  return from_bits2<typename Elem<T>::T2>(and_or<Elem<T>::kMask16>(sh >= 0 ? (w >> sh) : (w << -sh), Elem<T>::kMagic16));
}
// The same with the shift of nibble 0 as a product with `up` = 2^kPos, of
// which the compiler must not know that it is one: it then runs beside the
// ALUs, on the multipliers.
template <class T>
__device__ __forceinline__ typename Elem<T>::T2 code16(uint32_t w, int i, uint32_t up) {
  if (i != 0) return code16<T>(w, i);
  return from_bits2<typename Elem<T>::T2>(and_or<Elem<T>::kMask16>(w * up, Elem<T>::kMagic16));
}

// Whether a group of the cache (s and z as a pair) holds no numbers.
template <class T>
__device__ __forceinline__ bool no_numbers(uint32_t par) {
  return (~par & Elem<T>::kExp) == 0u || (~par & (Elem<T>::kExp << 16)) == 0u;
}

// 16 x 8 x 16 product with f32 accumulation.
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight elements (x0..x7) as the pairs (x0,x4), (x1,x5), (x2,x6), (x3,x7):
// the order in which one shift and mask takes the nibbles out of a word.
__device__ __forceinline__ uint4 pair_order(uint4 v) {
  uint4 o;
  o.x = __byte_perm(v.x, v.z, 0x5410);
  o.y = __byte_perm(v.x, v.z, 0x7632);
  o.z = __byte_perm(v.y, v.w, 0x5410);
  o.w = __byte_perm(v.y, v.w, 0x7632);
  return o;
}

// 2^x.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// mbar_wait for waits that are short and many: the clock is looked at once in
// 64 tries, since reading it costs more than such a wait.  CTA scope also on
// barriers that a cluster's peer arrives on: what those announce is in shared
// or tensor memory (an acquire at cluster scope took some 1000 cycles each).
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*abort) return false;
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit) {
        *abort = 1;
        return false;
      }
    }
  }
}

// The same for waits that are long: sleeps between the tries, so that the
// polling does not take issue slots and ALU cycles from the warps at work
// (eight warps polling took a third of a SM's ALU cycles).
__device__ __forceinline__ bool wait_bar_idle(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  uint64_t t0 = 0;
  while (!mbar_try_wait(bar, parity)) {
    __nanosleep(64);
    if (*abort) return false;
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, limit));
}

// One untiled copy global -> shared that completes on `bar` (16-byte aligned
// addresses, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Arguments of the q4tp product (checked by the C entry; strides in elements).
struct LinearArgs {
  const void* x;
  long long ldx;
  int tokens;
  const uint8_t* nibbles;
  const uint8_t* rungs;
  const float* tab;
  int rows, n;
  const void* bias;
  int act;
  const void* residual;
  long long ldr;
  void* y;
  long long ldy;
  unsigned* status;
};

// Arguments of the attention over the cache.
struct AttnArgs {
  const void* q;
  long long q_ts, q_hs;  // elements between query tokens and between heads
  int tq;
  const uint8_t* cache;
  long long pages;
  int heads, group, page_size;
  const int* table;
  int table_stride;
  const int* kv_lens;
  const int* q_starts;  // null: one query a sequence
  int seqs, max_q;
  float scale_log2;  // scale * log2(e)
  void* out;         // [tq][heads * group][dim]
  int4* cuts;        // workspace: a share's cut item for the join: (first query row, first row of the
                     // block, head << 9 | rows, share of its last piece); no rows: nothing to join
  float* part;       // workspace: pieces of cut items
  uint32_t up;       // 2^kPos of T (see code16)
  unsigned* status;
  bool first = true, last = true;  // the launch has the call's first, last sequence
};

// Zeros for the output rows that are no sequence's: before the first one's,
// after the last one's and past max_q of their own.  By `ctas` CTAs of a
// launch, this one number `cta`; a.q_starts is given.
template <class T, int D>
__device__ __forceinline__ void zero_other_rows(const AttnArgs& a, int cta, int ctas) {
  auto start = [&](int i) { return min(max(a.q_starts[i], 0), a.tq); };
  auto zero = [&](int row) {
    const int n = a.heads * a.group * (D / 8);  // 16 bytes each
    uint4* dst = static_cast<uint4*>(a.out) + (long long)row * n;
    for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = uint4{};
  };
  if (a.first)
    for (int r = cta, end = start(0); r < end; r += ctas) zero(r);
  if (a.last)
    for (int r = start(a.seqs) + cta; r < a.tq; r += ctas) zero(r);
  for (int b = cta; b < a.seqs; b += ctas)
    for (int r = start(b), end = start(b + 1), i = a.max_q; i < end - r; ++i) zero(r + i);
}

// The driver's tensor-map encoder (null when it cannot be had).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Shares of a launch at most, and bytes of the workspace before the pieces.
constexpr int kShares = 2560;
constexpr size_t kCutBytes = kShares * sizeof(int4);

// Geometry of the cache: blocks of 16 tokens, each
//   K codes [16][dim / 2], K (scale, offset) [16][dim / 32], V codes, V (scale, offset).
constexpr int KV_BLOCK = 16;
__host__ __device__ constexpr int kv_block_bytes(int dim) { return 20 * dim; }
__host__ __device__ constexpr int kv_param_off(int dim) { return 8 * dim; }
__host__ __device__ constexpr int kv_value_off(int dim) { return 10 * dim; }

// (s, z) pairs of the value of token t of sequence b: what the copies of the
// attention kernels read (an entry of the table outside the pool: page 0).
template <int D>
__device__ __forceinline__ const uint32_t* value_params(const AttnArgs& a, int b, int head, int t) {
  const unsigned e = (unsigned)a.table[(long long)b * a.table_stride + t / a.page_size];
  const long long page = e < (unsigned long long)a.pages ? (long long)e : 0;
  const int bpp = a.page_size / KV_BLOCK;
  const uint8_t* blk = a.cache + ((page * a.heads + head) * bpp + t / KV_BLOCK % bpp) * (long long)kv_block_bytes(D);
  return reinterpret_cast<const uint32_t*>(blk + kv_value_off(D) + kv_param_off(D) + t % KV_BLOCK * (D / 8));
}

}  // namespace gq
