// The 4-bit key/value cache, written and read back.
//
// A group is 32 consecutive channels of one token's key (or value) of one
// head.  With lo and hi its smallest and largest value,
//   s = T((hi - lo) / 15),  z = T(lo - 16 s),
//   c = clamp(rint((x - z) / s), 16, 31) - 16,   value = T(z + s (16 + c)).
// The offset z belongs to the code 16 + c and not to c because 16 + c is an
// element of T whose top four mantissa bits are the code: a code becomes its
// value by an AND, an OR and one fused multiply-add with one rounding, and
// every reader gets the same bits.  The codes are chosen against the rounded
// s and z, so rounding them costs no more than the clamp at the ends.
// A group with a NaN or an infinity, or whose s or z leaves T's range
// (f16: groups within +-20000 cannot), is stored with s = z = NaN and reads
// back as NaN.
//
// Both kernels move each byte once: four lanes share a group (16 bytes of T
// a lane), a thread does the key and the value of its place, so that the
// slot is looked up once and two loads are in flight.
#include "serve.cuh"

namespace gq {
namespace {

struct CacheShape {
  uint8_t* base;
  long long pages;
  int heads, dim, page_size;
};

// Byte address of the block that holds `slot` for `head`; null when the slot
// is not in the pool (negative slots mark padding).
__device__ __forceinline__ uint8_t* block_of(const CacheShape& c, long long slot, int head) {
  const long long page = slot < 0 ? -1 : slot / c.page_size;
  if (page < 0 || page >= c.pages) return nullptr;
  const int off = (int)(slot - page * c.page_size);
  const int bpp = c.page_size / KV_BLOCK;
  return c.base + ((page * c.heads + head) * bpp + off / KV_BLOCK) * (long long)kv_block_bytes(c.dim);
}

// Quantises the eight elements of one lane (four lanes a group): the word of
// codes, and the group's (s, z) in `par`.
template <class T>
__device__ __forceinline__ uint32_t quantise8(uint4 raw, uint32_t& par) {
  using T2 = typename Elem<T>::T2;
  const T2 a = from_bits2<T2>(raw.x), b = from_bits2<T2>(raw.y), c = from_bits2<T2>(raw.z), d = from_bits2<T2>(raw.w);
  const float2 mn2 = Elem<T>::to2(__hmin2_nan(__hmin2_nan(a, b), __hmin2_nan(c, d)));
  const float2 mx2 = Elem<T>::to2(__hmax2_nan(__hmax2_nan(a, b), __hmax2_nan(c, d)));
  // A NaN on either side must survive: x + 0 * y keeps it where fminf drops it.
  float lo = fminf(mn2.x, mn2.y), hi = fmaxf(mx2.x, mx2.y);
  if (mn2.x != mn2.x || mn2.y != mn2.y) lo = hi = __int_as_float(0x7fffffff);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float l2 = __shfl_xor_sync(0xffffffffu, lo, o), h2 = __shfl_xor_sync(0xffffffffu, hi, o);
    const bool nan = l2 != l2 || lo != lo;
    lo = nan ? __int_as_float(0x7fffffff) : fminf(lo, l2);
    hi = nan ? __int_as_float(0x7fffffff) : fmaxf(hi, h2);
  }
  T st = Elem<T>::from(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
  float s = Elem<T>::to(st);
  T zt = Elem<T>::from(__fsub_rn(lo, __fmul_rn(16.0f, s)));
  float z = Elem<T>::to(zt);
  uint32_t w = 0;
  if (isfinite(s) && isfinite(z)) {
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    const float2 f[4] = {Elem<T>::to2(a), Elem<T>::to2(b), Elem<T>::to2(c), Elem<T>::to2(d)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float q0 = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(f[i].x, z), r)), 16.f), 31.f);
      const float q1 = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(f[i].y, z), r)), 16.f), 31.f);
      w |= ((uint32_t)q0 - 16u) << (8 * i);
      w |= ((uint32_t)q1 - 16u) << (8 * i + 4);
    }
    par = (uint32_t)*reinterpret_cast<uint16_t*>(&st) | ((uint32_t)*reinterpret_cast<uint16_t*>(&zt) << 16);
  } else {
    par = 0x7fff7fffu;  // NaN in both types
  }
  return w;
}

// The eight values of a word of codes, in order.
template <class T>
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t par) {
  using T2 = typename Elem<T>::T2;
  const T2 s2 = from_bits2<T2>(__byte_perm(par, par, 0x1010)), z2 = from_bits2<T2>(__byte_perm(par, par, 0x3232));
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = bits2(__hfma2(code16<T>(w, i), s2, z2));  // values i and i + 4
  uint4 o;
  o.x = __byte_perm(p[0], p[1], 0x5410);
  o.y = __byte_perm(p[2], p[3], 0x5410);
  o.z = __byte_perm(p[0], p[1], 0x7632);
  o.w = __byte_perm(p[2], p[3], 0x7632);
  return o;
}

struct Strides {
  long long kt, kh, vt, vh;  // elements between tokens and between heads
};

// A place: (token, head, eight channels).  per = heads * dim / 8 a token.
template <class T>
__global__ void __launch_bounds__(256)
    k_kv4_write(CacheShape c, const T* __restrict__ k, const T* __restrict__ v, Strides st,
                const long long* __restrict__ slots, int tokens, int per) {
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long total = (long long)tokens * per;
  const long long tok = id / per;
  const bool in = id < total;
  const int at = (int)(id - tok * per), cpr = c.dim / 8;
  const int head = at / cpr, ch = at % cpr;
  uint8_t* blk = in ? block_of(c, slots[tok], head) : nullptr;
  uint4 rk{}, rv{};
  if (blk != nullptr) {
    rk = *reinterpret_cast<const uint4*>(k + tok * st.kt + head * st.kh + ch * 8);
    rv = *reinterpret_cast<const uint4*>(v + tok * st.vt + head * st.vh + ch * 8);
  }
  // The four lanes of a group are always active together (dim % 32 == 0).
  uint32_t pk, pv;
  const uint32_t wk = quantise8<T>(rk, pk), wv = quantise8<T>(rv, pv);
  if (blk == nullptr) return;
  const int row = (int)(slots[tok] % KV_BLOCK);  // page_size is a multiple of the block
  uint8_t* kb = blk + row * (c.dim / 2) + ch * 4;
  *reinterpret_cast<uint32_t*>(kb) = wk;
  *reinterpret_cast<uint32_t*>(kb + kv_value_off(c.dim)) = wv;
  if ((ch & 3) == 0) {
    uint8_t* pb = blk + kv_param_off(c.dim) + row * (c.dim / 8) + ch;
    *reinterpret_cast<uint32_t*>(pb) = pk;
    *reinterpret_cast<uint32_t*>(pb + kv_value_off(c.dim)) = pv;
  }
}

template <class T>
__global__ void __launch_bounds__(256)
    k_kv4_read(CacheShape c, const long long* __restrict__ slots, int tokens, int per, T* __restrict__ k,
               T* __restrict__ v) {
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= (long long)tokens * per) return;
  const long long tok = id / per;
  const int at = (int)(id - tok * per), cpr = c.dim / 8;
  const int head = at / cpr, ch = at % cpr;
  const long long slot = slots[tok];
  const uint8_t* blk = block_of(c, slot, head);
  uint4 ok{}, ov{};
  if (blk != nullptr) {
    const int row = (int)(slot % KV_BLOCK);
    const uint8_t* kb = blk + row * (c.dim / 2) + ch * 4;
    const uint8_t* pb = blk + kv_param_off(c.dim) + row * (c.dim / 8) + (ch & ~3);
    const uint32_t wk = *reinterpret_cast<const uint32_t*>(kb);
    const uint32_t wv = *reinterpret_cast<const uint32_t*>(kb + kv_value_off(c.dim));
    const uint32_t pk = *reinterpret_cast<const uint32_t*>(pb);
    const uint32_t pv = *reinterpret_cast<const uint32_t*>(pb + kv_value_off(c.dim));
    ok = values8<T>(wk, pk);
    ov = values8<T>(wv, pv);
  }
  reinterpret_cast<uint4*>(k)[id] = ok;
  reinterpret_cast<uint4*>(v)[id] = ov;
}

}  // namespace

gptq_status kv4_write_run(int dtype, uint8_t* cache, long long pages, int heads, int dim, int page_size,
                          const void* k, const void* v, long long kt, long long kh, long long vt, long long vh,
                          const long long* slots, int tokens, cudaStream_t s) {
  if (tokens == 0) return GPTQ_OK;
  const CacheShape c{cache, pages, heads, dim, page_size};
  const Strides st{kt, kh, vt, vh};
  const int per = heads * (dim / 8);
  const unsigned grid = (unsigned)(((long long)tokens * per + 255) / 256);
  GQ_PROF(K_KV4_WRITE, s);
  if (dtype == GPTQ_BF16)
    k_kv4_write<<<grid, 256, 0, s>>>(c, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, st, slots, tokens, per);
  else
    k_kv4_write<<<grid, 256, 0, s>>>(c, (const __half*)k, (const __half*)v, st, slots, tokens, per);
  GQ_LAUNCHED();
  return GPTQ_OK;
}

gptq_status kv4_read_run(int dtype, const uint8_t* cache, long long pages, int heads, int dim, int page_size,
                         const long long* slots, int tokens, void* k, void* v, cudaStream_t s) {
  if (tokens == 0) return GPTQ_OK;
  const CacheShape c{const_cast<uint8_t*>(cache), pages, heads, dim, page_size};
  const int per = heads * (dim / 8);
  const unsigned grid = (unsigned)(((long long)tokens * per + 255) / 256);
  GQ_PROF(K_KV4_READ, s);
  if (dtype == GPTQ_BF16)
    k_kv4_read<<<grid, 256, 0, s>>>(c, slots, tokens, per, (__nv_bfloat16*)k, (__nv_bfloat16*)v);
  else
    k_kv4_read<<<grid, 256, 0, s>>>(c, slots, tokens, per, (__half*)k, (__half*)v);
  GQ_LAUNCHED();
  return GPTQ_OK;
}

}  // namespace gq
