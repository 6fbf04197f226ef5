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
// a lane), a thread does the key and the value of its place, so that two
// loads are in flight for each.  Nothing orders the stores of one place
// against another's: the slots of a write have to differ.  A block looks its tokens' slots up once, into
// shared memory: the divisions of a 64-bit slot would otherwise be most of
// what a place costs.  They are bound by the memory: 131072 tokens of 8 heads
// of 128 read back in 122 us, 5.78 TB/s of codes and values together, and
// 16001 tokens written and read back in 37 us, 4.68 TB/s.
#include "rotary.cuh"

namespace gq {
namespace {

struct CacheShape {
  uint8_t* base;
  long long pages;
  int heads, dim, page_size;
};

constexpr int MAXTOK = 128;  // tokens of one CTA at most: a token has at least eight places

// Byte address of the block that holds `slot` for head 0; null when the slot
// is not in the pool (negative slots mark padding).
__device__ __forceinline__ uint8_t* block_of(const CacheShape& c, long long slot) {
  if (slot < 0) return nullptr;
  const int bpp = c.page_size / KV_BLOCK;
  const long long blk = slot / KV_BLOCK;
  // (A 32-bit division is a quarter of a 64-bit one.)
  const long long page = blk >> 32 ? blk / bpp : (long long)((uint32_t)blk / (uint32_t)bpp);
  if (page >= c.pages) return nullptr;
  return c.base + (page * c.heads * bpp + (blk - page * bpp)) * (long long)kv_block_bytes(c.dim);
}

// What a CTA knows of its tokens.
struct Tokens {
  uint8_t* blk[MAXTOK];
  int row[MAXTOK];
};

__device__ __forceinline__ void look_up(Tokens& t, const CacheShape& c, const long long* slots, long long tok0, int n) {
  if ((int)threadIdx.x < n) {
    const long long slot = slots[tok0 + threadIdx.x];
    t.blk[threadIdx.x] = block_of(c, slot);
    t.row[threadIdx.x] = (int)(slot & (KV_BLOCK - 1));  // page_size is a multiple of the block
  }
  __syncthreads();
}

// Quantises the eight elements of one lane (four lanes a group): the word of
// codes, and the group's (s, z) in `par`.
template <class T>
__device__ __forceinline__ uint32_t quantise8(uint4 raw, uint32_t& par) {
  using T2 = typename Elem<T>::T2;
  const T2 a = from_bits2<T2>(raw.x), b = from_bits2<T2>(raw.y), c = from_bits2<T2>(raw.z), d = from_bits2<T2>(raw.w);
  T2 mn = __hmin2_nan(__hmin2_nan(a, b), __hmin2_nan(c, d));
  T2 mx = __hmax2_nan(__hmax2_nan(a, b), __hmax2_nan(c, d));
  // Both ends in one pair, (lo, -hi), for the steps across the lanes.
  const uint32_t n = bits2(mn), x = bits2(mx) ^ 0x80008000u;
  T2 e = __hmin2_nan(from_bits2<T2>(__byte_perm(n, x, 0x5410)), from_bits2<T2>(__byte_perm(n, x, 0x7632)));
  e = __hmin2_nan(e, from_bits2<T2>(__shfl_xor_sync(0xffffffffu, bits2(e), 1)));
  e = __hmin2_nan(e, from_bits2<T2>(__shfl_xor_sync(0xffffffffu, bits2(e), 2)));
  const float2 ends = Elem<T>::to2(e);
  const float lo = ends.x, hi = -ends.y;
  T st = Elem<T>::from(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
  float s = Elem<T>::to(st);
  T zt = Elem<T>::from(__fsub_rn(lo, __fmul_rn(16.0f, s)));
  float z = Elem<T>::to(zt);
  uint32_t w = 0;
  if (isfinite(s) && isfinite(z)) {
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    const float2 f[4] = {Elem<T>::to2(a), Elem<T>::to2(b), Elem<T>::to2(c), Elem<T>::to2(d)};
    // The clamp's ends are integers, so that it may come before the rounding;
    // adding 3 * 2^22 then rounds to the nearest even and leaves the integer
    // in the low bits.
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float q0 = fminf(fmaxf(__fmul_rn(__fsub_rn(f[i].x, z), r), 16.f), 31.f);
      const float q1 = fminf(fmaxf(__fmul_rn(__fsub_rn(f[i].y, z), r), 16.f), 31.f);
      q[2 * i] = __float_as_uint(__fadd_rn(q0, 12582912.f));
      q[2 * i + 1] = __float_as_uint(__fadd_rn(q1, 12582912.f));
    }
    const uint32_t even = __byte_perm(__byte_perm(q[0], q[2], 0x0040), __byte_perm(q[4], q[6], 0x0040), 0x5410);
    const uint32_t odd = __byte_perm(__byte_perm(q[1], q[3], 0x0040), __byte_perm(q[5], q[7], 0x0040), 0x5410);
    w = (even & 0x0f0f0f0fu) | ((odd << 4) & 0xf0f0f0f0u);
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

// A place: (token, head, eight channels).  per = heads * dim / 8 a token; a CTA
// has `take` tokens, place i of them is token i / per (per_inv = ceil(2^32 /
// per): exact for the places of a CTA, which are less than 2^16 or one token's).
template <class T>
__global__ void __launch_bounds__(256)
    k_kv4_write(CacheShape c, const T* __restrict__ k, const T* __restrict__ v, Strides st,
                const long long* __restrict__ slots, int tokens, int per, uint32_t per_inv, int take) {
  __shared__ Tokens ts;
  const long long tok0 = (long long)blockIdx.x * take;
  const int n = (int)min((long long)take, tokens - tok0);
  const int cl = c.dim == 256 ? 5 : c.dim == 128 ? 4 : 3;  // log2(dim / 8)
  const long long head_bytes = (long long)(c.page_size / KV_BLOCK) * kv_block_bytes(c.dim);
  const int total = n * per;
  int i = threadIdx.x, tok, head, ch;
  uint4 rk{}, rv{};
  // A place's elements are loaded ahead: the first one's while the slots are
  // looked up, the others' while the one before is quantised.
  auto load = [&] {
    const bool in = i < total;
    tok = take == 1 || !in ? 0 : (int)__umulhi((uint32_t)i, per_inv);
    const int at = in ? i - tok * per : 0;
    head = at >> cl, ch = at & ((1 << cl) - 1);
    if (in) {
      rk = *reinterpret_cast<const uint4*>(k + (tok0 + tok) * st.kt + head * st.kh + ch * 8);
      rv = *reinterpret_cast<const uint4*>(v + (tok0 + tok) * st.vt + head * st.vh + ch * 8);
    }
  };
  load();
  look_up(ts, c, slots, tok0, n);
#pragma unroll 1
  while ((i & ~31) < total) {
    uint8_t* blk = i < total ? ts.blk[tok] : nullptr;
    const int row = ts.row[tok], ch0 = ch;
    if (blk != nullptr) blk += head * head_bytes;
    const uint4 k8 = rk, v8 = rv;
    i += 256;
    load();
    // The four lanes of a group always come together (dim % 32 == 0).
    uint32_t pk, pv;
    const uint32_t wk = quantise8<T>(k8, pk), wv = quantise8<T>(v8, pv);
    if (blk != nullptr) {
      uint8_t* kb = blk + row * (c.dim / 2) + ch0 * 4;
      *reinterpret_cast<uint32_t*>(kb) = wk;
      *reinterpret_cast<uint32_t*>(kb + kv_value_off(c.dim)) = wv;
      if ((ch0 & 3) == 0) {
        uint8_t* pb = blk + kv_param_off(c.dim) + row * (c.dim / 8) + ch0;
        *reinterpret_cast<uint32_t*>(pb) = pk;
        *reinterpret_cast<uint32_t*>(pb + kv_value_off(c.dim)) = pv;
      }
    }
  }
}

template <class T>
__global__ void __launch_bounds__(256)
    k_kv4_read(CacheShape c, const long long* __restrict__ slots, int tokens, int per, uint32_t per_inv, int take,
               T* __restrict__ k, T* __restrict__ v) {
  __shared__ Tokens ts;
  const long long tok0 = (long long)blockIdx.x * take;
  const int n = (int)min((long long)take, tokens - tok0);
  look_up(ts, c, slots, tok0, n);
  const int cl = c.dim == 256 ? 5 : c.dim == 128 ? 4 : 3;  // log2(dim / 8)
  const long long head_bytes = (long long)(c.page_size / KV_BLOCK) * kv_block_bytes(c.dim);
  const int total = n * per;
  uint4* ko = reinterpret_cast<uint4*>(k) + tok0 * per;
  uint4* vo = reinterpret_cast<uint4*>(v) + tok0 * per;
#pragma unroll 4
  for (int i = threadIdx.x; i < total; i += 256) {
    const int tok = take == 1 ? 0 : (int)__umulhi((uint32_t)i, per_inv);
    const int at = i - tok * per, head = at >> cl, ch = at & ((1 << cl) - 1);
    const uint8_t* blk = ts.blk[tok];
    uint4 ok{}, ov{};
    if (blk != nullptr) {
      blk += head * head_bytes;
      const int row = ts.row[tok];
      const uint8_t* kb = blk + row * (c.dim / 2) + ch * 4;
      const uint8_t* pb = blk + kv_param_off(c.dim) + row * (c.dim / 8) + (ch & ~3);
      const uint32_t wk = *reinterpret_cast<const uint32_t*>(kb);
      const uint32_t wv = *reinterpret_cast<const uint32_t*>(kb + kv_value_off(c.dim));
      const uint32_t pk = *reinterpret_cast<const uint32_t*>(pb);
      const uint32_t pv = *reinterpret_cast<const uint32_t*>(pb + kv_value_off(c.dim));
      ok = values8<T>(wk, pk);
      ov = values8<T>(wv, pv);
    }
    __stcs(ko + i, ok);
    __stcs(vo + i, ov);
  }
}

// The write with rotary positions on its way: q turned into y, k turned into
// the cache (rounded to T first, so that the codes are those of a turned key
// that k_kv4_write is given), v as it is.  A lane has a token and eight channels and
// walks over heads, so that its sines and
// cosines serve them all; in the half layout the other channels of its pairs
// are another lane's, which hands them over (dim / 8 lanes of a warp are a
// head's).  A lane reads and writes its own octets only: y may be q itself.
// Measured: 8001 tokens of 32 query and 8 key heads of 128 in 41.1 us, 4.2 TB/s
// (55 % of the issue slots, memory 41 % busy, neither of them its limit: a warp waits for
// its loads); 64 tokens 3.5 us, one 3.5.
struct TurnedHeads {
  const void* q;
  long long qt, qh;
  int q_heads;
  void* y;
  long long yt, yh;
  const void* k;
  const void* v;
  Strides st;
};

template <class T, bool HALF>
__global__ void __launch_bounds__(256)
    k_kv4_write_rotary(CacheShape c, TurnedHeads io, RotaryArgs a, const long long* __restrict__ slots, int tokens, int take) {
  const int cl = c.dim == 256 ? 5 : c.dim == 128 ? 4 : 3;  // log2(dim / 8)
  const int i = (int)(blockIdx.x * 256 + threadIdx.x), ch = (i & ((1 << cl) - 1)) * 8;
  const bool in = i >> cl < tokens;
  const int tok = in ? i >> cl : tokens - 1;
  const int h0 = (int)blockIdx.y * take, h1 = min(h0 + take, io.q_heads + c.heads);
  const bool turns = ch < a.rot, second = HALF && ch >= a.rot / 2;
  const int step = turns ? a.rot / 16 : 0, lane = threadIdx.x % 32, partner = second ? lane - step : lane + step;
  float co[8], si[8];
  const long long position = a.positions[tok];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float2 t{0.f, 0.f};
    if (turns && (HALF || k < 4)) t = turn_of(a, position, HALF ? (second ? ch - a.rot / 2 : ch) + k : ch / 2 + k);
    co[k] = t.x, si[k] = HALF && !second ? -t.y : t.y;
  }
  auto turned8 = [&](uint4 x) {
    uint4 o;
    if (HALF) {
      uint4 p;
      p.x = __shfl_sync(0xffffffffu, x.x, partner), p.y = __shfl_sync(0xffffffffu, x.y, partner);
      p.z = __shfl_sync(0xffffffffu, x.z, partner), p.w = __shfl_sync(0xffffffffu, x.w, partner);
      o = turn_half<T>(x, p, co, si);
    } else {
      o = turn_pairs<T>(x, co, si);
    }
    return turns ? o : x;
  };
  // The cache's heads come first: they take longest.
  const int kv1 = min(h1, c.heads);
  if (h0 < kv1) {
    const long long slot = slots[tok];
    const T* kp = static_cast<const T*>(io.k) + tok * io.st.kt + ch;
    const T* vp = static_cast<const T*>(io.v) + tok * io.st.vt + ch;
    uint4 rk = *reinterpret_cast<const uint4*>(kp + h0 * io.st.kh), rv = *reinterpret_cast<const uint4*>(vp + h0 * io.st.vh);
    const long long head_bytes = (long long)(c.page_size / KV_BLOCK) * kv_block_bytes(c.dim);
    const int row = (int)(slot & (KV_BLOCK - 1));  // page_size is a multiple of the block
    uint8_t* blk = in ? block_of(c, slot) : nullptr;
    const bool stored = blk != nullptr;
    blk += h0 * head_bytes + row * (c.dim / 2) + ch / 2;
    const int par = kv_param_off(c.dim) + row * (c.dim / 8) + ch / 8 - (row * (c.dim / 2) + ch / 2);
#pragma unroll 2
    for (int h = h0; h < kv1; ++h, blk += head_bytes) {
      const uint4 k8 = turned8(rk), v8 = rv;
      if (h + 1 < kv1) {  // ahead: under the quantisation
        rk = *reinterpret_cast<const uint4*>(kp + (h + 1) * io.st.kh);
        rv = *reinterpret_cast<const uint4*>(vp + (h + 1) * io.st.vh);
      }
      uint32_t pk, pv;
      const uint32_t wk = quantise8<T>(k8, pk), wv = quantise8<T>(v8, pv);
      if (stored) {
        *reinterpret_cast<uint32_t*>(blk) = wk;
        *reinterpret_cast<uint32_t*>(blk + kv_value_off(c.dim)) = wv;
        if (ch % 32 == 0) {
          *reinterpret_cast<uint32_t*>(blk + par) = pk;
          *reinterpret_cast<uint32_t*>(blk + par + kv_value_off(c.dim)) = pv;
        }
      }
    }
  }
  const T* q = static_cast<const T*>(io.q) + tok * io.qt + ch;
  T* y = static_cast<T*>(io.y) + tok * io.yt + ch;
#pragma unroll 4
  for (int h = max(h0 - c.heads, 0); h < h1 - c.heads; ++h) {
    const uint4 o = turned8(*reinterpret_cast<const uint4*>(q + h * io.qh));
    if (in) *reinterpret_cast<uint4*>(y + h * io.yh) = o;
  }
}

// Tokens a CTA: four places a thread where that still gives every SM its eight
// CTAs, else one.  Measured, 131072 tokens of 8 heads of 128 read back: two
// places a thread 128.6 us, four 122.1, eight 121.0, sixteen 122.6; 16001
// tokens written and read: 37.5, 36.8, 37.8, 43.7.
struct Split {
  int take;
  unsigned grid;
  uint32_t per_inv;
};

Split split_of(int tokens, int per) {
  const long long places = (long long)tokens * per;
  const int want = places >= 152ll * 8 * 1024 ? 4 * 256 : 256;
  Split s;
  s.take = std::min(std::max(want / per, 1), MAXTOK);
  s.grid = (unsigned)((tokens + s.take - 1) / s.take);
  s.per_inv = (uint32_t)(((1ull << 32) + per - 1) / per);
  return s;
}

}  // namespace

gptq_status kv4_write_run(int dtype, uint8_t* cache, long long pages, int heads, int dim, int page_size,
                          const void* k, const void* v, long long kt, long long kh, long long vt, long long vh,
                          const long long* slots, int tokens, cudaStream_t s) {
  if (tokens == 0) return GPTQ_OK;
  const CacheShape c{cache, pages, heads, dim, page_size};
  const Strides st{kt, kh, vt, vh};
  const int per = heads * (dim / 8);
  const Split p = split_of(tokens, per);
  GQ_PROF(K_KV4_WRITE, s);
  if (dtype == GPTQ_BF16)
    k_kv4_write<<<p.grid, 256, 0, s>>>(c, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, st, slots, tokens, per, p.per_inv, p.take);
  else
    k_kv4_write<<<p.grid, 256, 0, s>>>(c, (const __half*)k, (const __half*)v, st, slots, tokens, per, p.per_inv, p.take);
  GQ_LAUNCHED();
  return GPTQ_OK;
}

gptq_status kv4_write_rotary_run(int dtype, bool half, uint8_t* cache, long long pages, int heads, int page_size,
                                 const void* q, long long qt, long long qh, int q_heads, const void* k, const void* v,
                                 long long kt, long long kh, long long vt, long long vh, const long long* slots,
                                 int tokens, const RotaryArgs& a, void* y, long long yt, long long yh, cudaStream_t s) {
  if (tokens == 0) return GPTQ_OK;
  const CacheShape c{cache, pages, heads, a.dim, page_size};
  const TurnedHeads io{q, qt, qh, q_heads, y, yt, yh, k, v, Strides{kt, kh, vt, vh}};
  const long long threads = (long long)tokens * (a.dim / 8);
  // Heads a thread: as many as leave every SM 1024 threads, sixteen at most.
  // Measured, 32 + 8 heads of 128 (2048 / 1024 / 512 / 256 threads an SM): 500 tokens
  // 8.1 / 6.2 / 6.0 / 8.0 us, 1000 9.3 / 7.6 / 8.5 / 10.3, 2000 11.8 / 11.2 / 13.0 / 13.0;
  // 8001 tokens with sixteen heads 41.2, with eight 44.5.
  const int every = q_heads + heads;
  const int take = (int)std::min<long long>(std::max<long long>(threads * every / (num_sms() * 1024ll), 1), 16);
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)((every + take - 1) / take));
  GQ_PROF(K_KV4_WRITE_ROTARY, s);
  if (dtype == GPTQ_BF16) {
    if (half) k_kv4_write_rotary<__nv_bfloat16, true><<<grid, 256, 0, s>>>(c, io, a, slots, tokens, take);
    else k_kv4_write_rotary<__nv_bfloat16, false><<<grid, 256, 0, s>>>(c, io, a, slots, tokens, take);
  } else {
    if (half) k_kv4_write_rotary<__half, true><<<grid, 256, 0, s>>>(c, io, a, slots, tokens, take);
    else k_kv4_write_rotary<__half, false><<<grid, 256, 0, s>>>(c, io, a, slots, tokens, take);
  }
  GQ_LAUNCHED();
  return GPTQ_OK;
}

gptq_status kv4_read_run(int dtype, const uint8_t* cache, long long pages, int heads, int dim, int page_size,
                         const long long* slots, int tokens, void* k, void* v, cudaStream_t s) {
  if (tokens == 0) return GPTQ_OK;
  const CacheShape c{const_cast<uint8_t*>(cache), pages, heads, dim, page_size};
  const int per = heads * (dim / 8);
  const Split p = split_of(tokens, per);
  GQ_PROF(K_KV4_READ, s);
  if (dtype == GPTQ_BF16)
    k_kv4_read<<<p.grid, 256, 0, s>>>(c, slots, tokens, per, p.per_inv, p.take, (__nv_bfloat16*)k, (__nv_bfloat16*)v);
  else
    k_kv4_read<<<p.grid, 256, 0, s>>>(c, slots, tokens, per, p.per_inv, p.take, (__half*)k, (__half*)v);
  GQ_LAUNCHED();
  return GPTQ_OK;
}

}  // namespace gq
