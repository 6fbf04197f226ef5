// Attention over the 4-bit cache for many queries a sequence (prompt chunks),
// on tcgen05.
//
// A CTA owns 256 query rows -- (query, head of the key head's group) pairs --
// as two tiles A and B of 128, and walks the keys they see in steps of 128
// tokens.  With so many rows the products bound it (4 * 128 * D flop a row
// and step), and the decoding of the codes, done once for both tiles, and the
// exponentials run beside them:
//   warps 0-3, 4-7  softmax of tile A, B: a row a thread.  S from tensor
//                   memory (twice: maximum, then exponentials), P written
//                   back over it in T, the operand A of the second product;
//   warps 8-10, 11-13  decode K, V of a step into shared memory in 128-byte
//                   swizzled rows of tokens (K is then a K-major operand, V
//                   an N-major one: no transpose);
//   warp 14         copies the step's cache blocks (untiled bulk copies);
//   warp 15         issues the products: S_A, S_B of the next step between
//                   O_A += P_A V and O_B += P_B V, so that one tile's
//                   softmax runs under the other's products.
// Tensor memory: S_A, S_B (128 columns each, P over their first half), O_A,
// O_B (D columns each).
// The running maximum is only raised (and O rescaled, by its rows' threads,
// after the step's commit has shown the last product done) when it would
// grow by more than 2^8; exponentials stay within that and nothing is lost.
// Channels keep the order in which the nibbles come out (0 4 1 5 2 6 3 7 of
// every eight): q is stored to match, and the output is read back through it.
#include "serve.cuh"

namespace gq {
namespace {

constexpr int CK = 128;     // keys a step
constexpr int CROWS = 256;  // query rows a CTA
constexpr int CTHREADS = 512;
constexpr float kNone = -1e30f;

template <class T>
struct MmaFormat;
template <>
struct MmaFormat<__nv_bfloat16> {
  static constexpr uint32_t k = 1u;
};
template <>
struct MmaFormat<__half> {
  static constexpr uint32_t k = 0u;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// For what is in tensor memory (ordered by the tcgen05 fences).
__device__ __forceinline__ void arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Descriptor of an N-major operand, 128-byte swizzle: rows of 64 elements
// (one a token), 8 rows in 1024 bytes; `lead` bytes between the 64-element
// halves of N.
__device__ __forceinline__ uint64_t ndesc(uint32_t saddr, uint32_t lead) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Byte offset of 16-byte piece p (0 .. 7) of row r in a swizzled tile.
__device__ __forceinline__ uint32_t swz(int r, int p) { return (uint32_t)(r * 128 + ((p ^ (r & 7)) * 16)); }

template <int D>
struct ChunkSmem {  // byte offsets; 1024-byte aligned operands
  static constexpr int kTile = CK * D * 2;           // K, V, and a tile of Q
  static constexpr int kRaw = (CK / KV_BLOCK) * kv_block_bytes(D);
  static constexpr int q = 0;                        // two tiles
  static constexpr int k = q + 2 * kTile;            // two steps
  static constexpr int v = k + 2 * kTile;            // one
  static constexpr int raw = v + kTile;              // two steps
  static constexpr int bytes = raw + 2 * kRaw + 1024;
};

template <class T, int D>
__global__ void __launch_bounds__(CTHREADS, 1) k_kv4_chunk(AttnArgs a, int nblk_max, WaitCfg wc) {
  using T2 = typename Elem<T>::T2;
  using S = ChunkSmem<D>;
  constexpr int BB = kv_block_bytes(D), HALVES = D / 64;
  constexpr uint32_t kO = 256;  // tensor memory: S_A 0, S_B 128, O_A 256, O_B 256 + D
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t qfull, kfull[2], kempty[2], vfull, vempty, rawfull[2], rawempty[2], sfull[2],
      pfull[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  const int b = (int)blockIdx.y, head = (int)blockIdx.x, rb = nblk_max - 1 - (int)blockIdx.z;  // long rows first
  const int q0 = min(max(a.q_starts[b], 0), a.tq);
  const int nq = min(min(max(a.q_starts[b + 1], q0), a.tq) - q0, a.max_q);
  const int len = (int)min((long long)max(a.kv_lens[b], 0), (long long)a.table_stride * a.page_size);
  const long long all = (long long)nq * a.group;
  const long long r0 = (long long)rb * CROWS;
  if (r0 >= all) return;
  const int rows = (int)min((long long)CROWS, all - r0);
  const int vis = max(0, min(len, len - nq + (int)((r0 + rows - 1) / a.group) + 1));  // keys the last row sees
  const int steps = (vis + CK - 1) / CK;
  const bool two = rows > 128;

  if (threadIdx.x == 0) {
    mbar_init(&qfull, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 96), mbar_init(&kempty[i], 1);
      mbar_init(&rawfull[i], 1), mbar_init(&rawempty[i], 6);
      mbar_init(&sfull[i], 1), mbar_init(&pfull[i], 128);
    }
    mbar_init(&vfull, 96), mbar_init(&vempty, 1);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 15) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Registers: 128 a thread at launch (512 threads); a softmax thread keeps a
  // row of scores, 2 * 128 * 184 + 2 * 128 * 72 = 65536 in all.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int x = warp / 4, rt = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = (uint32_t)(128 * x) + lanes, to = kO + (uint32_t)(D * x) + lanes;
    const bool mine = 128 * x + rt < rows;
    const long long rr = r0 + min(128 * x + rt, rows - 1);
    const int qi = (int)(rr / a.group), hq = head * a.group + (int)(rr % a.group);
    const int last = mine ? len - nq + qi : -1;
    // The row's q, in the nibbles' order of channels.
    {
      const T* qp = static_cast<const T*>(a.q) + (long long)(q0 + qi) * a.q_ts + (long long)hq * a.q_hs;
      const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale: -q
      uint8_t* tile = smem + S::q + x * S::kTile;
#pragma unroll
      for (int c0 = 0; c0 < D / 8; c0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = mine ? *reinterpret_cast<const uint4*>(qp + 8 * (c0 + c)) : uint4{};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 o = pair_order(v[c]);
          o.x ^= flip, o.y ^= flip, o.z ^= flip, o.w ^= flip;
          *reinterpret_cast<uint4*>(tile + c0 / 8 * (CK * 128) + swz(rt, c)) = o;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&qfull);
    }
    // (Not 0: a hidden key is a score of -inf, and -inf times 0 is no number.)
    const float sl = fmaxf(fabsf(a.scale_log2), 1e-30f);
    float m = kNone, l = 0.f;
    bool ok = true;
    if (x == 0 || two) {
#pragma unroll 1
      for (int j = 0; j < steps && ok; ++j) {
        if (!(ok = wait_bar_warp(&sfull[x], (uint32_t)j & 1u, abort, wc.ns))) break;
        tc_fence_after();
        uint32_t v[4][32];  // the row's scores, in registers from here on
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32u * (uint32_t)c, v[c]);
        tmem_ld_wait();
        const int lim = last - j * CK;  // last visible column of the step
        if (__any_sync(0xffffffffu, lim < CK - 1)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i > lim) v[c][i] = 0xff800000u;  // -inf
        }
        float t4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          t4[c] = max3(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]), -INFINITY);
#pragma unroll
          for (int i = 2; i < 32; i += 2) t4[c] = max3(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]), t4[c]);
        }
        const float top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
        if (__any_sync(0xffffffffu, sl * (top - m) > 8.f)) {
          const float nm = fmaxf(m, top), f = ex2(sl * (m - nm));
          m = nm;
          l *= f;
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t w[16];
              tmem_ld16(to + (uint32_t)c, w);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
              tmem_st16(to + (uint32_t)c, w);
            }
          }
        }
        const float ms = sl * m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float e0 = ex2(fmaf(sl, __uint_as_float(v[c][2 * i]), -ms)),
                        e1 = ex2(fmaf(sl, __uint_as_float(v[c][2 * i + 1]), -ms));
            sum[2 * i & 3] += e0;
            sum[(2 * i + 1) & 3] += e1;
            p[i] = bits2(Elem<T>::make2(e0, e1));
          }
          tmem_st16(ts + 16u * (uint32_t)c, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
        tc_fence_before();
        arrive_relaxed(&pfull[x]);
      }
      // The output, once the last product is done.
      if (ok && steps > 0) ok = wait_bar_warp(&sfull[x], (uint32_t)steps & 1u, abort, wc.ns);
      if (ok) {
        tc_fence_after();
        const float inv = l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing: zeros
        T* dst = static_cast<T*>(a.out) + ((long long)(q0 + qi) * a.heads * a.group + hq) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t v[16];
          if (steps > 0) {
            tmem_ld16(to + (uint32_t)c, v);
            tmem_ld_wait();
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = inv != 0.f ? __uint_as_float(v[8 * h + i]) * inv : 0.f;
            uint4 o;  // columns 0 .. 7 hold channels 0 4 1 5 2 6 3 7
            o.x = bits2(Elem<T>::make2(e[0], e[2]));
            o.y = bits2(Elem<T>::make2(e[4], e[6]));
            o.z = bits2(Elem<T>::make2(e[1], e[3]));
            o.w = bits2(Elem<T>::make2(e[5], e[7]));
            if (mine) *reinterpret_cast<uint4*>(dst + c + 8 * h) = o;
          }
        }
        tc_fence_before();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  }
  if (warp >= 8 && warp < 14) {
    // Three warps decode K, three V.  A thread takes 32 channels (one group)
    // of a token at a time: 16 bytes of codes to 64 bytes; it stays with its
    // group and its token's place among eight, so that its addresses advance
    // by constants.  Lanes of the upper half of the channels store their
    // pieces in another order: eight lanes then meet no bank twice.
    const int dt = (threadIdx.x - 256) % 96;
    const bool isv = warp >= 11;
    constexpr int GR = D / 32, TSTEP = 96 / GR;  // groups a token; tokens between a thread's pieces
    const int grp = dt % GR, tok0 = dt / GR;
    const bool swap = GR == 4 && grp >= 2;
    const int rot = swap ? 2 : 0;
    uint32_t off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      off[u] = (uint32_t)(grp / 2 * (CK * 128)) + swz(tok0, grp % 2 * 4 + (u ^ rot));
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < steps && ok; ++j) {
      const int st = j & 1;
      if (!(ok = wait_bar_warp(&rawfull[st], (uint32_t)(j >> 1) & 1u, abort, wc.ns))) break;
      ok = isv ? wait_bar_warp(&vempty, ((uint32_t)j & 1u) ^ 1u, abort, wc.ns)
               : wait_bar_warp(&kempty[st], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort, wc.ns);
      if (!ok) break;
      const uint8_t* raw = smem + S::raw + st * S::kRaw + (isv ? kv_value_off(D) : 0);
      uint8_t* tile = smem + (isv ? S::v : S::k + st * S::kTile);
      const int seen = vis - j * CK;  // tokens of the step that some row sees
#pragma unroll 3
      for (int tok = tok0; tok < CK; tok += TSTEP) {
        const uint8_t* blk = raw + tok / KV_BLOCK * BB;
        uint4 codes = *reinterpret_cast<const uint4*>(blk + tok % KV_BLOCK * (D / 2) + grp * 16);
        uint32_t par = *reinterpret_cast<const uint32_t*>(blk + kv_param_off(D) + tok % KV_BLOCK * (D / 8) + grp * 4);
        if (tok >= seen) par = 0u;  // past what any row sees: no value, whatever is there
        if (GR == 4) {
          const uint4 c = codes;
          codes.x = swap ? c.z : c.x, codes.y = swap ? c.w : c.y;
          codes.z = swap ? c.x : c.z, codes.w = swap ? c.y : c.w;
        }
        const T2 s2 = from_bits2<T2>(__byte_perm(par, par, 0x1010)), z2 = from_bits2<T2>(__byte_perm(par, par, 0x3232));
        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
        uint8_t* dst = tile + (tok - tok0) * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint4 o;
          o.x = bits2(__hfma2(code16<T>(w[u], 0, a.up), s2, z2));
          o.y = bits2(__hfma2(code16<T>(w[u], 1), s2, z2));
          o.z = bits2(__hfma2(code16<T>(w[u], 2), s2, z2));
          o.w = bits2(__hfma2(code16<T>(w[u], 3), s2, z2));
          *reinterpret_cast<uint4*>(dst + off[u]) = o;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(isv ? &vfull : &kfull[st]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&rawempty[st]);
    }
  }
  if (warp == 14) {
    if (!wc.no_loads) {
      const int bpp = a.page_size / KV_BLOCK, nb = (vis + KV_BLOCK - 1) / KV_BLOCK;
      const int* trow = a.table + (long long)b * a.table_stride;
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const int st = j & 1, blk = j * (CK / KV_BLOCK) + lane;
        const bool in = lane < CK / KV_BLOCK && blk < nb;
        const unsigned e = in ? (unsigned)trow[blk / bpp] : 0u;  // an entry outside the pool reads page 0
        const long long page = e < (unsigned long long)a.pages ? (long long)e : 0;
        if (!wait_bar_warp(&rawempty[st], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort, wc.ns)) break;
        if (lane == 0) mbar_expect_tx(&rawfull[st], (uint32_t)(min(CK / KV_BLOCK, nb - j * (CK / KV_BLOCK)) * BB));
        __syncwarp();
        if (in)
          bulk_load(smem_u32(smem + S::raw + st * S::kRaw + lane * BB),
                    a.cache + ((page * a.heads + head) * bpp + blk % bpp) * (long long)BB, BB, &rawfull[st]);
      }
    }
  } else if (warp == 15) {
    uint32_t one;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(one));
    constexpr uint32_t fmt = MmaFormat<T>::k;
    constexpr uint32_t ids = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(CK >> 3) << 17) | (8u << 24);
    constexpr uint32_t idp = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
    const uint64_t qd = sdesc(smem_u32(smem + S::q)), kd = sdesc(smem_u32(smem + S::k));
    const uint64_t vd = ndesc(smem_u32(smem + S::v), CK * 128);
    auto score = [&](int x, int st) {  // S_x = Q_x K^T
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss((uint32_t)(128 * x), qd + (uint64_t)((x * S::kTile + h * CK * 128 + 32 * k) >> 4),
                 kd + (uint64_t)((st * S::kTile + h * CK * 128 + 32 * k) >> 4), ids, (h || k) ? 1u : 0u);
    };
    auto value = [&](int x, int j) {  // O_x += P_x V
#pragma unroll
      for (int k = 0; k < CK / 16; ++k)
        mma_ts(kO + (uint32_t)(D * x), (uint32_t)(128 * x + 8 * k), vd + (uint64_t)((2048 * k) >> 4), idp,
               (j || k) ? 1u : 0u);
    };
    bool ok = steps > 0 && wait_bar_warp(&qfull, 0u, abort, wc.ns) && wait_bar_warp(&kfull[0], 0u, abort, wc.ns);
    if (ok) {
      tc_fence_after();
      if (one) {
        score(0, 0);
        mma_commit(&sfull[0]);
        if (two) {
          score(1, 0);
          mma_commit(&sfull[1]);
        }
        mma_commit(&kempty[0]);
      }
    }
#pragma unroll 1
    for (int j = 0; j < steps && ok; ++j) {
      const int nx = (j + 1) & 1;
      const bool more = j + 1 < steps;
      if (more && !(ok = wait_bar_warp(&kfull[nx], (uint32_t)((j + 1) >> 1) & 1u, abort, wc.ns))) break;
      if (!(ok = wait_bar_warp(&vfull, (uint32_t)j & 1u, abort, wc.ns))) break;
      if (!(ok = wait_bar_warp(&pfull[0], (uint32_t)j & 1u, abort, wc.ns))) break;
      tc_fence_after();
      if (one) {
        value(0, j);
        if (!two) mma_commit(&vempty);
        if (more) score(0, nx);
        mma_commit(&sfull[0]);
        if (!two && more) mma_commit(&kempty[nx]);
      }
      if (two) {
        if (!(ok = wait_bar_warp(&pfull[1], (uint32_t)j & 1u, abort, wc.ns))) break;
        tc_fence_after();
        if (one) {
          value(1, j);
          mma_commit(&vempty);
          if (more) score(1, nx);
          mma_commit(&sfull[1]);
          if (more) mma_commit(&kempty[nx]);
        }
      }
      __syncwarp();
    }
    if (!ok && steps > 0) {
      // Whatever was issued has to end before the memory is given back.
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 200000ull) {
      }
    }
  }
  __syncthreads();
  if (abort_sh) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, 2u);
  }
  tc_fence_after();
  if (warp == 15)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base_sh), "r"(512u) : "memory");
}

template <class T, int D>
gptq_status chunk_launch(const AttnArgs& a, cudaStream_t s) {
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_chunk<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkSmem<D>::bytes));
    return GPTQ_OK;
  }));
  const long long nblk = ((long long)a.max_q * a.group + CROWS - 1) / CROWS;
  constexpr int kSeqs = 65535;
  for (int b0 = 0; b0 < a.seqs; b0 += kSeqs) {
    AttnArgs p = a;
    p.seqs = a.seqs - b0 < kSeqs ? a.seqs - b0 : kSeqs;
    p.table += (long long)b0 * a.table_stride;
    p.kv_lens += b0;
    p.q_starts += b0;
    GQ_PROF(K_KV4_CHUNK, s);
    k_kv4_chunk<T, D><<<dim3((unsigned)a.heads, (unsigned)p.seqs, (unsigned)nblk), CTHREADS, ChunkSmem<D>::bytes, s>>>(
        p, (int)nblk, wait_cfg());
    GQ_LAUNCHED();
  }
  return GPTQ_OK;
}

}  // namespace

gptq_status kv4_chunk_run(int dtype, int dim, const AttnArgs& a, cudaStream_t s) {
  if (dim == 64)
    return dtype == GPTQ_BF16 ? chunk_launch<__nv_bfloat16, 64>(a, s) : chunk_launch<__half, 64>(a, s);
  return dtype == GPTQ_BF16 ? chunk_launch<__nv_bfloat16, 128>(a, s) : chunk_launch<__half, 128>(a, s);
}

}  // namespace gq
