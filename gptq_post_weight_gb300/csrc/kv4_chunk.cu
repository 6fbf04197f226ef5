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
// The (sequence, row block, key head) tiles and their steps form one list, of
// which each of the persistent CTAs takes an equal, contiguous share: a tile
// inside one share is finished there, a cut one leaves its maximum, sum and
// unnormalised output (f32) in the workspace, and k_kv4_chunk_join adds the
// pieces in the order of the list.
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
constexpr int CLIST = 2048;  // (sequence, row block) pairs of one launch at most
constexpr int CSTART = 3;    // what a tile's start and end cost, in steps
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

// One (sequence, row block) pair.
struct Pair {
  int q0, nq, len, r0, rows, vis, steps;
};
__device__ __forceinline__ Pair pair_of(const AttnArgs& a, int b, int rb) {
  Pair t;
  t.q0 = min(max(a.q_starts[b], 0), a.tq);
  t.nq = min(min(max(a.q_starts[b + 1], t.q0), a.tq) - t.q0, a.max_q);
  t.len = (int)min((long long)max(a.kv_lens[b], 0), (long long)a.table_stride * a.page_size);
  t.r0 = rb * CROWS;
  t.rows = max(0, min(CROWS, t.nq * a.group - t.r0));
  t.vis = t.rows > 0 ? max(0, min(t.len, t.len - t.nq + (t.r0 + t.rows - 1) / a.group + 1)) : 0;
  t.steps = (t.vis + CK - 1) / CK;
  return t;
}
// Units of a tile in the list: its steps (one that writes zeros if its rows
// see nothing), and CSTART for its start and end.
__device__ __forceinline__ int units_of(const Pair& t) { return t.rows > 0 ? max(t.steps, 1) + CSTART : 0; }

// pref[i] = units of one head before pair i = (sequence i / nblk, row block
// i % nblk); pref[pairs] = all.  By every thread of the CTA.
__device__ void pair_prefix(const AttnArgs& a, int nblk, long long* pref, long long* scratch) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, pairs = a.seqs * nblk;
  long long before = 0;
  for (int p0 = 0; p0 < pairs; p0 += CTHREADS) {
    const int p = p0 + tid;
    const long long mine = p < pairs ? units_of(pair_of(a, p / nblk, p % nblk)) : 0;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    long long base = before + inc - mine;
    for (int w = 0; w < CTHREADS / 32; ++w) {
      if (w < warp) base += scratch[w];
      before += scratch[w];
    }
    if (p < pairs) pref[p] = base;
    __syncthreads();
  }
  if (tid == 0) pref[pairs] = before;
  __syncthreads();
}

// A piece of the list: units up to `next`; steps j0 .. j1 - 1 of a tile (none
// where j1 == 0).
struct Piece {
  Pair t;
  int b, head, j0, j1;
  bool whole;
  long long next;
};
__device__ __forceinline__ Piece piece_at(const AttnArgs& a, int nblk, const long long* pref, long long u, long long uend) {
  int lo = 0, hi = a.seqs * nblk - 1;  // the last pair that starts at or before u
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (pref[mid] * a.heads <= u) lo = mid; else hi = mid - 1;
  }
  Piece p;
  p.b = lo / nblk;
  p.t = pair_of(a, p.b, lo % nblk);
  const int n = units_of(p.t);
  const long long rem = u - pref[lo] * a.heads;
  int at;
  if (rem >> 31 == 0) {
    p.head = (int)((unsigned)rem / (unsigned)n);
    at = (int)((unsigned)rem % (unsigned)n);
  } else {
    p.head = (int)(rem / n);
    at = (int)(rem % n);
  }
  const int end = (int)min((long long)n, at + (uend - u));
  p.next = u + (end - at);
  p.j0 = max(at - CSTART, 0);
  p.j1 = max(end - CSTART, 0);
  p.whole = p.j0 == 0 && p.j1 == n - CSTART;
  return p;
}

constexpr size_t piece_floats(int dim) { return (size_t)CROWS * (dim + 2); }

template <class T, int D>
__global__ void __launch_bounds__(CTHREADS, 1) k_kv4_chunk(AttnArgs a, int nblk, WaitCfg wc) {
  using T2 = typename Elem<T>::T2;
  using S = ChunkSmem<D>;
  constexpr int BB = kv_block_bytes(D), HALVES = D / 64;
  constexpr uint32_t kO = 256;  // tensor memory: S_A 0, S_B 128, O_A 256, O_B 256 + D
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t qfull, kfull[2], kempty[2], vfull, vempty, rawfull[2], rawempty[2], sfull[2],
      pfull[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ long long pref[CLIST + 1], scratch[CTHREADS / 32];
  __shared__ int abort_sh;
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

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
  pair_prefix(a, nblk, pref, scratch);
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_kv4_chunk_join may set itself up
  const long long W = pref[a.seqs * nblk] * a.heads;
  const long long shares = min(W, (long long)gridDim.x);  // no share is empty
  const bool has = blockIdx.x < shares;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.seqs * nblk; i += CTHREADS) a.list[i] = pref[i];  // for the join
  const long long ubeg = has ? W * blockIdx.x / shares : 0, uend = has ? W * (blockIdx.x + 1) / shares : 0;

  // Registers: 128 a thread at launch (512 threads); a softmax thread keeps a
  // row of scores, 2 * 128 * 184 + 2 * 128 * 72 = 65536 in all.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int x = warp / 4, rt = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = (uint32_t)(128 * x) + lanes, to = kO + (uint32_t)(D * x) + lanes;
    // (Not 0: a hidden key is a score of -inf, and -inf times 0 is no number.)
    const float sl = fmaxf(fabsf(a.scale_log2), 1e-30f);
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale: -q
    uint32_t sph = 0u, qph = 0u;  // phases of sfull[x], qfull
    bool ok = true;
#pragma unroll 1
    for (long long u = ubeg; u < uend && ok;) {
      // What the steps need of the piece; the rest is looked up again for the
      // output, to leave the registers to the scores.
      int last, j, j1;
      bool active;
      {
        const Piece pc = piece_at(a, nblk, pref, u, uend);
        if (pc.j1 == 0) {  // no steps of the tile in this share
          u = pc.next;
          continue;
        }
        const bool mine = 128 * x + rt < pc.t.rows;
        const int rr = pc.t.r0 + min(128 * x + rt, pc.t.rows - 1);
        const int qi = rr / a.group, hq = pc.head * a.group + rr % a.group;
        last = mine ? pc.t.len - pc.t.nq + qi : -1;
        j = pc.j0;
        j1 = min(pc.j1, pc.t.steps);  // (a tile that sees nothing: no steps)
        active = x == 0 || pc.t.rows > 128;
        // The row's q, in the nibbles' order of channels.
        const T* qp = static_cast<const T*>(a.q) + (long long)(pc.t.q0 + qi) * a.q_ts + (long long)hq * a.q_hs;
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
        // Nobody is a piece ahead of the others.
        if (!(ok = wait_bar_warp(&qfull, qph, abort, wc.ns))) break;
        qph ^= 1u;
      }
      float m = kNone, l = 0.f;
      bool began = false;
#pragma unroll 1
      for (; active && j < j1; ++j) {
        if (!(ok = wait_bar_warp(&sfull[x], sph, abort, wc.ns))) break;
        sph ^= 1u;
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
          if (began) {
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
        began = true;
      }
      // The output, once the last product is done.
      if (ok && began) {
        ok = wait_bar_warp(&sfull[x], sph, abort, wc.ns);
        sph ^= 1u;
      }
      if (!ok) break;
      tc_fence_after();
      const Piece pc = piece_at(a, nblk, pref, u, uend);
      u = pc.next;
      if (!active) continue;
      const bool mine = 128 * x + rt < pc.t.rows;
      const int rr = pc.t.r0 + min(128 * x + rt, pc.t.rows - 1);
      const int qi = rr / a.group, hq = pc.head * a.group + rr % a.group;
      const float inv = l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing: zeros
      T* dst = static_cast<T*>(a.out) + ((long long)(pc.t.q0 + qi) * a.heads * a.group + hq) * D;
      float* part = a.part + ((size_t)blockIdx.x * 2 + (pc.j0 == 0 ? 1 : 0)) * piece_floats(D);
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t v[16];
        if (began) {
          tmem_ld16(to + (uint32_t)c, v);
          tmem_ld_wait();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float e[8];  // columns 0 .. 7 hold channels 0 4 1 5 2 6 3 7
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = l != 0.f ? __uint_as_float(v[8 * h + (i < 4 ? 2 * i : 2 * i - 7)]) : 0.f;
          if (!mine) continue;
          if (pc.whole) {
            uint4 o;
            o.x = bits2(Elem<T>::make2(e[0] * inv, e[1] * inv));
            o.y = bits2(Elem<T>::make2(e[2] * inv, e[3] * inv));
            o.z = bits2(Elem<T>::make2(e[4] * inv, e[5] * inv));
            o.w = bits2(Elem<T>::make2(e[6] * inv, e[7] * inv));
            *reinterpret_cast<uint4*>(dst + c + 8 * h) = o;
          } else {
            float4* o = reinterpret_cast<float4*>(part + (size_t)(128 * x + rt) * D + c + 8 * h);
            o[0] = float4{e[0], e[1], e[2], e[3]};
            o[1] = float4{e[4], e[5], e[6], e[7]};
          }
        }
      }
      if (!pc.whole && mine)
        *reinterpret_cast<float2*>(part + (size_t)CROWS * D + 2 * (128 * x + rt)) = float2{m, l};
      tc_fence_before();
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
    int n = 0;  // steps so far
#pragma unroll 1
    for (long long u = ubeg; u < uend && ok;) {
      const Piece pc = piece_at(a, nblk, pref, u, uend);
      u = pc.next;
#pragma unroll 1
      for (int j = pc.j0; j < min(pc.j1, pc.t.steps); ++j, ++n) {
        const int st = n & 1;
        if (!(ok = wait_bar_warp(&rawfull[st], (uint32_t)(n >> 1) & 1u, abort, wc.ns))) break;
        ok = isv ? wait_bar_warp(&vempty, ((uint32_t)n & 1u) ^ 1u, abort, wc.ns)
                 : wait_bar_warp(&kempty[st], ((uint32_t)(n >> 1) & 1u) ^ 1u, abort, wc.ns);
        if (!ok) break;
        const uint8_t* raw = smem + S::raw + st * S::kRaw + (isv ? kv_value_off(D) : 0);
        uint8_t* tile = smem + (isv ? S::v : S::k + st * S::kTile);
        const int seen = pc.t.vis - j * CK;  // tokens of the step that some row sees
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
  }
  if (warp == 14) {
    if (!wc.no_loads) {
      const int bpp = a.page_size / KV_BLOCK;
      bool ok = true;
      int n = 0;
#pragma unroll 1
      for (long long u = ubeg; u < uend && ok;) {
        const Piece pc = piece_at(a, nblk, pref, u, uend);
        u = pc.next;
        const int nb = (pc.t.vis + KV_BLOCK - 1) / KV_BLOCK;
        const int* trow = a.table + (long long)pc.b * a.table_stride;
#pragma unroll 1
        for (int j = pc.j0; j < min(pc.j1, pc.t.steps); ++j, ++n) {
          const int st = n & 1, blk = j * (CK / KV_BLOCK) + lane;
          const bool in = lane < CK / KV_BLOCK && blk < nb;
          const unsigned e = in ? (unsigned)trow[blk / bpp] : 0u;  // an entry outside the pool reads page 0
          const long long page = e < (unsigned long long)a.pages ? (long long)e : 0;
          if (!(ok = wait_bar_warp(&rawempty[st], ((uint32_t)(n >> 1) & 1u) ^ 1u, abort, wc.ns))) break;
          if (lane == 0) mbar_expect_tx(&rawfull[st], (uint32_t)(min(CK / KV_BLOCK, nb - j * (CK / KV_BLOCK)) * BB));
          __syncwarp();
          if (in)
            bulk_load(smem_u32(smem + S::raw + st * S::kRaw + lane * BB),
                      a.cache + ((page * a.heads + pc.head) * bpp + blk % bpp) * (long long)BB, BB, &rawfull[st]);
        }
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
    bool ok = true;
    int n = 0;                               // steps so far
    uint32_t qph = 0u, pph[2] = {0u, 0u};    // phases of qfull, pfull
#pragma unroll 1
    for (long long u = ubeg; u < uend && ok;) {
      const Piece pc = piece_at(a, nblk, pref, u, uend);
      u = pc.next;
      if (pc.j1 == 0) continue;
      const int count = min(pc.j1, pc.t.steps) - pc.j0;
      const bool two = pc.t.rows > 128;
      if (!(ok = wait_bar_warp(&qfull, qph, abort, wc.ns))) break;
      qph ^= 1u;
      if (count <= 0) continue;
      if (!(ok = wait_bar_warp(&kfull[n & 1], (uint32_t)(n >> 1) & 1u, abort, wc.ns))) break;
      tc_fence_after();
      if (one) {
        score(0, n & 1);
        mma_commit(&sfull[0]);
        if (two) {
          score(1, n & 1);
          mma_commit(&sfull[1]);
        }
        mma_commit(&kempty[n & 1]);
      }
#pragma unroll 1
      for (int j = 0; j < count; ++j, ++n) {
        const int nx = (n + 1) & 1;
        const bool more = j + 1 < count;
        if (more && !(ok = wait_bar_warp(&kfull[nx], (uint32_t)((n + 1) >> 1) & 1u, abort, wc.ns))) break;
        if (!(ok = wait_bar_warp(&vfull, (uint32_t)n & 1u, abort, wc.ns))) break;
        if (!(ok = wait_bar_warp(&pfull[0], pph[0], abort, wc.ns))) break;
        pph[0] ^= 1u;
        tc_fence_after();
        if (one) {
          value(0, j);
          if (!two) mma_commit(&vempty);
          if (more) score(0, nx);
          mma_commit(&sfull[0]);
          if (!two && more) mma_commit(&kempty[nx]);
        }
        if (two) {
          if (!(ok = wait_bar_warp(&pfull[1], pph[1], abort, wc.ns))) break;
          pph[1] ^= 1u;
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
    }
    if (!ok) {
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

// Adds the pieces of a tile that more than one CTA shared: a CTA takes 32
// rows of a (pair, head) tile, a warp a row at a time.
template <class T, int D>
__global__ void __launch_bounds__(256) k_kv4_chunk_join(AttnArgs a, int nblk, int grid) {
  const int p = (int)blockIdx.x / a.heads, head = (int)blockIdx.x % a.heads;
  const Pair t = pair_of(a, p / nblk, p % nblk);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the list and the pieces are there
  const int r1 = min(t.rows, ((int)blockIdx.y + 1) * 32);
  if ((int)blockIdx.y * 32 >= r1) return;
  // The shares of the first and the last step.
  const int n = units_of(t);
  const long long W = a.list[a.seqs * nblk] * a.heads, u0 = a.list[p] * a.heads + (long long)head * n;
  const long long shares = min(W, (long long)grid);
  const int first = (int)(((u0 + CSTART + 1) * shares - 1) / W), lastc = (int)(((u0 + n) * shares - 1) / W);
  if (first == lastc) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const float sl = fmaxf(fabsf(a.scale_log2), 1e-30f);
  for (int r = (int)blockIdx.y * 32 + warp; r < r1; r += 8) {
    float top = kNone, den = 0.f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int c = first; c <= lastc; ++c) {
      const float* s = a.part + ((size_t)c * 2 + (c == first ? 1 : 0)) * piece_floats(D);
      const float2 ml = *reinterpret_cast<const float2*>(s + (size_t)CROWS * D + 2 * r);
      const float nt = fmaxf(top, ml.x), fo = ex2(sl * (top - nt)), fn = ex2(sl * (ml.x - nt));
      top = nt;
      den = den * fo + ml.y * fn;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] = acc[i] * fo + s[(size_t)r * D + lane + 32 * i] * fn;
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    const int rr = t.r0 + r;
    T* dst = static_cast<T*>(a.out) +
             ((long long)(t.q0 + rr / a.group) * a.heads * a.group + head * a.group + rr % a.group) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dst[lane + 32 * i] = Elem<T>::from(acc[i] * inv);
  }
}

template <class T, int D>
gptq_status chunk_launch(const AttnArgs& a, cudaStream_t s) {
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_chunk<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkSmem<D>::bytes));
    return GPTQ_OK;
  }));
  const int nblk = (int)(((long long)a.max_q * a.group + CROWS - 1) / CROWS);
  const int per = CLIST / nblk;  // sequences of a launch
  for (int b0 = 0; b0 < a.seqs; b0 += per) {
    AttnArgs p = a;
    p.seqs = a.seqs - b0 < per ? a.seqs - b0 : per;
    p.table += (long long)b0 * a.table_stride;
    p.kv_lens += b0;
    p.q_starts += b0;
    const int grid = num_sms();
    {
      GQ_PROF(K_KV4_CHUNK, s);
      k_kv4_chunk<T, D><<<grid, CTHREADS, ChunkSmem<D>::bytes, s>>>(p, nblk, wait_cfg());
      GQ_LAUNCHED();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.seqs * nblk * a.heads), CROWS / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    GQ_PROF(K_KV4_JOIN, s);
    GQ_CUDA(cudaLaunchKernelEx(&cfg, k_kv4_chunk_join<T, D>, p, nblk, grid));
  }
  return GPTQ_OK;
}

}  // namespace

size_t kv4_chunk_ws_bytes(int dim) { return kListBytes + (size_t)num_sms() * 2 * piece_floats(dim) * 4; }

gptq_status kv4_chunk_run(int dtype, int dim, const AttnArgs& a, cudaStream_t s) {
  if (dim == 64)
    return dtype == GPTQ_BF16 ? chunk_launch<__nv_bfloat16, 64>(a, s) : chunk_launch<__half, 64>(a, s);
  return dtype == GPTQ_BF16 ? chunk_launch<__nv_bfloat16, 128>(a, s) : chunk_launch<__half, 128>(a, s);
}

}  // namespace gq
