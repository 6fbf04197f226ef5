// Attention over the 4-bit cache for many queries a sequence (prompt chunks),
// on tcgen05.
//
// A CTA owns 256 query rows -- (query, head of the key head's group) pairs --
// as two tiles A and B of 128, and walks the keys they see in steps of 128
// tokens.  With so many rows the products bound it (4 * 128 * D flop a row
// and step), and the decoding of the codes, done once for both tiles, and the
// exponentials run beside them:
//   warps 0-7, 8-15 softmax of tile A, B: half a row (64 scores) a thread.  The
//                   halves exchange their maxima through shared memory; P goes
//                   back over S in T, the operand A of the second product;
//   warps 16-19, 20-23  decode K, V of a step into shared memory in 128-byte
//                   swizzled rows of tokens (K is then a K-major operand, V
//                   an N-major one: no transpose);
//   warp 24         copies the step's cache blocks (untiled bulk copies);
//   warp 25         issues the products: S_A, S_B of the next step between
//                   O_A += P_A V and O_B += P_B V, so that one tile's
//                   softmax runs under the other's products.
// The (sequence, row block, key head) tiles and their steps form one list, of
// which each of the persistent CTAs takes an equal, contiguous share: a tile
// inside one share is finished there, a cut one leaves its maximum, sum and
// unnormalised output (f32) in the workspace, and k_kv4_chunk_join adds the
// pieces in the order of the list.
// Measured: 2 sequences of 2048 queries of 32 heads (8 key heads of 128),
// contexts to 8192: 335 us, 0.90 PFLOP/s, the tensor cores 46 % busy.  A step
// of a tile is a chain of 3650 cycles (maximum 440, exchange 180, exponentials
// 1400, products 1250 and their waits), of which two tiles overlap; tensor
// memory has no room for a third.
// Heads of 256 have one tile of 128 rows and steps of 64 keys: their outputs
// take half of tensor memory, and K and V of a step are as large as with 128
// keys of 128 (48 sequences of 7 queries of 8 x 16 heads, contexts to 4000: 217
// us, three times as fast as sixteen rows at a time on mma.sync).
// Tensor memory: S_A, S_B (128 columns each; P of each half of the keys over
// the first 32 columns of its scores), O_A, O_B (D columns each).
// The running maximum is only raised (and O rescaled, by its rows' threads,
// after the step's commit has shown the last product done) when it would
// grow by more than 2^8; exponentials stay within that and nothing is lost.
// Channels keep the order in which the nibbles come out (0 4 1 5 2 6 3 7 of
// every eight): q is stored to match, and the output is read back through it.
#include "serve.cuh"

namespace gq {
namespace {

// Keys a step, and query rows a CTA: heads of 256 leave tensor and shared
// memory for half of both.
template <int D>
constexpr int kKeys = D == 256 ? 64 : 128;
template <int D>
constexpr int kRows = D == 256 ? 128 : 256;
constexpr int CTHREADS = 896;
constexpr int CLIST = 512;   // (sequence, row block) pairs of one launch at most
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

// Two f32 numbers as one operand.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// Scores past column `lim` count nothing.
__device__ __forceinline__ void hide(uint32_t (&v)[32], int lim) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i > lim) v[i] = 0xff800000u;  // -inf
}

// Barrier of tile x's 256 softmax threads, AND-reducing: they go on or leave
// together.
__device__ __forceinline__ bool tile_all(int x, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.and.pred po, %2, 256, pi;\n"
      " selp.u32 %0, 1, 0, po;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(1 + x)
      : "memory");
  return r != 0u;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
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

// 16 bytes of shared memory in one load.
__device__ __forceinline__ uint4 load128(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p))
               : "memory");
  return v;
}

// Byte offset of 16-byte piece p (0 .. 7) of row r in a swizzled tile.
__device__ __forceinline__ uint32_t swz(int r, int p) { return (uint32_t)(r * 128 + ((p ^ (r & 7)) * 16)); }

template <int D>
struct ChunkSmem {  // byte offsets; 1024-byte aligned operands
  static constexpr int CK = kKeys<D>;
  static constexpr int kQTile = 128 * D * 2, kTile = CK * D * 2;  // a tile of Q; K or V of a step
  // Codes come in units of 128 groups (of K and of V): a group a decoding thread.
  static constexpr int kTokens = 128 / (D / 32), kUnits = CK / kTokens, kBlocks = kTokens / KV_BLOCK;
  static constexpr int kRaw = kBlocks * kv_block_bytes(D);
  static constexpr int q = 0;                                // its tiles
  static constexpr int k = q + kRows<D> / 128 * kQTile;      // two steps
  static constexpr int v = k + 2 * kTile;            // two steps
  static constexpr int raw = v + 2 * kTile;          // the units of one step
  static constexpr int bytes = raw + kUnits * kRaw + 1024;
};

// One (sequence, row block) pair.
struct Pair {
  int q0, nq, len, r0, rows, vis, steps;
};
template <int D>
__device__ __forceinline__ Pair pair_of(const AttnArgs& a, int b, int rb) {
  Pair t;
  t.q0 = min(max(a.q_starts[b], 0), a.tq);
  t.nq = min(min(max(a.q_starts[b + 1], t.q0), a.tq) - t.q0, a.max_q);
  t.len = (int)min((long long)max(a.kv_lens[b], 0), (long long)a.table_stride * a.page_size);
  t.r0 = rb * kRows<D>;
  t.rows = max(0, min(kRows<D>, t.nq * a.group - t.r0));
  t.vis = t.rows > 0 ? max(0, min(t.len, t.len - t.nq + (t.r0 + t.rows - 1) / a.group + 1)) : 0;
  t.steps = (t.vis + kKeys<D> - 1) / kKeys<D>;
  return t;
}
// The first token that some of the rows does not see.
__device__ __forceinline__ int open_end(const AttnArgs& a, const Pair& t) { return max(0, t.len - t.nq + t.r0 / a.group + 1); }
// Units of a tile in the list: its steps (one that writes zeros if its rows
// see nothing), and CSTART for its start and end.
__device__ __forceinline__ int units_of(const Pair& t) { return t.rows > 0 ? max(t.steps, 1) + CSTART : 0; }

// pref[i] = units of one head before pair i = (sequence i / nblk, row block
// i % nblk); pref[pairs] = all.  By every thread of the CTA.
template <int D>
__device__ void pair_prefix(const AttnArgs& a, int nblk, long long* pref, long long* scratch) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, pairs = a.seqs * nblk;
  long long before = 0;
  for (int p0 = 0; p0 < pairs; p0 += CTHREADS) {
    const int p = p0 + tid;
    const long long mine = p < pairs ? units_of(pair_of<D>(a, p / nblk, p % nblk)) : 0;
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
template <int D>
__device__ __forceinline__ Piece piece_at(const AttnArgs& a, int nblk, const long long* pref, long long u, long long uend) {
  int lo = 0, hi = a.seqs * nblk - 1;  // the last pair that starts at or before u
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (pref[mid] * a.heads <= u) lo = mid; else hi = mid - 1;
  }
  Piece p;
  p.b = lo / nblk;
  p.t = pair_of<D>(a, p.b, lo % nblk);
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

constexpr size_t piece_floats(int dim);

// A value that is no number must not meet the probability of 0 of a row that
// does not see its token: it was decoded as 0, and the rows that do see it get
// their NaN here, over what the CTA has written of each of its pieces.  By the
// softmax warps (the others have given registers away), after the steps.  (The
// share is worked out again, from what the compiler does not see through: kept
// in registers for this, which no call with numbers in its cache comes to, it
// cost the steps 2 % of their time.)
template <class T, int D>
__device__ __forceinline__ void spoil_pieces(const AttnArgs& a, int nblk, const volatile long long* prefix, int* first) {
  uint32_t cta, ctas;
  asm volatile("mov.u32 %0, %%ctaid.x;\n mov.u32 %1, %%nctaid.x;" : "=r"(cta), "=r"(ctas));
  const long long* pref = const_cast<const long long*>(prefix);
  const long long W = prefix[a.seqs * nblk] * a.heads, shares = min(W, (long long)ctas), uend = W * (cta + 1) / shares;
#pragma unroll 1
  for (long long u = W * cta / shares; u < uend;) {
    const Piece pc = piece_at<D>(a, nblk, pref, u, uend);
    u = pc.next;
    if (pc.j1 == 0) continue;
    if (threadIdx.x < D / 32) first[threadIdx.x] = INT_MAX;
    asm volatile("bar.sync 3, 512;" ::: "memory");
    const int end = min(pc.t.vis, pc.j1 * kKeys<D>);
#pragma unroll 1
    for (int t = max(open_end(a, pc.t), pc.j0 * kKeys<D>) + (int)threadIdx.x; t < end; t += 512) {
      const uint32_t* par = value_params<D>(a, pc.b, pc.head, t);
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i)
        if (no_numbers<T>(par[i])) atomicMin(&first[i], t);
    }
    asm volatile("bar.sync 3, 512;" ::: "memory");
    float* part = a.part + ((size_t)cta * 2 + (pc.j0 == 0 ? 1 : 0)) * piece_floats(D);
#pragma unroll 1
    for (int i = threadIdx.x; i < pc.t.rows * (D / 8); i += 512) {
      const int row = i / (D / 8), c = i % (D / 8) * 8, rr = pc.t.r0 + row, qi = rr / a.group;
      if (pc.t.len - pc.t.nq + qi < first[c / 32]) continue;
      if (pc.whole) {
        T* dst = static_cast<T*>(a.out) + ((long long)(pc.t.q0 + qi) * a.heads * a.group + pc.head * a.group + rr % a.group) * D;
        *reinterpret_cast<uint4*>(dst + c) = uint4{0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu};
      } else {
        float4* o = reinterpret_cast<float4*>(part + (size_t)row * D + c);
        o[0] = o[1] = float4{NAN, NAN, NAN, NAN};
      }
    }
    asm volatile("bar.sync 3, 512;" ::: "memory");
  }
}

constexpr int rows_of(int dim) { return dim == 256 ? kRows<256> : kRows<128>; }
constexpr size_t piece_floats(int dim) { return (size_t)rows_of(dim) * (dim + 2); }

// TURNS: no sequence has more than 128 rows; the two tiles hold the same rows
// and take turns at the steps, so that two chains run for them too, and join
// at the end of a piece (112 rows of 128, 8 sequences to 32000: 168 -> 144 us;
// of 64, 48 sequences: 674 -> 523; decoding is then the longer part).
template <class T, int D, bool TURNS>
__global__ void __launch_bounds__(CTHREADS, 1) k_kv4_chunk(AttnArgs a, int nblk, WaitCfg wc) {
  using T2 = typename Elem<T>::T2;
  using S = ChunkSmem<D>;
  constexpr int BB = kv_block_bytes(D), HALVES = D / 64, CK = kKeys<D>;
  constexpr uint32_t kO = 256;  // tensor memory: S_A 0, S_B 128, O_A 256, O_B 256 + D
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t qfull, kfull[2], kempty[2], vfull[2], vempty[2], rawfull[4], rawempty[4], sfull[2],
      pfull[2], mfull;
  __shared__ uint32_t tmem_base_sh;
  __shared__ long long pref[CLIST + 1], scratch[CTHREADS / 32];
  __shared__ int abort_sh;
  __shared__ int spoiled, spoiled_at[D / 32];  // see spoil_pieces
  __shared__ float2 other[128];  // maximum and sum of tile B's half of the steps
  __shared__ float xmax[2][2][2][128];  // [turn][tile][half][row]: what a row's halves tell each other
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    mbar_init(&qfull, 513), mbar_init(&mfull, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 128), mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 128), mbar_init(&vempty[i], 1);
      mbar_init(&sfull[i], 1), mbar_init(&pfull[i], 256);
    }
    for (int i = 0; i < S::kUnits; ++i) mbar_init(&rawfull[i], 1), mbar_init(&rawempty[i], 8);
    abort_sh = 0, spoiled = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 25) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  pair_prefix<D>(a, nblk, pref, scratch);
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_kv4_chunk_join may set itself up
  const long long W = pref[a.seqs * nblk] * a.heads;
  const long long shares = min(W, (long long)gridDim.x);  // no share is empty
  const bool has = blockIdx.x < shares;
  if (threadIdx.x == 0) a.cuts[blockIdx.x] = int4{};  // nothing to join
  const long long ubeg = has ? W * blockIdx.x / shares : 0, uend = has ? W * (blockIdx.x + 1) / shares : 0;

  // Registers: 72 a thread at launch, 896 * 72 = 64512; then the softmax warps
  // 80, the decoding ones 72, the last four 40: 4 * 128 * 80 + 2 * 128 * 72 +
  // 128 * 40 = 64512.
  if (warp < 16) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    const int x = warp / 8, half = warp / 4 % 2, rt = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = (uint32_t)(128 * x) + lanes, to = kO + (uint32_t)(D * x + D / 2 * half) + lanes;
    // (Not 0: a hidden key is a score of -inf, and -inf times 0 is no number.)
    const float sl = fmaxf(fabsf(a.scale_log2), 1e-30f);
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale: -q
    uint32_t sph = 0u, qph = 0u, mph = 0u;  // phases of sfull[x], qfull, mfull
    uint32_t par = 0u;            // of the exchange buffer
    bool ok = true;
#pragma unroll 1
    for (long long u = ubeg; u < uend;) {
      // What the steps need of the piece; the rest is looked up again for the
      // output, to leave the registers to the scores.
      int last, j, j1;
      {
        const Piece pc = piece_at<D>(a, nblk, pref, u, uend);
        if (pc.j1 == 0) {  // no steps of the tile in this share
          u = pc.next;
          continue;
        }
        const int row = (TURNS ? 0 : 128 * x) + rt;
        const bool mine = row < pc.t.rows;
        const int rr = pc.t.r0 + min(row, pc.t.rows - 1);
        const int qi = rr / a.group, hq = pc.head * a.group + rr % a.group;
        last = mine ? pc.t.len - pc.t.nq + qi - CK / 2 * half : -1 - CK / 2 * half;  // among this thread's columns
        j = pc.j0 + (TURNS ? x : 0);
        j1 = min(pc.j1, pc.t.steps);  // (a tile that sees nothing: no steps)
        if (!TURNS && 128 * x >= pc.t.rows && x > 0) j = j1;  // nothing for tile B
        // Half of the row's q, in the nibbles' order of channels.
        const T* qp = static_cast<const T*>(a.q) + (long long)(pc.t.q0 + qi) * a.q_ts + (long long)hq * a.q_hs +
                      D / 2 * half;
        uint8_t* tile = smem + S::q + x * S::kQTile;
        constexpr int QC = D / 16 < 8 ? D / 16 : 8;  // pieces at a time
#pragma unroll 1
        for (int c0 = 0; c0 < D / 16 && x < kRows<D> / 128; c0 += QC) {
          uint4 v[QC];
#pragma unroll
          for (int c = 0; c < QC; ++c) v[c] = mine ? *reinterpret_cast<const uint4*>(qp + 8 * (c0 + c)) : uint4{};
#pragma unroll
          for (int c = 0; c < QC; ++c) {
            const int at = D / 16 * half + c0 + c;
            uint4 o = pair_order(v[c]);
            o.x ^= flip, o.y ^= flip, o.z ^= flip, o.w ^= flip;
            *reinterpret_cast<uint4*>(tile + at / 8 * (128 * 128) + swz(rt, at % 8)) = o;
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&qfull);
        // Nobody is a piece ahead of the others.
        ok = tile_all(x, wait_bar_warp(&qfull, qph, abort, wc.ns));
        if (!ok) break;
        qph ^= 1u;
      }
      float m = kNone, l = 0.f;
      bool began = false;
#pragma unroll 1
      for (; j < j1; j += TURNS ? 2 : 1) {
        ok = wait_bar_warp(&sfull[x], sph, abort, wc.ns);
        sph ^= 1u;
        const int lim = last - j * CK;  // last visible column of this half
        const bool masked = __any_sync(0xffffffffu, lim < CK / 2 - 1);
        float top = -INFINITY;
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < CK / 64; ++c) {
            uint32_t v[32];
            tmem_ld32(ts + (uint32_t)(CK / 2 * half) + 32u * (uint32_t)c, v);
            tmem_ld_wait();
            if (masked) hide(v, lim - 32 * c);
            float t2[2] = {top, fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]))};
#pragma unroll
            for (int i = 2; i < 32; i += 2)
              t2[i / 2 & 1] = max3(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), t2[i / 2 & 1]);
            top = fmaxf(t2[0], t2[1]);
          }
          xmax[par][x][half][rt] = top;
        }
        if (!(ok = tile_all(x, ok))) break;
        top = fmaxf(top, xmax[par][x][half ^ 1][rt]);
        par ^= 1u;
        // Both halves of a row decide alike: they see the same numbers.
        if (__any_sync(0xffffffffu, sl * (top - m) > 8.f)) {
          const float nm = fmaxf(m, top), f = ex2(sl * (m - nm));
          m = nm;
          l *= f;
          if (began) {
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              uint32_t w[16];
              tmem_ld16(to + (uint32_t)c, w);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
              tmem_st16(to + (uint32_t)c, w);
            }
          }
        }
        // Two at a time: p = 2^(sl s - sl m).
        const float ms = -sl * m;
        const uint64_t sl2 = pack2(sl, sl), ms2 = pack2(ms, ms);
        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < CK / 64; ++c) {
          // (Read again: a row of 128 does not leave registers enough for the
          // number of warps that hide these latencies.)
          uint32_t v[32], p[16];
          tmem_ld32(ts + (uint32_t)(CK / 2 * half) + 32u * (uint32_t)c, v);
          tmem_ld_wait();
          if (masked) hide(v, lim - 32 * c);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = unpack2(fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sl2, ms2));
            const float e0 = ex2(e.x), e1 = ex2(e.y);
            sum2[i & 1] = add2(sum2[i & 1], pack2(e0, e1));
            p[i] = bits2(Elem<T>::make2(e0, e1));
          }
          tmem_st16(ts + (uint32_t)(CK / 2 * half) + 16u * (uint32_t)c, p);
        }
        const float2 s0 = unpack2(sum2[0]), s1 = unpack2(sum2[1]);
        l += (s0.x + s0.y) + (s1.x + s1.y);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_relaxed(&pfull[x]);
        began = true;
      }
      if (!ok) break;
      // The output, once the last product is done; the halves' sums meet.
      if (began) {
        ok = wait_bar_warp(&sfull[x], sph, abort, wc.ns);
        sph ^= 1u;
      }
      xmax[par][x][half][rt] = l;
      if (!(ok = tile_all(x, ok))) break;
      l += xmax[par][x][half ^ 1][rt];
      par ^= 1u;
      float fa = 1.f, fb = 0.f;  // weights of the tiles' outputs
      const Piece pc = piece_at<D>(a, nblk, pref, u, uend);
      u = pc.next;
      if (TURNS) {
        if (x == 1) {
          if (half == 0) {
            other[rt] = float2{m, l};
            tc_fence_before();
            mbar_arrive(&mfull);
          }
          continue;  // (the next piece's q waits for tile A's threads)
        }
        ok = tile_all(x, wait_bar_warp(&mfull, mph, abort, wc.ns));
        if (!ok) break;
        mph ^= 1u;
        const float2 ml = other[rt];
        const float nm = fmaxf(m, ml.x);
        fa = ex2(sl * (m - nm)), fb = ex2(sl * (ml.x - nm));
        l = l * fa + ml.y * fb;
        m = nm;
      }
      tc_fence_after();
      if (threadIdx.x == 0 && pc.j0 == 0 && !pc.whole) {  // a cut tile's first piece: the join's work
        const long long w = pref[a.seqs * nblk] * a.heads, n = min(w, (long long)gridDim.x);
        const int lastc = (int)(((u + units_of(pc.t) - CSTART - pc.j1) * n - 1) / w);  // its last unit's share
        a.cuts[blockIdx.x] = int4{pc.t.q0, pc.t.r0, pc.head << 9 | pc.t.rows, lastc};
      }
      if (x > 0 && pc.t.rows <= 128) continue;
      const bool mine = 128 * x + rt < pc.t.rows;
      const int rr = pc.t.r0 + min(128 * x + rt, pc.t.rows - 1);
      const int qi = rr / a.group, hq = pc.head * a.group + rr % a.group;
      const float inv = l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing: zeros
      T* dst = static_cast<T*>(a.out) + ((long long)(pc.t.q0 + qi) * a.heads * a.group + hq) * D + D / 2 * half;
      float* part = a.part + ((size_t)blockIdx.x * 2 + (pc.j0 == 0 ? 1 : 0)) * piece_floats(D);
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t v[16];
        if (began) {
          tmem_ld16(to + (uint32_t)c, v);
          tmem_ld_wait();
        }
        if (TURNS && min(pc.j1, pc.t.steps) - pc.j0 > 1) {  // tile B had a step: so had this one
          uint32_t w[16];
          tmem_ld16(to + (uint32_t)(D + c), w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = __float_as_uint(__uint_as_float(v[i]) * fa + __uint_as_float(w[i]) * fb);
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
            float4* o = reinterpret_cast<float4*>(part + (size_t)(128 * x + rt) * D + D / 2 * half + c + 8 * h);
            o[0] = float4{e[0], e[1], e[2], e[3]};
            o[1] = float4{e[4], e[5], e[6], e[7]};
          }
        }
      }
      if (!pc.whole && mine && half == 0)
        *reinterpret_cast<float2*>(part + (size_t)kRows<D> * D + 2 * (128 * x + rt)) = float2{m, l};
      tc_fence_before();
    }
  } else if (warp < 24) {
    // Four warps decode K, four V: a thread takes 32 channels (one group) of
    // a token of each unit, 16 bytes of codes to 64 bytes.  Lanes of the upper
    // half of the channels store their pieces in another order: eight lanes
    // then meet no bank twice.
    const int dt = threadIdx.x & 127;
    const bool isv = warp >= 20;
    constexpr int GR = D / 32;  // groups a token
    const int grp = dt % GR, tok = dt / GR;
    const int turn = GR == 8 ? grp / 2 : GR == 4 ? grp / 2 * 2 : 0;
    uint32_t off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      off[u] = (uint32_t)(grp / 2 * (CK * 128)) + swz(tok, grp % 2 * 4 + (u ^ turn));
    const uint8_t* from = smem + S::raw + tok / KV_BLOCK * BB + (isv ? kv_value_off(D) : 0);
    const uint8_t* from_codes = from + tok % KV_BLOCK * (D / 2) + grp * 16;
    const uint8_t* from_par = from + kv_param_off(D) + tok % KV_BLOCK * (D / 8) + grp * 4;
    uint64_t* full = isv ? vfull : kfull;
    uint64_t* empty = isv ? vempty : kempty;
    bool ok = true;
    int n = 0;  // steps so far
#pragma unroll 1
    for (long long u = ubeg; u < uend && ok;) {
      const Piece pc = piece_at<D>(a, nblk, pref, u, uend);
      u = pc.next;
      const int open = open_end(a, pc.t) - tok;  // tokens from this thread's on that every row sees
#pragma unroll 1
      for (int j = pc.j0; j < min(pc.j1, pc.t.steps); ++j, ++n) {
        const int st = n & 1;
        if (!(ok = wait_bar_warp(&empty[st], ((uint32_t)(n >> 1) & 1u) ^ 1u, abort, wc.ns))) break;
        uint8_t* tile = smem + (isv ? S::v : S::k) + st * S::kTile;
        const int seen = pc.t.vis - j * CK - tok;  // tokens from this thread's on that some row sees
#pragma unroll 1
        for (int q = 0; q < S::kUnits; ++q) {
          if (!(ok = wait_bar_warp(&rawfull[q], (uint32_t)n & 1u, abort, wc.ns))) break;
          uint4 codes = load128(from_codes + q * S::kRaw);
          uint32_t par = *reinterpret_cast<const uint32_t*>(from_par + q * S::kRaw);
          if (j * CK + q * S::kTokens >= open) {
            if (q * S::kTokens >= seen) {
              par = 0u;  // past what any row sees: no value, whatever is there
            } else if (isv && no_numbers<T>(par)) {
              par = 0u;
              spoiled = 1;
            }
          }
          if (GR >= 4) {
            const bool two = (turn & 2) != 0;
            const uint4 c = codes;
            codes.x = two ? c.z : c.x, codes.y = two ? c.w : c.y;
            codes.z = two ? c.x : c.z, codes.w = two ? c.y : c.w;
          }
          if (GR == 8) {
            const bool one = (turn & 1) != 0;
            const uint4 c = codes;
            codes.x = one ? c.y : c.x, codes.y = one ? c.x : c.y;
            codes.z = one ? c.w : c.z, codes.w = one ? c.z : c.w;
          }
          const T2 s2 = from_bits2<T2>(__byte_perm(par, par, 0x1010)), z2 = from_bits2<T2>(__byte_perm(par, par, 0x3232));
          const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
          uint8_t* dst = tile + q * S::kTokens * 128;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 o;
            o.x = bits2(__hfma2(code16<T>(w[e], 0, a.up), s2, z2));
            o.y = bits2(__hfma2(code16<T>(w[e], 1), s2, z2));
            o.z = bits2(__hfma2(code16<T>(w[e], 2), s2, z2));
            o.w = bits2(__hfma2(code16<T>(w[e], 3), s2, z2));
            *reinterpret_cast<uint4*>(dst + off[e]) = o;
            // Not before this store, which needs both loads: an arrival does not wait
            // for loads in flight, and the next copy overtook them (one unit of a warp
            // in some 10 million held the next step's tokens).  After all four stores
            // it costs 1 to 2 % more.
            if (e == 0) {
              __syncwarp();
              if (lane == 0) mbar_arrive(&rawempty[q]);
            }
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        mbar_arrive(&full[st]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  }
  if (warp == 24) {
    if (!wc.no_loads) {
      const int bpp = a.page_size / KV_BLOCK;
      bool ok = true;
      int n = 0;
#pragma unroll 1
      for (long long u = ubeg; u < uend && ok;) {
        const Piece pc = piece_at<D>(a, nblk, pref, u, uend);
        u = pc.next;
        const int nb = (pc.t.vis + KV_BLOCK - 1) / KV_BLOCK;
        const int* trow = a.table + (long long)pc.b * a.table_stride;
#pragma unroll 1
        for (int j = pc.j0; j < min(pc.j1, pc.t.steps); ++j, ++n) {
          const int blk = j * (CK / KV_BLOCK) + lane;
          const bool in = lane < CK / KV_BLOCK && blk < nb;
          const unsigned e = in ? (unsigned)trow[blk / bpp] : 0u;  // an entry outside the pool reads page 0
          const long long page = e < (unsigned long long)a.pages ? (long long)e : 0;
          const uint8_t* src = a.cache + ((page * a.heads + pc.head) * bpp + blk % bpp) * (long long)BB;
#pragma unroll 1
          for (int q = 0; q < S::kUnits; ++q) {
            if (!(ok = wait_bar_warp(&rawempty[q], ((uint32_t)n & 1u) ^ 1u, abort, wc.ns))) break;
            const int have = min(max(nb - j * (CK / KV_BLOCK) - q * S::kBlocks, 0), S::kBlocks);
            if (lane == 0) {
              if (have > 0)
                mbar_expect_tx(&rawfull[q], (uint32_t)(have * BB));
              else
                mbar_arrive(&rawfull[q]);  // nothing of the unit is seen
            }
            __syncwarp();
            if (in && lane / S::kBlocks == q)
              bulk_load(smem_u32(smem + S::raw + lane * BB), src, BB, &rawfull[q]);
          }
          if (!ok) break;
        }
      }
    }
  } else if (warp == 25) {
    const bool one = elect_one();
    constexpr uint32_t fmt = MmaFormat<T>::k;
    constexpr uint32_t ids = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(CK >> 3) << 17) | (8u << 24);
    constexpr uint32_t idp = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
    const uint64_t qd = sdesc(smem_u32(smem + S::q)), kd = sdesc(smem_u32(smem + S::k));
    const uint64_t vd0 = ndesc(smem_u32(smem + S::v), CK * 128);
    auto score = [&](int x, int st) {  // S_x = Q_x K^T
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss((uint32_t)(128 * x), qd + (uint64_t)((x * S::kQTile + h * 128 * 128 + 32 * k) >> 4),
                 kd + (uint64_t)((st * S::kTile + h * CK * 128 + 32 * k) >> 4), ids, (h || k) ? 1u : 0u);
    };
    auto value = [&](int x, int st, int j) {  // O_x += P_x V
      const uint64_t vd = vd0 + (uint64_t)((st * S::kTile) >> 4);
#pragma unroll
      for (int k = 0; k < CK / 16; ++k)
        mma_ts(kO + (uint32_t)(D * x), (uint32_t)(128 * x + k / (CK / 32) * (CK / 2) + k % (CK / 32) * 8), vd + (uint64_t)((2048 * k) >> 4), idp,
               (j || k) ? 1u : 0u);
    };
    bool ok = true;
    int n = 0;                               // steps so far
    uint32_t qph = 0u, pph[2] = {0u, 0u};    // phases of qfull, pfull
#pragma unroll 1
    for (long long u = ubeg; u < uend && ok;) {
      const Piece pc = piece_at<D>(a, nblk, pref, u, uend);
      u = pc.next;
      if (pc.j1 == 0) continue;
      const int count = min(pc.j1, pc.t.steps) - pc.j0;
      const bool two = pc.t.rows > 128;
      // This warp takes part: pieces without steps wait for nothing of it, and
      // two of them ahead the phase's parity would be the old one again.
      if (lane == 0) mbar_arrive(&qfull);
      if (!(ok = wait_bar_warp(&qfull, qph, abort, wc.ns))) break;
      qph ^= 1u;
      if (count <= 0) continue;
      if (!(ok = wait_bar_warp(&kfull[n & 1], (uint32_t)(n >> 1) & 1u, abort, wc.ns))) break;
      tc_fence_after();
      if (TURNS) {
        // Steps in turn: the next but one's scores behind a step's output.
        auto begin = [&](int x, int st) {
          score(x, st);
          mma_commit(&sfull[x]);
          mma_commit(&kempty[st]);
        };
        if (one) begin(0, n & 1);
        __syncwarp();
        if (count > 1) {
          if (!(ok = wait_bar_warp(&kfull[(n + 1) & 1], (uint32_t)((n + 1) >> 1) & 1u, abort, wc.ns))) break;
          tc_fence_after();
          if (one) begin(1, (n + 1) & 1);
          __syncwarp();
        }
#pragma unroll 1
        for (int j = 0; j < count; ++j, ++n) {
          const int x = j & 1, st = n & 1;
          if (!(ok = wait_bar_warp(&vfull[st], (uint32_t)(n >> 1) & 1u, abort, wc.ns))) break;
          if (!(ok = wait_bar_warp(&pfull[x], pph[x], abort, wc.ns))) break;
          pph[x] ^= 1u;
          tc_fence_after();
          if (one) {
            value(x, st, j > 1);
            mma_commit(&vempty[st]);
            if (j + 2 >= count) mma_commit(&sfull[x]);
          }
          __syncwarp();
          if (j + 2 < count) {
            if (!(ok = wait_bar_warp(&kfull[st], (uint32_t)((n + 2) >> 1) & 1u, abort, wc.ns))) break;
            tc_fence_after();
            if (one) begin(x, st);
            __syncwarp();
          }
        }
        continue;
      }
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
        if (!(ok = wait_bar_warp(&vfull[n & 1], (uint32_t)(n >> 1) & 1u, abort, wc.ns))) break;
        if (!(ok = wait_bar_warp(&pfull[0], pph[0], abort, wc.ns))) break;
        pph[0] ^= 1u;
        tc_fence_after();
        if (one) {
          value(0, n & 1, j);
          if (!two) mma_commit(&vempty[n & 1]);
          if (more) score(0, nx);
          mma_commit(&sfull[0]);
          if (!two && more) mma_commit(&kempty[nx]);
        }
        if (two) {
          if (!(ok = wait_bar_warp(&pfull[1], pph[1], abort, wc.ns))) break;
          pph[1] ^= 1u;
          tc_fence_after();
          if (one) {
            value(1, n & 1, j);
            mma_commit(&vempty[n & 1]);
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
  if (__builtin_expect(spoiled != 0, 0) && warp < 16) spoil_pieces<T, D>(a, nblk, pref, spoiled_at);
  tc_fence_after();
  if (warp == 25)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base_sh), "r"(512u) : "memory");
}

// Adds the pieces of the tiles that more than one CTA shared: block (c, i)
// those of the tile whose first piece share c ends with, sixteen rows of it
// (heads of 256: eight), a warp RW, whose pieces come through shared memory
// four at a time.
template <class T, int D>
__global__ void __launch_bounds__(128) k_kv4_chunk_join(AttnArgs a) {
  constexpr int RW = D == 256 ? 2 : 4;
  __shared__ __align__(16) float batch[4][4 * RW][D];  // [warp][piece, row]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, first = (int)blockIdx.x;
  zero_other_rows<T, D>(a, (int)(blockIdx.y * gridDim.x + blockIdx.x), (int)(gridDim.x * gridDim.y));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the cuts and the pieces are there
  const int4 cut = a.cuts[first];
  const int head = cut.z >> 9, rows = cut.z & 511, lastc = cut.w;
  const int r0 = ((int)blockIdx.y * 4 + warp) * RW;
  if (r0 >= rows) return;
  const float sl = fmaxf(fabsf(a.scale_log2), 1e-30f);
  auto slot = [&](int c) { return a.part + ((size_t)c * 2 + (c == first ? 1 : 0)) * piece_floats(D); };
  float top = kNone, den = 0.f;  // of row r0 + lane % RW
  float acc[RW][D / 32];
#pragma unroll
  for (int k = 0; k < RW; ++k)
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[k][i] = 0.f;
#pragma unroll 1
  for (int c0 = first; c0 <= lastc; c0 += 4) {
    const int pieces = min(4, lastc + 1 - c0);  // (rows past the tile's are the workspace's all the same)
    for (int i = lane; i < pieces * RW * (D / 4); i += 32)
      cp_async16(&batch[warp][i / (D / 4)][i % (D / 4) * 4],
                 slot(c0 + i / (RW * (D / 4))) + (size_t)(r0 + i / (D / 4) % RW) * D + i % (D / 4) * 4);
    float2 ml{kNone, 0.f};
    if (lane < RW * pieces)
      ml = *reinterpret_cast<const float2*>(slot(c0 + lane / RW) + (size_t)kRows<D> * D + 2 * (r0 + lane % RW));
    float nt = fmaxf(ml.x, top);
#pragma unroll
    for (int x = RW; x < 32; x <<= 1) nt = fmaxf(nt, __shfl_xor_sync(0xffffffffu, nt, x));
    const float f = ex2(sl * (ml.x - nt)), fo = ex2(sl * (top - nt));
    float l = ml.y * f;
#pragma unroll
    for (int x = RW; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    top = nt;
    den = fmaf(den, fo, l);
    cp_async_wait_all();
    __syncwarp();
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const float fk = __shfl_sync(0xffffffffu, fo, k);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[k][i] *= fk;
    }
    for (int c = 0; c < pieces; ++c)
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, RW * c + k);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[k][i] = fmaf(batch[warp][RW * c + k][lane + 32 * i], fk, acc[k][i]);
      }
    __syncwarp();  // the batch is read
  }
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    const float dk = __shfl_sync(0xffffffffu, den, k);
    if (r0 + k >= rows) continue;
    const float inv = dk != 0.f ? 1.f / dk : 0.f;  // a row that sees nothing: zeros
    const int rr = cut.y + r0 + k;
    T* dst = static_cast<T*>(a.out) +
             ((long long)(cut.x + rr / a.group) * a.heads * a.group + head * a.group + rr % a.group) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dst[lane + 32 * i] = Elem<T>::from(acc[k][i] * inv);
  }
}

template <class T, int D, bool TURNS>
gptq_status chunk_launch(const AttnArgs& a, cudaStream_t s) {
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_chunk<T, D, TURNS>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkSmem<D>::bytes));
    return GPTQ_OK;
  }));
  const int nblk = (int)(((long long)a.max_q * a.group + kRows<D> - 1) / kRows<D>);
  const int per = CLIST / nblk;  // sequences of a launch
  for (int b0 = 0; b0 < a.seqs; b0 += per) {
    AttnArgs p = a;
    p.seqs = a.seqs - b0 < per ? a.seqs - b0 : per;
    p.table += (long long)b0 * a.table_stride;
    p.kv_lens += b0;
    p.q_starts += b0;
    p.first = b0 == 0, p.last = b0 + p.seqs == a.seqs;
    const int grid = num_sms();
    {
      GQ_PROF(K_KV4_CHUNK, s);
      k_kv4_chunk<T, D, TURNS><<<grid, CTHREADS, ChunkSmem<D>::bytes, s>>>(p, nblk, wait_cfg());
      GQ_LAUNCHED();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, 16);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    GQ_PROF(K_KV4_JOIN, s);
    GQ_CUDA(cudaLaunchKernelEx(&cfg, k_kv4_chunk_join<T, D>, p));
  }
  return GPTQ_OK;
}

}  // namespace

size_t kv4_chunk_ws_bytes(int dim) { return kCutBytes + (size_t)num_sms() * 2 * piece_floats(dim) * 4; }

template <class T>
static gptq_status chunk_dim(int dim, const AttnArgs& a, cudaStream_t s) {
  const bool turns = (long long)a.max_q * a.group <= 128;
  if (dim == 64) return turns ? chunk_launch<T, 64, true>(a, s) : chunk_launch<T, 64, false>(a, s);
  if (dim == 128) return turns ? chunk_launch<T, 128, true>(a, s) : chunk_launch<T, 128, false>(a, s);
  return chunk_launch<T, 256, false>(a, s);
}

gptq_status kv4_chunk_run(int dtype, int dim, const AttnArgs& a, cudaStream_t s) {
  return dtype == GPTQ_BF16 ? chunk_dim<__nv_bfloat16>(dim, a, s) : chunk_dim<__half>(dim, a, s);
}

}  // namespace gq
