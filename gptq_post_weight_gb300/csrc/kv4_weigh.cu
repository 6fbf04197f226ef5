// What the queries of an attention call looked at: for every cached token the
// sum of its attention weights, added to a running total.
//
//   weights[b][h][t] += sum over rows r of exp(scale q_r k_t - lse_r)
//
// The logarithm of each row's sum comes from the attention itself, so that one
// pass over the keys is all it takes, and nothing of a token's sum depends on
// another token.
//
// The product is transposed, S^T = K Q^T on tcgen05: 128 keys are the rows of a
// tile (the lanes of tensor memory), the query rows its columns.  A thread that
// reads its lane then has one key's scores, and the sum over the query rows
// stays in its registers: no maximum, no exchange between lanes, and no second
// product.  A CTA fills an SM and is a line of workers; two tiles (256 keys) make
// a step:
//   crews        decode codes into 128-byte swizzled rows (operand A), once for
//                all query rows, 16 warps (many rows: 8) that take turns at the
//                tiles;
//   the last     issues the products, several steps ahead of the sums;
//   the first    8 warps (many rows: 16) take exponentials and sums, a lane
//                quarter a warp, a team for each tile of a step (many rows: two,
//                half of the columns each).
// Few rows a sequence and key head (!MANY: one column tile): a CTA takes a
// contiguous share of the list of (sequence, key head, step), a crew's next codes
// are on their way in registers, and q (operand B, in the order in which the
// nibbles come out; warp 24) stays while the head does.
// Many: steps go round the CTAs, and for each of them all the rows' tiles that
// see it come by, which the crews bring between the keys.  Where the steps are too
// few for the SMs, or a last round of them nearly empty, their rows are cut into
// parts: each leaves its sums in the workspace, and k_kv4_weigh_join adds them in
// order.
//
// Measured: 48 sequences of up to 16384 tokens, 8 key heads of 128 with 8 query
// heads each, one new token: 88.5 us, 3.4 TB/s of codes and weights.  No unit is at its
// limit (issue slots 59 %, a third of that the decoding's arithmetic; memory 34 %): the
// warps wait for one another and for their codes.  2 sequences of 2048
// queries of 32 heads, contexts to 8192: 250 us, 0.60 PFLOP/s; issue slots 63 %, shared
// memory 51, tensor cores 33, ex2 34, none of them a limit either: the products run two
// steps' sums ahead at most.  (A quarter of the exponentials as a polynomial
// made that 287: the unit for them is not what is waited for.)  One prompt's last 64
// queries of 32 heads of 64 over 4001 tokens: 9.6 us.
#include "serve.cuh"

namespace gq {
namespace {

constexpr int WKEYS = 128;           // keys of a tile; two tiles are a step, one a team
// (Registers go by eights a thread: without the warp that brings q, 80 and not 72.)
constexpr int wthreads(bool many) { return many ? 800 : 832; }
constexpr int WSEQS = 512;           // sequences of a launch at most
constexpr int WROWS = 8;             // rows' tiles whose logarithms are kept (more than WD + 2)
constexpr int WD = 4;                // steps' sums in tensor memory at most
// Tiles of keys in shared memory: a place is always the same crew's.
template <int D>
constexpr int kTurns = D == 256 ? 2 : 4;
template <int D>
constexpr int kMostRows = D == 256 ? 64 : 128;  // query rows of a tile (shared memory)

struct WeighArgs {
  const float* lse;
  float* weights;
  int nt;    // columns of a tile: a multiple of 16
  int nd;    // steps' sums in tensor memory
  int split;        // MANY: parts that a step's rows are cut into at most
  float* part;      // their sums, `apart` floats from part to part, laid out like the weights
  long long apart;
};

// wait_bar_warp, suspended for up to a microsecond a try: 26 warps that look again
// at once take the issue slots of the ones at work.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  uint64_t t0 = 0;
  bool ok = true;
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (done != 0u) break;
    if (*abort) {
      ok = false;
      break;
    }
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit) {
      *abort = 1;
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ bool look_at(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0u;
}
// Waits on three barriers at once.
__device__ __forceinline__ bool wait_three(uint64_t* x, uint32_t xp, uint64_t* y, uint32_t yp, uint64_t* z, uint32_t zp,
                                           volatile int* abort, uint64_t limit) {
  const bool ok = (look_at(x, xp) & look_at(y, yp) & look_at(z, zp)) ||
                  (wait_bar(x, xp, abort, limit) && wait_bar(y, yp, abort, limit) && wait_bar(z, zp, abort, limit));
  return __all_sync(0xffffffffu, ok);
}

// The four products of 64 channels: A and B 32 bytes on per 16 of them; first: overwrite D.
__device__ __forceinline__ void mma_keys(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool first) {
  asm volatile(
      "{\n .reg .pred p, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n setp.eq.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.u64 a1, %1, 2;\n add.u64 a2, %1, 4;\n add.u64 a3, %1, 6;\n"
      " add.u64 b1, %2, 2;\n add.u64 b2, %2, 4;\n add.u64 b3, %2, 6;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)first)
      : "memory");
}

// A sequence: first query row, queries, keys, query rows of a key head, steps of two key tiles.
struct WSeq {
  int q0, nq, len, rows, steps;
};
__device__ __forceinline__ WSeq wseq_of(const AttnArgs& a, int b) {
  WSeq s;
  s.q0 = a.q_starts != nullptr ? min(max(a.q_starts[b], 0), a.tq) : b;
  s.nq = a.q_starts != nullptr ? min(min(max(a.q_starts[b + 1], s.q0), a.tq) - s.q0, a.max_q) : 1;
  s.len = (int)min((long long)max(a.kv_lens[b], 0), (long long)a.table_stride * a.page_size);
  s.rows = s.nq * a.group;
  s.steps = s.nq > 0 ? (s.len + 2 * WKEYS - 1) / (2 * WKEYS) : 0;
  return s;
}

// x / y of numbers that mostly fit 32 bits, where a division is a quarter as long.
__device__ __forceinline__ long long quotient(long long x, int y) {
  return x >> 31 ? x / y : (long long)((unsigned)x / (unsigned)y);
}

// Query rows before the first one that sees key k.  (Cut off at 0 before the
// product: nq * group is at most 2^30, len * group is not.)
__device__ __forceinline__ int rows_before(const AttnArgs& a, const WSeq& s, int k) {
  return max(k - s.len + s.nq, 0) * a.group;
}
// The first tile of query rows that sees a key of a step.
__device__ __forceinline__ int first_rows(const AttnArgs& a, const WSeq& s, int step, int nt) {
  return rows_before(a, s, step * 2 * WKEYS) / nt;
}

// A CTA's walk over the list of (sequence, key head, step).
template <bool MANY>
struct Walk {
  const AttnArgs& a;
  const long long* pref;
  long long u, end;
  int b, head, step;
  WSeq s;
  int split, nt, seg, lo, hi;  // MANY: part of the rows, its tiles of them

  __device__ __forceinline__ Walk(const AttnArgs& args, const long long* prefix, const WeighArgs& w, int rows_of_tile)
      : a(args), pref(prefix), split(w.split), nt(rows_of_tile), seg(0), lo(0), hi(1) {
    const long long W = pref[a.seqs];
    if (MANY) {
      u = blockIdx.x;
      end = W * split;
    } else {
      u = W * blockIdx.x / gridDim.x;
      end = W * (blockIdx.x + 1) / gridDim.x;
    }
    find();
  }
  __device__ __forceinline__ bool there() const { return u < end; }
  __device__ __forceinline__ void find() {
#pragma unroll 1
    for (; u < end; u += gridDim.x) {
      const long long item = MANY && split > 1 ? quotient(u, split) : u;
      int below = 0, last = a.seqs - 1;  // the last sequence that starts at or before the item
      while (below < last) {
        const int mid = (below + last + 1) / 2;
        if (pref[mid] <= item) below = mid; else last = mid - 1;
      }
      b = below;
      s = wseq_of(a, b);
      const long long rem = item - pref[b];
      head = (int)quotient(rem, s.steps);
      step = (int)(rem - (long long)head * s.steps);
      if (!MANY) return;
      const int first = first_rows(a, s, step, nt), n = (s.rows + nt - 1) / nt - first;
      lo = first, hi = first + n;
      if (split == 1) return;
      const int parts = min(split, n);
      seg = (int)(u - item * split);
      lo = first + (int)((unsigned)(n * seg) / (unsigned)parts);  // (less than 2^24 tiles, sixteen parts)
      hi = first + (int)((unsigned)(n * (seg + 1)) / (unsigned)parts);
      if (seg < parts) return;  // (else fewer tiles of rows than parts: none here)
    }
  }
  // Steps from this one on that are neighbours in one head, `most` at most.
  __device__ __forceinline__ int run(int most) const { return MANY ? 1 : (int)min((long long)min(most, s.steps - step), end - u); }
  // On by so many steps of a run.  Whether the next one has other query rows.
  __device__ __forceinline__ bool next(int n = 1) {
    if (MANY) {
      u += gridDim.x;
      find();
      return true;
    }
    u += n;
    if ((step += n) < s.steps) return false;
    step = 0;
    if (++head == a.heads) find();
    return true;
  }
};

template <class T, int D, bool MANY>
__global__ void __launch_bounds__(wthreads(MANY), 1) k_kv4_weigh(AttnArgs a, WeighArgs w, WaitCfg wc) {
  using T2 = typename Elem<T>::T2;
  constexpr int WTHREADS = wthreads(MANY), MMA = WTHREADS / 32 - 1;  // the warp that issues the products
  constexpr int SUM = MANY ? 16 : 8;  // warps that sum
  constexpr int HALVES = D / 64, ATILE = WKEYS * D * 2, TURNS = kTurns<D>, CREW = MANY ? 128 : 512 / TURNS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t afull[TURNS], aempty[TURNS / 2], qfull[2], qempty[2], dfull[WD], dempty[WD];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ long long pref[WSEQS + 1], scratch[26];
  // Of each row of a tile: minus its logarithm of the sum (-inf past the end: its
  // exponentials are 0), and the last key that it sees.  Written with the tile, read
  // by the sums, which may be WD steps behind the products, those two tiles behind
  // the writer: a place's last readers are long gone.
  __shared__ __align__(16) float nlse[WROWS][128];
  __shared__ int lastkey[WROWS][128];
  __shared__ float other[2][2][WKEYS];  // MANY: [turn][tile] sums of the second half of the columns
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int nt = MANY ? kMostRows<D> : w.nt, qtile = nt * D * 2;
  uint8_t* asm_ = smem;                  // tiles of keys
  uint8_t* qsm = smem + TURNS * ATILE;   // two tiles of query rows

  if (threadIdx.x == 0) {
    for (int i = 0; i < TURNS; ++i) mbar_init(&afull[i], CREW);
    for (int i = 0; i < TURNS / 2; ++i) mbar_init(&aempty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&qfull[i], MANY ? 256 : 32), mbar_init(&qempty[i], 1);
    for (int i = 0; i < WD; ++i) mbar_init(&dfull[i], 1), mbar_init(&dempty[i], SUM);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  {  // pref[b]: items before sequence b
    long long before = 0;
    for (int p0 = 0; p0 < a.seqs; p0 += WTHREADS) {
      const int p = p0 + (int)threadIdx.x;
      const long long mine = p < a.seqs ? (long long)a.heads * wseq_of(a, p).steps : 0;
      long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) scratch[warp] = inc;
      __syncthreads();
      long long base = before + inc - mine;
      for (int x = 0; x < WTHREADS / 32; ++x) {
        if (x < warp) base += scratch[x];
        before += scratch[x];
      }
      if (p < a.seqs) pref[p] = base;
      __syncthreads();
    }
    if (threadIdx.x == 0) pref[a.seqs] = before;
    __syncthreads();
  }
  tc_fence_after();

  struct Row {
    float nlse;
    int last;
  };
  auto row_of = [&](const Walk<MANY>& it, int r, bool in) {
    Row row{-INFINITY, -1};
    if (in && r < it.s.rows) {
      const int qi = r / a.group;
      row.nlse = -w.lse[((long long)it.s.q0 + qi) * a.heads * a.group + it.head * a.group + r % a.group];
      row.last = it.s.len - it.s.nq + qi;
    }
    return row;
  };
  if (warp < SUM) {
    const int team = warp / 4 % 2, key = threadIdx.x & 127;
    const int part = MANY ? warp / 8 : 0, c0 = MANY ? part * (nt / 2) : 0;  // of the columns
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const long long cap = (long long)a.table_stride * a.page_size;
    const float scale = a.scale_log2;  // (here the plain scale: see the launch)
    const uint64_t scale2 = pack2(scale, scale), log2e2 = pack2(1.4426950408889634f, 1.4426950408889634f);
    int d = 0, qn = MANY ? -1 : 0, turn = 0;
    uint32_t dph = 0u;
    bool ok = true;
    Walk<MANY> it(a, pref, w, nt);
    while (it.there()) {
      const int k0 = (2 * it.step + team) * WKEYS, t = k0 + key;
      uint64_t sum2[2] = {0ull, 0ull};
      float masked_sum = 0.f;
      // Rows before this one do not see some key of the tile that is there.
      const int open = rows_before(a, it.s, min(k0 + WKEYS, it.s.len) - 1);
#pragma unroll 1
      for (int rt = MANY ? it.lo : 0; rt < (MANY ? it.hi : 1); ++rt) {
        if (MANY) ++qn;
        const int r0 = MANY ? rt * nt + c0 : 0, have = min(MANY ? nt / 2 : nt, it.s.rows - r0);
        const bool masked = r0 < open;
        if (!(ok = wait_long(&dfull[d], dph, abort, wc.ns))) break;
        tc_fence_after();
        const uint32_t ts = (uint32_t)((2 * d + team) * nt + c0) + lanes;
        const float* nl = nlse[qn % WROWS] + c0;
        const int* lk = lastkey[qn % WROWS] + c0;
        if (!masked) {
          auto some = [&](auto& v, int c) {
            constexpr int N = sizeof(v) / 16;
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const float4 l = *reinterpret_cast<const float4*>(nl + c + 4 * k);  // (the same for every lane)
              const float2 e = unpack2(mul2(fma2(pack2(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1])), scale2,
                                                 pack2(l.x, l.y)), log2e2));
              const float2 f = unpack2(mul2(fma2(pack2(__uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3])), scale2,
                                                 pack2(l.z, l.w)), log2e2));
              sum2[0] = add2(sum2[0], pack2(ex2(e.x), ex2(e.y)));
              sum2[1] = add2(sum2[1], pack2(ex2(f.x), ex2(f.y)));
            }
          };
          int c = 0;
          if (MANY) {
            // Sixteen columns on their way while sixteen are summed.
            uint32_t v[16], u[16];
            tmem_ld16(ts, v);
            tmem_ld_wait();
#pragma unroll 1
            for (; c + 32 <= have; c += 32) {
              tmem_ld16(ts + (uint32_t)c + 16u, u);
              some(v, c);
              tmem_ld_wait();
              if (c + 32 < have) tmem_ld16(ts + (uint32_t)c + 32u, v);
              some(u, c + 16);
              tmem_ld_wait();
            }
          }
#pragma unroll 1
          for (; c + 8 < have; c += 16) {
            uint32_t v[16];
            tmem_ld16(ts + (uint32_t)c, v);
            tmem_ld_wait();
            some(v, c);
          }
          if (c < have) {
            uint32_t v[8];
            tmem_ld8(ts + (uint32_t)c, v);
            tmem_ld_wait();
            some(v, c);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < have; c += 16) {
            uint32_t v[16];
            tmem_ld16(ts + (uint32_t)c, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float e = fmaf(__uint_as_float(v[k]), scale, nl[c + k]) * 1.4426950408889634f;
              if (t <= lk[c + k]) masked_sum += ex2(e);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&dempty[d]);
        if (++d == w.nd) d = 0, dph ^= 1u;
      }
      if (!MANY && !ok) break;
      const float2 x = unpack2(sum2[0]), y = unpack2(sum2[1]);
      float sum = ((x.x + x.y) + (y.x + y.y)) + masked_sum;
      if (MANY) {
        // (A warp whose wait has run out comes here all the same: a tile's warps leave together.)
        if (part == 1) other[turn][team][key] = sum;
        if (!(ok = tile_all(team, ok))) break;
        sum += other[turn][team][key];
        turn ^= 1;
      }
      const long long at = ((long long)it.b * a.heads + it.head) * cap + t;
      // The only addition to this place of the launch: its order is no question,
      // and the total need not come here.
      if (t < it.s.len && part == 0) {
        if (MANY && w.split > 1)
          w.part[it.seg * w.apart + at] = sum;
        else
          atomicAdd(w.weights + at, sum);
      }
      if (it.next() && !MANY) ++qn;
    }
  } else if (warp < 24) {
    // Crew number c has tile c % 2 of every step, or, where there are four, of
    // every second one.
    constexpr int CREWS = (24 - SUM) * 32 / CREW;
    const int ct = (int)threadIdx.x - SUM * 32, crew = ct / CREW, dt = ct % CREW, half = crew & 1;
    constexpr int GR = D / 32, STRIDE = CREW / GR, U = WKEYS / STRIDE;  // groups a key; keys between a thread's; its keys
    // A warp's lanes: eight that store together have four keys of two neighbouring
    // groups, whose pieces meet no bank twice.
    const int l3 = lane >> 3;
    const int grp = (lane & 1) | (GR == 8 ? l3 << 1 : GR == 4 ? (l3 & 1) << 1 : 0);
    const int tok = dt / 32 * (32 / GR) + ((lane >> 1 & 3) | (GR == 2 ? l3 << 2 : GR == 4 ? (l3 & 2) << 1 : 0));
    uint32_t off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      off[u] = (uint32_t)(grp / 2 * (WKEYS * 128) + tok * 128 + (((grp % 2 * 4 + u) ^ (tok & 7)) * 16));
    const int bpp = a.page_size / KV_BLOCK, jump = STRIDE / KV_BLOCK / bpp, rest = STRIDE / KV_BLOCK % bpp;
    const uint8_t* mine = a.cache + tok % KV_BLOCK * (D / 2) + grp * 16;
    const int par_off = kv_param_off(D) + tok % KV_BLOCK * (D / 8) + grp * 4 - (tok % KV_BLOCK * (D / 2) + grp * 16);
    constexpr int B = U < 4 ? U : 4;  // of its keys at a time
    uint4 codes[B];
    uint32_t par[B];
    // The thread's codes of its crew's tile of a step.  Nothing is asked about keys
    // past the end: their rows of the product go nowhere, and what stands in the
    // table for them is looked at like any other entry.
    auto fetch = [&](const Walk<MANY>& it, int x0) {
      const uint32_t blk = (uint32_t)((2 * it.step + half) * WKEYS + tok + x0 * STRIDE) / KV_BLOCK;
      int page = (int)(blk / (uint32_t)bpp), in = (int)(blk % (uint32_t)bpp);
      const int* row = a.table + (long long)it.b * a.table_stride;
#pragma unroll
      for (int x = 0; x < B; ++x) {
        const unsigned e = (unsigned)row[min(page, a.table_stride - 1)];  // (an entry outside the pool reads page 0)
        // (A pool has less than 2^32 blocks of 1280 bytes and more.)
        const uint32_t at = ((e < (unsigned long long)a.pages ? e : 0u) * (uint32_t)a.heads + (uint32_t)it.head) * (uint32_t)bpp + (uint32_t)in;
        const uint8_t* src = mine + (unsigned long long)at * kv_block_bytes(D);
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(codes[x].x), "=r"(codes[x].y), "=r"(codes[x].z), "=r"(codes[x].w)
                     : "l"(src));
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(par[x]) : "l"(src + par_off));
        page += jump;
        if ((in += rest) >= bpp) in -= bpp, ++page;
      }
    };
    // MANY: from a thread's piece of a tile of rows to its next one.
    const int apart = 256 / (D / 8), gmore = apart % a.group;
    const long long more = apart / a.group * a.q_ts + gmore * a.q_hs, wrap = a.q_ts - a.group * a.q_hs;
    static_assert(MANY || B == U, "codes ahead are a whole tile's");
    int i = 0, qn = 0;
    bool ok = true;
    Walk<MANY> it(a, pref, w, nt), ahead = it;
    if (CREWS == 4 && crew >= 2 && ahead.there()) ahead.next();
    if (!MANY && !wc.no_loads && ahead.there()) fetch(ahead, 0);
    for (; it.there() && ok && !wc.no_loads; it.next(), ++i) {
      if (CREWS == 2 || (i & 1) == crew / 2) {
        // Its place, and which use of it this is.
        const int as = (TURNS == 4 ? i % 2 * 2 : 0) + half, use = TURNS == 4 ? i / 2 : i;
        if (MANY) fetch(it, 0);  // (kept through the query rows' tiles, the codes would be spilled)
        if (!(ok = wait_long(&aempty[as / 2], ((uint32_t)use & 1u) ^ 1u, abort, wc.ns))) break;
        uint8_t* tile = asm_ + as * ATILE;
#pragma unroll
        for (int x0 = 0; x0 < U; x0 += B) {
          if (x0 > 0) fetch(it, x0);
#pragma unroll
          for (int x = 0; x < B; ++x) {
            const T2 s2 = from_bits2<T2>(__byte_perm(par[x], par[x], 0x1010)), z2 = from_bits2<T2>(__byte_perm(par[x], par[x], 0x3232));
            const uint32_t cw[4] = {codes[x].x, codes[x].y, codes[x].z, codes[x].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4 o;
              o.x = bits2(__hfma2(code16<T>(cw[e], 0, a.up), s2, z2));
              o.y = bits2(__hfma2(code16<T>(cw[e], 1), s2, z2));
              o.z = bits2(__hfma2(code16<T>(cw[e], 2), s2, z2));
              o.w = bits2(__hfma2(code16<T>(cw[e], 3), s2, z2));
              *reinterpret_cast<uint4*>(tile + (x0 + x) * STRIDE * 128 + off[e]) = o;
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&afull[as]);
        if (!MANY) {
          ahead.next();
          if (CREWS == 4 && ahead.there()) ahead.next();
          if (ahead.there()) fetch(ahead, 0);
        }
      }
      if (MANY) {
#pragma unroll 1
        for (int rt = it.lo; rt < it.hi; ++rt, ++qn) {
          // Sixteen bytes of each of P rows, one division for all of them.
          constexpr int C = D / 8, APART = 256 / C, P = kMostRows<D> / APART;  // pieces of a row; rows between a thread's
          const int r0 = ct / C, c = ct % C, first = rt * nt + r0;
          int g = first % a.group;
          const T* src = static_cast<const T*>(a.q) + ((long long)it.s.q0 + first / a.group) * a.q_ts +
                         (long long)(it.head * a.group + g) * a.q_hs + c * 8;
          uint4 v[P];
#pragma unroll
          for (int k = 0; k < P; ++k) {
            v[k] = uint4{};
            if (first + k * APART < it.s.rows) v[k] = *reinterpret_cast<const uint4*>(src);
            src += more;
            if ((g += gmore) >= a.group) g -= a.group, src += wrap;
          }
          const Row row = row_of(it, rt * nt + ct, ct < nt);
          // (Before the place is free.)
          if (!(ok = wait_long(&qempty[qn & 1], ((uint32_t)(qn >> 1) & 1u) ^ 1u, abort, wc.ns))) break;
          uint8_t* dst = qsm + (qn & 1) * qtile + c / 8 * (nt * 128) + r0 * 128 + (((c & 7) ^ (r0 & 7)) * 16);
#pragma unroll
          for (int k = 0; k < P; ++k) *reinterpret_cast<uint4*>(dst + k * APART * 128) = pair_order(v[k]);
          if (ct < nt) nlse[qn % WROWS][ct] = row.nlse, lastkey[qn % WROWS][ct] = row.last;
          fence_proxy_async_smem();
          mbar_arrive(&qfull[qn & 1]);
        }
      }
    }
  } else if (warp != MMA) {
    if (!wc.no_loads) {  // the query rows of each head
      int qn = 0;
      for (Walk<MANY> it(a, pref, w, nt); it.there(); it.next(it.run(1 << 30)), ++qn) {
        if (!wait_long(&qempty[qn & 1], ((uint32_t)(qn >> 1) & 1u) ^ 1u, abort, wc.ns)) break;
        uint8_t* dst = qsm + (qn & 1) * qtile;
        constexpr int C = D / 8;  // 16-byte pieces of a row
#pragma unroll 4
        for (int p = lane; p < nt * C; p += 32) {
          const int r = p / C, c = p % C;
          uint4 v{};
          if (r < it.s.rows)
            v = pair_order(*reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.q) + ((long long)it.s.q0 + r / a.group) * a.q_ts +
                (long long)(it.head * a.group + r % a.group) * a.q_hs + c * 8));
          *reinterpret_cast<uint4*>(dst + c / 8 * (nt * 128) + r * 128 + (((c & 7) ^ (r & 7)) * 16)) = v;
        }
        for (int r = lane; r < nt; r += 32) {
          const Row row = row_of(it, r, true);
          nlse[qn % WROWS][r] = row.nlse, lastkey[qn % WROWS][r] = row.last;
        }
        fence_proxy_async_smem();
        mbar_arrive(&qfull[qn & 1]);
      }
    }
  } else {
    const bool one = elect_one();
    const uint32_t idesc = (1u << 4) | (MmaFormat<T>::k << 7) | (MmaFormat<T>::k << 10) | ((uint32_t)(nt >> 3) << 17) | (8u << 24);
    const uint64_t ad = sdesc(smem_u32(asm_)), qd = sdesc(smem_u32(qsm));
    // Every step goes through this warp's loop, and beside 25 others an instruction
    // of it takes some ten cycles and a look at a barrier 200: three barriers are
    // looked at together, a step is two tiles of keys, and nothing of the list is
    // looked up but where a run of steps ends.
    const uint32_t halfa = WKEYS * 128 >> 4, halfb = (uint32_t)nt * 128 >> 4;
    int as = 0, d = 0, qn = 0;
    uint32_t dph = 1u, aph = 0u;
    bool ok = true, fresh = true;
    Walk<MANY> it(a, pref, w, nt);
    while (it.there() && ok) {
      // Steps of one head, or rows' tiles of one step.
      const int n = MANY ? it.hi - it.lo : it.run(1 << 30);
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        if (MANY || fresh) {
          // The rows' tile before this one is read by what has been issued.
          if (one && qn > 0) mma_commit(&qempty[(qn - 1) & 1]);
          __syncwarp();
          if (!(ok = wait_bar_warp(&qfull[qn & 1], (uint32_t)(qn >> 1) & 1u, abort, wc.ns))) break;
          ++qn;
          fresh = false;
        }
        if (!(ok = wait_three(&afull[as], aph, &afull[as + 1], aph, &dempty[d], dph, abort, wc.ns))) break;
        tc_fence_after();
        if (one) {
          const uint64_t at = ad + (uint32_t)(as * (ATILE >> 4)), bt = qd + (uint32_t)(((qn - 1) & 1) * (qtile >> 4));
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              mma_keys((uint32_t)((2 * d + x) * nt), at + (uint32_t)(x * (ATILE >> 4)) + h * halfa, bt + h * halfb, idesc, h == 0);
          mma_commit(&dfull[d]);
          if (!MANY || k == n - 1) mma_commit(&aempty[as / 2]);
        }
        if (++d == w.nd) d = 0, dph ^= 1u;
        if (!MANY || k == n - 1)
          if ((as += 2) == TURNS) as = 0, aph ^= 1u;
      }
      if (!ok) break;
      it.next(n);
      fresh = true;  // (a run ends where the head does)
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
    // Copies still in flight land in this CTA's shared memory: give them time.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, 2u);
  }
  tc_fence_after();
  if (warp == MMA)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base_sh), "r"(512u) : "memory");
}

// The parts of a step's rows added to the weights, in order.  A CTA a step.
__global__ void __launch_bounds__(2 * WKEYS) k_kv4_weigh_join(AttnArgs a, WeighArgs w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  const int step = (int)blockIdx.x, head = (int)blockIdx.y, b = (int)blockIdx.z, t = step * 2 * WKEYS + (int)threadIdx.x;
  const WSeq s = wseq_of(a, b);
  if (s.nq == 0 || t >= s.len) return;
  const int parts = min(w.split, (s.rows + w.nt - 1) / w.nt - first_rows(a, s, step, w.nt));
  const long long at = ((long long)b * a.heads + head) * a.table_stride * a.page_size + t;
  float sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) sum += w.part[i * w.apart + at];
  w.weights[at] += sum;
}

// Query rows of a tile.  Up to as many a sequence and key head stay in shared
// memory (measured, 16 sequences to 16384, 128 rows of 128: 101 us, brought again for
// each step, as tiles of many are, 115).
int many_rows(int dim) { return dim == 256 ? kMostRows<256> : kMostRows<128>; }

// Parts that a step's rows are cut into: the least time of the CTA with the most
// to do, in tiles of rows (four of them at least a part; a part costs two more, for
// its keys).  The lengths are on the device: the table's width is what is looked at, so that
// short contexts in a wide table are cut too little.  Measured, 8 x 4 heads of 128, 2048
// queries over 2048 tokens: 57 us in a table of 2048 places, 102 in one of 32768 and more;
// 512 queries: 23 and 33.
int split_of(int dim, int heads, int group, int max_q, int seqs, long long max_len) {
  const long long rows = (long long)max_q * group;
  if (rows <= many_rows(dim)) return 1;
  const long long tiles = (rows + many_rows(dim) - 1) / many_rows(dim);
  const long long steps = (max_len + 2 * WKEYS - 1) / (2 * WKEYS) * heads;  // of a sequence
  const long long sms = num_sms();
  if (steps >= 16 * sms || steps * std::min(seqs, WSEQS) >= 16 * sms) return 1;
  const long long items = steps * std::min(seqs, WSEQS);
  int best = 1;
  long long least = -1;
  for (int k = 1; k <= 16 && (k == 1 || tiles >= 4 * k); ++k) {
    const long long time = (items * k + sms - 1) / sms * ((tiles + k - 1) / k + 2) + (k > 1 ? 4 : 0);
    if (least < 0 || time < least) least = time, best = k;
  }
  return best;
}

template <class T, int D, bool MANY>
gptq_status weigh_launch(const AttnArgs& a, const float* lse, float* weights, int nt, int split, float* part,
                         cudaStream_t s) {
  constexpr int most = 1024 + kTurns<D> * WKEYS * D * 2 + 2 * kMostRows<D> * D * 2;
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_weigh<T, D, MANY>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    return GPTQ_OK;
  }));
  const long long head_places = (long long)a.table_stride * a.page_size;
  WeighArgs w{lse, weights, nt, std::min(WD, 256 / nt), split, part, head_places * a.heads * std::min(a.seqs, WSEQS)};
  const size_t smem = 1024 + (size_t)kTurns<D> * WKEYS * D * 2 + (size_t)2 * nt * D * 2;
  const long long steps = ((long long)a.table_stride * a.page_size + 2 * WKEYS - 1) / (2 * WKEYS);
  for (int b0 = 0; b0 < a.seqs; b0 += WSEQS) {
    AttnArgs p = a;
    p.seqs = std::min(a.seqs - b0, WSEQS);
    p.table += (long long)b0 * a.table_stride;
    p.kv_lens += b0;
    w.weights = weights + (long long)b0 * a.heads * a.table_stride * a.page_size;
    if (a.q_starts != nullptr) {
      p.q_starts += b0;
    } else {
      p.q = static_cast<const T*>(a.q) + b0 * a.q_ts;
      p.tq = p.seqs;
      w.lse = lse + (long long)b0 * a.heads * a.group;
    }
    const unsigned grid = (unsigned)std::min<long long>(num_sms(), std::min<long long>(steps * a.heads, 1 << 20) * p.seqs * split);
    {
      GQ_PROF(K_KV4_WEIGH, s);
      k_kv4_weigh<T, D, MANY><<<grid, wthreads(MANY), smem, s>>>(p, w, wait_cfg());
      GQ_LAUNCHED();
    }
    if (split == 1) continue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)steps, (unsigned)a.heads, (unsigned)p.seqs);
    cfg.blockDim = dim3(2 * WKEYS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    GQ_PROF(K_KV4_JOIN, s);
    GQ_CUDA(cudaLaunchKernelEx(&cfg, k_kv4_weigh_join, p, w));
  }
  return GPTQ_OK;
}

template <class T, int D>
gptq_status weigh_dim(const AttnArgs& a, const float* lse, float* weights, int split, float* part, cudaStream_t s) {
  const long long rows = (long long)a.max_q * a.group;
  if (rows > kMostRows<D>) return weigh_launch<T, D, true>(a, lse, weights, kMostRows<D>, split, part, s);
  return weigh_launch<T, D, false>(a, lse, weights, (int)(rows + 15) / 16 * 16, 1, nullptr, s);
}

template <class T>
gptq_status weigh_t(int dim, const AttnArgs& a, const float* lse, float* weights, int split, float* part, cudaStream_t s) {
  if (dim == 64) return weigh_dim<T, 64>(a, lse, weights, split, part, s);
  if (dim == 128) return weigh_dim<T, 128>(a, lse, weights, split, part, s);
  return weigh_dim<T, 256>(a, lse, weights, split, part, s);
}

}  // namespace

size_t kv4_weigh_ws_bytes(int dim, int heads, int group, int max_q, int seqs, long long max_len) {
  const int k = split_of(dim, heads, group, max_q, seqs, max_len);
  return k == 1 ? 0 : (size_t)k * std::min(seqs, WSEQS) * heads * max_len * 4;
}

// `scale` as it is: a score less its logarithm is rounded once, at its own size,
// before the change of base (in base 2 throughout, the logarithms' rounding
// alone was 3e-7 of a weight).
gptq_status kv4_weigh_run(int dtype, int dim, const AttnArgs& a, float scale, const float* lse, float* weights, void* ws,
                          cudaStream_t s) {
  AttnArgs p = a;
  p.scale_log2 = scale;
  const int split = split_of(dim, a.heads, a.group, a.max_q, a.seqs, (long long)a.table_stride * a.page_size);
  return dtype == GPTQ_BF16 ? weigh_t<__nv_bfloat16>(dim, p, lse, weights, split, static_cast<float*>(ws), s)
                            : weigh_t<__half>(dim, p, lse, weights, split, static_cast<float*>(ws), s);
}

}  // namespace gq
