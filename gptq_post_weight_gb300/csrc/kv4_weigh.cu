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
// product.  A CTA fills an SM and is a line of workers:
//   warp 16      copies the key halves of a tile's eight cache blocks;
//   warps 8-15   decode them into 128-byte swizzled rows (operand A), once for
//                all query rows, and bring the rows' q (operand B), in the
//                order in which the nibbles come out;
//   warp 17      issues the products, four tiles of sums ahead in tensor memory;
//   warps 0-7    exponentials and sums, two teams of a lane quarter a warp.
// Few rows a sequence and key head (!MANY: one column tile): a CTA takes a
// contiguous share of the list of (sequence, key head, key tile), q stays while
// the head does, and the teams take turns at the tiles.  Many: key tiles go
// round the CTAs, and for each of them all the rows' tiles that see it come by,
// a half of the columns a team.
#include "serve.cuh"

namespace gq {
namespace {

constexpr int WKEYS = 128;           // keys of a tile
constexpr int WTHREADS = 576;
constexpr int WSEQS = 512;           // sequences of a launch at most
constexpr int WRAW = 4;              // tiles of codes in flight at most
constexpr int WD = 4;                // tiles of sums in tensor memory
template <int D>
constexpr int kMostRows = D == 256 ? 64 : 128;  // query rows of a tile (shared memory)

template <class T>
struct WFormat;
template <>
struct WFormat<__nv_bfloat16> {
  static constexpr uint32_t k = 1u;
};
template <>
struct WFormat<__half> {
  static constexpr uint32_t k = 0u;
};

struct WeighArgs {
  const float* lse;
  float* weights;
  int nt;    // columns of a tile: a multiple of 16
  int nraw;  // tiles of codes in flight
};

__device__ __forceinline__ uint64_t pair2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// Barrier of a team's 128 threads, AND-reducing: they go on or leave together.
__device__ __forceinline__ bool team_all(int team, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.and.pred po, %2, 128, pi;\n"
      " selp.u32 %0, 1, 0, po;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(1 + team)
      : "memory");
  return r != 0u;
}
// The same for both teams.
__device__ __forceinline__ bool teams_all(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.and.pred po, 3, 256, pi;\n"
      " selp.u32 %0, 1, 0, po;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0u;
}

__device__ __forceinline__ void mma_keys(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

// A sequence: first query row, queries, keys, query rows of a key head, key tiles.
struct WSeq {
  int q0, nq, len, rows, tiles;
};
__device__ __forceinline__ WSeq wseq_of(const AttnArgs& a, int b) {
  WSeq s;
  s.q0 = a.q_starts != nullptr ? min(max(a.q_starts[b], 0), a.tq) : b;
  s.nq = a.q_starts != nullptr ? min(min(max(a.q_starts[b + 1], s.q0), a.tq) - s.q0, a.max_q) : 1;
  s.len = (int)min((long long)max(a.kv_lens[b], 0), (long long)a.table_stride * a.page_size);
  s.rows = s.nq * a.group;
  s.tiles = s.nq > 0 ? (s.len + WKEYS - 1) / WKEYS : 0;
  return s;
}

// A CTA's walk over the list of (sequence, key head, key tile).
template <bool MANY>
struct Walk {
  const AttnArgs& a;
  const long long* pref;
  long long u, end;
  int b, head, tile;
  WSeq s;

  __device__ __forceinline__ Walk(const AttnArgs& args, const long long* prefix) : a(args), pref(prefix) {
    const long long W = pref[a.seqs];
    if (MANY) {
      u = blockIdx.x;
      end = W;
    } else {
      u = W * blockIdx.x / gridDim.x;
      end = W * (blockIdx.x + 1) / gridDim.x;
    }
    find();
  }
  __device__ __forceinline__ bool there() const { return u < end; }
  __device__ __forceinline__ void find() {
    if (u >= end) return;
    int lo = 0, hi = a.seqs - 1;  // the last sequence that starts at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (pref[mid] <= u) lo = mid; else hi = mid - 1;
    }
    b = lo;
    s = wseq_of(a, b);
    const long long rem = u - pref[b];
    head = (int)(rem / s.tiles);
    tile = (int)(rem % s.tiles);
  }
  // Whether the next item has other query rows.
  __device__ __forceinline__ bool next() {
    if (MANY) {
      u += gridDim.x;
      find();
      return true;
    }
    ++u;
    if (++tile < s.tiles) return false;
    tile = 0;
    if (++head == a.heads) find();
    return true;
  }
  // The first tile of query rows that sees a key of this tile.
  __device__ __forceinline__ int first_rows(int nt) const {
    return max((tile * WKEYS - s.len + s.nq) * a.group, 0) / nt;
  }
};

template <class T, int D, bool MANY>
__global__ void __launch_bounds__(WTHREADS, 1) k_kv4_weigh(AttnArgs a, WeighArgs w, WaitCfg wc) {
  using T2 = typename Elem<T>::T2;
  constexpr int HALVES = D / 64, RB = 10 * D, RAW = WKEYS / KV_BLOCK * RB, ATILE = WKEYS * D * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t rawfull[WRAW], rawempty[WRAW], afull[2], aempty[2], qfull[2], qempty[2], dfull[WD],
      dempty[WD];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ long long pref[WSEQS + 1], scratch[WTHREADS / 32];
  __shared__ __align__(16) float nlse[2][2][128];  // [team][turn][row]: minus its logarithm of the sum
  __shared__ int lastkey[2][2][128];               // the last key it sees
  __shared__ float other[2][WKEYS];                // MANY: team 1's sums
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int nt = w.nt, qtile = nt * D * 2;
  uint8_t* asm_ = smem;                     // two tiles of keys
  uint8_t* qsm = smem + 2 * ATILE;          // two tiles of query rows
  uint8_t* raw = qsm + 2 * qtile;           // tiles of codes

  if (threadIdx.x == 0) {
    for (int i = 0; i < WRAW; ++i) mbar_init(&rawfull[i], 1), mbar_init(&rawempty[i], 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&afull[i], 256), mbar_init(&aempty[i], 1);
      mbar_init(&qfull[i], 256), mbar_init(&qempty[i], 1);
    }
    for (int i = 0; i < WD; ++i) mbar_init(&dfull[i], 1), mbar_init(&dempty[i], MANY ? 8 : 4);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 17) {
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
      const long long mine = p < a.seqs ? (long long)a.heads * wseq_of(a, p).tiles : 0;
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

  if (warp < 8) {
    const int team = warp / 4, key = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int c0 = MANY ? team * (nt / 2) : 0, cn = MANY ? nt / 2 : nt;  // this team's columns
    const long long cap = (long long)a.table_stride * a.page_size;
    const float scale = a.scale_log2;  // (here the plain scale: see the launch)
    const uint64_t scale2 = pair2(scale, scale), log2e2 = pair2(1.4426950408889634f, 1.4426950408889634f);
    int d = 0, turn = 0;
    uint32_t dph = 0u;
    bool ok = true, fresh = true;
    int i = 0;
    // Row r of the rows' tile rt: what this team needs of it, into the buffer of `turn`.
    auto look_up = [&](const Walk<MANY>& it, int rt) {
      if (key < cn) {
        const int rr = rt * nt + c0 + key, qi = rr / a.group;
        const bool in = rr < it.s.rows;
        const long long at = ((long long)it.s.q0 + qi) * a.heads * a.group + it.head * a.group + rr % a.group;
        nlse[team][turn][key] = in ? -w.lse[at] : 0.f;
        lastkey[team][turn][key] = in ? it.s.len - it.s.nq + qi : -1;
      }
    };
    for (Walk<MANY> it(a, pref); it.there() && ok; ++i) {
      const bool mine = MANY || (i & 1) == team;
      const int t = it.tile * WKEYS + key;
      float* out = w.weights + ((long long)it.b * a.heads + it.head) * cap + t;
      const float old = mine && t < it.s.len && (!MANY || team == 0) ? *out : 0.f;
      uint64_t sum2[2] = {0ull, 0ull};
      float masked_sum = 0.f;
      const int rt1 = MANY ? (it.s.rows + nt - 1) / nt : 1;
      for (int rt = MANY ? it.first_rows(nt) : 0; rt < rt1; ++rt) {
        if (mine) {
          if (MANY || fresh) {
            turn ^= 1;
            look_up(it, rt);
          }
          fresh = false;
          // (A row sees at least the keys of the rows before it.)
          const int r0 = rt * nt + c0, have = min(cn, it.s.rows - r0);
          const int first_last = it.s.len - it.s.nq + r0 / a.group;
          ok = team_all(team, wait_bar_warp(&dfull[d], dph, abort, wc.ns));
          if (!ok) break;
          tc_fence_after();
          const bool masked = it.tile * WKEYS + WKEYS - 1 > first_last;
          const uint32_t ts = (uint32_t)(d * nt + c0) + lanes;
          const float* nl = nlse[team][turn];
          const int* lk = lastkey[team][turn];
          for (int c = 0; c < have; c += 16) {
            uint32_t v[16];
            tmem_ld16(ts + (uint32_t)c, v);
            tmem_ld_wait();
            if (!masked && c + 16 <= have) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float2 l = *reinterpret_cast<const float2*>(nl + c + 2 * k);
                const uint64_t e2 = mul2(fma2(pair2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), scale2,
                                              pair2(l.x, l.y)), log2e2);
                const float2 e = both(e2);
                sum2[k & 1] = add2(sum2[k & 1], pair2(ex2(e.x), ex2(e.y)));
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float e = fmaf(__uint_as_float(v[k]), scale, nl[c + k]) * 1.4426950408889634f;
                if (t <= lk[c + k] && c + k < have) masked_sum += ex2(e);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(&dempty[d]);
        }
        if (++d == WD) d = 0, dph ^= 1u;
      }
      const float2 x = both(sum2[0]), y = both(sum2[1]);
      float sum = ((x.x + x.y) + (y.x + y.y)) + masked_sum;
      if (MANY) {
        if (team == 1) other[i & 1][key] = sum;
        if (!(ok = teams_all(ok))) break;
        sum += other[i & 1][key];
      }
      if (ok && mine && t < it.s.len && (!MANY || team == 0)) *out = old + sum;
      if (it.next()) fresh = true;
    }
  } else if (warp < 16) {
    const int dt = (int)threadIdx.x - 256;
    constexpr int GR = D / 32, STEP = 256 / GR;  // groups a key; keys between a thread's
    const int grp = dt % GR, tok = dt / GR;
    // (As in the attention for prompt chunks: eight lanes' pieces meet no bank twice.)
    const int order = GR == 8 ? grp / 2 : GR == 4 ? grp / 2 * 2 : 0;
    uint32_t off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      off[u] = (uint32_t)(grp / 2 * (WKEYS * 128) + tok * 128 + (((grp % 2 * 4 + (u ^ order)) ^ (tok & 7)) * 16));
    const uint8_t* from_codes = raw + tok / KV_BLOCK * RB + tok % KV_BLOCK * (D / 2) + grp * 16;
    const uint8_t* from_par = raw + tok / KV_BLOCK * RB + kv_param_off(D) + tok % KV_BLOCK * (D / 8) + grp * 4;
    int i = 0, rs = 0, qn = 0;
    uint32_t rph = 0u;
    bool ok = true, fresh = true;
    for (Walk<MANY> it(a, pref); it.there() && ok; ++i) {
      if (!(ok = wait_bar_warp(&aempty[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u, abort, wc.ns))) break;
      if (!(ok = wait_bar_warp(&rawfull[rs], rph, abort, wc.ns))) break;
      uint8_t* tile = asm_ + (i & 1) * ATILE;
#pragma unroll
      for (int x = 0; x < WKEYS / STEP; ++x) {
        const int at = rs * RAW + x * (STEP / KV_BLOCK) * RB;
        uint4 codes;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(codes.x), "=r"(codes.y), "=r"(codes.z), "=r"(codes.w)
                     : "r"(smem_u32(from_codes + at))
                     : "memory");
        const uint32_t par = *reinterpret_cast<const uint32_t*>(from_par + at);
        if (GR >= 4) {
          const bool two = (order & 2) != 0;
          const uint4 c = codes;
          codes.x = two ? c.z : c.x, codes.y = two ? c.w : c.y;
          codes.z = two ? c.x : c.z, codes.w = two ? c.y : c.w;
        }
        if (GR == 8) {
          const bool one = (order & 1) != 0;
          const uint4 c = codes;
          codes.x = one ? c.y : c.x, codes.y = one ? c.x : c.y;
          codes.z = one ? c.w : c.z, codes.w = one ? c.z : c.w;
        }
        const T2 s2 = from_bits2<T2>(__byte_perm(par, par, 0x1010)), z2 = from_bits2<T2>(__byte_perm(par, par, 0x3232));
        const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 o;
          o.x = bits2(__hfma2(code16<T>(cw[e], 0, a.up), s2, z2));
          o.y = bits2(__hfma2(code16<T>(cw[e], 1), s2, z2));
          o.z = bits2(__hfma2(code16<T>(cw[e], 2), s2, z2));
          o.w = bits2(__hfma2(code16<T>(cw[e], 3), s2, z2));
          *reinterpret_cast<uint4*>(tile + x * STEP * 128 + off[e]) = o;
        }
      }
      // Behind the stores, which need what was loaded: a copy into the place may follow at once.
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&rawempty[rs]);
      mbar_arrive(&afull[i & 1]);
      if (++rs == w.nraw) rs = 0, rph ^= 1u;
      const int rt1 = MANY ? (it.s.rows + nt - 1) / nt : 1;
      for (int rt = MANY ? it.first_rows(nt) : 0; rt < rt1 && (MANY || fresh); ++rt, ++qn) {
        if (!(ok = wait_bar_warp(&qempty[qn & 1], ((uint32_t)(qn >> 1) & 1u) ^ 1u, abort, wc.ns))) break;
        uint8_t* dst = qsm + (qn & 1) * qtile;
        constexpr int C = D / 8;  // 16-byte pieces of a row
#pragma unroll 4
        for (int p = dt; p < nt * C; p += 256) {
          const int r = p / C, c = p % C, rr = rt * nt + r;
          uint4 v{};
          if (rr < it.s.rows)
            v = pair_order(*reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.q) + ((long long)it.s.q0 + rr / a.group) * a.q_ts +
                (long long)(it.head * a.group + rr % a.group) * a.q_hs + c * 8));
          *reinterpret_cast<uint4*>(dst + c / 8 * (nt * 128) + r * 128 + (((c & 7) ^ (r & 7)) * 16)) = v;
        }
        fence_proxy_async_smem();
        mbar_arrive(&qfull[qn & 1]);
      }
      fresh = false;
      if (!ok) break;
      if (it.next()) fresh = true;
    }
  } else if (warp == 16) {
    if (!wc.no_loads) {
      const int bpp = a.page_size / KV_BLOCK;
      int rs = 0;
      uint32_t rph = 1u;
      // The page of a lane's block, one item ahead.
      auto page_of = [&](const Walk<MANY>& it) {
        const int blk = it.tile * (WKEYS / KV_BLOCK) + lane;
        return it.there() && lane < WKEYS / KV_BLOCK && blk * KV_BLOCK < it.s.len
                   ? (unsigned)a.table[(long long)it.b * a.table_stride + blk / bpp]
                   : 0u;
      };
      Walk<MANY> it(a, pref);
      unsigned entry = page_of(it);
      while (it.there()) {
        const int blk = it.tile * (WKEYS / KV_BLOCK) + lane;
        const int have = min(WKEYS / KV_BLOCK, (it.s.len + KV_BLOCK - 1) / KV_BLOCK - it.tile * (WKEYS / KV_BLOCK));
        // (An entry outside the pool reads page 0.)
        const long long page = entry < (unsigned long long)a.pages ? (long long)entry : 0;
        const uint8_t* src = a.cache + ((page * a.heads + it.head) * bpp + blk % bpp) * (long long)kv_block_bytes(D);
        it.next();
        entry = page_of(it);
        if (!wait_bar_warp(&rawempty[rs], rph, abort, wc.ns)) break;
        if (lane == 0) mbar_expect_tx(&rawfull[rs], (uint32_t)(have * RB));
        __syncwarp();
        if (lane < have) bulk_load(smem_u32(raw + rs * RAW + lane * RB), src, RB, &rawfull[rs]);
        if (++rs == w.nraw) rs = 0, rph ^= 1u;
      }
    }
  } else {
    const bool one = elect_one();
    const uint32_t idesc = (1u << 4) | (WFormat<T>::k << 7) | (WFormat<T>::k << 10) | ((uint32_t)(nt >> 3) << 17) | (8u << 24);
    const uint64_t ad = sdesc(smem_u32(asm_)), qd = sdesc(smem_u32(qsm));
    int i = 0, d = 0, qn = 0;
    uint32_t dph = 1u;
    bool ok = true, fresh = true;
    for (Walk<MANY> it(a, pref); it.there() && ok; ++i) {
      if (!(ok = wait_bar_warp(&afull[i & 1], (uint32_t)(i >> 1) & 1u, abort, wc.ns))) break;
      const int rt1 = MANY ? (it.s.rows + nt - 1) / nt : 1;
      for (int rt = MANY ? it.first_rows(nt) : 0; rt < rt1; ++rt) {
        if (MANY || fresh) {
          // The rows' tile before this one is read by what has been issued.
          if (one && qn > 0) mma_commit(&qempty[(qn - 1) & 1]);
          __syncwarp();
          if (!(ok = wait_bar_warp(&qfull[qn & 1], (uint32_t)(qn >> 1) & 1u, abort, wc.ns))) break;
          ++qn;
          fresh = false;
        }
        if (!(ok = wait_bar_warp(&dempty[d], dph, abort, wc.ns))) break;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_keys((uint32_t)(d * nt), ad + (uint64_t)(((i & 1) * ATILE + h * WKEYS * 128 + 32 * k) >> 4),
                       qd + (uint64_t)((((qn - 1) & 1) * qtile + h * nt * 128 + 32 * k) >> 4), idesc, (h || k) ? 1u : 0u);
          mma_commit(&dfull[d]);
        }
        __syncwarp();
        if (++d == WD) d = 0, dph ^= 1u;
      }
      if (!ok) break;
      if (one) mma_commit(&aempty[i & 1]);
      __syncwarp();
      if (it.next()) fresh = true;
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
  if (warp == 17)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base_sh), "r"(512u) : "memory");
}

template <class T, int D, bool MANY>
gptq_status weigh_launch(const AttnArgs& a, const float* lse, float* weights, int nt, cudaStream_t s) {
  constexpr int RAW = WKEYS / KV_BLOCK * 10 * D, ATILE = WKEYS * D * 2, most = 217 << 10;
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_weigh<T, D, MANY>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    return GPTQ_OK;
  }));
  const int fixed = 1024 + 2 * ATILE + 2 * nt * D * 2;
  WeighArgs w{lse, weights, nt, std::min((most - fixed) / RAW, WRAW)};
  const size_t smem = fixed + (size_t)w.nraw * RAW;
  const long long tiles = ((long long)a.table_stride * a.page_size + WKEYS - 1) / WKEYS;
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
    const unsigned grid = (unsigned)std::min<long long>(num_sms(), std::min<long long>(tiles * a.heads, 1 << 20) * p.seqs);
    GQ_PROF(K_KV4_WEIGH, s);
    k_kv4_weigh<T, D, MANY><<<grid, WTHREADS, smem, s>>>(p, w, wait_cfg());
    GQ_LAUNCHED();
  }
  return GPTQ_OK;
}

template <class T, int D>
gptq_status weigh_dim(const AttnArgs& a, const float* lse, float* weights, cudaStream_t s) {
  const long long rows = (long long)a.max_q * a.group;
  if (rows > kMostRows<D>) return weigh_launch<T, D, true>(a, lse, weights, kMostRows<D>, s);
  return weigh_launch<T, D, false>(a, lse, weights, (int)(rows + 15) / 16 * 16, s);
}

template <class T>
gptq_status weigh_t(int dim, const AttnArgs& a, const float* lse, float* weights, cudaStream_t s) {
  if (dim == 64) return weigh_dim<T, 64>(a, lse, weights, s);
  if (dim == 128) return weigh_dim<T, 128>(a, lse, weights, s);
  return weigh_dim<T, 256>(a, lse, weights, s);
}

}  // namespace

// `scale` as it is: a score less its logarithm is rounded once, at its own size,
// before the change of base (in base 2 throughout, the logarithms' rounding
// alone was 3e-7 of a weight).
gptq_status kv4_weigh_run(int dtype, int dim, const AttnArgs& a, float scale, const float* lse, float* weights, cudaStream_t s) {
  AttnArgs p = a;
  p.scale_log2 = scale;
  return dtype == GPTQ_BF16 ? weigh_t<__nv_bfloat16>(dim, p, lse, weights, s) : weigh_t<__half>(dim, p, lse, weights, s);
}

}  // namespace gq
