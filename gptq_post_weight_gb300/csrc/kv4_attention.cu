// Attention over the 4-bit key/value cache.
//
// o = softmax(scale q K^T + causal mask) V per query head, in one pass over
// the keys with a running maximum and sum; K and V become elements of T in
// registers, one AND/OR and half a fused multiply-add a value, straight into
// the A fragments of the tensor cores (16 x 8 x 16, f32 sums).
//
// Bytes bound it (5/8 byte a key or value channel), so the work is cut to
// keep every SM loading: the (sequence, key head, row block) items and their
// chunks of 128 tokens form one list, and each CTA takes an equal, contiguous
// share of it.  An item inside one share is finished there; a cut one leaves
// its running maximum, sum and unnormalised output (f32) in the workspace,
// and k_kv4_join adds the pieces in the order of the list.  The cut depends
// on the lengths alone: results do not change from run to run.
//
// Measured: 48 sequences of up to 16384 tokens, 8 key heads of 128 with 8
// query heads each, one new token: 129 us, 4.2 TB/s of cache; the vector ALU
// (codes to values: two instructions a pair, at half rate) is then 62 % busy
// and the memory 64 %.  16 sequences of 5 drafted tokens over up to 4001
// tokens, 20 rows of 64: 27.3 us, three CTAs an SM waiting on their own
// chains of products and shuffles.  One token over 1000: 5.2 us.
//
// Rows of a block are (query, head of the key head's group) pairs, so that a
// key is decoded once for every head that shares it.  Each of a CTA's four
// warps streams its own blocks of 16 tokens through a ring of bulk copies,
// two at a time, and keeps its own maximum, sum and output; they meet at the
// item's end.
//
// Fragments.  The products are transposed, S^T = K q^T and O^T = V^T P^T:
// tokens (or value channels) are the 16 rows and the query rows the 8
// columns, so that a group of up to 8 heads wastes nothing and a thread's
// sums are half as many as with the query rows as rows of 16.  A tile of P
// turns from S^T's sums to the B fragment by one movmatrix.  Row r of eight
// stands for token r ^ (r >> 1 & 1) (which spreads the value rows over the
// banks), and the channel order inside the products is the order in which
// the nibbles come out: lane t of a quad owns whole words of a token's row,
// and q is loaded to match.  For the values lane g owns channels g D/8 ..
// + D/8 - 1, two a row tile.
#include "serve.cuh"

namespace gq {
gptq_status kv4_chunk_run(int dtype, int dim, const AttnArgs& a, cudaStream_t s);
size_t kv4_chunk_ws_bytes(int dim);

namespace {

constexpr int AW = 4;            // warps
constexpr int ATHREADS = 32 * AW;
constexpr int ACH = 32 * AW;     // tokens per chunk of the work list
constexpr int ASEQS = 1024;      // sequences per launch at most
constexpr float kNone = -1e30f;  // running maximum of a row that has seen nothing

struct Seq {
  int q0, nq, len;  // first query row, queries, keys
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s;
  if (a.q_starts != nullptr) {
    s.q0 = min(max(a.q_starts[b], 0), a.tq);
    s.nq = min(min(max(a.q_starts[b + 1], s.q0), a.tq) - s.q0, a.max_q);
  } else {
    s.q0 = b;
    s.nq = 1;
  }
  const long long cap = (long long)a.table_stride * a.page_size;
  s.len = (int)min((long long)max(a.kv_lens[b], 0), cap);
  return s;
}

// Row blocks and chunks of a sequence (an empty one keeps a chunk, whose
// item writes its zeros).
template <int MR>
__device__ __forceinline__ int blocks_of(const AttnArgs& a, const Seq& s) {
  return (s.nq * a.group + MR - 1) / MR;
}
__device__ __forceinline__ int chunks_of(const Seq& s) { return max(1, (s.len + ACH - 1) / ACH); }

// pref[b] = chunks of all items before sequence b; pref[seqs] = all.
template <int MR>
__device__ void work_prefix(const AttnArgs& a, long long* pref, long long* scratch) {
  constexpr int PER = ASEQS / ATHREADS;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  long long mine[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    mine[i] = sum;
    if (b < a.seqs) {
      const Seq s = seq_of(a, b);
      sum += (long long)a.heads * blocks_of<MR>(a, s) * chunks_of(s);
    }
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  long long base = inc - sum;
  for (int w = 0; w < warp; ++w) base += scratch[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    if (b < a.seqs) pref[b] = base + mine[i];
    if (b == a.seqs - 1) pref[a.seqs] = base + sum;
  }
  __syncthreads();
}

template <int D>
constexpr size_t slot_floats(int mr) {
  return (size_t)mr * (D + 2);
}

// The sequence of chunk u of the list.
__device__ __forceinline__ int seq_at(const AttnArgs& a, const long long* pref, long long u) {
  int lo = 0, hi = a.seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (pref[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A piece of an item: chunks c0 .. c1 - 1 of nch of a row block.
struct Item {
  int b, head, r0, rows, c0, c1, nch;
};

// A value that is no number must not meet the probability of 0 of a row that
// does not see its token: it counted nothing, and the rows that do see it get
// their NaN here, over the sums of row r at row(r), or over its output where row(r)
// is null.  By the whole CTA.
template <class T, int D, class Row>
__device__ __forceinline__ void spoil_item(const AttnArgs& a, const Seq& sq, const Item& it, int* first, Row row) {
  if (threadIdx.x < D / 32) first[threadIdx.x] = INT_MAX;
  __syncthreads();
  const int open = max(0, sq.len - sq.nq + it.r0 / a.group + 1);  // the first token that some row does not see
  const int end = min(it.c1 * ACH, min(sq.len, sq.len - sq.nq + (it.r0 + it.rows - 1) / a.group + 1));
#pragma unroll 1
  for (int t = max(open, it.c0 * ACH) + (int)threadIdx.x; t < end; t += ATHREADS) {
    const uint32_t* par = value_params<D>(a, it.b, it.head, t);
#pragma unroll 1
    for (int i = 0; i < D / 32; ++i)
      if (no_numbers<T>(par[i])) atomicMin(&first[i], t);
  }
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < it.rows * (D / 2); i += ATHREADS) {
    const int r = i / (D / 2), d = i % (D / 2) * 2, rr = it.r0 + r, qi = rr / a.group;
    if (sq.len - sq.nq + qi < first[d / 32]) continue;
    float* sums = row(r);
    if (sums != nullptr)
      *reinterpret_cast<float2*>(sums + d) = float2{NAN, NAN};
    else
      *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + ((long long)(sq.q0 + qi) * a.heads * a.group +
                                                             it.head * a.group + rr % a.group) * D + d) = 0x7fff7fffu;
  }
  __syncthreads();
}

// The same for every item of a CTA's share, after its steps.  (The share is
// worked out again, from what the compiler does not see through, so that no
// register is kept for this, which no call with numbers in its cache comes to.)
template <class T, int D, int NQ>
__device__ __forceinline__ void spoil_items(const AttnArgs& a, const volatile long long* prefix, int* first) {
  constexpr int MR = 8 * NQ;
  uint32_t cta, ctas;
  asm volatile("mov.u32 %0, %%ctaid.x;\n mov.u32 %1, %%nctaid.x;" : "=r"(cta), "=r"(ctas));
  const long long* pref = const_cast<const long long*>(prefix);
  const long long W = prefix[a.seqs], shares = min(W, (long long)ctas), uend = W * (cta + 1) / shares;
#pragma unroll 1
  for (long long u = W * cta / shares; u < uend;) {
    const int b = seq_at(a, pref, u);
    const Seq sq = seq_of(a, b);
    const int nch = chunks_of(sq), nblk = blocks_of<MR>(a, sq);
    const long long rem = u - pref[b];
    const int item = (int)(rem / nch), c0 = (int)(rem % nch);
    const Item it{b, item / nblk, item % nblk * MR, min(MR, sq.nq * a.group - item % nblk * MR), c0,
                  (int)min((long long)nch, c0 + (uend - u)), nch};
    float* part = a.part + ((size_t)cta * 2 + (c0 == 0 ? 1 : 0)) * slot_floats<D>(MR);
    spoil_item<T, D>(a, sq, it, first, [&](int r) {
      return it.c0 == 0 && it.c1 == it.nch ? nullptr : part + r * D;
    });
    u += it.c1 - it.c0;
  }
}

// First channel of word w of quad lane t (keys): lanes own 16-byte pieces.
template <int D>
__device__ __forceinline__ int word_channel(int t, int w) {
  return D == 64 ? 16 * t + 8 * w : 128 * (w / 4) + 32 * t + 8 * (w % 4);
}

// The transposed 8 x 8 tile of 16-bit elements.
__device__ __forceinline__ uint32_t turn8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Two floats at this CTA's address `at`, read in the cluster's CTA `rank`.
__device__ __forceinline__ float2 peer2(uint32_t at, uint32_t rank) {
  float2 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %2, %3;\n ld.shared::cluster.v2.f32 {%0, %1}, [a];\n}\n"
      : "=f"(v.x), "=f"(v.y)
      : "r"(at), "r"(rank)
      : "memory");
  return v;
}

// CTAs an SM that the registers are cut to.
constexpr int resident(int dim, int nq) { return dim * nq <= 128 ? 4 : dim * nq <= 192 ? 3 : 2; }

// NQ: column tiles of eight query rows; ST: pairs of blocks in a warp's ring.
// CL = 0: equal shares of the list.  CL > 0: blockIdx.y is the sequence, and
// CL CTAs of a cluster share each item of it and join its pieces themselves.
// SEV: a sequence may have several queries, of which one sees a key that
// another does not (one query a sequence keeps the kernel without what that
// takes, which was 2 % of the time of 48 sequences to 16384 tokens).
// LSE: a.lse is given (its test and its logarithm in every instance were 1 % of that
// time, 129.7 us and not 128.3).
template <class T, int D, int NQ, int ST, int CL, bool SEV, bool LSE>
__global__ void __launch_bounds__(ATHREADS, resident(D, NQ))
    k_kv4_attention(AttnArgs a, WaitCfg wc) {
  using T2 = typename Elem<T>::T2;
  constexpr int MR = 8 * NQ, NW = D / 32, BB = kv_block_bytes(D), PB = 2 * BB;
  constexpr int DV = D / 8;  // value channels per lane
  constexpr int OS = D + 4;  // row stride of a warp's output in shared memory
  static_assert(ST * PB >= MR * OS * 4, "a warp's output goes through its ring");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[AW * ST];
  __shared__ long long pref[ASEQS + 1];
  __shared__ long long scratch[AW];
  __shared__ float mls[AW][MR][2];
  __shared__ int spoiled, spoiled_at[D / 32];  // SEV: see spoil_item
  __shared__ int abort_sh;
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  uint8_t* ring = smem + warp * ST * PB;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_kv4_join may set itself up
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&full[warp * ST + s], 1);
    if (warp == 0) abort_sh = 0, spoiled = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  long long u = 0, uend = 1;
  if (CL == 0) {
    work_prefix<MR>(a, pref, scratch);
    const long long W = pref[a.seqs];
    const long long shares = min(W, (long long)gridDim.x);  // no share is empty
    if (threadIdx.x == 0) a.cuts[blockIdx.x] = int4{};  // nothing to join
    if (blockIdx.x >= shares) return;
    u = W * blockIdx.x / shares;
    uend = W * (blockIdx.x + 1) / shares;
  } else {
    __syncthreads();
  }
  const uint32_t rank = CL ? blockIdx.x % max(CL, 1) : 0u;
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale: -q
  const float sl = fabsf(a.scale_log2);
  int slot = 0;  // of the ring: the next copy to wait for
  uint32_t phase = 0u;
  const int perm = g ^ ((g >> 1) & 1);                                // token of row g
  const int ta = 2 * t + (t & 1), tb = 2 * t + 1 - (t & 1);           // tokens of rows 2t, 2t + 1

  while (u < uend) {
    // The item of chunk u.
    const int b = CL == 0 ? seq_at(a, pref, u) : (int)blockIdx.y;
    const Seq sq = seq_of(a, b);
    const int nch = chunks_of(sq);
    int c0, c1, head, r0;
    if (CL == 0) {
      const int nblk = blocks_of<MR>(a, sq);
      const long long rem = u - pref[b];
      const int item = (int)(rem / nch);
      c0 = (int)(rem % nch);
      c1 = (int)min((long long)nch, c0 + (uend - u));
      head = item / nblk, r0 = (item % nblk) * MR;
    } else {
      if (a.q_starts != nullptr && sq.nq == 0) {  // the whole cluster
        zero_other_rows<T, D>(a, (int)(blockIdx.y * gridDim.x + blockIdx.x), (int)(gridDim.x * gridDim.y));
        return;
      }
      c0 = (int)(nch * rank / max(CL, 1)), c1 = (int)(nch * (rank + 1) / max(CL, 1));
      head = (int)blockIdx.x / max(CL, 1), r0 = 0;  // one row block
    }
    const int rows = min(MR, sq.nq * a.group - r0);
    const int first_pos = sq.len - sq.nq + r0 / a.group;  // last key the block's first row sees
    const int vis = min(sq.len, sq.len - sq.nq + (r0 + rows - 1) / a.group + 1);  // keys the last row sees
    const int tok_end = min(c1 * ACH, vis);
    // This warp's blocks: j0 + 2 warp, + 1, then + 2 AW, ...
    const int j0 = c0 * (ACH / 16), nb_all = max(0, (tok_end + 15) / 16 - j0);
    const int nb = 2 * (nb_all / (2 * AW)) + min(max(nb_all % (2 * AW) - 2 * warp, 0), 2);
    // Copies: a pair of blocks at a time, one copy where they lie in one page.
    const int bpp = a.page_size / KV_BLOCK;
    const int* trow = a.table + (long long)b * a.table_stride;
    const uint8_t* src0 = a.cache + (long long)head * bpp * BB;
    const long long page_bytes = (long long)a.heads * bpp * BB;
    const int jump = 2 * AW / bpp, jrest = 2 * AW % bpp;
    int ip = (j0 + 2 * warp) / bpp, iin = (j0 + 2 * warp) % bpp, islot = slot, left = nb;
    // Of the next pair, loaded a round ahead; `entry2` where it crosses pages.
    int entry = left > 0 ? trow[ip] : 0, entry2 = left > 1 && iin + 1 >= bpp ? trow[ip + 1] : 0;
    auto place = [&](int e, int in) {  // an entry outside the pool reads page 0: never outside the buffer
      return src0 + ((unsigned)e < (unsigned long long)a.pages ? (long long)e : 0) * page_bytes + in * BB;
    };
    auto issue = [&]() {
      uint64_t* bar = &full[warp * ST + islot];
      const uint32_t dst = smem_u32(ring + islot * PB);
      if (lane == 0) {
        if (left == 1 || iin + 1 < bpp) {
          const uint32_t bytes = left == 1 ? BB : PB;
          mbar_expect_tx(bar, bytes);
          bulk_load(dst, place(entry, iin), bytes, bar);
        } else {
          mbar_expect_tx(bar, PB);
          bulk_load(dst, place(entry, iin), BB, bar);
          bulk_load(dst + BB, place(entry2, 0), BB, bar);
        }
      }
      if (++islot == ST) islot = 0;
      left -= 2;
      ip += jump;
      iin += jrest;
      if (iin >= bpp) iin -= bpp, ++ip;
      if (left > 0) entry = trow[ip];
      if (left > 1 && iin + 1 >= bpp) entry2 = trow[ip + 1];
    };
    if (!wc.no_loads)
      for (int i = 0; i < ST && left > 0; ++i) issue();
    if (CL && a.q_starts != nullptr)  // (elsewhere the join's, before it waits)
      zero_other_rows<T, D>(a, (int)(blockIdx.y * gridDim.x + blockIdx.x), (int)(gridDim.x * gridDim.y));

    // q, in the order of the key words: column g of each tile.
    uint32_t qb[NQ][NW][4];
    int last[NQ][2];  // last key that columns 2t, 2t + 1 see (-1: none)
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int rr = r0 + min(8 * n + g, rows - 1);
      const T* qp = static_cast<const T*>(a.q) + (long long)(sq.q0 + rr / a.group) * a.q_ts +
                    (long long)(head * a.group + rr % a.group) * a.q_hs;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint4 x = pair_order(*reinterpret_cast<const uint4*>(qp + word_channel<D>(t, w)));
        qb[n][w][0] = x.x ^ flip; qb[n][w][1] = x.y ^ flip; qb[n][w][2] = x.z ^ flip; qb[n][w][3] = x.w ^ flip;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        last[n][e] = r < rows ? sq.len - sq.nq + (r0 + r) / a.group : -1;
      }
    }
    float o[NQ][DV / 2][4], mx[NQ][2], sum[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      mx[n][0] = mx[n][1] = kNone;
      sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < DV / 2; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

    int tok0 = (j0 + 2 * warp) * 16;
#pragma unroll 1
    for (int i = 0; i < nb; i += 2, tok0 += 32 * AW) {
      const bool two = i + 1 < nb;
      if (!wait_bar_warp(&full[warp * ST + slot], phase, abort, wc.ns)) break;
      const uint8_t* pair = ring + slot * PB;
      if (++slot == ST) slot = 0, phase ^= 1u;

      // Scores of 32 tokens: sums (token g, columns 2t, 2t + 1), (token g + 8, ...).
      float s[2][NQ][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[k][n][0] = s[k][n][1] = s[k][n][2] = s[k][n][3] = 0.f;
        const uint8_t* kp = pair + k * BB + perm * (D / 2);
        const uint32_t* pp = reinterpret_cast<const uint32_t*>(pair + k * BB + kv_param_off(D)) + perm * (D / 32);
#pragma unroll
        for (int c = 0; c < (NW + 3) / 4; ++c) {
          uint32_t w[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(kp + 8 * e * (D / 2) + t * 8);
              w[e][0] = v.x; w[e][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(kp + 8 * e * (D / 2) + c * 64 + t * 16);
              w[e][0] = v.x; w[e][1] = v.y; w[e][2] = v.z; w[e][3] = v.w;
            }
          }
          // A lane's words of a token lie in one group.
          const int grp = D == 64 ? t / 2 : 4 * c + t;
          T2 s2[2], z2[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t par = pp[8 * e * (D / 32) + grp];
            s2[e] = from_bits2<T2>(__byte_perm(par, par, 0x1010));
            z2[e] = from_bits2<T2>(__byte_perm(par, par, 0x3232));
          }
#pragma unroll
          for (int q = 0; q < (NW < 4 ? NW : 4); ++q) {
            uint32_t v[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int p = 0; p < 4; ++p) v[e][p] = bits2(__hfma2(code16<T>(w[e][q], p, a.up), s2[e], z2[e]));
            const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]};
            const uint32_t a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              mma16816<T>(s[k][n], a0, qb[n][4 * c + q][0], qb[n][4 * c + q][1]);
              mma16816<T>(s[k][n], a1, qb[n][4 * c + q][2], qb[n][4 * c + q][3]);
            }
          }
        }
      }

      // Mask (only where a token of the two blocks is hidden from some row),
      // running maximum, exponentials.
      const bool hidden = tok0 + (two ? 31 : 15) > first_pos || !two;
      uint32_t pb[2][NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float nm[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (hidden) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (tok0 + 16 * k + 8 * h + perm > last[n][e] || (k == 1 && !two)) s[k][n][2 * h + e] = -INFINITY;
          }
          nm[e] = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) nm[e] = fmaxf(nm[e], __shfl_xor_sync(0xffffffffu, nm[e], x));
        }
        if (__any_sync(0xffffffffu, nm[0] > mx[n][0] || nm[1] > mx[n][1])) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            nm[e] = fmaxf(nm[e], mx[n][e]);
            f[e] = ex2(sl * (mx[n][e] - nm[e]));
            sum[n][e] *= f[e];
            mx[n][e] = nm[e];
          }
#pragma unroll
          for (int i2 = 0; i2 < DV / 2; ++i2) {
            o[n][i2][0] *= f[0]; o[n][i2][1] *= f[1];
            o[n][i2][2] *= f[0]; o[n][i2][3] *= f[1];
          }
        }
        const float m0 = sl * mx[n][0], m1 = sl * mx[n][1];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = ex2(fmaf(sl, s[k][n][2 * h], -m0)), y = ex2(fmaf(sl, s[k][n][2 * h + 1], -m1));
            if (hidden) {  // (-inf times a scale of 0 is no number)
              if (s[k][n][2 * h] == -INFINITY) x = 0.f;
              if (s[k][n][2 * h + 1] == -INFINITY) y = 0.f;
            }
            sum[n][0] += x;
            sum[n][1] += y;
            pb[k][n][h] = turn8x8(bits2(Elem<T>::make2(x, y)));
          }
      }

      // A group without numbers of a token that some row does not see must not meet
      // that row's probability of 0: it counts nothing, and the rows that see the
      // first such token get their NaN at the item's end.  (A warp has one such
      // pair of blocks an item, its last: the rows of a block are at most 32 tokens
      // apart and a warp's pairs 128.  The fence for the copies into this ring is
      // the one at the item's end.)
      if (SEV && hidden) {
        uint2* at = reinterpret_cast<uint2*>(const_cast<uint8_t*>(pair) + lane / 16 * BB + kv_value_off(D) + kv_param_off(D) +
                                             lane % 16 * (D / 8));
        uint2 par[D / 64];
        bool nan = false;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          par[i] = at[i];
          nan = nan || no_numbers<T>(par[i].x) || no_numbers<T>(par[i].y);
        }
        nan = nan && tok0 + lane > first_pos && tok0 + lane < sq.len;
        if (__builtin_expect(__any_sync(0xffffffffu, nan), 0)) {
#pragma unroll 1
          for (int i = 0; i < D / 32 && nan; ++i) {
            uint32_t* p = reinterpret_cast<uint32_t*>(at) + i;
            if (no_numbers<T>(*p)) *p = 0u;
          }
          if (lane == 0) spoiled = 1;
          __syncwarp();
        }
      }

      // Values: lane (g, t) takes channels g DV .. of the tokens of rows 2t,
      // 2t + 1 (and + 8).  Tokens past the end count nothing, whatever the
      // page holds.
      const bool tail = tok0 + 32 > sq.len || !two;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint8_t* vp = pair + k * BB + kv_value_off(D) + g * (DV / 2);
        const uint32_t* pp = reinterpret_cast<const uint32_t*>(pair + k * BB + kv_value_off(D) + kv_param_off(D)) + g * DV / 32;
        uint32_t w[4][DV / 8];  // tokens ta, tb, ta + 8, tb + 8
        T2 s2[2], z2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t par[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = 8 * h + (e ? tb : ta);
            const uint8_t* src = vp + tok * (D / 2);
            if (DV / 8 == 1) {
              w[2 * h + e][0] = *reinterpret_cast<const uint32_t*>(src);
            } else if (DV / 8 == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              w[2 * h + e][0] = v.x; w[2 * h + e][DV / 8 - 1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              w[2 * h + e][0] = v.x; w[2 * h + e][(DV / 8) / 4] = v.y;
              w[2 * h + e][(DV / 8) / 2] = v.z; w[2 * h + e][DV / 8 - 1] = v.w;
            }
            par[e] = pp[tok * (D / 32)];
            if (tail && (tok0 + 16 * k + tok >= sq.len || (k == 1 && !two))) par[e] = 0u;
          }
          s2[h] = from_bits2<T2>(__byte_perm(par[0], par[1], 0x5410));
          z2[h] = from_bits2<T2>(__byte_perm(par[0], par[1], 0x7632));
        }
#pragma unroll
        for (int v = 0; v < DV / 8; ++v) {
          uint32_t d[2][8];  // [tokens, tokens + 8][channel]
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = __byte_perm(w[2 * h][v], w[2 * h + 1][v], 0x5410),
                           y = __byte_perm(w[2 * h][v], w[2 * h + 1][v], 0x7632);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              d[h][e] = bits2(__hfma2(code16<T>(x, e, a.up), s2[h], z2[h]));
              d[h][4 + e] = bits2(__hfma2(code16<T>(y, e, a.up), s2[h], z2[h]));
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t av[4] = {d[0][2 * e], d[0][2 * e + 1], d[1][2 * e], d[1][2 * e + 1]};
#pragma unroll
            for (int n = 0; n < NQ; ++n) mma16816<T>(o[n][4 * v + e], av, pb[k][n][0], pb[k][n][1]);
          }
        }
      }
      __syncwarp();
      if (left > 0) issue();
    }

    // The four warps' maxima, sums and outputs meet; the outputs go through
    // the rings, which are empty here.
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[n][e] += __shfl_xor_sync(0xffffffffu, sum[n][e], x);
        if (g == 0) {
          mls[warp][8 * n + 2 * t + e][0] = mx[n][e];
          mls[warp][8 * n + 2 * t + e][1] = sum[n][e];
        }
        float* dst = reinterpret_cast<float*>(ring) + (8 * n + 2 * t + e) * OS + g * DV;
#pragma unroll
        for (int i = 0; i < DV / 2; ++i)
          *reinterpret_cast<float2*>(dst + 2 * i) = float2{o[n][i][e], o[n][i][2 + e]};
      }
    __syncthreads();
    const bool whole = CL == 0 && c0 == 0 && c1 == nch;
    float* part = CL ? nullptr : a.part + ((size_t)blockIdx.x * 2 + (c0 == 0 ? 1 : 0)) * slot_floats<D>(MR);
    for (int r = warp; r < rows; r += AW) {
      float top = mls[0][r][0], f[AW], den = 0.f;
#pragma unroll
      for (int w = 1; w < AW; ++w) top = fmaxf(top, mls[w][r][0]);
#pragma unroll
      for (int w = 0; w < AW; ++w) {
        f[w] = ex2(sl * (mls[w][r][0] - top));
        den += mls[w][r][1] * f[w];
      }
      const float inv = den != 0.f ? 1.f / den : 0.f;  // a row that sees nothing: zeros
      const int rr = r0 + r;
      T* dst = static_cast<T*>(a.out) +
               ((long long)(sq.q0 + rr / a.group) * a.heads * a.group + head * a.group + rr % a.group) * D;
#pragma unroll
      for (int d = 2 * lane; d < D; d += 64) {
        float2 v{0.f, 0.f};
#pragma unroll
        for (int w = 0; w < AW; ++w) {
          const float2 x = *reinterpret_cast<const float2*>(smem + (size_t)w * ST * PB + (r * OS + d) * 4);
          v.x = fmaf(x.x, f[w], v.x);
          v.y = fmaf(x.y, f[w], v.y);
        }
        if (CL)  // over warp 0's, which only this thread reads
          *reinterpret_cast<float2*>(smem + (r * OS + d) * 4) = v;
        else if (whole)
          *reinterpret_cast<T2*>(dst + d) = Elem<T>::make2(v.x * inv, v.y * inv);
        else
          *reinterpret_cast<float2*>(part + r * D + d) = v;
      }
      __syncwarp();
      if (LSE && CL == 0 && whole && lane == 0)
        a.lse[(long long)(sq.q0 + rr / a.group) * a.heads * a.group + head * a.group + rr % a.group] = log_sum(sl, top, den);
      if (CL && lane == 0) {
        mls[0][r][0] = top;
        mls[0][r][1] = den;
      } else if (!whole && lane == 0) {
        part[MR * D + 2 * r] = top;
        part[MR * D + 2 * r + 1] = den;
      }
    }
    if (SEV && CL && __builtin_expect(spoiled != 0, 0)) {
      __syncthreads();
      const Item it{b, head, r0, rows, c0, c1, nch};
      spoil_item<T, D>(a, sq, it, spoiled_at, [&](int r) { return reinterpret_cast<float*>(smem) + r * OS; });
      __syncthreads();
    }
    if (CL) {
      // The pieces of the cluster's CTAs, in the order of the ranks.
      cluster_sync_all();
      for (int r = (int)rank * AW + warp; r < rows; r += CL * AW) {
        float f[CL ? CL : 1], den = 0.f, top = kNone;
        float2 ml[CL ? CL : 1];
#pragma unroll
        for (int c = 0; c < CL; ++c) ml[c] = peer2(smem_u32(&mls[0][r][0]), (uint32_t)c);
#pragma unroll
        for (int c = 0; c < CL; ++c) top = fmaxf(top, ml[c].x);
#pragma unroll
        for (int c = 0; c < CL; ++c) {
          f[c] = ex2(sl * (ml[c].x - top));
          den += ml[c].y * f[c];
        }
        const float inv = den != 0.f ? 1.f / den : 0.f;  // a row that sees nothing: zeros
        const long long at = (long long)(sq.q0 + r / a.group) * a.heads * a.group + head * a.group + r % a.group;
        if (LSE && lane == 0) a.lse[at] = log_sum(sl, top, den);
        T* dst = static_cast<T*>(a.out) + at * D;
#pragma unroll
        for (int d = 2 * lane; d < D; d += 64) {
          float2 v{0.f, 0.f};
#pragma unroll
          for (int c = 0; c < CL; ++c) {
            const float2 x = peer2(smem_u32(smem + (r * OS + d) * 4), (uint32_t)c);
            v.x = fmaf(x.x, f[c], v.x);
            v.y = fmaf(x.y, f[c], v.y);
          }
          *reinterpret_cast<T2*>(dst + d) = Elem<T>::make2(v.x * inv, v.y * inv);
        }
      }
      cluster_sync_all();  // nobody leaves while its pieces are read
      break;
    }
    u += c1 - c0;
    if (c0 == 0 && c1 < nch && threadIdx.x == 0) {  // the cut's first piece: the join's work
      const long long W = pref[a.seqs], shares = min(W, (long long)gridDim.x);
      const int lastc = (int)(((u + nch - c1) * shares - 1) / W);  // the share of the last chunk
      a.cuts[blockIdx.x] = int4{sq.q0, r0, head << 9 | rows, lastc};
    }
    if (__syncthreads_or(abort_sh)) break;  // the whole CTA leaves together
    fence_proxy_async_smem();               // the rings take copies again
    __syncwarp();
  }
  __syncthreads();
  if (SEV && CL == 0 && __builtin_expect(spoiled != 0, 0)) spoil_items<T, D, NQ>(a, pref, spoiled_at);
  if (abort_sh) {
    // Copies in flight land in this CTA's ring: give them time.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, 2u);
  }
}

// Adds the pieces of the items that more than one CTA shared: block (c, y)
// those of the item whose first piece share c ends with, rows 4 y .. 4 y + 3,
// a warp a row.  A row's pieces come through shared memory, a batch of JB at a
// time: one latency a batch (loaded one after the other into registers they
// took 0.25 us each, 16 us of a context of 8000 tokens in 63 pieces).
template <class T, int D, int NQ>
__global__ void __launch_bounds__(ATHREADS) k_kv4_join(AttnArgs a) {
  constexpr int MR = 8 * NQ, JB = D == 256 ? 8 : 16;
  __shared__ __align__(16) float batch[AW][JB][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = (int)blockIdx.y * AW + warp, first = (int)blockIdx.x;
  if (a.q_starts != nullptr)
    zero_other_rows<T, D>(a, (int)(blockIdx.y * gridDim.x + blockIdx.x), (int)(gridDim.x * gridDim.y));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the cuts and the pieces are there
  const int4 cut = a.cuts[first];
  const int head = cut.z >> 9, rows = cut.z & 511, lastc = cut.w;
  if (r >= rows) return;
  const float sl = fabsf(a.scale_log2);
  auto slot = [&](int c) { return a.part + ((size_t)c * 2 + (c == first ? 1 : 0)) * slot_floats<D>(MR); };
  float top = kNone, den = 0.f, acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int c0 = first; c0 <= lastc; c0 += JB) {
    const int n = min(JB, lastc + 1 - c0);
    for (int i = lane; i < n * (D / 4); i += 32)
      cp_async16(&batch[warp][i / (D / 4)][i % (D / 4) * 4], slot(c0 + i / (D / 4)) + r * D + i % (D / 4) * 4);
    float2 ml{kNone, 0.f};
    if (lane < n) ml = *reinterpret_cast<const float2*>(slot(c0 + lane) + MR * D + 2 * r);
    float nt = ml.x;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) nt = fmaxf(nt, __shfl_xor_sync(0xffffffffu, nt, x));
    nt = fmaxf(nt, top);
    const float f = ex2(sl * (ml.x - nt)), fo = ex2(sl * (top - nt));
    float l = ml.y * f;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    top = nt;
    den = fmaf(den, fo, l);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= fo;
    cp_async_wait_all();
    __syncwarp();
    for (int k = 0; k < n; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(batch[warp][k][lane + 32 * i], fk, acc[i]);
    }
    __syncwarp();  // the batch is read
  }
  const float inv = den != 0.f ? 1.f / den : 0.f;  // a row that sees nothing: zeros
  const int rr = cut.y + r;
  const long long at = (long long)(cut.x + rr / a.group) * a.heads * a.group + head * a.group + rr % a.group;
  if (lane == 0 && a.lse != nullptr) a.lse[at] = log_sum(sl, top, den);
  T* dst = static_cast<T*>(a.out) + at * D;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) dst[lane + 32 * i] = Elem<T>::from(acc[i] * inv);
}

// Pairs of blocks in a warp's ring: two keep the copies ahead; with four
// column tiles the outputs need four.
template <int NQ>
constexpr int stages() {
  return NQ > 2 ? NQ : 2;
}

// Few rows, few items and short contexts: a cluster of ACL CTAs an item joins
// its own pieces, in one launch.  Measured, one new token, 8 key heads of 128,
// clusters against shares and a join: 1 sequence of 1000 tokens 5.4 and 7.5 us,
// of 8000 tokens 12.3 and 13.6, of 16000 tokens 19.6 and 17.7; 8 sequences of
// 1000 tokens 7.5 and 9.6, of 8000 17.4 and 20.4, of 16000 39.5 and 37.0.  The
// lengths are on the device, so the table's width is what is looked at.
constexpr int ACL = 8;
constexpr int kClusterTokens = 8192;

// More rows a sequence than a CTA of this file takes go to the tcgen05 kernel
// (kv4_chunk.cu).  Measured, 8 key heads of 128, tcgen05 kernel and this one:
// 16 sequences of up to 8000 tokens, 32 rows 86 and 88 us, 48 rows 87 and 141,
// 128 rows 80 and 263; one sequence of 8000, 32 rows 27 and 23, 48 rows 28 and
// 28, 128 rows 30 and 44; of 1000, 48 rows 17 and 13 (its start costs more).
// Heads of 256, 112 rows: 48 sequences to 4000, 217 and 633; one of 4000, 33
// and 34.  (The rows alone decide: for one short sequence of 33 to 48 rows this
// kernel would be the faster by those 4 us.)
bool kv4_is_chunk(int dim, int group, int max_q, bool single) {
  const long long rows = (long long)max_q * group;
  return !single && rows > 32 && rows <= (dim == 256 ? 128 : 256) * 512;
}

// What a call launches and what it needs for that.
struct Plan {
  bool chunk, cluster;
  int nq;            // column tiles
  long long shares;  // of the largest launch
  size_t ws;
};
Plan plan_of(int dim, int heads, int group, int max_q, int seqs, bool single, long long max_len) {
  Plan p{};
  const long long rows = (long long)max_q * group;
  p.chunk = kv4_is_chunk(dim, group, max_q, single);
  if (p.chunk) {
    p.ws = kv4_chunk_ws_bytes(dim);
    return p;
  }
  p.nq = rows <= 8 ? 1 : rows <= 16 || dim == 256 ? 2 : rows <= 24 ? 3 : 4;
  const long long resident_ctas = (long long)num_sms() * resident(dim, p.nq);
  p.cluster = rows <= 8 && max_len <= kClusterTokens && (long long)seqs * heads * ACL <= resident_ctas;
  if (p.cluster) return p;
  // No more shares than the longest contexts the table allows have chunks.
  const long long blocks = (rows + 8 * p.nq - 1) / (8 * p.nq);
  // (A step at a time: at the arguments' limits the product passes 64 bits.)
  p.shares = std::min(resident_ctas, (long long)kShares);
  long long most = std::min((long long)std::min(seqs, ASEQS) * heads, p.shares);
  most = std::min(most * blocks, p.shares);
  p.shares = std::min(most * ((max_len + ACH - 1) / ACH), p.shares);
  p.ws = kCutBytes + (size_t)p.shares * 2 * 8 * p.nq * (dim + 2) * 4;
  return p;
}

template <class T, int D, int NQ, int CL, bool SEV, bool LSE>
struct Kernel {
  static constexpr int ST = stages<NQ>(), smem = AW * ST * 2 * kv_block_bytes(D);
  static constexpr auto fn = k_kv4_attention<T, D, NQ, ST, CL, SEV, LSE>;
  static_assert(resident(D, NQ) * (smem + 12288) <= 233472, "the CTAs that the registers leave room for fit");
  static gptq_status ready() {
    static DeviceOnce attr;
    return attr.run([](int) -> gptq_status {
      GQ_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
      return GPTQ_OK;
    });
  }
};

template <class T, int D, bool SEV, bool LSE>
gptq_status attn_cluster(const AttnArgs& a, cudaStream_t s) {
  using K = Kernel<T, D, 1, ACL, SEV, LSE>;
  GQ_TRY(K::ready());
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.heads * ACL), (unsigned)a.seqs);
  cfg.blockDim = dim3(ATHREADS);
  cfg.dynamicSmemBytes = K::smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ACL;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  GQ_PROF(K_KV4_ATTENTION, s);
  GQ_CUDA(cudaLaunchKernelEx(&cfg, K::fn, a, wait_cfg()));
  return GPTQ_OK;
}

template <class T, int D, int NQ, bool SEV, bool LSE>
gptq_status attn_launch(const AttnArgs& a, long long shares, cudaStream_t s) {
  using K = Kernel<T, D, NQ, 0, SEV, LSE>;
  GQ_TRY(K::ready());
  const int seqs = a.seqs;
  for (int b0 = 0; b0 < seqs; b0 += ASEQS) {
    AttnArgs p = a;
    p.seqs = seqs - b0 < ASEQS ? seqs - b0 : ASEQS;
    p.table += (long long)b0 * a.table_stride;
    p.kv_lens += b0;
    p.first = b0 == 0, p.last = b0 + p.seqs == seqs;
    if (a.q_starts != nullptr) {
      p.q_starts += b0;
    } else {
      p.q = static_cast<const T*>(a.q) + b0 * a.q_ts;
      p.out = static_cast<T*>(a.out) + (long long)b0 * a.heads * a.group * D;
      if (a.lse != nullptr) p.lse = a.lse + (long long)b0 * a.heads * a.group;
      p.tq = p.seqs;
    }
    {
      GQ_PROF(K_KV4_ATTENTION, s);
      K::fn<<<(unsigned)shares, ATHREADS, K::smem, s>>>(p, wait_cfg());
      GQ_LAUNCHED();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)shares, 2 * NQ);
    cfg.blockDim = dim3(ATHREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    GQ_PROF(K_KV4_JOIN, s);
    GQ_CUDA(cudaLaunchKernelEx(&cfg, k_kv4_join<T, D, NQ>, p));
  }
  return GPTQ_OK;
}

template <class T, int D, bool SEV, bool LSE>
gptq_status attn_rows(const AttnArgs& a, const Plan& p, cudaStream_t s) {
  if (p.cluster) return attn_cluster<T, D, SEV, LSE>(a, s);
  if (p.nq == 1) return attn_launch<T, D, 1, SEV, LSE>(a, p.shares, s);
  if (p.nq == 2) return attn_launch<T, D, 2, SEV, LSE>(a, p.shares, s);
  if (p.nq == 3) return attn_launch<T, D, D == 256 ? 2 : 3, SEV, LSE>(a, p.shares, s);
  return attn_launch<T, D, D == 256 ? 2 : 4, SEV, LSE>(a, p.shares, s);
}

template <class T, bool SEV, bool LSE>
gptq_status attn_dim(int dim, const AttnArgs& a, const Plan& p, cudaStream_t s) {
  if (dim == 64) return attn_rows<T, 64, SEV, LSE>(a, p, s);
  if (dim == 128) return attn_rows<T, 128, SEV, LSE>(a, p, s);
  return attn_rows<T, 256, SEV, LSE>(a, p, s);
}
template <class T, bool LSE>
gptq_status attn_queries(int dim, const AttnArgs& a, const Plan& p, cudaStream_t s) {
  return a.max_q > 1 ? attn_dim<T, true, LSE>(dim, a, p, s) : attn_dim<T, false, LSE>(dim, a, p, s);
}
template <class T>
gptq_status attn_sums(int dim, const AttnArgs& a, const Plan& p, cudaStream_t s) {
  return a.lse != nullptr ? attn_queries<T, true>(dim, a, p, s) : attn_queries<T, false>(dim, a, p, s);
}

}  // namespace

size_t kv4_attention_ws_bytes(int dim, int heads, int group, int max_q, int seqs, bool single, long long max_len) {
  return plan_of(dim, heads, group, max_q, seqs, single, max_len).ws;
}

__global__ void __launch_bounds__(256) k_no_sums(float* lse, long long n) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i < n) lse[i] = -INFINITY;
}

// -inf for n rows that no sequence has.
gptq_status kv4_no_sums_run(float* lse, long long n, cudaStream_t s) {
  GQ_PROF(K_KV4_JOIN, s);
  k_no_sums<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(lse, n);
  GQ_LAUNCHED();
  return GPTQ_OK;
}

gptq_status kv4_attention_run(int dtype, int dim, const AttnArgs& a, cudaStream_t s) {
  if (a.seqs == 0 || a.tq == 0) return GPTQ_OK;
  const Plan p = plan_of(dim, a.heads, a.group, a.max_q, a.seqs, a.q_starts == nullptr,
                         (long long)a.table_stride * a.page_size);
  if (p.chunk) return kv4_chunk_run(dtype, dim, a, s);
  return dtype == GPTQ_BF16 ? attn_sums<__nv_bfloat16>(dim, a, p, s) : attn_sums<__half>(dim, a, p, s);
}

}  // namespace gq
