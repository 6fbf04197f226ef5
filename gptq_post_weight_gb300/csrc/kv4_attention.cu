// Attention over the 4-bit key/value cache.
//
// o = softmax(scale q K^T + causal mask) V per query head, in one pass over
// the keys with a running maximum and sum; K and V become elements of T in
// registers, one AND/OR and half a fused multiply-add a value, straight into
// the B fragments of the tensor cores (16 x 8 x 16, f32 sums).
//
// Bytes bound it (5/8 byte a key or value channel), so the work is cut to
// keep every SM loading: the (sequence, key head, row block) items and their
// chunks of 64 tokens form one list, and each CTA takes an equal, contiguous
// share of it.  An item inside one share is finished there; a cut one leaves
// its running maximum, sum and unnormalised output (f32) in the workspace,
// and k_kv4_join adds the pieces in the order of the list.  The cut depends
// on the lengths alone: results do not change from run to run.
//
// Rows of a block are (query, head of the key head's group) pairs, so that a
// key is decoded once for every head that shares it.  Each of a CTA's four
// warps streams its own blocks of 16 tokens through a ring of bulk copies
// and keeps its own maximum, sum and output; they meet at the item's end.
//
// Fragments.  Within a block, key column n of the 16 x 8 products stands for
// token n ^ (n >> 1 & 1) (which spreads the value rows over the banks), and
// the channel order inside the products is the order in which the nibbles
// come out: lane t of a quad owns whole words of a token's row, and q is
// loaded to match.  For the values lane g owns channels g D/8 .. + D/8 - 1.
#include "serve.cuh"

namespace gq {
namespace {

constexpr int AW = 4;            // warps
constexpr int ATHREADS = 32 * AW;
constexpr int ACH = 16 * AW;     // tokens per chunk of the work list
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// First channel of word w of quad lane t (keys): lanes own 16-byte pieces.
template <int D>
__device__ __forceinline__ int word_channel(int t, int w) {
  return D == 64 ? 16 * t + 8 * w : 128 * (w / 4) + 32 * t + 8 * (w % 4);
}

template <class T, int D, int MT, int ST>
__global__ void __launch_bounds__(ATHREADS)
    k_kv4_attention(AttnArgs a, WaitCfg wc) {
  using T2 = typename Elem<T>::T2;
  constexpr int MR = 16 * MT, NW = D / 32, BB = kv_block_bytes(D);
  constexpr int DV = D / 8;  // value channels per lane and n-tiles
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[AW * ST];
  __shared__ long long pref[ASEQS + 1];
  __shared__ long long scratch[AW];
  __shared__ float mls[AW][MR][2];
  __shared__ int abort_sh;
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  uint8_t* ring = smem + warp * ST * BB;
  float* osum = reinterpret_cast<float*>(smem + AW * ST * BB);  // [MR][D + 4]

  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&full[warp * ST + s], 1);
    if (warp == 0) abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  work_prefix<MR>(a, pref, scratch);
  const long long W = pref[a.seqs];
  const long long shares = min(W, (long long)gridDim.x);  // no share is empty
  if (blockIdx.x >= shares) return;
  long long u = W * blockIdx.x / shares;
  const long long uend = W * (blockIdx.x + 1) / shares;
  int cnt = 0;  // copies this warp has waited for (slot cnt % ST)

  while (u < uend) {
    // The item of chunk u.
    int lo = 0, hi = a.seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (pref[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    const Seq sq = seq_of(a, b);
    const int nblk = blocks_of<MR>(a, sq), nch = chunks_of(sq);
    const long long rem = u - pref[b];
    const int item = (int)(rem / nch), c0 = (int)(rem % nch);
    const int c1 = (int)min((long long)nch, c0 + (uend - u));
    const int head = item / nblk, r0 = (item % nblk) * MR;
    const int rows = min(MR, sq.nq * a.group - r0);
    const int vis = min(sq.len, sq.len - sq.nq + (r0 + rows - 1) / a.group + 1);  // keys the last row sees
    const int tok_end = min(c1 * ACH, vis);
    // This warp's blocks: j0 + warp, + AW, ...
    const int j0 = c0 * AW, nb_all = max(0, (tok_end + 15) / 16 - j0);
    const int nb = max(0, (nb_all - warp + AW - 1) / AW);
    const int* trow = a.table + (long long)b * a.table_stride;
    const int bpp = a.page_size / KV_BLOCK;
    auto issue = [&](int i) {  // copy of this warp's i-th block into ring slot (cnt + i) % ST
      const int j = j0 + warp + AW * i;
      const int slot = (cnt + i) % ST;
      // An entry outside the pool reads page 0: never outside the buffer.
      const unsigned e = (unsigned)trow[j / bpp];
      const long long page = e < (unsigned long long)a.pages ? (long long)e : 0;
      mbar_expect_tx(&full[warp * ST + slot], BB);
      bulk_load(smem_u32(ring + slot * BB), a.cache + ((page * a.heads + head) * bpp + j % bpp) * (long long)BB, BB,
                &full[warp * ST + slot]);
    };
    if (lane == 0 && !wc.no_loads)
      for (int i = 0; i < ST && i < nb; ++i) issue(i);

    // q, in the order of the key words; rows g and g + 8 of each m-tile.
    uint32_t qa[MT][NW][8];
    int last[MT][2];  // last key the row sees (-1: none)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const T* qp[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = m * 16 + g + 8 * e, rr = r0 + min(r, rows - 1);
        last[m][e] = r < rows ? sq.len - sq.nq + rr / a.group : -1;
        qp[e] = static_cast<const T*>(a.q) + (long long)(sq.q0 + rr / a.group) * a.q_ts +
                (long long)(head * a.group + rr % a.group) * a.q_hs;
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int ch = word_channel<D>(t, w);
        const uint4 x = pair_order(*reinterpret_cast<const uint4*>(qp[0] + ch));
        const uint4 y = pair_order(*reinterpret_cast<const uint4*>(qp[1] + ch));
        qa[m][w][0] = x.x; qa[m][w][1] = y.x; qa[m][w][2] = x.y; qa[m][w][3] = y.y;
        qa[m][w][4] = x.z; qa[m][w][5] = y.z; qa[m][w][6] = x.w; qa[m][w][7] = y.w;
      }
    }
    float o[MT][DV][4], mx[MT][2], sum[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m][0] = mx[m][1] = kNone;
      sum[m][0] = sum[m][1] = 0.f;
#pragma unroll
      for (int j = 0; j < DV; ++j) o[m][j][0] = o[m][j][1] = o[m][j][2] = o[m][j][3] = 0.f;
    }

    for (int i = 0; i < nb; ++i) {
      const int slot = (cnt + i) % ST;
      if (!wait_bar_warp(&full[warp * ST + slot], (uint32_t)((cnt + i) / ST) & 1u, abort, wc.ns)) break;
      const uint8_t* blk = ring + slot * BB;
      const int tok0 = (j0 + warp + AW * i) * 16;

      // Scores of 16 tokens.
      float s[MT][2][4];
#pragma unroll
      for (int a2 = 0; a2 < 2; ++a2) {
        const int kt = 8 * a2 + (g ^ ((g >> 1) & 1));
#pragma unroll
        for (int m = 0; m < MT; ++m) s[m][a2][0] = s[m][a2][1] = s[m][a2][2] = s[m][a2][3] = 0.f;
        const uint8_t* kp = blk + kt * (D / 2);
        const uint32_t* pp = reinterpret_cast<const uint32_t*>(blk + kv_param_off(D)) + kt * (D / 32);
        uint32_t w[NW];
        if (D == 64) {
          const uint2 v = *reinterpret_cast<const uint2*>(kp + t * 8);
          w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
          for (int c = 0; c < NW / 4; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(kp + c * 64 + t * 16);
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
          }
        }
#pragma unroll
        for (int k = 0; k < NW; ++k) {
          const uint32_t par = pp[word_channel<D>(t, k) / 32];
          const T2 s2 = from_bits2<T2>(__byte_perm(par, par, 0x1010));
          const T2 z2 = from_bits2<T2>(__byte_perm(par, par, 0x3232));
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = bits2(__hfma2(code16<T>(w[k], e), s2, z2));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t a0[4] = {qa[m][k][0], qa[m][k][1], qa[m][k][2], qa[m][k][3]};
            const uint32_t a1[4] = {qa[m][k][4], qa[m][k][5], qa[m][k][6], qa[m][k][7]};
            mma16816<T>(s[m][a2], a0, v[0], v[1]);
            mma16816<T>(s[m][a2], a1, v[2], v[3]);
          }
        }
      }

      // Mask, running maximum, exponentials.
      const int ta = tok0 + 2 * t + (t & 1), tb = tok0 + 2 * t + 1 - (t & 1);  // tokens of columns 2t, 2t + 1
      uint32_t pa[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float nm[2] = {mx[m][0], mx[m][1]};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int a2 = 0; a2 < 2; ++a2) {
            float& x = s[m][a2][2 * e];
            float& y = s[m][a2][2 * e + 1];
            x = ta + 8 * a2 <= last[m][e] ? x * a.scale_log2 : -INFINITY;
            y = tb + 8 * a2 <= last[m][e] ? y * a.scale_log2 : -INFINITY;
            nm[e] = fmaxf(nm[e], fmaxf(x, y));
          }
          nm[e] = fmaxf(nm[e], __shfl_xor_sync(0xffffffffu, nm[e], 1));
          nm[e] = fmaxf(nm[e], __shfl_xor_sync(0xffffffffu, nm[e], 2));
        }
        if (__any_sync(0xffffffffu, nm[0] > mx[m][0] || nm[1] > mx[m][1])) {
          const float f0 = ex2(mx[m][0] - nm[0]), f1 = ex2(mx[m][1] - nm[1]);
          sum[m][0] *= f0;
          sum[m][1] *= f1;
#pragma unroll
          for (int j = 0; j < DV; ++j) {
            o[m][j][0] *= f0; o[m][j][1] *= f0;
            o[m][j][2] *= f1; o[m][j][3] *= f1;
          }
          mx[m][0] = nm[0];
          mx[m][1] = nm[1];
        }
#pragma unroll
        for (int a2 = 0; a2 < 2; ++a2)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = ex2(s[m][a2][2 * e] - mx[m][e]), y = ex2(s[m][a2][2 * e + 1] - mx[m][e]);
            sum[m][e] += x + y;
            pa[m][2 * a2 + e] = bits2(Elem<T>::make2(x, y));
          }
      }

      // Values: lane (g, t) takes channels g DV .. of the four tokens of its
      // columns.  Tokens past the end count nothing, whatever the page holds.
#pragma unroll
      for (int wv = 0; wv < DV / 8; ++wv) {
        uint32_t b0[8], b1[8];
#pragma unroll
        for (int a2 = 0; a2 < 2; ++a2) {
          const int va = 8 * a2 + 2 * t + (t & 1), vb = 8 * a2 + 2 * t + 1 - (t & 1);
          const uint8_t* vp = blk + kv_value_off(D) + (g * DV / 2 + wv * 4);
          const uint32_t wa = *reinterpret_cast<const uint32_t*>(vp + va * (D / 2));
          const uint32_t wb = *reinterpret_cast<const uint32_t*>(vp + vb * (D / 2));
          const uint32_t* pp = reinterpret_cast<const uint32_t*>(blk + kv_value_off(D) + kv_param_off(D)) +
                               (g * DV + wv * 8) / 32;
          const uint32_t pA = tok0 + va < sq.len ? pp[va * (D / 32)] : 0u;
          const uint32_t pB = tok0 + vb < sq.len ? pp[vb * (D / 32)] : 0u;
          const T2 s2 = from_bits2<T2>(__byte_perm(pA, pB, 0x5410)), z2 = from_bits2<T2>(__byte_perm(pA, pB, 0x7632));
          const uint32_t x = __byte_perm(wa, wb, 0x5410), y = __byte_perm(wa, wb, 0x7632);
          uint32_t* dst = a2 == 0 ? b0 : b1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dst[e] = bits2(__hfma2(code16<T>(x, e), s2, z2));
            dst[4 + e] = bits2(__hfma2(code16<T>(y, e), s2, z2));
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int m = 0; m < MT; ++m) mma16816<T>(o[m][wv * 8 + e], pa[m], b0[e], b1[e]);
      }
      __syncwarp();
      if (lane == 0 && i + ST < nb) issue(i + ST);
    }
    cnt += nb;

    // The four warps' maxima, sums and outputs meet.
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[m][e] += __shfl_xor_sync(0xffffffffu, sum[m][e], 1);
        sum[m][e] += __shfl_xor_sync(0xffffffffu, sum[m][e], 2);
        if (t == 0) {
          mls[warp][m * 16 + g + 8 * e][0] = mx[m][e];
          mls[warp][m * 16 + g + 8 * e][1] = sum[m][e];
        }
      }
    __syncthreads();
    for (int w = 0; w < AW; ++w) {
      if (warp == w) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = m * 16 + g + 8 * e;
            const float top = fmaxf(fmaxf(mls[0][r][0], mls[1][r][0]), fmaxf(mls[2][r][0], mls[3][r][0]));
            const float f = ex2(mx[m][e] - top);
            float* d0 = osum + r * (D + 4) + 2 * t * DV;
#pragma unroll
            for (int j = 0; j < DV; ++j) {
              const float x = o[m][j][2 * e] * f, y = o[m][j][2 * e + 1] * f;
              d0[j] = w == 0 ? x : d0[j] + x;
              d0[DV + j] = w == 0 ? y : d0[DV + j] + y;
            }
          }
      }
      __syncthreads();
    }
    const bool whole = c0 == 0 && c1 == nch;
    float* slot = a.part + ((size_t)blockIdx.x * 2 + (c0 == 0 ? 1 : 0)) * slot_floats<D>(MR);
    for (int r = warp; r < rows; r += AW) {
      const float top = fmaxf(fmaxf(mls[0][r][0], mls[1][r][0]), fmaxf(mls[2][r][0], mls[3][r][0]));
      float den = 0.f;
#pragma unroll
      for (int w = 0; w < AW; ++w) den += mls[w][r][1] * ex2(mls[w][r][0] - top);
      const float* src = osum + r * (D + 4);
      if (whole) {
        const float inv = den != 0.f ? 1.f / den : 0.f;  // a row that sees nothing: zeros
        T* dst = static_cast<T*>(a.out) +
                 ((long long)(sq.q0 + (r0 + r) / a.group) * a.heads * a.group + head * a.group + (r0 + r) % a.group) * D;
        for (int d = 2 * lane; d < D; d += 64)
          *reinterpret_cast<T2*>(dst + d) = Elem<T>::make2(src[d] * inv, src[d + 1] * inv);
      } else {
        for (int d = lane; d < D; d += 32) slot[r * D + d] = src[d];
        if (lane == 0) {
          slot[MR * D + 2 * r] = top;
          slot[MR * D + 2 * r + 1] = den;
        }
      }
    }
    u += c1 - c0;
    if (__syncthreads_or(abort_sh)) break;  // the whole CTA leaves together
  }
  __syncthreads();
  if (abort_sh) {
    // Copies in flight land in this CTA's ring: give them time.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, 2u);
  }
}

// Adds the pieces of an item that more than one CTA shared.  One CTA per
// (key head, row block) and sequence; a warp per row.
template <class T, int D, int MT>
__global__ void __launch_bounds__(ATHREADS) k_kv4_join(AttnArgs a, int grid) {
  constexpr int MR = 16 * MT;
  __shared__ long long pref[ASEQS + 1];
  __shared__ long long scratch[AW];
  work_prefix<MR>(a, pref, scratch);
  const int b = (int)blockIdx.y, item = (int)blockIdx.x;
  const Seq sq = seq_of(a, b);
  const int nblk = blocks_of<MR>(a, sq), nch = chunks_of(sq);
  if (item >= a.heads * nblk) return;
  const long long W = pref[a.seqs], u0 = pref[b] + (long long)item * nch;
  const long long shares = min(W, (long long)grid);
  const int first = (int)(((u0 + 1) * shares - 1) / W), lastc = (int)(((u0 + nch) * shares - 1) / W);
  if (first == lastc) return;
  const int head = item / nblk, r0 = (item % nblk) * MR, rows = min(MR, sq.nq * a.group - r0);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto slot = [&](int c) { return a.part + ((size_t)c * 2 + (c == first ? 1 : 0)) * slot_floats<D>(MR); };
  for (int r = warp; r < rows; r += AW) {
    float top = kNone;
    for (int c = first; c <= lastc; ++c) top = fmaxf(top, slot(c)[MR * D + 2 * r]);
    float den = 0.f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
    for (int c = first; c <= lastc; ++c) {
      const float* p = slot(c);
      const float f = ex2(p[MR * D + 2 * r] - top);
      den += p[MR * D + 2 * r + 1] * f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] += p[r * D + lane + 32 * i] * f;
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    T* dst = static_cast<T*>(a.out) +
             ((long long)(sq.q0 + (r0 + r) / a.group) * a.heads * a.group + head * a.group + (r0 + r) % a.group) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dst[lane + 32 * i] = Elem<T>::from(acc[i] * inv);
  }
}

template <int D, int MT>
constexpr int stages() {
  return D == 64 ? 8 : (D == 128 ? 6 : 4);
}

// Shares of the work list: three CTAs a SM (two for dim 256).
int shares_of(int dim) { return num_sms() * (dim == 256 ? 2 : 3); }

template <class T, int D, int MT>
gptq_status attn_launch(AttnArgs a, cudaStream_t s) {
  constexpr int ST = stages<D, MT>();
  constexpr int smem = AW * ST * kv_block_bytes(D) + 16 * MT * (D + 4) * 4;
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_attention<T, D, MT, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    return GPTQ_OK;
  }));
  const int seqs = a.seqs;
  for (int b0 = 0; b0 < seqs; b0 += ASEQS) {
    AttnArgs p = a;
    p.seqs = seqs - b0 < ASEQS ? seqs - b0 : ASEQS;
    p.table += (long long)b0 * a.table_stride;
    p.kv_lens += b0;
    if (a.q_starts != nullptr) {
      p.q_starts += b0;
    } else {
      p.q = static_cast<const T*>(a.q) + b0 * a.q_ts;
      p.out = static_cast<T*>(a.out) + (long long)b0 * a.heads * a.group * D;
    }
    const int shares = shares_of(D);
    {
      GQ_PROF(K_KV4_ATTENTION, s);
      k_kv4_attention<T, D, MT, ST><<<shares, ATHREADS, smem, s>>>(p, wait_cfg());
      GQ_LAUNCHED();
    }
    const long long items = (long long)a.heads * (((long long)a.max_q * a.group + 16 * MT - 1) / (16 * MT));
    GQ_PROF(K_KV4_JOIN, s);
    k_kv4_join<T, D, MT><<<dim3((unsigned)items, (unsigned)p.seqs), ATHREADS, 0, s>>>(p, shares);
    GQ_LAUNCHED();
  }
  return GPTQ_OK;
}

template <class T, int D>
gptq_status attn_rows(const AttnArgs& a, cudaStream_t s) {
  if (D <= 128 && (long long)a.max_q * a.group > 16) return attn_launch<T, D, D <= 128 ? 2 : 1>(a, s);
  return attn_launch<T, D, 1>(a, s);
}

template <class T>
gptq_status attn_dim(int dim, const AttnArgs& a, cudaStream_t s) {
  if (dim == 64) return attn_rows<T, 64>(a, s);
  if (dim == 128) return attn_rows<T, 128>(a, s);
  return attn_rows<T, 256>(a, s);
}

}  // namespace

size_t kv4_attention_ws_bytes(int dim) { return (size_t)shares_of(dim) * 2 * 32 * (dim + 2) * 4; }

gptq_status kv4_attention_run(int dtype, int dim, const AttnArgs& a, cudaStream_t s) {
  if (a.seqs == 0 || a.tq == 0) return GPTQ_OK;
  return dtype == GPTQ_BF16 ? attn_dim<__nv_bfloat16>(dim, a, s) : attn_dim<__half>(dim, a, s);
}

}  // namespace gq
