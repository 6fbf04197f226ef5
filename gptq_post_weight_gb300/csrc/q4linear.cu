// y = act(x W^T + bias) + residual with W in q4tp codes.
//
// Few tokens (k_q4_few).  The product reads every weight once and does little
// with it, so the bytes bound it: half a byte a weight, a rung per 32.  The
// codes enter the tensor cores as they are: an A fragment takes two nibbles
// of a word by one shift and mask, as whole numbers of the element type, and
// the products of one 32-column group (two 16 x 8 x 16 steps) are exact sums
// of code times x in f32.  The group's scale (f32, from the row's ladder)
// multiplies that sum once, so no weight is rounded to 16 bits and a weight
// costs no arithmetic of its own but its share of the shift and mask.
//   bf16: code c is the number 128 + c (0x4300 | c);
//   f16:  code c is the subnormal c 2^-24, its scale 2^24 s.
// The sum starts at -(128 + 8) sum(x) (bf16; -8 2^-24 sum(x) for f16), which
// takes the offset of the nibble off again (f32: the cancellation costs some
// 2^-18 of the result; sums that are no finite number are taken again without
// it, see sum_again).
//
// A CTA is four or eight warps of 16 rows and a slice of the columns; the CTAs of a
// cluster share the rows and split the columns, and add their sums over
// distributed shared memory in rank order.  A warp keeps its own ring of
// boxes of 16 rows x 256 columns (2 KB, 128-byte swizzle, TMA), read back by
// ldmatrix: its 8 x 16-byte matrices are eight rows of one group's codes,
// and hand lane (row, t) word t of it (one and two tokens: see k_q4_few).
// The slice of x sits in shared memory in the order in which the nibbles come
// out.  Measured: one token, 4096 x 4096 8.0 us, 5120 x 17408 18.4 us (2.6
// TB/s of codes and rungs; 6 000 of 30 000 cycles load ladders, rungs and x,
// 4 000 join the cluster, and a box takes a warp 1400, shared by the ALU's
// shifts and masks, the products and the shared-memory reads of twelve warps).
//
// The gated product (GATED): act(x Wg^T + bg) * (x Wu^T + bu) with W the gate's
// rows and then as many of the up projection.  A tile's rows come in sixteens,
// in turns of the gate and of the same outputs of the up projection (wrow), so
// that the two sums of an output are in one warp's reach when a tile is
// written out, in all three kernels; what differs from the plain product is
// that map, boxes of 16 rows for the codes, and the end.
// Both sums enter the product, and with them the rounding of their weights: in
// bf16 above 8 tokens the error against 64 bits was 0.0029 of the result, where
// a result rounded once has 0.0017.  The weights of a gated product are therefore
// f16 numbers there too (their row's power of two is taken out in any case), and
// x enters as f16 times a power of two a token (k_q4_scale_x): eight bits of
// significand fit f16's eleven, down to 2^-32 of the token's largest element.  In
// f16 itself eleven bits raised the error from 0.00021 to 0.00036; there half of the
// columns' weights (0 to 127 of every 256) enter with what their rounding leaves (FINE:
// 0.00026).
// Measured, 14336 outputs, n = 4096, weights from memory: one token 18.9 us (3.5 TB/s), 2, 4
// and 8 tokens 22.6, 31.5 and 34.2, 45 tokens 49 us (224 tiles on 152 SMs: two rounds of the
// plain product's one), of f16 60, 4096 tokens 651 us, 1.48 PFLOP/s (tensor cores 64 %: with
// 4096 columns a tile's end is a quarter of it), of f16 1045.  Two plain products and a
// multiplication take 41 us for 45 tokens and 783 for 4096, in either type.
#include <cooperative_groups.h>

#include <type_traits>

#include "serve.cuh"

namespace gq {
namespace {

constexpr int FBOX = 16 * 128;    // 16 rows x 256 columns of codes
constexpr int FST = 4;            // boxes in flight per warp
constexpr int FTAB = 36;          // ladder stride in shared memory; entry 32 is a zero
constexpr size_t kFewSmem = 225 << 10;  // dynamic shared memory of a CTA at most

template <class T>
struct CodeNum;
template <>
struct CodeNum<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;
  static constexpr float kInit = -136.0f, kScale = 1.0f;
};
template <>
struct CodeNum<__half> {
  static constexpr uint32_t kMagic = 0u;
  static constexpr float kInit = -8.0f / 16777216.0f, kScale = 16777216.0f;
};

template <class T>
__device__ __forceinline__ uint32_t code_num(uint32_t w, int i) {
  return and_or<0x000F000Fu>(w >> (4 * i), CodeNum<T>::kMagic);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

}  // namespace

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case GPTQ_ACT_RELU: return v > 0.f ? v : (v != v ? v : 0.f);
    case GPTQ_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case GPTQ_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
      return v / (1.f + expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
    case GPTQ_ACT_SILU: return v / (1.f + expf(-v));
    default: return v;
  }
}

namespace {

// The weight row of local row r of a tile whose rows start at row0 (a multiple
// of 32).  Gated: sixteen rows of the gate, the same sixteen of the up
// projection, the next ones; the tile has half as many outputs, from row0 / 2.
// (Past the gate's end its sixteens run into the up projection's rows: nothing
// of that is written out.)
template <bool GATED>
__device__ __forceinline__ int wrow(const LinearArgs& a, int row0, int r) {
  if (!GATED) return row0 + r;
  return row0 / 2 + (r / 32 * 16 + r % 16) + (r / 16 % 2 ? a.rows / 2 : 0);
}

// The epilogue of eight outputs: rows r .. r + 7 of a token (r a multiple of
// 8), with 16-byte accesses where the rows of y and the residual allow it.
template <class T>
__device__ __forceinline__ void residual8(const LinearArgs& a, int tok, int r, bool vec, uint4& raw) {
  if (a.residual != nullptr && vec) raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + (size_t)tok * a.ldr + r);
}
__device__ __forceinline__ bool rows_vec(const LinearArgs& a, int r) {
  return r + 8 <= a.rows && a.ldy % 8 == 0 && (a.residual == nullptr || a.ldr % 8 == 0);
}
template <class T>
__device__ __forceinline__ void add8(float (&v)[8], uint4 raw) {
  using T2 = typename Elem<T>::T2;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Elem<T>::to2(from_bits2<T2>(w[i]));
    v[2 * i] += f.x;
    v[2 * i + 1] += f.y;
  }
}
// `raw`: the residual as residual8 loaded it (vec only).
template <class T>
__device__ __forceinline__ void finish8(const LinearArgs& a, int tok, int r, bool vec, float (&v)[8], uint4 raw) {
  if (vec) {
    if (a.bias != nullptr) add8<T>(v, *reinterpret_cast<const uint4*>(static_cast<const T*>(a.bias) + r));
    if (a.act != GPTQ_ACT_NONE) {
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {  // (the case of k_q4_mid, side by side: one at a time 20.5 us, eight 20.1, four 19.9)
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = activate(v[k], a.act);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = v[k + 4], v[k + 4] = x[k];
      }
    }
    if (a.residual != nullptr) add8<T>(v, raw);
    uint4 o;
    o.x = bits2(Elem<T>::make2(v[0], v[1]));
    o.y = bits2(Elem<T>::make2(v[2], v[3]));
    o.z = bits2(Elem<T>::make2(v[4], v[5]));
    o.w = bits2(Elem<T>::make2(v[6], v[7]));
    *reinterpret_cast<uint4*>(static_cast<T*>(a.y) + (size_t)tok * a.ldy + r) = o;
  } else {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float x = v[0];
#pragma unroll
      for (int k = 0; k < 7; ++k) v[k] = v[k + 1];
      if (r + i < a.rows) {
        if (a.bias != nullptr) x += Elem<T>::to(static_cast<const T*>(a.bias)[r + i]);
        x = activate(x, a.act);
        if (a.residual != nullptr) x += Elem<T>::to(static_cast<const T*>(a.residual)[(size_t)tok * a.ldr + r + i]);
        static_cast<T*>(a.y)[(size_t)tok * a.ldy + r + i] = Elem<T>::from(x);
      }
    }
  }
}

// The activation of a gate, by the approximate exponential and reciprocal: each good to
// 2^-22 of the result, and for a negative v the exponent's rounding at its own size, some
// 1.5 |v| 2^-24 (SiLU; of the tanh form's u 6 |u| 2^-24), comes on top.  With a full
// division an output took some forty instructions, which the writing warps of k_q4_many
// share their issue slots for.
__device__ __forceinline__ float gate(float v, int act) {
  if (act != GPTQ_ACT_SILU && act != GPTQ_ACT_GELU_TANH) return activate(v, act);
  const float u = act == GPTQ_ACT_SILU ? v : 1.5957691216057308f * (v + 0.044715f * v * v * v);
  return __fdividef(v, 1.f + ex2(-1.4426950408889634f * u));
}

// The sum of a token and a weight row, weight by weight.
template <class T>
__device__ __noinline__ float row_sum(const T* x, const uint8_t* nibbles, const uint8_t* rungs, const float* tab, int n) {
  float sum = 0.f;
#pragma unroll 1
  for (int k = 0; k < n / GROUP; ++k) {
    const float s = rungs[k] < 32 ? tab[rungs[k]] : 0.f;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const int b = nibbles[k * 16 + i];
      sum = fmaf((float)((b & 15) - 8) * s, Elem<T>::to(x[k * 32 + 2 * i]), sum);
      sum = fmaf((float)((b >> 4) - 8) * s, Elem<T>::to(x[k * 32 + 2 * i + 1]), sum);
    }
  }
  return sum;
}

// Sums of rows r .. r + 7 that are no finite number, again: an infinite x times a
// weight and times what its rounding left may be infinity minus infinity (FINE).
template <class T>
__device__ __forceinline__ void sums_again(const LinearArgs& a, int tok, int r, int rows, float (&v)[8]) {
  bool finite = true;
#pragma unroll
  for (int k = 0; k < 8; ++k) finite = finite && fabsf(v[k]) < INFINITY;
  if (__builtin_expect(finite, 1)) return;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (r + k < rows && !(fabsf(v[k]) < INFINITY))
      v[k] = row_sum<T>(static_cast<const T*>(a.x) + (size_t)tok * a.ldx, a.nibbles + (size_t)(r + k) * (a.n / 2),
                        a.rungs + (size_t)(r + k) * (a.n / GROUP), a.tab + (size_t)(r + k) * 32, a.n);
}

// Eight gated outputs, r .. r + 7 of a token, of the sums g of the gate and u of
// the up projection; times `ts` (see LinearArgs::x_scale).
template <class T, bool FINE>
__device__ __forceinline__ void finish_gated8(const LinearArgs& a, int tok, int r, float (&g)[8], float (&u)[8], float ts) {
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] *= ts, u[k] *= ts;
  const int outs = a.rows / 2;
  if (FINE) {
    sums_again<T>(a, tok, r, outs, g);
    sums_again<T>(a, tok, outs + r, a.rows, u);
  }
  const T* bias = static_cast<const T*>(a.bias);
  T* y = static_cast<T*>(a.y) + (size_t)tok * a.ldy + r;
  if (r + 8 <= outs && a.ldy % 8 == 0 && outs % 8 == 0) {
    if (bias != nullptr) {
      add8<T>(g, *reinterpret_cast<const uint4*>(bias + r));
      add8<T>(u, *reinterpret_cast<const uint4*>(bias + outs + r));
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {  // (as in finish8)
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = gate(g[k], a.act);
#pragma unroll
      for (int k = 0; k < 4; ++k) g[k] = g[k + 4], g[k + 4] = x[k];
    }
    uint4 o;
    o.x = bits2(Elem<T>::make2(g[0] * u[0], g[1] * u[1]));
    o.y = bits2(Elem<T>::make2(g[2] * u[2], g[3] * u[3]));
    o.z = bits2(Elem<T>::make2(g[4] * u[4], g[5] * u[5]));
    o.w = bits2(Elem<T>::make2(g[6] * u[6], g[7] * u[7]));
    *reinterpret_cast<uint4*>(y) = o;
  } else {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float x = g[0], w = u[0];
#pragma unroll
      for (int k = 0; k < 7; ++k) g[k] = g[k + 1], u[k] = u[k + 1];
      if (r + i < outs) {
        if (bias != nullptr) x += Elem<T>::to(bias[r + i]), w += Elem<T>::to(bias[outs + r + i]);
        y[i] = Elem<T>::from(gate(x, a.act) * w);
      }
    }
  }
}

// v += eight sums at this CTA's address `at`, of the cluster's CTA `rank`.
__device__ __forceinline__ void add_peer8(float (&v)[8], uint32_t at, int rank) {
  const uint32_t ra = mapa_u32(at, (uint32_t)rank);
  float4 p, q;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w) : "r"(ra) : "memory");
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w) : "r"(ra + 16u) : "memory");
  v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
  v[4] += q.x; v[5] += q.y; v[6] += q.z; v[7] += q.w;
}

// reduce_finish of a gated tile.
template <class T, int ROWS, bool FINE>
__device__ __forceinline__ void reduce_finish_gated(const LinearArgs& a, const float* part, int rank, int nrank, int nthreads,
                                                    int ntok, int tok0, int row0) {
  for (int i = rank * nthreads + threadIdx.x; i < ntok * (ROWS / 16); i += nrank * nthreads) {
    const int tok = i / (ROWS / 16), o = i % (ROWS / 16) * 8, r = row0 / 2 + o;
    if (r >= a.rows / 2) continue;
    const float* gate = part + tok * ROWS + o / 16 * 32 + o % 16;
    float g[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.f;
    if (nrank > 1) {
      for (int k = 0; k < nrank; ++k) {
        add_peer8(g, smem_u32(gate), k);
        add_peer8(u, smem_u32(gate + 16), k);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = gate[e], u[e] = gate[16 + e];
    }
    finish_gated8<T, FINE>(a, tok0 + tok, r, g, u, a.x_scale != nullptr ? a.x_scale[tok0 + tok] : 1.f);
  }
}

// Sums of a row tile in shared memory, [token][ROWS], of this CTA or of
// the `nrank` CTAs of its cluster (added in rank order, each rank finishing
// its share of the outputs).
template <class T, int ROWS>
__device__ __forceinline__ void reduce_finish(const LinearArgs& a, const float* part, int rank, int nrank, int nthreads,
                                              int ntok, int tok0, int row0) {
  for (int i = rank * nthreads + threadIdx.x; i < ntok * (ROWS / 8); i += nrank * nthreads) {
    const int tok = tok0 + i / (ROWS / 8), r = row0 + i % (ROWS / 8) * 8;
    if (r >= a.rows) continue;
    const bool vec = rows_vec(a, r);
    uint4 raw{};
    residual8<T>(a, tok, r, vec, raw);
    float v[8];
    if (nrank > 1) {
      const uint32_t la = smem_u32(part + i * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
      for (int k = 0; k < nrank; ++k) add_peer8(v, la, k);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = part[i * 8 + e];
    }
    finish8<T>(a, tok, r, vec, v, raw);
  }
}

// ---------------------------------------------------------------- few tokens

// The eight rungs of box b of a row (0xff: past the end).
__device__ __forceinline__ uint2 box_rungs(const LinearArgs& a, int row, int b, int gpr) {
  uint2 r{0xffffffffu, 0xffffffffu};
  const int g0 = 8 * b;
  if (row >= a.rows || g0 >= gpr) return r;
  const uint8_t* p = a.rungs + (size_t)row * gpr + g0;
  if (gpr % 8 == 0) return *reinterpret_cast<const uint2*>(p);
  r.x = r.y = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x |= (g0 + i < gpr ? (uint32_t)p[i] : 0xffu) << (8 * i);
    r.y |= (g0 + 4 + i < gpr ? (uint32_t)p[4 + i] : 0xffu) << (8 * i);
  }
  return r;
}

// The lane's sums in `part` that are no finite number, again from the slice of
// x and the weights, weight by weight.  (Where it is comes from the special
// registers once more, opaque to the compiler: kept from the kernel's start,
// it cost two tokens a tenth of their time.)
template <class T, int TT, int FROWS, bool GATED>
__device__ __forceinline__ void sum_again(const LinearArgs& a, int boxes, float* part) {
  uint32_t tid, bx, by, bz;
  asm volatile("mov.u32 %0, %%tid.x;\n mov.u32 %1, %%ctaid.x;\n mov.u32 %2, %%ctaid.y;\n mov.u32 %3, %%ctaid.z;"
               : "=r"(tid), "=r"(bx), "=r"(by), "=r"(bz));
  const int g = tid % 32 / 4, t = tid % 4, gpr = a.n / GROUP;
  const int row = tid / 32 * 16 + (TT <= 2 ? (g >> 1) | ((g & 1) << 2) : g);  // as in k_q4_few
  const int grp0 = (int)by * boxes * 8, groups = min(boxes * 8, gpr - grp0);
#pragma unroll 1
  for (int e = 0; e < 4; ++e) {
    const int tok = TT <= 2 ? t / 2 : 2 * t + (e & 1), r = row + (e >> 1) * 8;
    if (tok >= TT || (TT <= 2 && (e | t) % 2 != 0)) continue;  // not this lane's
    const int token = (int)bz * TT + tok, rr = wrow<GATED>(a, (int)bx * FROWS, r);
    if (token >= a.tokens || rr >= a.rows || fabsf(part[tok * FROWS + r]) < INFINITY) continue;
    const T* x = static_cast<const T*>(a.x) + (size_t)token * a.ldx + (size_t)grp0 * 32;
    const uint8_t* nibbles = a.nibbles + ((size_t)rr * gpr + grp0) * 16;
    const uint8_t* rungs = a.rungs + (size_t)rr * gpr + grp0;
    float sum = 0.f;
#pragma unroll 1
    for (int k = 0; k < groups; ++k) {
      const float s = rungs[k] < 32 ? a.tab[(size_t)rr * 32 + rungs[k]] : 0.f;
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int b = nibbles[k * 16 + i];
        sum = fmaf((float)((b & 15) - 8) * s, Elem<T>::to(x[k * 32 + 2 * i]), sum);
        sum = fmaf((float)((b >> 4) - 8) * s, Elem<T>::to(x[k * 32 + 2 * i + 1]), sum);
      }
    }
    part[tok * FROWS + r] = sum;
  }
}

// Floats of shared memory a group for its starting sums, and a warp for the
// scales that its lanes look up for one another.
template <int TT>
constexpr int kInitFloats = TT <= 2 ? TT : 16;
template <int TT>
constexpr int kScaleFloats = TT <= 2 ? 0 : 128;

// TT: tokens of a block (1, 2, 4 or 8); FW warps.
//
// With one or two tokens the eight columns of a product would be six or seven
// empty ones.  There a column is (token, group mod 4) instead: lane t of a
// quad puts group t's codes into its own four of the sixteen places of K, the
// column of group c holds x in the places of lane c and zeros elsewhere, and
// one accumulator collects the sums of four groups.  Their scales are then
// two factors a lane and half a box, looked up by the lane that needs them,
// where one column takes 32 multiply-adds and an exchange through shared
// memory.  Measured, one token, 5120 x 17408: 16.9 us against 17.8.
template <class T, int TT, int FW, bool GATED>
__global__ void __launch_bounds__(32 * FW)
    k_q4_few(const __grid_constant__ CUtensorMap wmap, LinearArgs a, int boxes, WaitCfg wc) {
  static_assert(TT <= 8, "one token tile");
  constexpr int FROWS = 16 * FW, NTHR = 32 * FW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[FW * FST];
  __shared__ int abort_sh;
  volatile int* abort = &abort_sh;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int gpr = a.n / GROUP;
  const int rank = (int)blockIdx.y, nrank = (int)gridDim.y;  // the cluster's split of the columns
  const int row0 = (int)blockIdx.x * FROWS, tok0 = (int)blockIdx.z * TT;
  const int ntok = min(TT, a.tokens - tok0);
  const int box0 = rank * boxes;
  const int nbox = min(boxes, (gpr + 7) / 8 - box0);
  const int grp0 = box0 * 8;

  // Ring | x slice | starting sums | ladders | scales of a warp's box | rungs of the slice
  uint8_t* ring = smem + warp * FST * FBOX;
  uint4* xs = reinterpret_cast<uint4*>(smem + FW * FST * FBOX);               // [group][TT][4]
  float4* init = reinterpret_cast<float4*>(xs + (size_t)boxes * 8 * TT * 4);  // [group][4]: tokens 2t, 2t+1, twice
  float* init1 = reinterpret_cast<float*>(init);                              // (to two tokens: [token][group])
  float* tabs = init1 + (size_t)boxes * 8 * kInitFloats<TT>;
  float* sc = tabs + FROWS * FTAB + warp * kScaleFloats<TT>;                             // [16][8]
  uint2* rung = reinterpret_cast<uint2*>(tabs + FROWS * FTAB + FW * kScaleFloats<TT>);  // [boxes][row]

  if (lane == 0) {
    for (int s = 0; s < FST; ++s) mbar_init(&full[warp * FST + s], 1);
    if (warp == 0) abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
    if (!wc.no_loads)
      for (int s = 0; s < FST && s < nbox; ++s) {
        mbar_expect_tx(&full[warp * FST + s], FBOX);
        tma_load_2d(smem_u32(ring + s * FBOX), &wmap, (box0 + s) * 128, wrow<GATED>(a, row0, warp * 16), &full[warp * FST + s]);
      }
  }

  // The rows' ladders, the slice's rungs and x in the order of the nibbles:
  // the loads go out together, since their latency is all that this costs.
  float4 tv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = threadIdx.x + i * NTHR, wr = wrow<GATED>(a, row0, at / 8);
    tv[i] = wr < a.rows ? *reinterpret_cast<const float4*>(a.tab + (size_t)wr * 32 + at % 8 * 4) : float4{};
  }
  {
    const int r = threadIdx.x / 2;  // two threads a row
    for (int b0 = threadIdx.x % 2; b0 < nbox; b0 += 8) {
      uint2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = b0 + 2 * i < nbox ? box_rungs(a, wrow<GATED>(a, row0, r), box0 + b0 + 2 * i, gpr) : uint2{};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b0 + 2 * i < nbox)  // a rung above 31 is entry 32 of its ladder: 0
          rung[(b0 + 2 * i) * FROWS + r] = uint2{__vminu4(v[i].x, 0x20202020u), __vminu4(v[i].y, 0x20202020u)};
    }
  }
  const T* x = static_cast<const T*>(a.x);
  // Lanes 4 i .. 4 i + 3 hold one group of a token and sum it.
  const int chunks = nbox * 8 * TT * 4;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < chunks; i0 += 4 * NTHR) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = i0 + i * NTHR, tok = at / 4 % TT, grp = at / (4 * TT);
      v[i] = uint4{};
      if (at < chunks && tok < ntok && grp0 + grp < gpr)
        v[i] = *reinterpret_cast<const uint4*>(x + (size_t)(tok0 + tok) * a.ldx + (size_t)(grp0 + grp) * 32 + at % 4 * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = i0 + i * NTHR, tok = at / 4 % TT, grp = at / (4 * TT);
      using T2 = typename Elem<T>::T2;
      const float2 f0 = Elem<T>::to2(from_bits2<T2>(v[i].x)), f1 = Elem<T>::to2(from_bits2<T2>(v[i].y)),
                   f2 = Elem<T>::to2(from_bits2<T2>(v[i].z)), f3 = Elem<T>::to2(from_bits2<T2>(v[i].w));
      float s = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (at < chunks) {
        xs[at] = pair_order(v[i]);
        if (at % 4 == 0) {
          if (TT <= 2) {
            init1[tok * boxes * 8 + grp] = s * CodeNum<T>::kInit;
          } else {
            float* d = reinterpret_cast<float*>(init + grp * 4 + tok / 2) + tok % 2;
            d[0] = d[2] = s * CodeNum<T>::kInit;
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = threadIdx.x + i * NTHR;
    const float k = CodeNum<T>::kScale;
    *reinterpret_cast<float4*>(tabs + at / 8 * FTAB + at % 8 * 4) = float4{tv[i].x * k, tv[i].y * k, tv[i].z * k, tv[i].w * k};
    if (at % 8 == 0) tabs[at / 8 * FTAB + 32] = 0.f;
  }
  __syncthreads();

  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto refill = [&](int b, int st) {  // the stage that box b has left
    __syncwarp();
    if (lane == 0 && b + FST < nbox) {
      mbar_expect_tx(&full[warp * FST + st], FBOX);
      tma_load_2d(smem_u32(ring + st * FBOX), &wmap, (box0 + b + FST) * 128, wrow<GATED>(a, row0, warp * 16),
                  &full[warp * FST + st]);
    }
  };
  // Row of the box that lane g's first half of a fragment is (the other one
  // is 8 below): eight lanes' pieces of four groups then meet no bank twice.
  const int row = TT <= 2 ? (g >> 1) | ((g & 1) << 2) : g;

  if constexpr (TT <= 2) {
    const bool act = t == g % 4 && g / 4 < TT;  // this lane's places of its column hold x
    const uint4* xp = xs + (t * TT + (act ? g / 4 : 0)) * 4;
    const float2* ip = reinterpret_cast<const float2*>(init1 + (t / 2 < TT ? t / 2 : 0) * boxes * 8) + t % 2;
    const uint2* rp = rung + warp * 16 + row;
    const float* tl = tabs + (warp * 16 + row) * FTAB;
    const float* th = tl + 8 * FTAB;
    const uint32_t off = (uint32_t)(row * 128 + ((t ^ row) * 16));
    const int shift = 16 * (t % 2);
    uint4 xb[2][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) xb[i / 4][i % 4] = uint4{};
    int st = 0;
    uint32_t ph = 0u;
#pragma unroll 1
    for (int b = 0; b < nbox; ++b) {
      const uint2 rl = rp[0], rh = rp[8];
      rp += FROWS;
      const uint32_t wl[2] = {rl.x >> shift, rl.y >> shift}, wh[2] = {rh.x >> shift, rh.y >> shift};
      float sl[2][2], sh[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sl[h][0] = tl[wl[h] & 0xffu], sl[h][1] = tl[(wl[h] >> 8) & 0xffu];
        sh[h][0] = th[wh[h] & 0xffu], sh[h][1] = th[(wh[h] >> 8) & 0xffu];
      }
      if (act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) xb[i / 4][i % 4] = xp[i / 4 * 4 * TT * 4 + i % 4];
      }
      if (!wait_bar_warp(&full[warp * FST + st], ph, abort, wc.ns)) break;
      const uint8_t* box = ring + st * FBOX;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 c0 = *reinterpret_cast<const uint4*>(box + (off ^ (64u * h)));
        const uint4 c1 = *reinterpret_cast<const uint4*>(box + (off ^ (64u * h)) + 1024);
        const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
        const float2 i2 = ip[2 * h];
        float d[4] = {i2.x, i2.y, i2.x, i2.y};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t a0[4] = {code_num<T>(w0[u], 0), code_num<T>(w1[u], 0), code_num<T>(w0[u], 1),
                                  code_num<T>(w1[u], 1)};
          const uint32_t a1[4] = {code_num<T>(w0[u], 2), code_num<T>(w1[u], 2), code_num<T>(w0[u], 3),
                                  code_num<T>(w1[u], 3)};
          mma16816<T>(d, a0, xb[h][u].x, xb[h][u].y);
          mma16816<T>(d, a1, xb[h][u].z, xb[h][u].w);
        }
        acc[0] = fmaf(sl[h][1], d[1], fmaf(sl[h][0], d[0], acc[0]));
        acc[2] = fmaf(sh[h][1], d[3], fmaf(sh[h][0], d[2], acc[2]));
      }
      xp += 8 * TT * 4;
      ip += 4;
      refill(b, st);
      if (++st == FST) st = 0, ph ^= 1u;
    }
    // Columns 2t, 2t + 1 are two of the four groups of token t / 2.
    acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 1);
    acc[2] += __shfl_xor_sync(0xffffffffu, acc[2], 1);
  } else {
    // Scales: lane l looks up groups 4 (l % 2) .. + 3 of row l / 2 of each box.
    const int srow = lane / 2;
    const uint32_t* rp = reinterpret_cast<const uint32_t*>(rung + warp * 16 + srow) + lane % 2;
    const float* tp = tabs + (warp * 16 + srow) * FTAB;
    float4* sp = reinterpret_cast<float4*>(sc) + lane;
    const float4* sa = reinterpret_cast<const float4*>(sc) + g * 2;
    // Column g of a token tile: columns past the block's tokens repeat it, and
    // their sums are not used.
    const uint4* xp = xs + (TT < 8 ? g % TT : g) * 4 + t;
    const float4* ip = init + t;
    // ldmatrix: (rows 0-7, group c), (rows 8-15, group c), the same for c + 1.
    const int mrow = (lane & 7) + (lane & 8);
    uint32_t moff[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) moff[c] = (uint32_t)(mrow * 128 + (((2 * c + (lane >> 4)) ^ (mrow & 7)) * 16));
    int st = 0;
    uint32_t ph = 0u;
#pragma unroll 1
    for (int b = 0; b < nbox; ++b) {
      const uint32_t rg = *rp;
      rp += FROWS * 2;
      __syncwarp();
      *sp = float4{tp[rg & 0xffu], tp[(rg >> 8) & 0xffu], tp[(rg >> 16) & 0xffu], tp[rg >> 24]};
      if (!wait_bar_warp(&full[warp * FST + st], ph, abort, wc.ns)) break;
      const uint32_t base = smem_u32(ring + st * FBOX);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 s_lo = sa[h], s_hi = sa[16 + h];
        const float lo4[4] = {s_lo.x, s_lo.y, s_lo.z, s_lo.w}, hi4[4] = {s_hi.x, s_hi.y, s_hi.z, s_hi.w};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t w[4];
          ldmatrix4(w, base + moff[2 * h + p]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c = 4 * h + 2 * p + u;
            const uint32_t a0[4] = {code_num<T>(w[2 * u], 0), code_num<T>(w[2 * u + 1], 0), code_num<T>(w[2 * u], 1),
                                    code_num<T>(w[2 * u + 1], 1)};
            const uint32_t a1[4] = {code_num<T>(w[2 * u], 2), code_num<T>(w[2 * u + 1], 2), code_num<T>(w[2 * u], 3),
                                    code_num<T>(w[2 * u + 1], 3)};
            const float4 i4 = ip[c * 4];
            const uint4 xb = xp[c * TT * 4];
            float d[4] = {i4.x, i4.y, i4.z, i4.w};
            mma16816<T>(d, a0, xb.x, xb.y);
            mma16816<T>(d, a1, xb.z, xb.w);
            acc[0] = fmaf(lo4[2 * p + u], d[0], acc[0]);
            acc[1] = fmaf(lo4[2 * p + u], d[1], acc[1]);
            acc[2] = fmaf(hi4[2 * p + u], d[2], acc[2]);
            acc[3] = fmaf(hi4[2 * p + u], d[3], acc[3]);
          }
        }
      }
      ip += 8 * 4;
      xp += 8 * TT * 4;
      refill(b, st);
      if (++st == FST) st = 0, ph ^= 1u;
    }
  }
  __syncthreads();
  if (abort_sh) {
    // Copies still in flight land in this CTA's ring: give them time.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, 2u);
    __syncthreads();
  }

  // Sums to shared memory [token][row], added over the cluster's ranks in order.
  float* part = reinterpret_cast<float*>(smem);
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int tok = TT <= 2 ? t / 2 : 2 * t + (e & 1);
    if (tok < TT && (TT > 2 || (e | t) % 2 == 0)) {
      part[tok * FROWS + warp * 16 + row + (e >> 1) * 8] = acc[e];
      finite = finite && fabsf(acc[e]) < INFINITY;
    }
  }
  // An infinite x has an infinite offset, so that its sums are infinity minus
  // infinity (and the offsets of numbers near bf16's end leave f32's range).
  if (!finite) sum_again<T, TT, FROWS, GATED>(a, boxes, part);
  namespace cg = cooperative_groups;
  if (nrank > 1)
    cg::this_cluster().sync();
  else
    __syncthreads();
  if constexpr (GATED)
    reduce_finish_gated<T, FROWS, false>(a, part, rank, nrank, NTHR, ntok, tok0, row0);
  else
    reduce_finish<T, FROWS>(a, part, rank, nrank, NTHR, ntok, tok0, row0);
  if (nrank > 1) cg::this_cluster().sync();  // peers read this CTA's sums until here
}

// ---------------------------------------------------------------- many tokens

// D [rows][tokens] = W x^T on tcgen05 with the weights as operand A in tensor
// memory: a dequantising thread owns a row (a TMEM lane), turns 32 codes
// into 16 registers of T pairs and stores them to its lane, so a weight
// passes through no shared memory after its nibble and needs no swizzle; x
// (operand B) comes by TMA in 128-byte swizzled boxes of 64 columns.
//
// A weight is rounded once to T: with the row's scales divided by a power of
// two (the row's largest becomes 1 .. 2, restored in the epilogue, so that
// f16 keeps its 11 bits whatever the row's size) and split s = hi + lo,
//   w = fma(c, hi, c * lo)   with c = nibble - 8 exact,
// is the f32 product rounded to nearest but for a 2^-8 share of ties.
constexpr int QROWS = 128;           // weight rows per CTA (TMEM lanes)
constexpr int QK = 64;               // columns per stage
constexpr int QBOX = QROWS * 128;    // a box of codes: 128 rows x 256 columns
constexpr int QACOL = 256;           // columns 256 .. 511 hold eight stages of A (two boxes), filled and freed in
                                     // twos; 0 .. 255 the sums (the kernels take all 512, so they start at 0)
constexpr int QDEQ = 16;             // dequantising warps, warps 4 .. 19
constexpr int QTAB = 33;

template <class T>
struct Code8;  // nibble -> nibble - 8 as T
template <>
struct Code8<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u, kBias = 0x43084308u;  // 128 + c, 136
  static constexpr uint32_t kFormat = 1u;
};
template <>
struct Code8<__half> {
  static constexpr uint32_t kMagic = 0x64006400u, kBias = 0x64086408u;  // 1024 + c, 1032
  static constexpr uint32_t kFormat = 0u;
};

// 32 codes (one group of a row) times its scale (hi, lo as a pair of T).
template <class T>
__device__ __forceinline__ void dequant32(uint4 v, uint32_t s, uint32_t (&o)[16]) {
  using T2 = typename Elem<T>::T2;
  const T2 hi = from_bits2<T2>(__byte_perm(s, s, 0x1010)), lo = from_bits2<T2>(__byte_perm(s, s, 0x3232));
  const T2 bias = from_bits2<T2>(Code8<T>::kBias);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = w[i] >> 4;
    const uint32_t p[4] = {__byte_perm(w[i], h, 0x4400), __byte_perm(w[i], h, 0x5511), __byte_perm(w[i], h, 0x6622),
                           __byte_perm(w[i], h, 0x7733)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const T2 c = __hsub2(from_bits2<T2>(and_or<0x000F000Fu>(p[j], Code8<T>::kMagic)), bias);
      o[4 * i + j] = bits2(__hfma2(c, hi, __hmul2(c, lo)));
    }
  }
}

// The same with what the rounding left: o + rest is the product to some 21 bits.
template <class T>
__device__ __forceinline__ void dequant32(uint4 v, uint32_t s, uint32_t (&o)[16], uint32_t (&rest)[16]) {
  using T2 = typename Elem<T>::T2;
  const T2 hi = from_bits2<T2>(__byte_perm(s, s, 0x1010)), lo = from_bits2<T2>(__byte_perm(s, s, 0x3232));
  const T2 bias = from_bits2<T2>(Code8<T>::kBias);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = w[i] >> 4;
    const uint32_t p[4] = {__byte_perm(w[i], h, 0x4400), __byte_perm(w[i], h, 0x5511), __byte_perm(w[i], h, 0x6622),
                           __byte_perm(w[i], h, 0x7733)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const T2 c = __hsub2(from_bits2<T2>(and_or<0x000F000Fu>(p[j], Code8<T>::kMagic)), bias);
      const T2 full = __hfma2(c, hi, __hmul2(c, lo));
      o[4 * i + j] = bits2(full);
      rest[4 * i + j] = bits2(__hfma2(c, lo, __hfma2(c, hi, __hneg2(full))));
    }
  }
}

// mbar_arrive_relaxed on the pair leader's barrier.  What these arrivals
// announce (stores to tensor memory, finished reads of shared memory) is
// ordered by tcgen05.wait::st and the tcgen05 fences on both sides, or has been
// consumed; a releasing arrival waits for the thread's own loads from global
// memory as well, and those are the rungs of boxes to come (measured: 1400
// cycles from arrival to completed phase).
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_u32(smem_u32(bar), 0))
               : "memory");
}

// Non-blocking look at a barrier.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0u;
}

// Named barrier 1 over the 256 threads that write tiles out, AND-reducing.
__device__ __forceinline__ bool epi8_all(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n bar.red.and.pred po, 1, 256, pi;\n"
      " selp.u32 %0, 1, 0, po;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0u;
}

// The eight products of two stages: A at tensor-memory column a (8 columns
// per 16 of K), B at descriptors b0, b1 (32 bytes per 16 of K); first:
// overwrite D.
template <bool PAIR>
__device__ __forceinline__ void mma_two(uint32_t d, uint32_t a, uint64_t b0, uint64_t b1, uint32_t idesc, bool first) {
#define GQ_MMA(GROUP, A, B, P) " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [" A "], " B ", %4, " P ";\n"
#define GQ_MMA8(GROUP)                                                                            \
  asm volatile(                                                                                   \
      "{\n .reg .pred p, t;\n .reg .b32 a1, a2, a3, a4, a5, a6, a7;\n"                           \
      " .reg .b64 b1, b2, b3, c1, c2, c3;\n setp.eq.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n"      \
      " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n add.u32 a4, %1, 32;\n" \
      " add.u32 a5, %1, 40;\n add.u32 a6, %1, 48;\n add.u32 a7, %1, 56;\n"                       \
      " add.u64 b1, %2, 2;\n add.u64 b2, %2, 4;\n add.u64 b3, %2, 6;\n"                          \
      " add.u64 c1, %3, 2;\n add.u64 c2, %3, 4;\n add.u64 c3, %3, 6;\n"                          \
      GQ_MMA(GROUP, "%1", "%2", "p") GQ_MMA(GROUP, "a1", "b1", "t")                               \
      GQ_MMA(GROUP, "a2", "b2", "t") GQ_MMA(GROUP, "a3", "b3", "t")                               \
      GQ_MMA(GROUP, "a4", "%3", "t") GQ_MMA(GROUP, "a5", "c1", "t")                               \
      GQ_MMA(GROUP, "a6", "c2", "t") GQ_MMA(GROUP, "a7", "c3", "t") "}\n" ::"r"(d),               \
      "r"(a), "l"(b0), "l"(b1), "r"(idesc), "r"((uint32_t)first)                                  \
      : "memory")
  if (PAIR)
    GQ_MMA8("2");
  else
    GQ_MMA8("1");
#undef GQ_MMA8
#undef GQ_MMA
}

// Waits of the thread that issues the MMAs, on two barriers at once.
__device__ __forceinline__ bool wait_both(uint64_t* x, uint32_t xp, uint64_t* y, uint32_t yp, volatile int* abort,
                                          uint64_t limit) {
  if (mbar_test_wait(x, xp) & mbar_test_wait(y, yp)) return true;
  return wait_bar(x, xp, abort, limit) && wait_bar(y, yp, abort, limit);
}

// The rows' ladders as (hi, lo) pairs, and the powers of two taken out.  The
// dequantising threads: four a row, eight rungs each; barrier 2 is theirs.
// A row's largest rung comes to 1 to 2; of a gated product's, whose weights are f16
// numbers in either type, to 2^11 to 2^12: times 8 it still fits f16, and weights keep
// their eleven bits down to 2^-22 of it (with 1 to 2 they lost them from 2^-11 on).
template <class T, bool GATED>
__device__ __forceinline__ void load_ladders(const LinearArgs& a, int row0, uint32_t* tab, float* rowscale,
                                             float* rowmax) {
  const int i = threadIdx.x - 128, r = i % QROWS, part = i / QROWS, row = wrow<GATED>(a, row0, r);
  float s[8];
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float4 v{};
    if (row < a.rows) v = *reinterpret_cast<const float4*>(a.tab + (size_t)row * 32 + part * 8 + 4 * k);
    s[4 * k] = v.x; s[4 * k + 1] = v.y; s[4 * k + 2] = v.z; s[4 * k + 3] = v.w;
    m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
  rowmax[part * QROWS + r] = m;
  asm volatile("bar.sync 2, 512;" ::: "memory");  // also: nobody reads the last tile's ladders any more
  m = fmaxf(fmaxf(rowmax[r], rowmax[QROWS + r]), fmaxf(rowmax[2 * QROWS + r], rowmax[3 * QROWS + r]));
  // (2^-149 is the smallest power of two there is.)
  const int e = (m > 0.f && isfinite(m)) ? max(ilogbf(m) - (GATED ? 11 : 0), -149) : 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float v = scalbnf(s[k], -e);
    T hi = Elem<T>::from(v);
    T lo = Elem<T>::from(v - Elem<T>::to(hi));
    tab[r * QTAB + part * 8 + k] =
        (uint32_t)*reinterpret_cast<uint16_t*>(&hi) | ((uint32_t)*reinterpret_cast<uint16_t*>(&lo) << 16);
  }
  if (part == 0) {
    tab[r * QTAB + 32] = 0u;  // for a rung above 31, and past the row's end
    rowscale[r] = scalbnf(1.f, e);
  }
  asm volatile("bar.sync 2, 512;" ::: "memory");
}

// Rungs of groups g0 .. g0 + 3 of a row (given its first) as a word of bytes;
// 0xff past the end.
__device__ __forceinline__ uint32_t four_rungs(const uint8_t* row, bool in, int g0, int gpr) {
  if (!in || g0 >= gpr) return 0xffffffffu;
  if (gpr % 4 == 0) return *reinterpret_cast<const uint32_t*>(row + g0);
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v |= (g0 + i < gpr ? (uint32_t)row[g0 + i] : 0xffu) << (8 * i);
  return v;
}

// Stage j of a box for this thread's row r, from the box's bytes to tensor memory.
template <class T>
__device__ __forceinline__ void dequant_stage(const uint8_t* box, int r, int j, uint32_t rungs, const uint32_t* tab,
                                              uint32_t taddr) {
  const uint4 v0 = *reinterpret_cast<const uint4*>(box + r * 128 + (((2 * j) ^ (r & 7)) * 16));
  const uint4 v1 = *reinterpret_cast<const uint4*>(box + r * 128 + (((2 * j + 1) ^ (r & 7)) * 16));
  const uint32_t s0 = tab[r * QTAB + min(rungs & 0xffu, 32u)],
                 s1 = tab[r * QTAB + min((rungs >> 8) & 0xffu, 32u)];
  uint32_t o[16];
  dequant32<T>(v0, s0, o);
  tmem_st16(taddr, o);
  dequant32<T>(v1, s1, o);
  tmem_st16(taddr + 16, o);
}

// The same, and what the rounding left 32 columns on.
template <class T>
__device__ __forceinline__ void dequant_stage_both(const uint8_t* box, int r, int j, uint32_t rungs, const uint32_t* tab,
                                                   uint32_t taddr) {
#pragma unroll 1
  for (int g = 0; g < 2; ++g) {
    const uint4 v = *reinterpret_cast<const uint4*>(box + r * 128 + (((2 * j + g) ^ (r & 7)) * 16));
    const uint32_t s = tab[r * QTAB + min(rungs >> (8 * g) & 0xffu, 32u)];
    uint32_t o[16], rest[16];
    dequant32<T>(v, s, o, rest);
    tmem_st16(taddr + 16 * g, o);
    tmem_st16(taddr + 32 + 16 * g, rest);
  }
}

// What a dequantising warp does with the boxes 0 .. nbox - 1 of a tile, the
// first of which is box number `seq` of the kernel's life.  The sixteen warps
// are two teams that take turns at the boxes, and a team's two groups of four
// warps (the lane quarters) halve a box: a warp decodes two stages of its 32
// rows between looks at the barriers, always into the same columns of tensor
// memory.  (With one stage a look, looking cost as much as decoding.)
//
// FINE: the first half of each box (h == 0) is decoded with what the rounding of
// its weights leaves, one stage at a time in the columns of two: half of the
// weights then add no error.
template <class T, bool PAIR, int NS, bool GATED, bool FINE>  // NS: boxes in the ring
struct Dequant {
  int slot;        // of the next box of this team in the ring
  uint32_t phase;  // of its barrier
  uint32_t aphase;

  __device__ __forceinline__ Dequant() {
    slot = (threadIdx.x / 32 - 4) / 8 % NS;
    phase = 0u;
    aphase = 1u;
  }
  __device__ __forceinline__ bool tile(const LinearArgs& a, int row0, int box0, int nbox, int seq, const uint8_t* ring,
                                       const uint32_t* tab, uint64_t* nfull, uint64_t* nempty, uint64_t* afull,
                                       uint64_t* aempty, volatile int* abort, uint64_t limit) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int team = (warp - 4) / 8, h = (warp - 4) / 4 % 2, r = (warp & 3) * 32 + lane;
    const int half = 2 * team + h, gpr = a.n / GROUP;
    const uint32_t taddr = (uint32_t)(QACOL + 64 * half) + ((uint32_t)(r & ~31) << 16);
    const int wr = wrow<GATED>(a, row0, r);
    const bool in = wr < a.rows;
    const uint8_t* rungs = a.rungs + (size_t)(in ? wr : 0) * gpr;
    int b = (team ^ seq) & 1;
    int g0 = 8 * (box0 + b) + 4 * h;
    uint32_t q0 = four_rungs(rungs, in, g0, gpr), q1 = four_rungs(rungs, in, g0 + 16, gpr),
             q2 = four_rungs(rungs, in, g0 + 32, gpr);  // ahead: their loads come from far away
#pragma unroll 1
    for (; b < nbox; b += 2) {
      const uint32_t rg = q0;
      q0 = q1;
      q1 = q2;
      g0 += 16;
      q2 = four_rungs(rungs, in, g0 + 32, gpr);
      if (!wait_bar_warp(&nfull[slot], phase, abort, limit)) return false;
      const uint8_t* box = ring + slot * QBOX;
      const bool fine = FINE && h == 0;
#pragma unroll 1
      for (int k = 0; k < (fine ? 2 : 1); ++k) {
        // (Two uses of the place a box: its phases are even and odd by turns.)
        if (!wait_bar_warp(&aempty[half], fine ? (uint32_t)k ^ 1u : aphase, abort, limit)) return false;
        tc_fence_after();
        if (fine) {
          dequant_stage_both<T>(box, r, k, rg >> (16 * k), tab, taddr);
        } else {
#pragma unroll 1
          for (int u = 0; u < 2; ++u)
            dequant_stage<T>(box, r, 2 * h + u, rg >> (16 * u), tab, taddr + 32 * u);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_leader(&afull[half]);
          else
            mbar_arrive_relaxed(&afull[half]);
          if (!fine || k == 1) mbar_arrive_relaxed(&nempty[slot]);
        }
      }
      slot += 2;
      if (slot >= NS) {
        slot -= NS;
        phase ^= 1u;
      }
      aphase ^= 1u;
    }
    return true;
  }
};

// Copies of a box of codes (columns 256 b ..) of a tile's rows.
template <bool GATED>
__device__ __forceinline__ void load_box(const LinearArgs& a, uint32_t dst, const CUtensorMap* wmap, int b, int row0,
                                         uint64_t* bar) {
  if (GATED) {
#pragma unroll 1
    for (int r = 0; r < QROWS; r += 16) tma_load_2d(dst + r * 128, wmap, b * 128, wrow<true>(a, row0, r), bar);
  } else {
    tma_load_2d(dst, wmap, b * 128, row0, bar);
  }
}

// ---- up to some hundreds of tokens: one SM a tile, the columns split over a cluster

// Measured: 45 tokens, 14336 x 4096, GELU: 22.5 us, 112 tiles on 152 SMs.  A
// stage of 64 columns takes 575 cycles, all of them decoding (the vector ALU
// and the multiply-add pipe half busy each, 0.7 instructions a cycle); the
// tensor cores are 15 % busy.

constexpr int MNS = 4;     // boxes of codes
constexpr int MXS = 4;     // double stages of x (up to 128 tokens a tile; half of them above)
constexpr int MTN = 256;   // tokens per tile at most

// TO: type of the result (T, but for a gated product of bf16).
template <class T, bool GATED, class TO, bool FINE>
__global__ void __launch_bounds__(640, 1)
    k_q4_mid(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, LinearArgs a, int tn,
             int boxes, int nx, WaitCfg wc) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t nfull[MNS], nempty[MNS], xfull[MXS], xempty[MXS], afull[4], aempty[4], done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ float rowscale[QROWS], rowmax[4 * QROWS];
  volatile int* abort = &abort_sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int gpr = a.n / GROUP, nbox_all = (gpr + 7) / 8;
  const int rank = (int)blockIdx.z, nrank = (int)gridDim.z;
  const int row0 = (int)blockIdx.x * QROWS, tok0 = (int)blockIdx.y * tn;
  const int box0 = rank * boxes, nbox = max(0, min(boxes, nbox_all - box0));
  const int xbytes = tn * 128;
  uint8_t* nring = smem;
  uint8_t* xring = smem + MNS * QBOX;
  uint32_t* tab = reinterpret_cast<uint32_t*>(xring + 2 * nx * xbytes);

  if (threadIdx.x == 0) {
    for (int i = 0; i < MNS; ++i) mbar_init(&nfull[i], 1), mbar_init(&nempty[i], QDEQ / 2);
    for (int i = 0; i < MXS; ++i) mbar_init(&xfull[i], 1), mbar_init(&xempty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&afull[i], QDEQ / 4), mbar_init(&aempty[i], 1);
    mbar_init(&done, 1);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 0) {
    if (lane == 0 && !wc.no_loads) {
      int s = 0;
      uint32_t ph = 1u;
      for (int h = 0; h < 2 * nbox; ++h) {
        if (h % 2 == 0) {
          const int b = h / 2, k = b % MNS;
          if (!wait_bar(&nempty[k], ((uint32_t)(b / MNS) & 1u) ^ 1u, abort, wc.ns)) break;
          mbar_expect_tx(&nfull[k], QBOX);
          load_box<GATED>(a, smem_u32(nring + k * QBOX), &wmap, box0 + b, row0, &nfull[k]);
        }
        if (!wait_bar(&xempty[s], ph, abort, wc.ns)) break;
        mbar_expect_tx(&xfull[s], 2u * (uint32_t)xbytes);
        const uint32_t dst = smem_u32(xring + 2 * s * xbytes);
        tma_load_2d(dst, &xmap, box0 * 256 + h * 2 * QK, tok0, &xfull[s]);
        tma_load_2d(dst + (uint32_t)xbytes, &xmap, box0 * 256 + h * 2 * QK + QK, tok0, &xfull[s]);
        if (++s == nx) s = 0, ph ^= 1u;
      }
    }
  } else if (warp == 1) {
    // The whole warp walks the boxes, and everything it needs comes from the
    // loop counter: addresses stay in uniform registers, and few
    // instructions compete with the dequantising warps for the ALUs (a loop
    // that looked up each stage on its own took 650 cycles a stage).
    const bool one = elect_one();
    const uint32_t idesc = (1u << 4) | (Code8<T>::kFormat << 7) | (Code8<T>::kFormat << 10) |
                           ((uint32_t)(tn >> 3) << 17) | ((uint32_t)(QROWS >> 4) << 24);
    const uint64_t xdesc = sdesc(smem_u32(xring));
    const uint32_t step = (uint32_t)xbytes >> 4;
    bool ok = true;
    int xs = 0;
    uint32_t xph = 0u;
    for (int b = 0; b < nbox && ok; ++b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int as = 2 * (b & 1) + h;
        if (FINE && h == 0) {  // a stage and its rest, both times the stage's x
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (!(ok = wait_both(&xfull[xs], xph, &afull[as], (uint32_t)u, abort, wc.ns))) break;
            tc_fence_after();
            if (one) {
              const uint64_t xd = xdesc + (uint64_t)((2u * (uint32_t)xs + (uint32_t)u) * step);
              mma_two<false>(0u, QACOL + 64 * as, xd, xd, idesc, b == 0 && u == 0);
              if (u == 1) mma_commit(&xempty[xs]);
              mma_commit(&aempty[as]);
            }
          }
          if (!ok) break;
          if (++xs == nx) xs = 0, xph ^= 1u;
          continue;
        }
        if (!(ok = wait_both(&xfull[xs], xph, &afull[as], (uint32_t)(b >> 1) & 1u, abort, wc.ns))) break;
        tc_fence_after();
        if (one) {
          const uint64_t xd = xdesc + (uint64_t)(2u * (uint32_t)xs * step);
          mma_two<false>(0u, QACOL + 64 * as, xd, xd + step, idesc, b == 0 && h == 0);
          mma_commit(&xempty[xs]);
          mma_commit(&aempty[as]);
        }
        if (++xs == nx) xs = 0, xph ^= 1u;
      }
    }
    if (one) mma_commit(&done);
    if (!wait_bar(&done, 0u, abort, wc.ns)) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&done, 0u) && globaltimer() - t0 < wc.ns) {
      }
    }
  } else if (warp >= 4) {
    const int j = (warp - 4) / 4, q = warp & 3, r = q * 32 + lane;
    load_ladders<T, GATED>(a, row0, tab, rowscale, rowmax);
    Dequant<T, false, MNS, GATED, FINE> dq;
    bool ok = dq.tile(a, row0, box0, nbox, 0, nring, tab, nfull, nempty, afull, aempty, abort, wc.ns);
    // Sums to shared memory [token][row] (over the x ring: its MMAs are done).
    if (ok) ok = wait_bar_warp(&done, 0u, abort, wc.ns);
    if (ok) {
      tc_fence_after();
      float* part = reinterpret_cast<float*>(smem);
      const float sc = rowscale[r];
      for (int c = j * 16; c < tn; c += 64) {
        uint32_t v[16];
        tmem_ld16((uint32_t)c + ((uint32_t)(q * 32) << 16), v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          part[(c + i) * QROWS + r] = __uint_as_float(v[i]) * sc;
      }
      tc_fence_before();
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
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base_sh), "r"(512u) : "memory");
  namespace cg = cooperative_groups;
  if (nrank > 1) cg::this_cluster().sync();
  if constexpr (GATED)
    reduce_finish_gated<TO, QROWS, FINE>(a, reinterpret_cast<const float*>(smem), rank, nrank, 640, min(tn, a.tokens - tok0), tok0, row0);
  else
    reduce_finish<T, QROWS>(a, reinterpret_cast<const float*>(smem), rank, nrank, 640, min(tn, a.tokens - tok0), tok0, row0);
  if (nrank > 1) cg::this_cluster().sync();  // peers read this CTA's sums until here
}

// ---- many tokens: pairs of SMs, persistent

// Measured: 3840 tokens, 5120 x 17408: 371 us, 1.84 PFLOP/s (94 % of the plain
// library product's burst rate); 4096 tokens: 423, as the fifth round of tiles
// is a fifth full (486 when the power limit is reached).  A stage of 64
// columns takes 540 cycles, its products 512.

constexpr int PNS = 3;  // boxes of codes
constexpr int PXS = 4;  // double stages of x
constexpr int PTN = 256;  // tokens per tile at most

// Tile t: row tile t % mt (256 rows, a CTA each 128), token tile t / mt.
// Roles per CTA: warp 0 loads, warp 1 of the leader issues the MMAs of both,
// warps 4-19 dequantise, warps 20-27 write the tile out.  The sums are not
// doubled: eight stages of A and 256 tokens a tile keep the tensor cores busy
// through the tile (two sums of 160 tokens and four stages did not: 640
// cycles a stage), and the next tile's first stages are ready when the sums
// have been read.
template <class T, bool GATED, class TO, bool FINE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(896, 1)
    k_q4_many(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, LinearArgs a, int tn,
              int mt, int tiles, WaitCfg wc) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t nfull[PNS], nempty[PNS], xfull[PXS], xempty[PXS], afull[4], aempty[4],
      tfull, tempty, drain, scaled[4];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  // A tile's row scales, in turns of four: the ladders are at most three tiles
  // ahead of the sums (one box a tile: two in tensor memory, one waiting), and
  // `scaled` shows the warps that write out that a turn's have been stored.
  __shared__ float rowscale[4][QROWS], rowmax[4 * QROWS];
  volatile int* abort = &abort_sh;
  const uint32_t rank = cluster_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  const int gpr = a.n / GROUP, nbox = (gpr + 7) / 8;
  const int th = tn / 2, xbytes = th * 128;
  uint8_t* nring = smem;
  uint8_t* xring = smem + PNS * QBOX;
  uint32_t* tab = reinterpret_cast<uint32_t*>(xring + 2 * PXS * xbytes);

  if (threadIdx.x == 0) {
    for (int i = 0; i < PNS; ++i) mbar_init(&nfull[i], 1), mbar_init(&nempty[i], QDEQ / 2);
    for (int i = 0; i < PXS; ++i) mbar_init(&xfull[i], 1), mbar_init(&xempty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&afull[i], QDEQ / 2), mbar_init(&aempty[i], 1);
    mbar_init(&tfull, 1), mbar_init(&tempty, 512);
    mbar_init(&drain, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&scaled[i], 1);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();

  if (warp == 0) {
    if (lane == 0 && !wc.no_loads) {
      int box = 0, half = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += npairs) {
        const int row0 = (t % mt) * 2 * QROWS + (int)rank * QROWS, tok0 = (t / mt) * tn + (int)rank * th;
        for (int h = 0; h < 2 * nbox; ++h, ++half) {
          if (h % 2 == 0) {
            const int s = box % PNS;
            if (!(ok = wait_bar(&nempty[s], ((uint32_t)(box / PNS) & 1u) ^ 1u, abort, wc.ns))) break;
            mbar_expect_tx(&nfull[s], QBOX);
            load_box<GATED>(a, smem_u32(nring + s * QBOX), &wmap, h / 2, row0, &nfull[s]);
            ++box;
          }
          const int s = half % PXS;
          if (!(ok = wait_bar(&xempty[s], ((uint32_t)(half / PXS) & 1u) ^ 1u, abort, wc.ns))) break;
          if (rank == 0) mbar_expect_tx(&xfull[s], 4u * (uint32_t)xbytes);
          const uint32_t dst = smem_u32(xring + 2 * s * xbytes), bar = mapa_u32(smem_u32(&xfull[s]), 0);
          tma_load_2d_pair(dst, &xmap, h * 2 * QK, tok0, bar);
          tma_load_2d_pair(dst + (uint32_t)xbytes, &xmap, h * 2 * QK + QK, tok0, bar);
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {  // as in k_q4_mid
      const bool one = elect_one();
      const uint32_t idesc = (1u << 4) | (Code8<T>::kFormat << 7) | (Code8<T>::kFormat << 10) |
                             ((uint32_t)(tn >> 3) << 17) | ((uint32_t)((2 * QROWS) >> 4) << 24);
      const uint64_t xdesc = sdesc(smem_u32(xring));
      const uint32_t step = (uint32_t)xbytes >> 4;
      int box = 0, k = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += npairs, ++k) {
        if (!(ok = wait_bar(&tempty, ((uint32_t)k & 1u) ^ 1u, abort, wc.ns))) break;
        tc_fence_after();
        for (int b = 0; b < nbox && ok; ++b, ++box) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int xs = 2 * (box & 1) + h;  // x and A turn over together: two boxes
            const uint32_t ph = (uint32_t)(box >> 1) & 1u;
            if (FINE && h == 0) {  // as in k_q4_mid
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                if (!(ok = wait_both(&xfull[xs], ph, &afull[xs], (uint32_t)u, abort, wc.ns))) break;
                tc_fence_after();
                if (one) {
                  const uint64_t xd = xdesc + (uint64_t)((2u * (uint32_t)xs + (uint32_t)u) * step);
                  mma_two<true>(0u, QACOL + 64 * xs, xd, xd, idesc, b == 0 && u == 0);
                  if (u == 1) mma_commit_pair(&xempty[xs]);
                  mma_commit_pair(&aempty[xs]);
                }
              }
              if (!ok) break;
              continue;
            }
            if (!(ok = wait_both(&xfull[xs], ph, &afull[xs], ph, abort, wc.ns))) break;
            tc_fence_after();
            if (one) {
              const uint64_t xd = xdesc + (uint64_t)(2u * (uint32_t)xs * step);
              mma_two<true>(0u, QACOL + 64 * xs, xd, xd + step, idesc, b == 0 && h == 0);
              mma_commit_pair(&xempty[xs]);
              mma_commit_pair(&aempty[xs]);
            }
          }
        }
        if (ok && one) mma_commit_pair(&tfull);
      }
      if (one) mma_commit_pair(&drain);
      if (!wait_bar(&drain, 0u, abort, wc.ns)) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(&drain, 0u) && globaltimer() - t0 < wc.ns) {
        }
      }
    }
  } else if (warp >= 4 && warp < 4 + QDEQ) {
    Dequant<T, true, PNS, GATED, FINE> dq;
    int k = 0;
    bool ok = true;
    for (int t = pair; t < tiles; t += npairs, ++k) {
      const int row0 = (t % mt) * 2 * QROWS + (int)rank * QROWS;
      load_ladders<T, GATED>(a, row0, tab, rowscale[k & 3], rowmax);
      if (threadIdx.x == 128) mbar_arrive(&scaled[k & 3]);  // (behind load_ladders' last barrier)
      // After a wait has run out the warps only keep meeting at the ladders' barriers.
      if (ok) ok = dq.tile(a, row0, 0, nbox, k * nbox, nring, tab, nfull, nempty, afull, aempty, abort, wc.ns);
    }
  } else if (warp >= 4 + QDEQ) {
    // Two warps a lane quarter, each half of the tokens in sixteens: a row a
    // lane from tensor memory, turned in shared memory to 16 rows of a token
    // a lane for 16-byte accesses.  The residual of a sixteen is under way
    // before its sums are read.
    const int q = warp & 3, half = (warp - 4 - QDEQ) / 4, r = q * 32 + lane;
    float* turn = reinterpret_cast<float*>(tab + QROWS * QTAB) + (warp - 4 - QDEQ) * 16 * 36;
    const int tk = lane / 2, tr = q * 32 + lane % 2 * 16;  // this lane's token and rows after the turn
    int k = 0;
    for (int t = pair; t < tiles; t += npairs, ++k) {
      const int row0 = (t % mt) * 2 * QROWS + (int)rank * QROWS, tok0 = (t / mt) * tn;
      const int ntok = min(tn, a.tokens - tok0), c1 = min(ntok, half == 0 ? tn / 2 : tn);
      const bool v0 = rows_vec(a, row0 + tr), v1 = rows_vec(a, row0 + tr + 8);
      int c = half == 0 ? 0 : tn / 2;
      uint4 raw[2] = {};
      float ts = 1.f;
      auto fetch = [&](int cc) {
        if (GATED && a.x_scale != nullptr && cc + tk < c1) ts = a.x_scale[tok0 + cc + tk];
        if (!GATED && cc + tk < c1) {
          residual8<T>(a, tok0 + cc + tk, row0 + tr, v0, raw[0]);
          residual8<T>(a, tok0 + cc + tk, row0 + tr + 8, v1, raw[1]);
        }
      };
      fetch(c);
      // One thread looks; the others wait in the barrier.
      if (!epi8_all(threadIdx.x % 256 != 128 || (wait_bar_idle(&tfull, (uint32_t)k & 1u, abort, wc.ns) &&
                                                 wait_bar(&scaled[k & 3], (uint32_t)(k >> 2) & 1u, abort, wc.ns))))
        break;
      tc_fence_after();
      const float sc = rowscale[k & 3][r];
      for (; c < c1; c += 16) {
        uint32_t v[16];
        tmem_ld16((uint32_t)c + ((uint32_t)(q * 32) << 16), v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) turn[i * 36 + lane] = __uint_as_float(v[i]) * sc;
        __syncwarp();
        float w[2][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // Gated: eight rows of the gate, the same eight outputs of the up projection.
          const int at = GATED ? lane % 2 * 8 + i / 2 * 16 + i % 2 * 4 : lane % 2 * 16 + 4 * i;
          const float4 f = *reinterpret_cast<const float4*>(turn + tk * 36 + at);
          w[i / 2][i % 2 * 4] = f.x; w[i / 2][i % 2 * 4 + 1] = f.y;
          w[i / 2][i % 2 * 4 + 2] = f.z; w[i / 2][i % 2 * 4 + 3] = f.w;
        }
        __syncwarp();
        const uint4 now[2] = {raw[0], raw[1]};
        const float scale = ts;
        fetch(c + 16);
        if (GATED) {
          const int r8 = row0 / 2 + q * 16 + lane % 2 * 8;
          if (c + tk < c1 && r8 < a.rows / 2) finish_gated8<TO, FINE>(a, tok0 + c + tk, r8, w[0], w[1], scale);
        } else if (c + tk < c1) {
          if (row0 + tr < a.rows) finish8<T>(a, tok0 + c + tk, row0 + tr, v0, w[0], now[0]);
          if (row0 + tr + 8 < a.rows) finish8<T>(a, tok0 + c + tk, row0 + tr + 8, v1, w[1], now[1]);
        }
      }
      tc_fence_before();
      mbar_arrive_leader(&tempty);
    }
  }
  __syncthreads();
  if (abort_sh) {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
    if (threadIdx.x == 0 && a.status != nullptr) atomicOr(a.status, 2u);
  }
  tc_fence_before();
  cluster_sync_all();  // the leader's MMAs read the peer's memory until here
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base_sh), "r"(512u) : "memory");
}

// Codes [rows][n / 2] as boxes of 128 bytes (256 columns), 128-byte swizzle.
gptq_status make_code_map(CUtensorMap* m, const uint8_t* nib, int rows, int n, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return GPTQ_ERR_CUDA;
  cuuint64_t dims[2] = {(cuuint64_t)n / 2, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)n / 2};
  cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1u, 1u};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(nib), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GPTQ_OK : GPTQ_ERR_CUDA;
}

template <int TT, int FW>
size_t few_smem(int boxes) {
  constexpr int FROWS = 16 * FW;
  return 1024 + (size_t)FW * FST * FBOX + (size_t)boxes * 8 * (64 * TT + 4 * kInitFloats<TT>) +
         (size_t)(FROWS * FTAB + FW * kScaleFloats<TT>) * 4 + (size_t)FROWS * boxes * 8;
}

// A launch of k_q4_few with clusters of k CTAs.
template <class T, int TT, int FW>
struct FewLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  FewLaunch(unsigned rb, unsigned k, unsigned tz, size_t smem) {
    cfg.gridDim = dim3(rb, k, tz);
    cfg.blockDim = dim3(32 * FW);
    cfg.dynamicSmemBytes = smem;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = at[0].val.clusterDim.z = 1;
    at[0].val.clusterDim.y = k;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
};

constexpr int kFewSlots = 8;  // CTAs an SM at most
constexpr size_t few_slot_smem(int slots) { return 233472 / slots - 1536; }

template <class T, int TT, int FW, bool GATED>
gptq_status few_launch(const LinearArgs& a, cudaStream_t s) {
  constexpr int FROWS = 16 * FW;
  static DeviceOnce attr;
  static int active[9][kFewSlots + 1];  // clusters of k that run at once, by CTAs an SM
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_q4_few<T, TT, FW, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem));
    for (int k = 1; k <= 8; ++k)
      for (int n = 1; n <= kFewSlots; ++n) {
        FewLaunch<T, TT, FW> l(1, (unsigned)k, 1, std::min(few_slot_smem(n), kFewSmem));
        GQ_CUDA(cudaOccupancyMaxActiveClusters(&active[k][n], k_q4_few<T, TT, FW, GATED>, &l.cfg));
      }
    return GPTQ_OK;
  }));
  CUtensorMap m;
  GQ_TRY(make_code_map(&m, a.nibbles, a.rows, a.n, 16));
  const int nbox = (a.n / GROUP + 7) / 8;
  const int rb = (a.rows + FROWS - 1) / FROWS, tz = (a.tokens + TT - 1) / TT;
  // The split of the columns with the least time, among those whose slices
  // fit.  In units of the 500 cycles that a box costs the SM's quarter that
  // decodes it: no warp takes a box in less than two, and a CTA's start and
  // end (ladders, rungs, x; the sum over the cluster) take twenty.  Clusters
  // stay within a part of the GPU, so that fewer CTAs of large ones run at
  // once (6000 x 4096, one token: 94 clusters of eight 12.2 us, of four 8.9).
  int split = 0, boxes = 0;
  long long least = -1;
  const long long sms = num_sms(), clusters = (long long)rb * tz;
  for (int k = 8; k >= 1; --k) {
    const int bx = (nbox + k - 1) / k, sp = (nbox + bx - 1) / bx;
    const size_t smem = few_smem<TT, FW>(bx);
    if (smem > kFewSmem) break;
    int slots = kFewSlots;
    while (slots > 1 && smem > few_slot_smem(slots)) --slots;
    const long long room = active[sp][slots];
    if (room < 1) continue;
    const long long at_once = std::min((long long)slots, (clusters * sp + sms - 1) / sms) * FW / 4;
    const long long cost = ((clusters + room - 1) / room) * (bx * std::max(2ll, at_once) + 20);
    if (least < 0 || cost < least) least = cost, split = sp, boxes = bx;
  }
  if (split == 0) return GPTQ_ERR_SHAPE;
  FewLaunch<T, TT, FW> l((unsigned)rb, (unsigned)split, (unsigned)tz, few_smem<TT, FW>(boxes));
  l.cfg.stream = s;
  GQ_PROF(K_Q4_LINEAR, s);
  GQ_CUDA(cudaLaunchKernelEx(&l.cfg, k_q4_few<T, TT, FW, GATED>, m, a, boxes, wait_cfg()));
  return GPTQ_OK;
}

// Whether an eighth of the columns fits; blocks of four tokens always do.
template <int TT, int FW>
bool few_fits(const LinearArgs& a) {
  return few_smem<TT, FW>(((a.n / GROUP + 7) / 8 + 7) / 8) <= kFewSmem;
}

template <class T, bool GATED>
gptq_status few_tokens(const LinearArgs& a, cudaStream_t s) {
  if (a.tokens == 1) return few_launch<T, 1, 4, GATED>(a, s);
  if (a.tokens == 2) return few_launch<T, 2, 4, GATED>(a, s);
  if (a.tokens > 4 && few_fits<8, 8>(a)) return few_launch<T, 8, 8, GATED>(a, s);
  return few_launch<T, 4, 8, GATED>(a, s);
}

// x [tokens][n] of T as boxes of 64 columns, 128-byte swizzle.
gptq_status make_x_map(CUtensorMap* m, const LinearArgs& a, bool bf16, int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return GPTQ_ERR_CUDA;
  cuuint64_t dims[2] = {(cuuint64_t)a.n, (cuuint64_t)a.tokens};
  cuuint64_t strides[1] = {(cuuint64_t)a.ldx * 2u};
  cuuint32_t box[2] = {(cuuint32_t)QK, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1u, 1u};
  CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<void*>(a.x), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GPTQ_OK : GPTQ_ERR_CUDA;
}

// Shape of a launch of k_q4_mid: token tiles, tokens a tile, boxes a CTA,
// CTAs of a cluster; and the cycles it takes.
struct MidShape {
  int nt, tn, boxes, split;
  double cycles;
};

// Clusters of one to eight CTAs of k_q4_mid that run at once (a CTA fills an
// SM; clusters stay within a part of the GPU, so that 152 SMs hold 36 clusters
// of four, 23 of six and 15 of eight: 2048 x 4096, 45 tokens, in sixteen of
// eight took 25.2 us, in sixteen of six it takes 12.7).
template <class T, bool GATED, class TO, bool FINE>
gptq_status mid_clusters(const int** out) {
  static DeviceOnce attr;
  static int active[9];
  GQ_TRY(attr.run([](int) -> gptq_status {
    constexpr int most = 1024 + MNS * QBOX + 128 * 1024 + QROWS * QTAB * 4;
    GQ_CUDA(cudaFuncSetAttribute(k_q4_mid<T, GATED, TO, FINE>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    for (int k = 1; k <= 8; ++k) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(1, 1, (unsigned)k);
      cfg.blockDim = dim3(640);
      cfg.dynamicSmemBytes = most;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = at[0].val.clusterDim.y = 1;
      at[0].val.clusterDim.z = (unsigned)k;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      GQ_CUDA(cudaOccupancyMaxActiveClusters(&n, k_q4_mid<T, GATED, TO, FINE>, &cfg));
      active[k] = n < 1 ? 1 : n;
    }
    return GPTQ_OK;
  }));
  *out = active;
  return GPTQ_OK;
}

// The split of the columns with the least time.  A stage takes 575 cycles,
// more above 128 tokens a tile (x then streams through half the ring), a
// CTA's start and end 9000.
MidShape mid_shape(const LinearArgs& a, const int* active) {
  MidShape best{};
  const int nbox = (a.n / GROUP + 7) / 8, rb = (a.rows + QROWS - 1) / QROWS;
  const int nt = (a.tokens + MTN - 1) / MTN, tn = ((a.tokens + nt - 1) / nt + 15) / 16 * 16;
  const double stage = 575.0 + 3.3 * (tn > 128 ? tn - 128 : 0);
  for (int k = 1; k <= 8 && k <= nbox; ++k) {
    const int boxes = (nbox + k - 1) / k, split = (nbox + boxes - 1) / boxes;
    const long long rounds = ((long long)rb * nt + active[split] - 1) / active[split];
    // (In several rounds clusters wait for one another's places: 14336 x 4096,
    // 300 tokens in three rounds of pairs 60 us, in two of single CTAs 46.)
    if (split > 1 && rounds > 1) continue;
    const double cycles = (double)rounds * (boxes * 4 * stage + 9000.0);
    if (best.split == 0 || cycles < best.cycles) best = MidShape{nt, tn, boxes, split, cycles};
  }
  return best;
}

template <class T, bool GATED, class TO, bool FINE>
gptq_status mid_launch(const LinearArgs& a, const MidShape& ms, cudaStream_t s) {
  const int rb = (a.rows + QROWS - 1) / QROWS, nt = ms.nt, tn = ms.tn, boxes = ms.boxes, split = ms.split;
  const int nx = tn > 128 ? MXS / 2 : MXS;
  CUtensorMap wm, xm;
  GQ_TRY(make_code_map(&wm, a.nibbles, a.rows, a.n, GATED ? 16 : QROWS));
  GQ_TRY(make_x_map(&xm, a, std::is_same<T, __nv_bfloat16>::value, tn));
  size_t smem = 1024 + (size_t)MNS * QBOX + (size_t)2 * nx * tn * 128 + (size_t)QROWS * QTAB * 4;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)rb, (unsigned)nt, (unsigned)split);
  cfg.blockDim = dim3(640);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = (unsigned)split;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  GQ_PROF(K_Q4_MID, s);
  GQ_CUDA(cudaLaunchKernelEx(&cfg, k_q4_mid<T, GATED, TO, FINE>, wm, xm, a, tn, boxes, nx, wait_cfg()));
  return GPTQ_OK;
}

// Tokens per tile: the smallest multiple of 32 up to PTN that needs no more
// rounds of the pairs than the largest.  (Up to 256 tokens a stage's products
// take no longer than the decoding of its weights, so a round costs the same
// whatever the tile's width.)
int many_tile(int tokens, int mt, int pairs, long long& rounds) {
  auto need = [&](int tn) { return ((long long)mt * ((tokens + tn - 1) / tn) + pairs - 1) / pairs; };
  int best = PTN;
  rounds = need(PTN);
  for (int tn = PTN - 32; tn >= 32 && need(tn) == rounds; tn -= 32) best = tn;
  return best;
}

template <class T, bool GATED, class TO, bool FINE>
gptq_status many_launch(const LinearArgs& a, cudaStream_t s) {
  static DeviceOnce attr;
  constexpr int most = 1024 + PNS * QBOX + 2 * PXS * (PTN / 2) * 128 + QROWS * QTAB * 4 + 8 * 16 * 36 * 4;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_q4_many<T, GATED, TO, FINE>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    return GPTQ_OK;
  }));
  const int mt = (a.rows + 2 * QROWS - 1) / (2 * QROWS);
  const int pairs = num_sms() / 2;
  long long rounds;
  const int tn = many_tile(a.tokens, mt, pairs, rounds);
  const long long tiles = (long long)mt * ((a.tokens + tn - 1) / tn);
  if (tiles > (1ll << 30)) return GPTQ_ERR_SHAPE;
  CUtensorMap wm, xm;
  GQ_TRY(make_code_map(&wm, a.nibbles, a.rows, a.n, GATED ? 16 : QROWS));
  GQ_TRY(make_x_map(&xm, a, std::is_same<T, __nv_bfloat16>::value, tn / 2));
  const int np = tiles < pairs ? (int)tiles : pairs;
  const size_t smem = 1024 + (size_t)PNS * QBOX + (size_t)2 * PXS * (tn / 2) * 128 + (size_t)QROWS * QTAB * 4 +
                      8 * 16 * 36 * 4;
  GQ_PROF(K_Q4_MANY, s);
  k_q4_many<T, GATED, TO, FINE><<<2 * np, 896, smem, s>>>(wm, xm, a, tn, mt, (int)tiles, wait_cfg());
  GQ_LAUNCHED();
  return GPTQ_OK;
}

// Above 8 tokens: which of the two kernels.
template <class T, bool GATED, class TO, bool FINE>
gptq_status some_tokens(const LinearArgs& a, cudaStream_t s) {
  // Cycles of the two kernels as measured over 17 .. 4096 tokens (4096 x
  // 4096, 5120 x 17408, 14336 x 4096): mid_shape has the first's; a stage takes
  // 540 on a pair of SMs, which spends 13000 more on a tile.
  const int* active = nullptr;
  GQ_TRY((mid_clusters<T, GATED, TO, FINE>(&active)));
  const MidShape ms = mid_shape(a, active);
  long long rounds;
  many_tile(a.tokens, (a.rows + 2 * QROWS - 1) / (2 * QROWS), num_sms() / 2, rounds);
  // FINE decodes and multiplies half of the stages twice: 45 tokens, 14336 outputs of
  // 4096, 44.5 -> 55 us in the first (weights in the second-level cache), 4096 tokens 651 ->
  // 1050 in the other.  Measured with it, first and other: 14336 outputs of 4096, 128 tokens
  // 65 and 68 us, 256 97 and 94, 300 118 and 109 (the first is chosen), 512 149 and 138; 8704
  // of 5120, 200 tokens 52 and 54, 300 90 and 85 (the first is chosen); 4096 of 4096, 300
  // tokens 38 and 39, 700 92 and 80; 2048 of 8192, 512 tokens 54 and 62, 700 84 and 73.  With
  // 1024 columns the other's end is shorter than said here: 1000 outputs, 256 tokens 22
  // and 13 in either type, and the first is chosen.
  const double many = (double)rounds * ((a.n / GROUP + 7) / 8 * 4 * (FINE ? 870.0 : 540.0) + 13000.0);
  return ms.cycles * (FINE ? 1.25 : 1.0) <= many ? mid_launch<T, GATED, TO, FINE>(a, ms, s) : many_launch<T, GATED, TO, FINE>(a, s);
}

// Up to 8 tokens the few-token kernel is the faster (5120 x 17408: 18 / 27
// us for 1 / 8 tokens against 28); at 16 its blocks of x leave one CTA a SM
// (58 us against 29).
constexpr int kFewTokens = 8;

template <class T>
gptq_status linear_t(const LinearArgs& a, cudaStream_t s) {
  return a.tokens <= kFewTokens ? few_tokens<T, false>(a, s) : some_tokens<T, false, T, false>(a, s);
}

// x [tokens][n] of bf16 as f16 numbers times a power of two a token, which brings
// its largest finite element to 2^14 and above; infinities and NaN stay.  A CTA a
// token.
__global__ void __launch_bounds__(256) k_q4_scale_x(const __nv_bfloat16* __restrict__ x, long long ldx, int n,
                                                    __half* __restrict__ y, float* __restrict__ scale) {
  __shared__ uint32_t part[8];
  const int tok = (int)blockIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint4* src = reinterpret_cast<const uint4*>(x + tok * ldx);
  uint4* dst = reinterpret_cast<uint4*>(y + (size_t)tok * n);
  uint32_t most = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n / 8; i += 256) {
    const uint4 v = src[i];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = u[k] & 0x7fffu, hi = u[k] >> 16 & 0x7fffu;
      most = max(most, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) part[warp] = most;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) most = max(most, part[k]);
  const int up = min(141 - (int)(most >> 7), 126);  // to 2^14 .. 2^15
  const float f = __int_as_float((127 + up) << 23);
  if (threadIdx.x == 0) scale[tok] = __int_as_float((127 - up) << 23);
#pragma unroll 4
  for (int i = threadIdx.x; i < n / 8; i += 256) {
    const uint4 v = src[i];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 w = Elem<__nv_bfloat16>::to2(from_bits2<__nv_bfloat162>(u[k]));
      o[k] = bits2(Elem<__half>::make2(w.x * f, w.y * f));
    }
    dst[i] = uint4{o[0], o[1], o[2], o[3]};
  }
}

size_t scale_bytes(int tokens) { return round_up((size_t)tokens * 4, 256); }

}  // namespace

gptq_status q4tp_linear_run(int dtype, const LinearArgs& a, cudaStream_t s) {
  if (a.tokens == 0) return GPTQ_OK;
  return dtype == GPTQ_BF16 ? linear_t<__nv_bfloat16>(a, s) : linear_t<__half>(a, s);
}

size_t q4tp_gated_ws_bytes(int dtype, int tokens, int n) {
  return dtype == GPTQ_BF16 && tokens > kFewTokens ? scale_bytes(tokens) + (size_t)tokens * n * 2 : 0;
}

gptq_status q4tp_gated_run(int dtype, const LinearArgs& a, void* ws, cudaStream_t s) {
  if (a.tokens == 0) return GPTQ_OK;
  if (a.tokens <= kFewTokens) return dtype == GPTQ_BF16 ? few_tokens<__nv_bfloat16, true>(a, s) : few_tokens<__half, true>(a, s);
  if (dtype == GPTQ_F16) return some_tokens<__half, true, __half, true>(a, s);
  LinearArgs p = a;
  float* scale = static_cast<float*>(ws);
  __half* x = reinterpret_cast<__half*>(static_cast<char*>(ws) + scale_bytes(a.tokens));
  {
    GQ_PROF(K_Q4_SCALE_X, s);
    k_q4_scale_x<<<(unsigned)a.tokens, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(a.x), a.ldx, a.n, x, scale);
    GQ_LAUNCHED();
  }
  p.x = x, p.ldx = a.n, p.x_scale = scale;
  return some_tokens<__half, true, __nv_bfloat16, false>(p, s);
}

}  // namespace gq
