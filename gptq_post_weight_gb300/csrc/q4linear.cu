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
// 2^-18 of the result).
//
// A CTA is eight warps of 16 rows and a slice of the columns; the CTAs of a
// cluster share the rows and split the columns, and add their sums over
// distributed shared memory in rank order.  A warp keeps its own ring of
// boxes of 16 rows x 256 columns (2 KB, 128-byte swizzle, TMA), read back by
// ldmatrix: its 8 x 16-byte matrices are eight rows of one group's codes,
// and hand lane (row, t) word t of it.  The slice of x sits in shared memory
// in the order in which the nibbles come out.
#include <cooperative_groups.h>

#include "serve.cuh"

namespace gq {
namespace {

constexpr int FW = 8;             // warps
constexpr int FROWS = 16 * FW;    // rows per CTA
constexpr int FBOX = 16 * 128;    // 16 rows x 256 columns of codes
constexpr int FST = 4;            // boxes in flight per warp
constexpr int FTAB = 33;          // ladder stride in shared memory
constexpr int FMAX_SLICE = 32;    // boxes per CTA at most
constexpr int FMAX_XS = 96 << 10; // bytes of x in shared memory at most

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
  return ((w >> (4 * i)) & 0x000F000Fu) | CodeNum<T>::kMagic;
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
    case GPTQ_ACT_GELU_TANH: return 0.5f * v * (1.f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
    case GPTQ_ACT_SILU: return v / (1.f + expf(-v));
    default: return v;
  }
}

namespace {

// ---------------------------------------------------------------- few tokens

// NT: token tiles of eight; tt: tokens of this launch's token blocks.
template <class T, int NT>
__global__ void __launch_bounds__(32 * FW)
    k_q4_few(const __grid_constant__ CUtensorMap wmap, LinearArgs a, int tt, int boxes, WaitCfg wc) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[FW * FST];
  __shared__ int abort_sh;
  volatile int* abort = &abort_sh;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int gpr = a.n / GROUP;
  const int rank = (int)blockIdx.y, nrank = (int)gridDim.y;  // the cluster's split of the columns
  const int row0 = (int)blockIdx.x * FROWS, tok0 = (int)blockIdx.z * tt;
  const int ntok = min(tt, a.tokens - tok0);
  const int nbox_all = (gpr + 7) / 8;
  const int box0 = rank * boxes;
  const int nbox = max(0, min(boxes, nbox_all - box0));
  const int grp0 = box0 * 8;

  // Ring | x slice | x sums | ladders | scales of the warp's box
  uint8_t* ring = smem + warp * FST * FBOX;
  uint4* xs = reinterpret_cast<uint4*>(smem + FW * FST * FBOX);  // [group][token][4]
  float* xsum = reinterpret_cast<float*>(xs + (size_t)boxes * 8 * tt * 4);  // [group][8 NT]
  float* tabs = xsum + (size_t)boxes * 8 * 8 * NT;
  float* sc = tabs + FROWS * FTAB + warp * 128;  // [16][8]

  if (lane == 0) {
    for (int s = 0; s < FST; ++s) mbar_init(&full[warp * FST + s], 1);
    if (warp == 0) abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
    if (!wc.no_loads)
      for (int s = 0; s < FST && s < nbox; ++s) {
        mbar_expect_tx(&full[warp * FST + s], FBOX);
        tma_load_2d(smem_u32(ring + s * FBOX), &wmap, (box0 + s) * 128, row0 + warp * 16, &full[warp * FST + s]);
      }
  }

  // The rows' ladders and the slice of x, in the order of the nibbles; lanes
  // 4 i .. 4 i + 3 hold one group of a token and sum it.
  for (int i = threadIdx.x; i < FROWS * 32; i += 32 * FW) {
    const int r = i / 32;
    tabs[r * FTAB + i % 32] = row0 + r < a.rows ? a.tab[(size_t)(row0 + r) * 32 + i % 32] * CodeNum<T>::kScale : 0.f;
  }
  const T* x = static_cast<const T*>(a.x);
  const int chunks = nbox * 8 * 8 * NT * 4;
  for (int i = threadIdx.x; i < chunks; i += 32 * FW) {
    const int q = i % 4, tok = (i / 4) % (8 * NT), grp = i / (4 * 8 * NT);
    uint4 v{};
    if (tok < ntok && grp0 + grp < gpr)
      v = *reinterpret_cast<const uint4*>(x + (size_t)(tok0 + tok) * a.ldx + (size_t)(grp0 + grp) * 32 + q * 8);
    using T2 = typename Elem<T>::T2;
    const float2 f0 = Elem<T>::to2(from_bits2<T2>(v.x)), f1 = Elem<T>::to2(from_bits2<T2>(v.y)),
                 f2 = Elem<T>::to2(from_bits2<T2>(v.z)), f3 = Elem<T>::to2(from_bits2<T2>(v.w));
    float s = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (tok < tt) xs[(grp * tt + tok) * 4 + q] = pair_order(v);
    if (q == 0) xsum[grp * 8 * NT + tok] = s * CodeNum<T>::kInit;
  }
  __syncthreads();

  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

  // Scales: lane l looks up groups 4 (l % 2) .. + 3 of row l / 2 of each box.
  const int srow = lane / 2, sgrp = (lane % 2) * 4;
  const int wrow = row0 + warp * 16 + srow;
  const bool words = gpr % 4 == 0;
  auto load_rungs = [&](int b) -> uint32_t {  // four rungs; 0xff marks a group past the end
    const int g0 = (box0 + b) * 8 + sgrp;
    if (wrow >= a.rows || g0 >= gpr) return 0xffffffffu;
    const uint8_t* p = a.rungs + (size_t)wrow * gpr + g0;
    if (words) return *reinterpret_cast<const uint32_t*>(p);
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= (g0 + i < gpr ? (uint32_t)p[i] : 0xffu) << (8 * i);
    return r;
  };
  uint32_t rung_next = nbox > 0 ? load_rungs(0) : 0u;
  bool ok = true;
  for (int b = 0; b < nbox; ++b) {
    const int st = b % FST;
    const uint32_t rg = rung_next;
    if (b + 1 < nbox) rung_next = load_rungs(b + 1);
    __syncwarp();
    float4 s4;
    float* sp = &s4.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = (rg >> (8 * i)) & 0xffu;
      sp[i] = r < 32u ? tabs[(warp * 16 + srow) * FTAB + r] : 0.f;
    }
    *reinterpret_cast<float4*>(sc + srow * 8 + sgrp) = s4;
    ok = mbar_wait(&full[warp * FST + st], (uint32_t)(b / FST) & 1u, abort, wc.ns);
    if (!__all_sync(0xffffffffu, ok)) {
      ok = false;
      break;
    }
    __syncwarp();
    const uint32_t base = smem_u32(ring + st * FBOX);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 sa = *reinterpret_cast<const float4*>(sc + g * 8 + 4 * h);
      const float4 sb = *reinterpret_cast<const float4*>(sc + (g + 8) * 8 + 4 * h);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        // Matrices: (rows 0-7, group c), (rows 8-15, group c), the same for c + 1.
        const int c = 4 * h + 2 * p;
        const int mrow = (lane & 7) + (lane & 8), mgrp = c + (lane >> 4);
        uint32_t w[4];
        ldmatrix4(w, base + (uint32_t)(mrow * 128 + ((mgrp ^ (mrow & 7)) * 16)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int grp = b * 8 + c + u;
          const float s_lo = (p == 0) ? (u == 0 ? sa.x : sa.y) : (u == 0 ? sa.z : sa.w);
          const float s_hi = (p == 0) ? (u == 0 ? sb.x : sb.y) : (u == 0 ? sb.z : sb.w);
          const uint32_t a0[4] = {code_num<T>(w[2 * u], 0), code_num<T>(w[2 * u + 1], 0), code_num<T>(w[2 * u], 1),
                                  code_num<T>(w[2 * u + 1], 1)};
          const uint32_t a1[4] = {code_num<T>(w[2 * u], 2), code_num<T>(w[2 * u + 1], 2), code_num<T>(w[2 * u], 3),
                                  code_num<T>(w[2 * u + 1], 3)};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float2 init = *reinterpret_cast<const float2*>(xsum + grp * 8 * NT + 8 * j + 2 * t);
            float d[4] = {init.x, init.y, init.x, init.y};
            uint4 xb{};
            if (8 * j + g < tt) xb = xs[(grp * tt + 8 * j + g) * 4 + t];
            mma16816<T>(d, a0, xb.x, xb.y);
            mma16816<T>(d, a1, xb.z, xb.w);
            acc[j][0] = fmaf(s_lo, d[0], acc[j][0]);
            acc[j][1] = fmaf(s_lo, d[1], acc[j][1]);
            acc[j][2] = fmaf(s_hi, d[2], acc[j][2]);
            acc[j][3] = fmaf(s_hi, d[3], acc[j][3]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0 && b + FST < nbox) {
      mbar_expect_tx(&full[warp * FST + st], FBOX);
      tma_load_2d(smem_u32(ring + st * FBOX), &wmap, (box0 + b + FST) * 128, row0 + warp * 16,
                  &full[warp * FST + st]);
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
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      part[(8 * j + 2 * t + (e & 1)) * FROWS + warp * 16 + g + (e >> 1) * 8] = acc[j][e];
  namespace cg = cooperative_groups;
  if (nrank > 1)
    cg::this_cluster().sync();
  else
    __syncthreads();
  const int outs = ntok * FROWS;
  for (int i = rank * 32 * FW + threadIdx.x; i < outs; i += nrank * 32 * FW) {
    const int tok = i / FROWS, r = row0 + i % FROWS;
    float v = 0.f;
    if (nrank > 1) {
      const uint32_t la = smem_u32(part + i);
      for (int k = 0; k < nrank; ++k) {
        float o;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(mapa_u32(la, (uint32_t)k)) : "memory");
        v += o;
      }
    } else {
      v = part[i];
    }
    if (r < a.rows) {
      if (a.bias != nullptr) v += Elem<T>::to(static_cast<const T*>(a.bias)[r]);
      v = activate(v, a.act);
      const size_t tk = (size_t)(tok0 + tok);
      if (a.residual != nullptr) v += Elem<T>::to(static_cast<const T*>(a.residual)[tk * a.ldr + r]);
      static_cast<T*>(a.y)[tk * a.ldy + r] = Elem<T>::from(v);
    }
  }
  if (nrank > 1) cg::this_cluster().sync();  // peers read this CTA's sums until here
}

// Codes [rows][n / 2] bytes as boxes of 128 bytes x 16 rows.
gptq_status make_code_map(CUtensorMap* m, const uint8_t* nib, int rows, int n, int box_bytes, int box_rows,
                          CUtensorMapSwizzle sw) {
  auto fn = encode_fn();
  if (fn == nullptr) return GPTQ_ERR_CUDA;
  cuuint64_t dims[2] = {(cuuint64_t)n / 2, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)n / 2};
  cuuint32_t box[2] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1u, 1u};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(nib), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GPTQ_OK : GPTQ_ERR_CUDA;
}

size_t few_smem(int boxes, int tt, int nt) {
  size_t ring = (size_t)FW * FST * FBOX, xs = (size_t)boxes * 8 * tt * 64;
  size_t rest = ((size_t)boxes * 8 * 8 * nt + FROWS * FTAB + FW * 128) * 4;
  return 1024 + ring + xs + rest;
}

template <class T, int NT>
gptq_status few_launch(const LinearArgs& a, cudaStream_t s) {
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_q4_few<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 << 10));
    return GPTQ_OK;
  }));
  CUtensorMap m;
  GQ_TRY(make_code_map(&m, a.nibbles, a.rows, a.n, 128, 16, CU_TENSOR_MAP_SWIZZLE_128B));
  const int nbox = (a.n / GROUP + 7) / 8;
  const int rb = (a.rows + FROWS - 1) / FROWS;
  // About two CTAs a SM, and slices that fit in shared memory.
  int split = (2 * num_sms()) / rb;
  split = split < 1 ? 1 : (split > 8 ? 8 : split);
  while ((nbox + split - 1) / split > FMAX_SLICE) ++split;  // n <= 65536: at most 8
  int boxes = (nbox + split - 1) / split;
  split = (nbox + boxes - 1) / boxes;
  int tt = a.tokens < 8 * NT ? a.tokens : 8 * NT;
  while ((size_t)boxes * 8 * tt * 64 > (size_t)FMAX_XS) --tt;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)rb, (unsigned)split, (unsigned)((a.tokens + tt - 1) / tt));
  cfg.blockDim = dim3(32 * FW);
  cfg.dynamicSmemBytes = few_smem(boxes, tt, NT);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = (unsigned)split;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  GQ_PROF(K_Q4_LINEAR, s);
  GQ_CUDA(cudaLaunchKernelEx(&cfg, k_q4_few<T, NT>, m, a, tt, boxes, wait_cfg()));
  return GPTQ_OK;
}

template <class T>
gptq_status linear_t(const LinearArgs& a, cudaStream_t s) {
  if (a.tokens <= 8) return few_launch<T, 1>(a, s);
  return few_launch<T, 2>(a, s);
}

}  // namespace

gptq_status q4tp_linear_run(int dtype, const LinearArgs& a, cudaStream_t s) {
  if (a.tokens == 0) return GPTQ_OK;
  return dtype == GPTQ_BF16 ? linear_t<__nv_bfloat16>(a, s) : linear_t<__half>(a, s);
}

}  // namespace gq
