// Eviction from the 4-bit cache: each key head of a sequence keeps its last
// `recent` tokens and the heaviest of the others, in order, from place 0 on.
//
// k_kv4_select finds, for one head of one sequence, the weight of the last token
// kept (a radix selection over the weights' bits, eight at a time) and lists
// the places that stay; k_kv4_move carries their bytes.
//
// In place a token moves towards the front, over tokens that may have to move
// themselves.  The CTAs of a cluster share a head and go through its places in
// rounds: all loads of a round, a barrier, all its stores.  A later round reads
// behind what an earlier one wrote (a token comes from its own place or a
// later one), so that the barrier is all the order it takes.
#include "serve.cuh"

namespace gq {
namespace {

constexpr int SEL = 1024;  // threads that select

// Weights in the order of whole numbers; a NaN is the lightest, both zeros are one.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w);
  if (w != w) return 0u;
  if (w == 0.f) return 0x80000000u;
  return u >> 31 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int length_of(const EvictArgs& a, int b) {
  return (int)min((long long)max(a.kv_lens[b], 0), (long long)a.table_stride * a.page_size);
}

__global__ void __launch_bounds__(SEL) k_kv4_select(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_above[SEL / 32], warp_tie[SEL / 32];
  __shared__ uint32_t prefix_sh;
  __shared__ int need_sh;
  const int b = (int)(blockIdx.x / (unsigned)a.heads), tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int len = length_of(a, b), n = min(len, a.keep);
  const int old = max(len - min(a.recent, n), 0);  // up to here the weights decide
  const float* w = a.weights + (long long)blockIdx.x * a.table_stride * a.page_size;
  const long long out_cap = (long long)a.out_stride * a.page_size;
  int* kept = a.kept + (long long)blockIdx.x * a.keep;
  float* out_w = a.out_weights + (long long)blockIdx.x * out_cap;
  if (blockIdx.x % (unsigned)a.heads == 0 && tid == 0) a.out_lens[b] = n;
  for (int i = n + tid; i < a.keep; i += SEL) kept[i] = -1;
  for (long long i = n + tid; i < out_cap; i += SEL) out_w[i] = 0.f;
  if (len <= a.keep) {
    for (int i = tid; i < n; i += SEL) kept[i] = i, out_w[i] = w[i];
    return;
  }
  // The key of the last one kept, and how many equal to it are.
  uint32_t prefix = 0;
  int need = n - (len - old);
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < old; i += SEL) {
      const uint32_t k = weight_key(w[i]);
      if (shift == 24 || k >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&hist[k >> shift & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, left = need;
      while (hist[d] < left) left -= hist[d--];
      prefix_sh = prefix | (uint32_t)d << shift;
      need_sh = left;
    }
    __syncthreads();
    prefix = prefix_sh;
    need = need_sh;
  }
  const bool any = n > len - old;
  // The list, SEL places at a time.
  int at = 0, ties = 0;
  for (int i0 = 0; i0 < len; i0 += SEL) {
    const int i = i0 + tid;
    const float v = i < len ? w[i] : 0.f;
    const uint32_t k = weight_key(v);
    bool above = i < len && (i >= old || (any && k > prefix));
    const bool tie = any && i < old && k == prefix;
    const unsigned tie_mask = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_tie[warp] = __popc(tie_mask);
    __syncthreads();
    int before = ties + __popc(tie_mask & ((1u << lane) - 1));
    for (int x = 0; x < SEL / 32; ++x) {
      if (x < warp) before += warp_tie[x];
      ties += warp_tie[x];
    }
    above = above || (tie && before < need);
    const unsigned mask = __ballot_sync(0xffffffffu, above);
    if (lane == 0) warp_above[warp] = __popc(mask);
    __syncthreads();
    int place = at + __popc(mask & ((1u << lane) - 1));
    for (int x = 0; x < SEL / 32; ++x) {
      if (x < warp) place += warp_above[x];
      at += warp_above[x];
    }
    if (above) kept[place] = i, out_w[place] = v;
    __syncthreads();
  }
}

constexpr int MOVE = 256;  // threads that move, and pieces each has in flight
constexpr int PER = 8;
constexpr int CLU = 8;  // CTAs of a cluster

// Pieces of a block of 16 tokens, in the order of its bytes: 16 bytes of codes,
// a token's (s, z) pairs (8 or 16 bytes; heads of 256: two).
template <int D>
struct Pieces {
  static constexpr int codes = 16 * (D / 32), params = 16 * (D == 256 ? 2 : 1), half = codes + params, all = 2 * half;
  static constexpr int param_bytes = D == 64 ? 8 : 16;
  // The token of piece p of a block, and its bytes' offset from the block's start for token row 0.
  static __device__ __forceinline__ void at(int p, int& row, int& off, int& step, bool& wide) {
    const int v = p >= half, q = v ? p - half : p;
    if (q < codes) {
      row = q / (D / 32), off = q % (D / 32) * 16, step = D / 2, wide = true;
    } else {
      const int r = q - codes, per = D == 256 ? 2 : 1;
      row = r / per, off = kv_param_off(D) + r % per * 16, step = D / 8, wide = D != 64;
    }
    off += v ? kv_value_off(D) : 0;
  }
};

template <int D>
__device__ __forceinline__ uint8_t* block_at(const EvictArgs& a, const int* row, int head, int t, bool write) {
  const unsigned e = (unsigned)row[t / a.page_size];
  const bool in = e < (unsigned long long)a.pages;
  if (write && !in) return nullptr;  // dropped; a read outside the pool takes page 0
  const int bpp = a.page_size / KV_BLOCK;
  return a.cache + (((in ? (long long)e : 0) * a.heads + head) * bpp + t % a.page_size / KV_BLOCK) * (long long)kv_block_bytes(D);
}

template <int D, bool IN_PLACE>
__global__ void __launch_bounds__(MOVE) k_kv4_move(EvictArgs a) {
  using P = Pieces<D>;
  const int item = (int)(blockIdx.x / CLU), rank = (int)(blockIdx.x % CLU);
  const int b = item / a.heads, head = item % a.heads;
  const int len = length_of(a, b), n = min(len, a.keep);
  if (IN_PLACE && n == len) return;  // (the whole cluster)
  const int* from = a.table + (long long)b * a.table_stride;
  const int* to = a.out_table + (long long)b * a.out_stride;
  const int* kept = a.kept + (long long)item * a.keep;
  const long long total = (long long)((n + 15) / 16) * P::all;
  for (long long p0 = 0; p0 < total; p0 += (long long)CLU * MOVE * PER) {
    uint4 data[PER];
    uint8_t* dst[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const long long p = p0 + ((long long)rank * PER + i) * MOVE + threadIdx.x;
      dst[i] = nullptr;
      if (p >= total) continue;
      int row, off, step;
      bool wide;
      P::at((int)(p % P::all), row, off, step, wide);
      const int t = (int)(p / P::all) * 16 + row;
      if (t >= n) continue;
      const int src = kept[t];
      if (IN_PLACE && src == t) continue;
      uint8_t* d = block_at<D>(a, to, head, t, true);
      if (d == nullptr) continue;
      dst[i] = d + off + row * step;
      const uint8_t* s = block_at<D>(a, from, head, src, false) + off + src % 16 * step;
      if (wide) {
        data[i] = *reinterpret_cast<const uint4*>(s);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(s);
        data[i] = uint4{v.x, v.y, 0u, 0u};
      }
    }
    if (IN_PLACE) cluster_sync_all();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (dst[i] == nullptr) continue;
      const long long p = p0 + ((long long)rank * PER + i) * MOVE + threadIdx.x;
      int row, off, step;
      bool wide;
      P::at((int)(p % P::all), row, off, step, wide);
      if (wide)
        *reinterpret_cast<uint4*>(dst[i]) = data[i];
      else
        *reinterpret_cast<uint2*>(dst[i]) = uint2{data[i].x, data[i].y};
    }
  }
}

template <int D, bool IN_PLACE>
gptq_status move_launch(const EvictArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.seqs * a.heads * CLU));
  cfg.blockDim = dim3(MOVE);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CLU;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = IN_PLACE ? 1 : 0;
  GQ_PROF(K_KV4_MOVE, s);
  GQ_CUDA(cudaLaunchKernelEx(&cfg, k_kv4_move<D, IN_PLACE>, a));
  return GPTQ_OK;
}

}  // namespace

gptq_status kv4_evict_run(int dim, bool in_place, const EvictArgs& a, cudaStream_t s) {
  {
    GQ_PROF(K_KV4_SELECT, s);
    k_kv4_select<<<(unsigned)(a.seqs * a.heads), SEL, 0, s>>>(a);
    GQ_LAUNCHED();
  }
  if (dim == 64) return in_place ? move_launch<64, true>(a, s) : move_launch<64, false>(a, s);
  if (dim == 128) return in_place ? move_launch<128, true>(a, s) : move_launch<128, false>(a, s);
  return in_place ? move_launch<256, true>(a, s) : move_launch<256, false>(a, s);
}

}  // namespace gq
