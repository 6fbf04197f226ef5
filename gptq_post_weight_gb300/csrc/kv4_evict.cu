// Eviction from the 4-bit cache: each key head of a sequence keeps its last
// `recent` tokens and the heaviest of the others, in order, from place 0 on.
//
// k_kv4_select finds, for one head of one sequence, the weight of the last token
// kept (a radix selection over the weights' bits, eleven at a time: more bins
// than the exponent's alone, in which the first digits of most weights would
// meet) and lists the places that stay, a warp a stretch of them.
// k_kv4_move carries their bytes.
//
// In place a token moves towards the front, over tokens that may have to move
// themselves.  The CTAs of a cluster share a head and go through its places in
// rounds: all loads of a round, a barrier, all its stores.  A later round reads
// behind what an earlier one wrote (a token comes from its own place or a
// later one), so that the barrier is all the order it takes.
//
// Measured: 8 heads of 128, one sequence of 4096 tokens to 1024, in place: 13 us,
// two launches' latencies; of 32768 to 8192 42 us, of 131072 to 8192 148 (eight CTAs
// select).  48 sequences of up to 16384 tokens to 2000, into other
// pages: 88 us; the selection is some 32 of them (one CTA a head: 384 of unequal
// length on 152 SMs, 60 % of the issue slots), the moves 57 (72 % of the memory's
// cycles: a kept token is four pieces, of which the two of parameters are 16 bytes).
// Tables wider than the sequences cost: zeros for the weights past the end, and above
// 16640 places the selection of long heads (one sequence of 4096: 14.3 us in 32768
// places, 20.2 in 131072; 48 of 16384: 94.6 in 20032, 106 in 65536).
#include "serve.cuh"

namespace gq {
namespace {

constexpr int SBINS = 2048, SCAN = SBINS / 4;  // bins, and threads that look through them
constexpr int kStaged = 40 << 10;  // places of a head that are kept in shared memory at most

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

// STAGED: the keys of a head fit shared memory (else they are read again for each digit).
// SEL: threads.
template <bool STAGED, int SEL>
__global__ void __launch_bounds__(SEL) k_kv4_select(EvictArgs a, bool few) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[SBINS];
  __shared__ int2 part[SEL / 32];
  __shared__ uint32_t prefix_sh;
  __shared__ int need_sh;
  constexpr int W = SEL / 32;
  const int b = (int)(blockIdx.x / (unsigned)a.heads), tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int len = length_of(a, b), n = min(len, a.keep);
  const int old = max(len - min(a.recent, n), 0);  // up to here the weights decide
  const float* w = a.weights + (long long)blockIdx.x * a.table_stride * a.page_size;
  const long long out_cap = (long long)a.out_stride * a.page_size;
  int* kept = a.kept + (long long)blockIdx.x * a.keep;
  float* out_w = a.out_weights + (long long)blockIdx.x * out_cap;
  if (blockIdx.x % (unsigned)a.heads == 0 && tid == 0) a.out_lens[b] = n;
  for (int i = n + tid; i < a.keep; i += SEL) kept[i] = -1;
  if (len <= a.keep)
    for (int i = tid; i < n; i += SEL) kept[i] = i, out_w[i] = w[i];
  // k_kv4_move may set itself up.  (Not beside many heads: its CTAs would fill the SMs
  // whose heads are short, and start there, not where memory is idle: 113 us, not 92; beside
  // 1024 threads a head, 48 sequences to 20032, 104.5, not 101.7.)
  if (few) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (long long i = n + tid; i < out_cap; i += SEL) out_w[i] = 0.f;
  if (len <= a.keep) return;
  int need = n - (len - old);
  const bool any = need > 0;
  auto key = [&](int i) { return STAGED ? keys[i] : weight_key(w[i]); };
  if (STAGED && any) {
#pragma unroll 8
    for (int i = tid; i < len; i += SEL) keys[i] = weight_key(w[i]);
  }
  // The key of the last one kept, and how many of those equal to it stay.
  uint32_t prefix = 0;
  for (int shift = 21; any; shift = max(shift - 11, 0)) {
    const uint32_t mask = shift == 21 ? 0u : shift == 10 ? ~0u << 21 : ~0u << 10;  // the digits found
    const uint32_t bins = shift == 0 ? 1023u : 2047u;
    for (int i = tid; i < SBINS; i += SEL) hist[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (int i = tid; i < old; i += SEL) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&hist[k >> shift & bins], 1);
    }
    __syncthreads();
    // Keys in the bins above: a thread has four bins, from the highest down.
    const int4 mine = tid < SCAN ? reinterpret_cast<const int4*>(hist)[SCAN - 1 - tid] : int4{};
    const int sum = (mine.x + mine.y) + (mine.z + mine.w);
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) part[warp].x = inc;
    __syncthreads();
    int above = inc - sum;
    for (int x = 0; x < warp; ++x) above += part[x].x;
    if (above < need && need <= above + sum) {  // one thread's (threads without bins have a sum of 0)
      int d = 4 * (SCAN - 1 - tid) + 3;
      const int c[4] = {mine.w, mine.z, mine.y, mine.x};
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (d % 4 == 3 - x && above + c[x] < need) above += c[x], --d;
      prefix_sh = prefix | (uint32_t)d << shift;
      need_sh = need - above;
    }
    __syncthreads();
    prefix = prefix_sh;
    need = need_sh;
    if (shift == 0) break;
  }
  // A warp lists a stretch of the places: first how many stay before it.
  const int each = (len + W * 32 - 1) / (W * 32) * 32, i0 = min(warp * each, len), i1 = min(i0 + each, len);
  const int i2 = any ? min(i1, old) : i0;  // up to here the keys decide, from `old` on all stay
  int above = 0, ties = 0;
#pragma unroll 8
  for (int i = i0 + lane; i < i2; i += 32) {
    const uint32_t k = key(i);
    above += k > prefix;
    ties += k == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above) + max(i1 - max(i0, old), 0);
  ties = __reduce_add_sync(0xffffffffu, ties);
  __syncthreads();  // (part is read above)
  if (lane == 0) part[warp] = int2{above, ties};
  __syncthreads();
  int place = 0, tied = 0, all_ties = 0;
  for (int x = 0; x < W; ++x) {
    if (x < warp) place += part[x].x, tied += part[x].y;
    all_ties += part[x].y;
  }
  place += min(tied, need);
  const unsigned before = (1u << lane) - 1u;
  const bool some = all_ties > need;  // (else all of them stay: the same for every thread)
#pragma unroll 4
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const uint32_t k = i < i2 ? key(i) : 0u;
    bool stays = i < i1 && (i >= old || (i < i2 && k >= prefix));
    if (some) {
      const bool tie = i < i2 && k == prefix;
      const unsigned equal = __ballot_sync(0xffffffffu, tie);
      if (tie && tied + __popc(equal & before) >= need) stays = false;
      tied += __popc(equal);
    }
    const unsigned all = __ballot_sync(0xffffffffu, stays);
    if (stays) {
      const int at = place + __popc(all & before);
      kept[at] = i;
      // The weight from its key, without a load's latency, if it has one of its own.
      const uint32_t own = STAGED && any ? keys[i] : 0u;
      out_w[at] = own == 0u || own == 0x80000000u ? w[i] : __uint_as_float(own >> 31 ? own & ~(1u << 31) : ~own);
    }
    place += __popc(all);
  }
}

constexpr int MOVE = 256;  // threads that move
constexpr int CLU = 8;     // CTAs of a head

// Pieces of a block of 16 tokens, in the order of its bytes: 16 bytes of codes,
// a token's (s, z) pairs (8 or 16 bytes; heads of 256: two).
template <int D>
struct Pieces {
  static constexpr int blocks = D == 256 ? 4 : 8;  // of a CTA's round
  static constexpr int codes = 16 * (D / 32), params = 16 * (D == 256 ? 2 : 1), half = codes + params, all = 2 * half;
  static constexpr int each = blocks * all / MOVE;  // pieces of a thread: as many loads in flight
  // The token of piece p of a block, its bytes' offset from the block's start for
  // token 0, and bytes from token to token; whether it is sixteen.
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
__device__ __forceinline__ uint8_t* block_at(const EvictArgs& a, const int* row, int head, int blk, bool write) {
  const int bpp = a.page_size / KV_BLOCK, page = blk / bpp;
  const unsigned e = (unsigned)row[page];
  const bool in = e < (unsigned long long)a.pages;
  if (write && !in) return nullptr;  // dropped; a read outside the pool takes page 0
  return a.cache + (((in ? (long long)e : 0) * a.heads + head) * bpp + (blk - page * bpp)) * (long long)kv_block_bytes(D);
}

template <int D, bool IN_PLACE>
__global__ void __launch_bounds__(MOVE, 4) k_kv4_move(EvictArgs a) {
  using P = Pieces<D>;
  static_assert(P::blocks * P::all % MOVE == 0 && P::blocks * 16 <= MOVE, "a round is a thread's pieces");
  struct From {
    const uint8_t* block;  // null: stays where it is, or goes nowhere
    int row;
  };
  __shared__ From from[P::blocks * 16];
  __shared__ uint8_t* to[P::blocks];
  const int item = (int)(blockIdx.x / CLU), rank = (int)(blockIdx.x % CLU);
  const int b = item / a.heads, head = item % a.heads;
  const int len = length_of(a, b), n = min(len, a.keep), blocks = (n + 15) / 16;
  const int* table = a.table + (long long)b * a.table_stride;
  const int* out = a.out_table + (long long)b * a.out_stride;
  const int* kept = a.kept + (long long)item * a.keep;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the list is there
  if (IN_PLACE && n == len) return;                   // (the whole cluster)
  for (int b0 = 0; b0 < blocks; b0 += CLU * P::blocks) {
    const int first = b0 + rank * P::blocks, have = min(P::blocks, blocks - first);  // this CTA's blocks
    if ((int)threadIdx.x < P::blocks * 16) {
      const int lb = threadIdx.x / 16, t = first * 16 + (int)threadIdx.x;
      From f{nullptr, 0};
      if (t < n) {
        const int src = kept[t];
        uint8_t* dst = block_at<D>(a, out, head, first + lb, true);
        if (threadIdx.x % 16 == 0) to[lb] = dst;
        if (dst != nullptr && !(IN_PLACE && src == t)) f = From{block_at<D>(a, table, head, src / KV_BLOCK, false), src % KV_BLOCK};
      }
      from[threadIdx.x] = f;
    }
    __syncthreads();
    uint4 data[P::each];
#pragma unroll
    for (int i = 0; i < P::each; ++i) {
      const int l = i * MOVE + (int)threadIdx.x, lb = l / P::all;
      int row, off, step;
      bool wide;
      P::at(l - lb * P::all, row, off, step, wide);
      if (lb >= have) break;
      const From f = from[lb * 16 + row];
      if (f.block == nullptr) continue;
      const uint8_t* s = f.block + off + f.row * step;
      if (wide) {
        data[i] = *reinterpret_cast<const uint4*>(s);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(s);
        data[i].x = v.x, data[i].y = v.y;
      }
    }
    if (IN_PLACE) cluster_sync_all();
#pragma unroll
    for (int i = 0; i < P::each; ++i) {
      const int l = i * MOVE + (int)threadIdx.x, lb = l / P::all;
      int row, off, step;
      bool wide;
      P::at(l - lb * P::all, row, off, step, wide);
      if (lb >= have) break;
      if (from[lb * 16 + row].block == nullptr) continue;
      uint8_t* d = to[lb] + off + row * step;
      if (wide)
        *reinterpret_cast<uint4*>(d) = data[i];
      else
        *reinterpret_cast<uint2*>(d) = uint2{data[i].x, data[i].y};
    }
    __syncthreads();  // the lists are written again
  }
}

template <int D, bool IN_PLACE>
gptq_status move_launch(const EvictArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.seqs * a.heads * CLU));
  cfg.blockDim = dim3(MOVE);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CLU;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = IN_PLACE ? 2 : 1;
  GQ_PROF(K_KV4_MOVE, s);
  GQ_CUDA(cudaLaunchKernelEx(&cfg, k_kv4_move<D, IN_PLACE>, a));
  return GPTQ_OK;
}

}  // namespace

gptq_status kv4_evict_run(int dim, bool in_place, const EvictArgs& a, cudaStream_t s) {
  static DeviceOnce attr;
  GQ_TRY(attr.run([](int) -> gptq_status {
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_select<true, 1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStaged * 4));
    GQ_CUDA(cudaFuncSetAttribute(k_kv4_select<true, 512>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStaged * 4));
    return GPTQ_OK;
  }));
  const long long cap = (long long)a.table_stride * a.page_size;
  {
    GQ_PROF(K_KV4_SELECT, s);
    // Two CTAs of 1024 threads fit an SM; more heads start together where three of 512 and
    // their keys do (measured before the listing's last form: one sequence to 16384 19.4 us with
    // 1024 threads, 23 with 512; 48 of them 95 and 92, 48 to 4096 45 and 42).
    const unsigned grid = (unsigned)(a.seqs * a.heads), bytes = cap <= kStaged ? (unsigned)cap * 4 : 0;
    const bool few = grid <= 2u * (unsigned)num_sms();
    if (bytes == 0)
      k_kv4_select<false, 1024><<<grid, 1024, 0, s>>>(a, few);
    else if (few || bytes > 65 << 10)
      k_kv4_select<true, 1024><<<grid, 1024, bytes, s>>>(a, few);
    else
      k_kv4_select<true, 512><<<grid, 512, bytes, s>>>(a, false);
    GQ_LAUNCHED();
  }
  if (dim == 64) return in_place ? move_launch<64, true>(a, s) : move_launch<64, false>(a, s);
  if (dim == 128) return in_place ? move_launch<128, true>(a, s) : move_launch<128, false>(a, s);
  return in_place ? move_launch<256, true>(a, s) : move_launch<256, false>(a, s);
}

}  // namespace gq
