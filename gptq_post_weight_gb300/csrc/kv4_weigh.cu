// What the queries of an attention call looked at: for every cached token the
// sum of its attention weights, added to a running total.
//
//   weights[b][h][t] += sum over rows r of exp(scale q_r k_t - lse_r)
//
// The logarithm of each row's sum comes from the attention itself, so that one
// pass over the keys is all it takes, and nothing of a token's sum depends on
// another token.
#include "serve.cuh"

namespace gq {
namespace {

constexpr int WKEYS = 128;

// A thread has a key, decoded on the fly; the rows come by one at a time.
template <class T, int D>
__global__ void __launch_bounds__(WKEYS) k_kv4_weigh(AttnArgs a, const float* lse, float* weights, long long items, int tiles) {
  using T2 = typename Elem<T>::T2;
  __shared__ float q[D];
  const long long cap = (long long)a.table_stride * a.page_size;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int tile = (int)(it % tiles), head = (int)(it / tiles % a.heads), b = (int)(it / tiles / a.heads);
    const int q0 = a.q_starts ? min(max(a.q_starts[b], 0), a.tq) : b;
    const int nq = a.q_starts ? min(min(max(a.q_starts[b + 1], q0), a.tq) - q0, a.max_q) : 1;
    const int len = (int)min((long long)max(a.kv_lens[b], 0), cap);
    if (tile * WKEYS >= len || nq == 0) continue;
    const int t = tile * WKEYS + threadIdx.x;
    const uint32_t* par = value_params<D>(a, b, head, min(t, len - 1));
    par = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(par) - kv_value_off(D));
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(par) - kv_param_off(D) + (min(t, len - 1) % KV_BLOCK) * (D / 2 - D / 8);
    float sum = 0.f;
    for (int r = 0; r < nq * a.group; ++r) {
      const long long tok = q0 + r / a.group;
      const int hq = head * a.group + r % a.group;
      __syncthreads();
      for (int i = threadIdx.x; i < D; i += WKEYS) q[i] = Elem<T>::to(static_cast<const T*>(a.q)[tok * a.q_ts + hq * a.q_hs + i]);
      __syncthreads();
      if (t > len - nq + r / a.group || t >= len) continue;
      float s = 0.f;
      for (int w = 0; w < D / 8; ++w) {
        const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[w], p = par[w / 4];
        const T2 s2 = from_bits2<T2>(__byte_perm(p, p, 0x1010)), z2 = from_bits2<T2>(__byte_perm(p, p, 0x3232));
        for (int i = 0; i < 4; ++i) {
          const float2 v = Elem<T>::to2(__hfma2(code16<T>(c, i), s2, z2));
          s = fmaf(v.x, q[8 * w + i], fmaf(v.y, q[8 * w + i + 4], s));
        }
      }
      sum += exp2f(s * a.scale_log2 - lse[tok * a.heads * a.group + hq] * 1.4426950408889634f);
    }
    if (t < len) weights[((long long)b * a.heads + head) * cap + t] += sum;
  }
}

template <class T>
gptq_status weigh_t(int dim, const AttnArgs& a, const float* lse, float* weights, cudaStream_t s) {
  const int tiles = (int)(((long long)a.table_stride * a.page_size + WKEYS - 1) / WKEYS);
  const long long items = (long long)tiles * a.heads * a.seqs;
  const unsigned grid = (unsigned)std::min<long long>(items, num_sms() * 16);
  GQ_PROF(K_KV4_WEIGH, s);
  if (dim == 64) k_kv4_weigh<T, 64><<<grid, WKEYS, 0, s>>>(a, lse, weights, items, tiles);
  else if (dim == 128) k_kv4_weigh<T, 128><<<grid, WKEYS, 0, s>>>(a, lse, weights, items, tiles);
  else k_kv4_weigh<T, 256><<<grid, WKEYS, 0, s>>>(a, lse, weights, items, tiles);
  GQ_LAUNCHED();
  return GPTQ_OK;
}

}  // namespace

gptq_status kv4_weigh_run(int dtype, int dim, const AttnArgs& a, const float* lse, float* weights, cudaStream_t s) {
  return dtype == GPTQ_BF16 ? weigh_t<__nv_bfloat16>(dim, a, lse, weights, s) : weigh_t<__half>(dim, a, lse, weights, s);
}

}  // namespace gq
