// Rotary positions of [tokens][heads][dim] (rotary.cuh has the formula).
//
// A thread owns one token and sixteen channels of a head -- two octets that
// hold the same eight frequencies -- and walks over heads: the sines and
// cosines, some 200 instructions, are taken once for all of them, and what is
// left a head is two 16-byte loads, 32 multiplications and two stores.  Both
// octets of a pair are the thread's own, so that the call may write over its
// input.  Bytes bound it: 16001 tokens of 40 heads of 128 in 58.3 us, 5.6 TB/s
// read and written; one token 2.5 us.
#include "rotary.cuh"

namespace gq {
namespace {

struct RotaryIo {
  const void* x;
  long long xt, xh;  // elements between tokens and between heads
  void* y;
  long long yt, yh;
  int tokens, heads;
};

template <class T, bool HALF>
__global__ void __launch_bounds__(256) k_rotary(RotaryIo io, RotaryArgs a, int take) {
  const int units = a.dim / 16, i = (int)(blockIdx.x * 256 + threadIdx.x);
  const int tok = i / units, u = i - tok * units;
  if (tok >= io.tokens) return;
  const int h0 = (int)blockIdx.y * take, h1 = min(h0 + take, io.heads);
  // First channels of the two octets, and whether they turn.
  const int turning = a.rot / 16;
  int ca, cb;
  bool ra, rb;
  if (HALF) {
    ra = rb = u < turning;
    ca = ra ? 8 * u : 16 * u;
    cb = ra ? ca + a.rot / 2 : ca + 8;
  } else {
    ca = 8 * u, cb = ca + a.dim / 2;
    ra = ca < a.rot, rb = cb < a.rot;
  }
  const T* x = static_cast<const T*>(io.x) + tok * io.xt;
  T* y = static_cast<T*>(io.y) + tok * io.yt;
  if (!ra && !rb && io.x == io.y) return;  // in place: nothing to do
  float c[8], s[8], ns[8];
  const long long position = a.positions[tok];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float2 t{0.f, 0.f};
    if (HALF) {
      if (ra) t = turn_of(a, position, ca + k);
    } else if (k < 4 ? ra : rb) {
      t = turn_of(a, position, (k < 4 ? ca : cb) / 2 + k % 4);
    }
    c[k] = t.x, s[k] = t.y, ns[k] = -t.y;
  }
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const uint4 va = *reinterpret_cast<const uint4*>(x + h * io.xh + ca), vb = *reinterpret_cast<const uint4*>(x + h * io.xh + cb);
    uint4 oa, ob;
    if (HALF) {
      oa = turn_half<T>(va, vb, c, ns), ob = turn_half<T>(vb, va, c, s);
    } else {
      oa = turn_pairs<T>(va, c, s), ob = turn_pairs<T>(vb, c + 4, s + 4);
    }
    *reinterpret_cast<uint4*>(y + h * io.yh + ca) = ra ? oa : va;
    *reinterpret_cast<uint4*>(y + h * io.yh + cb) = rb ? ob : vb;
  }
}

}  // namespace

gptq_status rotary_run(int dtype, bool half, const void* x, long long xt, long long xh, int tokens, int heads,
                       const RotaryArgs& a, void* y, long long yt, long long yh, cudaStream_t s) {
  if (tokens == 0) return GPTQ_OK;
  const RotaryIo io{x, xt, xh, y, yt, yh, tokens, heads};
  const long long threads = (long long)tokens * (a.dim / 16);
  // Heads a thread: as many as leave every SM 512 threads, sixteen at most.
  // Measured, 32 heads of 128 (2048 / 1024 / 512 / 256 threads an SM): 1000 tokens 6.7 /
  // 6.7 / 5.0 / 5.5 us, 2000 11.3 / 7.4 / 6.8 / 7.6, 4000 11.5 / 10.5 / 9.3 / 9.5.
  const long long most = threads * heads / (num_sms() * 512ll);
  const int take = (int)std::min<long long>(std::max<long long>(most, 1), 16);
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)((heads + take - 1) / take));
  GQ_PROF(K_ROTARY, s);
  if (dtype == GPTQ_BF16) {
    if (half) k_rotary<__nv_bfloat16, true><<<grid, 256, 0, s>>>(io, a, take);
    else k_rotary<__nv_bfloat16, false><<<grid, 256, 0, s>>>(io, a, take);
  } else {
    if (half) k_rotary<__half, true><<<grid, 256, 0, s>>>(io, a, take);
    else k_rotary<__half, false><<<grid, 256, 0, s>>>(io, a, take);
  }
  GQ_LAUNCHED();
  return GPTQ_OK;
}

}  // namespace gq
