// Rotary positions: what the kernel of rotary.cu and the cache write of kv4.cu
// share.
//
// A pair (x0, x1) of channels with frequency f becomes, at position p,
//   y0 = x0 c - x1 s,   y1 = x1 c + x0 s,   c = gain cos(p f), s = gain sin(p f).
// f is held as a whole number of 2^64ths of a turn a position, so that p f
// modulo one turn is the low word of a 64-bit product: exact for every p, where
// 32-bit numbers would be off by whole radians past some hundred thousand
// positions, and four integer instructions, where the 64-bit pipe would need a
// multiplication at 1/64 of the 32-bit rate.  The turn's first 32 bits go to
// f32 and sincospif; the angle is off by at most pi 2^-25.
//   half layout:  pairs (i, i + rot / 2);  interleaved: (2 i, 2 i + 1).
#pragma once

#include "serve.cuh"

namespace gq {

struct RotaryArgs {
  int dim, rot;  // channels of a head, and how many of its first ones turn
  const long long* positions;
  const long long* turns;  // [rot / 2]
  float gain;
};

// cos and sin, times the gain, of frequency number i at a position.
__device__ __forceinline__ float2 turn_of(const RotaryArgs& a, long long position, int i) {
  const unsigned long long t = (unsigned long long)position * (unsigned long long)a.turns[i];
  float s, c;
  sincospif((float)(int)(t >> 32) * (1.0f / 2147483648.0f), &s, &c);
  return float2{c * a.gain, s * a.gain};
}

// One rounding order for every kernel, so that they give the same bits.
__device__ __forceinline__ float turned(float x, float other, float c, float s) {
  return __fmaf_rn(x, c, __fmul_rn(other, s));
}

// Eight channels (a, in pairs with those of b: half layout): a c + b s.
template <class T>
__device__ __forceinline__ uint4 turn_half(uint4 a, uint4 b, const float (&c)[8], const float (&s)[8]) {
  using T2 = typename Elem<T>::T2;
  const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = Elem<T>::to2(from_bits2<T2>(u[i])), y = Elem<T>::to2(from_bits2<T2>(v[i]));
    o[i] = bits2(Elem<T>::make2(turned(x.x, y.x, c[2 * i], s[2 * i]), turned(x.y, y.y, c[2 * i + 1], s[2 * i + 1])));
  }
  return uint4{o[0], o[1], o[2], o[3]};
}
// Four interleaved pairs.
template <class T>
__device__ __forceinline__ uint4 turn_pairs(uint4 a, const float* c, const float* s) {
  using T2 = typename Elem<T>::T2;
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = Elem<T>::to2(from_bits2<T2>(u[i]));
    o[i] = bits2(Elem<T>::make2(turned(x.x, x.y, c[i], -s[i]), turned(x.y, x.x, c[i], s[i])));
  }
  return uint4{o[0], o[1], o[2], o[3]};
}

}  // namespace gq
