// Rotary positions: what the kernel of rotary.cu and the cache write of kv4.cu
// share.
//
// A pair (x0, x1) of channels with frequency f becomes, at position p,
//   y0 = x0 c - x1 s,   y1 = x1 c + x0 s,   c = gain cos(p f), s = gain sin(p f).
// f is held as a whole number of 2^64ths of a turn a position, so that p f
// modulo one turn is the low word of a 64-bit product: exact for every p, where
// 32-bit numbers would be off by whole radians past some hundred thousand
// positions, and four integer instructions, where the 64-bit pipe would need a
// multiplication at 1/64 of the 32-bit rate.  The turn is rounded to 32 bits, and
// its nearest quarter taken off in whole numbers; the rest, an eighth of a turn at
// most, goes to f32: the angle is off by at most pi (2^-27 + 2^-32).
// (Of a whole turn in f32 that was pi 2^-25, and twice as many turned keys came to
// the other side of a bf16 number's middle as an exact angle sends there.)
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

// cos and sin, times the gain, of frequency number i at a position.  Both are Taylor's
// polynomials in the rest u (turns, |u| <= 1/8): of the sine to u^9, 2 pi in two numbers
// (1.2 2^-24 of it, by trying a million u), of the cosine to u^8, whose coefficient has nine tenths of
// the next term at the end of the range (1.5 2^-24).  (sincospif of the rest, which looks
// for the quarter once more, cost 1000 tokens of 32 heads 5.5 us, this 4.9.)
__device__ __forceinline__ float2 turn_of(const RotaryArgs& a, long long position, int i) {
  const unsigned long long t = (unsigned long long)position * (unsigned long long)a.turns[i];
  // Past the middle between two quarters the next one counts.
  const uint32_t q = (uint32_t)(t >> 32) + ((uint32_t)t >> 31) + (1u << 29);
  const float u = (float)((int)(q & ((1u << 30) - 1u)) - (1 << 29)) * 0x1p-32f, w = u * u;
  float s = fmaf(w, 42.058693944897634f, -76.70585975306136f);
  s = fmaf(w, fmaf(w, s, 81.60524927607504f), -41.341702240399755f);
  s = fmaf(u, 6.283185307179586f, u * fmaf(w, s, -1.7484555e-07f));
  float c = fmaf(w, 59.8730221f, -85.45681720669371f);
  c = fmaf(w, fmaf(w, fmaf(w, c, 64.93939402266828f), -19.739208802178716f), 1.f);
  const float x = q & 1u << 30 ? s : c, y = q & 1u << 30 ? c : s;
  return float2{__uint_as_float(__float_as_uint(x) ^ (q + (1u << 30) & 1u << 31)) * a.gain,
                __uint_as_float(__float_as_uint(y) ^ (q & 1u << 31)) * a.gain};
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
