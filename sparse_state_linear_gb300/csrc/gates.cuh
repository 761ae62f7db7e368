// gates.cuh -- softplus in float32, alone and for two channels per instruction:
// what the gates of the recurrence and the time steps of the selective scan are
// made of.
#pragma once

#include "packed.cuh"

namespace sdm {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// log2(1 + e) for e in [0, 1]: 2 log2(e) atanh(t) with t = e / (2 + e), as t
// times the degree-4 polynomial in t^2 that interpolates the rest at the
// Chebyshev points of [0, 1/9] (relative error 4e-9).  With the roundings the
// relative error is below 6.5 half steps for every e; the logarithm instruction
// has an absolute bound, which is not enough where the gate hardly decays.
constexpr float kLog0 = 2.88539004f, kLog1 = 0.961791694f, kLog2 = 0.577432871f,
                kLog3 = 0.403451949f, kLog4 = 0.406230867f;
__device__ __forceinline__ float log2p1_unit(float e) {
  const float t = e * rcp(e + 2.f), z = t * t;
  return t * fmaf(fmaf(fmaf(fmaf(kLog4, z, kLog3), z, kLog2), z, kLog1), z, kLog0);
}
// The packed forms take no immediates.  Their constants are made once, out of
// the compiler's sight: it would otherwise move them into registers again
// before every use (about seven of 42 instructions per element).
struct Constants {
  float2 log2e, one, two, k0, k1, k2, k3, k4;
};
__device__ __forceinline__ float2 hidden(float x) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %1};\n" : "=l"(r) : "f"(x));
  return float2_of(r);
}
__device__ __forceinline__ Constants constants() {
  return Constants{hidden(kLog2e), hidden(1.f),   hidden(2.f),   hidden(kLog0),
                   hidden(kLog1),  hidden(kLog2), hidden(kLog3), hidden(kLog4)};
}

// What the exponent of alpha is made of, for two channels: x = (za + bias)
// log2(e), e = 2^-|x| and softplus = max(x, 0) + log2(1 + e), as log2p1_unit.
// (The sum first: a bias times log2(e) would be rounded at its own size, which
// tells where za nearly cancels it.)
__device__ __forceinline__ void softplus_pair(const Constants& K, float2 za, float2 bias, float2& x,
                                              float2& e, float2& sp) {
  x = mul2(add2(za, bias), K.log2e);
  e = make_float2(ex2(-fabsf(x.x)), ex2(-fabsf(x.y)));
  const float2 d = add2(e, K.two);
  const float2 t = mul2(e, make_float2(rcp(d.x), rcp(d.y))), z = mul2(t, t);
  float2 p = fma2(K.k4, z, K.k3);
  p = fma2(p, z, K.k2);
  p = fma2(p, z, K.k1);
  p = fma2(p, z, K.k0);
  sp = fma2(p, t, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

}  // namespace sdm
