// packed.cuh -- float32 arithmetic in inline PTX: pairs of operations in one
// instruction (the packed forms of sm_100 on), 2^x, the reciprocal, and a
// maximum that keeps NaN.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace sdm {

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// Two float32 operations in one instruction (the packed forms of sm_100 on).
__device__ __forceinline__ uint64_t bits2(float2 a) { return *reinterpret_cast<uint64_t*>(&a); }
__device__ __forceinline__ float2 float2_of(uint64_t a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 ex2_pair(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
// The same on pairs that stay in one 64-bit register.
using Pair = uint64_t;
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair ex2_pair(Pair v) {
  Pair r;
  asm("{\n .reg .f32 a, b;\n mov.b64 {a, b}, %1;\n ex2.approx.ftz.f32 a, a;\n"
      " ex2.approx.ftz.f32 b, b;\n mov.b64 %0, {a, b};\n}\n"
      : "=l"(r)
      : "l"(v));
  return r;
}
__device__ __forceinline__ Pair rcp_pair(Pair v) {
  Pair r;
  asm("{\n .reg .f32 a, b;\n mov.b64 {a, b}, %1;\n rcp.approx.ftz.f32 a, a;\n"
      " rcp.approx.ftz.f32 b, b;\n mov.b64 %0, {a, b};\n}\n"
      : "=l"(r)
      : "l"(v));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// The larger of two numbers, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace sdm
