// rows.cuh -- four channels of a row, between memory (float32 or bf16) and pairs
// of float32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sdm {

// Four channels of a row in shared memory or registers.
__device__ __forceinline__ void load_row(const float* p, float2& lo, float2& hi) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  lo = make_float2(v.x, v.y);
  hi = make_float2(v.z, v.w);
}
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float2& lo, float2& hi) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  lo = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
  hi = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store_row(float* p, float2 lo, float2 hi) {
  *reinterpret_cast<float4*>(p) = make_float4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void store_row(__nv_bfloat16* p, float2 lo, float2 hi) {
  const __nv_bfloat162 a = __float22bfloat162_rn(lo), b = __float22bfloat162_rn(hi);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

}  // namespace sdm
