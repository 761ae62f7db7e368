// park.cuh -- tensor memory as a place for registers.
#pragma once

#include "tcgen05.cuh"

namespace sdm {

// Registers parked in tensor memory: the calling warp's 32 lanes of it, one
// 32-bit column per register, read back by the same threads.
__device__ __forceinline__ void park16(uint32_t taddr, const float2 (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x),
      "f"(v[3].y), "f"(v[4].x), "f"(v[4].y), "f"(v[5].x), "f"(v[5].y), "f"(v[6].x), "f"(v[6].y),
      "f"(v[7].x), "f"(v[7].y)
      : "memory");
}
__device__ __forceinline__ void parked() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
// Asked for; there after the wait, which the registers pass through so that no
// use of them precedes it.
__device__ __forceinline__ void ask16(uint32_t taddr, float2 (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y),
        "=f"(v[3].x), "=f"(v[3].y), "=f"(v[4].x), "=f"(v[4].y), "=f"(v[5].x), "=f"(v[5].y),
        "=f"(v[6].x), "=f"(v[6].y), "=f"(v[7].x), "=f"(v[7].y)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void ask4(uint32_t taddr, float2& lo, float2& hi) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(lo.x), "=f"(lo.y), "=f"(hi.x), "=f"(hi.y)
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void asked() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void here(float2 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i].x), "+f"(v[i].y) : : "memory");
}

}  // namespace sdm
