// residual_norm.cu -- residual addition and RMS-Norm, forward (16-, 32- or
// 8-bit output with scales) and backward.
//
//   s = round(x + residual),  inv = rsqrt(mean s^2 + eps),  n = s inv gamma;
//   8 bits: scale = max(max|n| / 448, 2^-126) of a row or a group of channels,
//   out = n / scale rounded to e4m3.
//   backward: w = dout gamma,  dx = ds + inv (w - s inv mean(w s inv)),
//   dgamma = sum over rows of dout s inv.
#include "common.cuh"
#include "internal.h"

namespace sdm {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kParts = 128;   // row groups whose gamma gradients are summed apart

// Lane sums over the block (every thread gets the result); `red` has room for
// one float per warp.
__device__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) v += red[i];
  return v;
}

__device__ __forceinline__ float rounded(float x, int dt) {
  return dt == SDM_BF16 ? __bfloat162float(__float2bfloat16_rn(x)) : x;
}
__device__ __forceinline__ void store_scalar(void* base, size_t i, int dt, float x) {
  if (dt == SDM_F32) {
    reinterpret_cast<float*>(base)[i] = x;
  } else if (dt == SDM_BF16) {
    reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(x);
  } else {
    uint16_t q;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(q) : "f"(0.f), "f"(x));
    reinterpret_cast<uint8_t*>(base)[i] = (uint8_t)(q & 0xff);
  }
}

struct Args {
  NormDims d;
  const void* x;
  const void* residual;
  const float* gamma;
  float eps;
  void* s;
  void* out;
  int out_dtype, group;
  float* scale;
  const void* dout;
  const void* ds;
  float* partial;
};

// One block per row, the row in shared memory.
__global__ void __launch_bounds__(256) forward_kernel(const Args P) {
  extern __shared__ float row[];
  __shared__ float red[8];
  const int D = P.d.D, dt = P.d.dtype;
  const size_t base = (size_t)blockIdx.x * D;
  float ss = 0.f;
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    float v = load_scalar(P.x, base + c, dt);
    if (P.residual) v = rounded(v + load_scalar(P.residual, base + c, dt), dt);
    row[c] = v;
    ss = fmaf(v, v, ss);
  }
  ss = block_sum(ss, red);
  const float inv = 1.f / sqrtf(ss / (float)D + P.eps);
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    if (P.s) store_scalar(P.s, base + c, dt, row[c]);
    row[c] = row[c] * inv * (P.gamma ? P.gamma[c] : 1.f);
    if (P.out_dtype != SDM_E4M3) store_scalar(P.out, base + c, P.out_dtype, row[c]);
  }
  if (P.out_dtype != SDM_E4M3) return;
  __syncthreads();
  const int group = P.group ? P.group : D, n = D / group, warp = threadIdx.x >> 5;
  for (int g = warp; g < n; g += 8) {
    uint32_t m = 0;   // as integers: a NaN is above every number
    for (int c = threadIdx.x & 31; c < group; c += 32)
      m = max(m, __float_as_uint(row[g * group + c]) & 0x7fffffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    const float amax = __uint_as_float(m);
    const float sc = amax != amax ? amax : fmaxf(amax / kE4m3Max, 1.17549435e-38f);
    for (int c = threadIdx.x & 31; c < group; c += 32)
      store_scalar(P.out, base + g * group + c, SDM_E4M3, row[g * group + c] / sc);
    if ((threadIdx.x & 31) == 0) P.scale[(size_t)blockIdx.x * n + g] = sc;
  }
}

__global__ void __launch_bounds__(256) backward_kernel(const Args P) {
  __shared__ float red[8];
  const int D = P.d.D, dt = P.d.dtype;
  const size_t base = (size_t)blockIdx.x * D;
  float ss = 0.f, dot = 0.f;
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    const float v = load_scalar(P.x, base + c, dt);
    ss = fmaf(v, v, ss);
    dot = fmaf(load_scalar(P.dout, base + c, dt) * (P.gamma ? P.gamma[c] : 1.f), v, dot);
  }
  ss = block_sum(ss, red);
  dot = block_sum(dot, red);
  const float inv = 1.f / sqrtf(ss / (float)D + P.eps), m = dot * inv / (float)D;
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    const float w = load_scalar(P.dout, base + c, dt) * (P.gamma ? P.gamma[c] : 1.f);
    const float hat = load_scalar(P.x, base + c, dt) * inv;
    float dx = inv * (w - hat * m);
    if (P.ds) dx += load_scalar(P.ds, base + c, dt);
    store_scalar(P.out, base + c, dt, dx);
  }
}

// dgamma, part k of the rows: needs dout and s as they were, so it runs before
// the kernel above (dx may be dout).
__global__ void __launch_bounds__(256) dgamma_kernel(const Args P) {
  __shared__ float red[8];
  const int D = P.d.D, dt = P.d.dtype;
  for (int c = threadIdx.x; c < D; c += blockDim.x) P.partial[(size_t)blockIdx.x * D + c] = 0.f;
  for (int r = blockIdx.x; r < P.d.rows; r += gridDim.x) {
    const size_t base = (size_t)r * D;
    float ss = 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      const float v = load_scalar(P.x, base + c, dt);
      ss = fmaf(v, v, ss);
    }
    ss = block_sum(ss, red);
    const float inv = 1.f / sqrtf(ss / (float)D + P.eps);
    for (int c = threadIdx.x; c < D; c += blockDim.x)
      P.partial[(size_t)blockIdx.x * D + c] +=
          load_scalar(P.dout, base + c, dt) * load_scalar(P.x, base + c, dt) * inv;
  }
}

__global__ void reduce_kernel(const float* partial, int parts, int D, float* dgamma) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= D) return;
  float a = 0.f;
  for (int k = 0; k < parts; ++k) a += partial[(size_t)k * D + c];
  dgamma[c] = a;
}

}  // namespace

size_t add_rmsnorm_workspace_bytes(const NormDims& d) {
  return (size_t)kParts * d.D * sizeof(float);
}

cudaError_t launch_add_rmsnorm(const NormDims& d, const void* x, const void* residual,
                               const float* gamma, float eps, void* s, void* out, int out_dtype,
                               int group, float* scale, cudaStream_t stream) {
  Args P{};
  P.d = d;
  P.x = x;
  P.residual = residual;
  P.gamma = gamma;
  P.eps = eps;
  P.s = s;
  P.out = out;
  P.out_dtype = out_dtype;
  P.group = group;
  P.scale = scale;
  const size_t smem = (size_t)d.D * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(forward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  forward_kernel<<<d.rows, 256, smem, stream>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_add_rmsnorm_backward(const NormDims& d, const void* s, const void* dout,
                                        const float* gamma, const void* ds, float eps, void* dx,
                                        float* dgamma, void* workspace, cudaStream_t stream) {
  Args P{};
  P.d = d;
  P.x = s;
  P.dout = dout;
  P.gamma = gamma;
  P.ds = ds;
  P.eps = eps;
  P.out = dx;
  P.partial = static_cast<float*>(workspace);
  const int parts = d.rows < kParts ? d.rows : kParts;
  if (dgamma) {
    if (parts > 0) dgamma_kernel<<<parts, 256, 0, stream>>>(P);
    reduce_kernel<<<(d.D + 127) / 128, 128, 0, stream>>>(P.partial, parts, d.D, dgamma);
  }
  if (d.rows > 0) backward_kernel<<<d.rows, 256, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace sdm
