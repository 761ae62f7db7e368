// residual_norm.cu -- residual addition and RMS-Norm, forward (16-, 32- or
// 8-bit output with scales) and backward.
//
//   s = round(x + residual),  inv = 1 / sqrt(mean s^2 + eps),  n = s inv gamma;
//   8 bits: scale = max(max|n| / 448, 2^-126) of a row or a group of channels,
//   out = n / scale rounded to e4m3.
//   backward: w = dout gamma,  dx = ds + inv (w - s inv mean(w s inv)),
//   dgamma = sum over rows of dout s inv.
//
// All of it is bound by the bytes of the rows, each read and written once: a
// row is held in the registers of a team of warps (eight channels a thread and
// step, 16 bytes of a bf16 tensor) between the reduction and the output.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace sdm {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kVec = 8;               // channels per thread and step

// ------------------------------------------------------------ eight channels
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
};
template <>
struct Eight<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo = reinterpret_cast<const float4*>(p)[0];
    hi = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = lo.x; f[1] = lo.y; f[2] = lo.z; f[3] = lo.w;
    f[4] = hi.x; f[5] = hi.y; f[6] = hi.z; f[7] = hi.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    lo = make_float4(f[0], f[1], f[2], f[3]);
    hi = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = lo;
    reinterpret_cast<float4*>(p)[1] = hi;
  }
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t q;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(q) : "f"(hi), "f"(lo));
  return q;
}

// ------------------------------------------------------------------ teams
// TW warps work on a row; a block has kTeams<TW> of them.
template <int TW>
constexpr int kTeams = TW < 8 ? 8 / TW : 1;
template <int TW>
constexpr int kBlock = kTeams<TW> * TW * 32;

// Sums over a team (every thread gets them).  `red` is the team's own, one slot
// per warp, and free for the next call after the barrier of the call after
// next: callers alternate between two.
template <int TW, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*red)[N], int team) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (TW == 1) return;
  const int w = (threadIdx.x >> 5) % TW;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[w][i] = v[i];
  named_bar_sync(1 + team, TW * 32);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
#pragma unroll
    for (int k = 0; k < TW; ++k) v[i] += red[k][i];
  }
}

// The largest over a team, of the bit patterns of |values|: a NaN is above
// every number.
template <int TW>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* red, int team) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (TW == 1) return v;
  if ((threadIdx.x & 31) == 0) red[(threadIdx.x >> 5) % TW] = v;
  named_bar_sync(1 + team, TW * 32);
#pragma unroll
  for (int k = 0; k < TW; ++k) v = max(v, red[k]);
  return v;
}

struct ForwardArgs {
  const void* x;
  const void* residual;
  const float* gamma;
  float eps;
  void* s;
  void* out;
  int out_dtype, group;
  float* scale;
  int rows, D;
};

template <typename T, int TW, int NV>
__global__ void __launch_bounds__(kBlock<TW>) forward_kernel(const ForwardArgs P) {
  __shared__ float red[2][kTeams<TW>][TW][1];
  __shared__ uint32_t redmax[2][kTeams<TW>][TW];
  const int team = threadIdx.x / (TW * 32), lane = threadIdx.x % (TW * 32), D = P.D;
  int flip = 0;
  for (long long row = (long long)blockIdx.x * kTeams<TW> + team; row < P.rows;
       row += (long long)gridDim.x * kTeams<TW>, flip ^= 1) {
    const size_t base = (size_t)row * D;
    Eight<T> s[NV], res[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        s[j].load(static_cast<const T*>(P.x) + base + c);
        if (P.residual) res[j].load(static_cast<const T*>(P.residual) + base + c);
      }
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        float f[8];
        s[j].get(f);
        if (P.residual) {
          float r[8];
          res[j].get(r);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += r[i];
          s[j].set(f);                     // rounds
          s[j].get(f);
        }
        if (P.s) s[j].store(static_cast<T*>(P.s) + base + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(f[i], f[i], ss[0]);
      }
    }
    team_sum<TW, 1>(ss, red[flip][team], team);
    const float inv = 1.f / sqrtf(ss[0] / (float)D + P.eps);
    // n, of the 8-bit output kept until the scale is known.
    float n[NV][8];
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        s[j].get(n[j]);
        Eight<float> g;
        if (P.gamma) g.load(P.gamma + c);
        float gm[8];
        g.get(gm);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[j][i] *= inv;
          if (P.gamma) n[j][i] *= gm[i];
        }
        if (P.out_dtype == SDM_BF16) {
          Eight<__nv_bfloat16> o;
          o.set(n[j]);
          o.store(static_cast<__nv_bfloat16*>(P.out) + base + c);
        } else if (P.out_dtype == SDM_F32) {
          Eight<float> o;
          o.set(n[j]);
          o.store(static_cast<float*>(P.out) + base + c);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(n[j][i]) & 0x7fffffffu);
        }
      }
    }
    if (P.out_dtype != SDM_E4M3) continue;
    if (P.group == 0) most = team_max<TW>(most, redmax[flip][team], team);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (P.group) {                       // 4, 8 or 16 neighbouring threads
        most = 0;
        if (c < D) {
#pragma unroll
          for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(n[j][i]) & 0x7fffffffu);
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        if (P.group >= 64) most = max(most, __shfl_xor_sync(0xffffffffu, most, 4));
        if (P.group >= 128) most = max(most, __shfl_xor_sync(0xffffffffu, most, 8));
      }
      const float amax = __uint_as_float(most);
      const float scale = amax != amax ? amax : fmaxf(amax / kE4m3Max, 1.17549435e-38f);
      const float by = 1.f / scale;
      if (c < D) {
        uint2 q;
        q.x = e4m3x2(n[j][0] * by, n[j][1] * by) | e4m3x2(n[j][2] * by, n[j][3] * by) << 16;
        q.y = e4m3x2(n[j][4] * by, n[j][5] * by) | e4m3x2(n[j][6] * by, n[j][7] * by) << 16;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(P.out) + base + c) = q;
        if (P.group) {
          if (c % P.group == 0) P.scale[(size_t)row * (D / P.group) + c / P.group] = scale;
        } else if (c == 0) {
          P.scale[row] = scale;
        }
      }
    }
  }
}

// ----------------------------------------------------------------- backward
struct BackwardArgs {
  const void* s;
  const void* dout;
  const float* gamma;
  const void* ds;
  float eps;
  void* dx;
  float* partial;      // [blocks][D], or null
  int rows, D;
};

// Threads keep their channels from row to row, so that the gradient of gamma
// is summed in registers; the teams of a block are added in shared memory at
// the end, the blocks by column_sums_kernel.
template <typename T, int TW, int NV>
__global__ void __launch_bounds__(kBlock<TW>) backward_kernel(const BackwardArgs P) {
  __shared__ float red[2][kTeams<TW>][TW][2];
  extern __shared__ float teams[];         // [kTeams - 1][TW * NV * 256]
  const int team = threadIdx.x / (TW * 32), lane = threadIdx.x % (TW * 32), D = P.D;
  float acc[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.f;
  int flip = 0;
  for (long long row = (long long)blockIdx.x * kTeams<TW> + team; row < P.rows;
       row += (long long)gridDim.x * kTeams<TW>, flip ^= 1) {
    const size_t base = (size_t)row * D;
    Eight<T> s[NV], d[NV], more[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        s[j].load(static_cast<const T*>(P.s) + base + c);
        d[j].load(static_cast<const T*>(P.dout) + base + c);
        if (P.ds) more[j].load(static_cast<const T*>(P.ds) + base + c);
      }
    }
    float v[2] = {0.f, 0.f};               // sum s^2, sum w s
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        float fs[8], fd[8], gm[8];
        s[j].get(fs);
        d[j].get(fd);
        Eight<float> g;
        if (P.gamma) g.load(P.gamma + c);
        g.get(gm);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[0] = fmaf(fs[i], fs[i], v[0]);
          v[1] = fmaf(P.gamma ? fd[i] * gm[i] : fd[i], fs[i], v[1]);
        }
      }
    }
    team_sum<TW, 2>(v, red[flip][team], team);
    const float inv = 1.f / sqrtf(v[0] / (float)D + P.eps), mean = v[1] * inv / (float)D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        float fs[8], fd[8], gm[8], fm[8];
        s[j].get(fs);
        d[j].get(fd);
        Eight<float> g;
        if (P.gamma) g.load(P.gamma + c);
        g.get(gm);
        if (P.ds) more[j].get(fm);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float hat = fs[i] * inv, w = P.gamma ? fd[i] * gm[i] : fd[i];
          acc[j][i] = fmaf(fd[i], hat, acc[j][i]);
          const float dx = inv * fmaf(-hat, mean, w);
          fs[i] = P.ds ? fm[i] + dx : dx;
        }
        Eight<T> o;
        o.set(fs);
        o.store(static_cast<T*>(P.dx) + base + c);
      }
    }
  }
  if (!P.partial) return;
  constexpr int kRow = TW * NV * 256;
  if (kTeams<TW> > 1) {
    if (team > 0)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          teams[(team - 1) * kRow + (j * TW * 32 + lane) * kVec + i] = acc[j][i];
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        for (int k = 0; k < kTeams<TW> - 1; ++k)
          acc[j][i] += teams[k * kRow + (j * TW * 32 + lane) * kVec + i];
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TW * 32 + lane) * kVec;
    if (c < D) {
      Eight<float> o;
      o.set(acc[j]);
      o.store(P.partial + (size_t)blockIdx.x * D + c);
    }
  }
}

// Sums of [parts][D] over the parts, always in the same order: 32 channels a
// block, each of 32 warps every 32nd part, then the warps.
__global__ void __launch_bounds__(1024)
    column_sums_kernel(const float* partial, int parts, int D, float* out) {
  __shared__ float warps[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int n = warp; n < parts; n += 32) a += __ldg(partial + (size_t)n * D + c);
  }
  warps[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && c < D) {
    float sum = 0.f;
    for (int w = 0; w < 32; ++w) sum += warps[w][lane];
    out[c] = sum;
  }
}

constexpr int kPartsPerSm = 2;
int most_parts() { return kPartsPerSm * device_limits().sms; }

template <typename T, int TW, int NV>
cudaError_t forward_as(const ForwardArgs& P, cudaStream_t stream) {
  const long long want = ((long long)P.rows + kTeams<TW> - 1) / kTeams<TW>;
  const long long most = 1 << 20;
  forward_kernel<T, TW, NV><<<(unsigned)(want < most ? want : most), kBlock<TW>, 0, stream>>>(P);
  return cudaGetLastError();
}

template <typename T, int TW, int NV>
cudaError_t backward_as(const BackwardArgs& P, float* dgamma, cudaStream_t stream) {
  const long long want = ((long long)P.rows + kTeams<TW> - 1) / kTeams<TW>;
  const int blocks = (int)(want < most_parts() ? want : most_parts());
  const int smem = (kTeams<TW> - 1) * TW * NV * 256 * (int)sizeof(float);
  backward_kernel<T, TW, NV><<<blocks, kBlock<TW>, dgamma ? smem : 0, stream>>>(P);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dgamma) return e;
  column_sums_kernel<<<(P.D + 31) / 32, 1024, 0, stream>>>(P.partial, blocks, P.D, dgamma);
  return cudaGetLastError();
}

// Calls f with the team for rows of D channels: up to 1024 channels a warp.
// Where there are too few rows to fill the GPU that way, up to 256 a warp: a
// row's latency is then that of fewer loads per thread.
template <class F>
cudaError_t with_team(int D, bool few, F f) {
  using std::integral_constant;
#define SDM_TEAM(tw, nv) return f(integral_constant<int, tw>{}, integral_constant<int, nv>{})
  if (few && D <= 4096) {
    if (D <= 256) SDM_TEAM(1, 1);
    if (D <= 512) SDM_TEAM(2, 1);
    if (D <= 1024) SDM_TEAM(4, 1);
    if (D <= 2048) SDM_TEAM(8, 1);
    SDM_TEAM(16, 1);
  }
  if (D <= 256) SDM_TEAM(1, 1);
  if (D <= 512) SDM_TEAM(1, 2);
  if (D <= 1024) SDM_TEAM(1, 4);
  if (D <= 2048) SDM_TEAM(2, 4);
  if (D <= 4096) SDM_TEAM(4, 4);
  if (D <= 8192) SDM_TEAM(8, 4);
  SDM_TEAM(16, 4);
#undef SDM_TEAM
}

bool few_rows(int rows) { return rows < 8 * device_limits().sms; }

}  // namespace

size_t add_rmsnorm_workspace_bytes(const NormDims& d) {
  return (size_t)most_parts() * d.D * sizeof(float);
}

cudaError_t launch_add_rmsnorm(const NormDims& d, const void* x, const void* residual,
                               const float* gamma, float eps, void* s, void* out, int out_dtype,
                               int group, float* scale, cudaStream_t stream) {
  const ForwardArgs P{x, residual, gamma, eps, s, out, out_dtype, group, scale, d.rows, d.D};
  return with_team(d.D, few_rows(d.rows), [&](auto tw, auto nv) {
    return d.dtype == SDM_BF16
               ? forward_as<__nv_bfloat16, decltype(tw)::value, decltype(nv)::value>(P, stream)
               : forward_as<float, decltype(tw)::value, decltype(nv)::value>(P, stream);
  });
}

cudaError_t launch_add_rmsnorm_backward(const NormDims& d, const void* s, const void* dout,
                                        const float* gamma, const void* ds, float eps, void* dx,
                                        float* dgamma, void* workspace, cudaStream_t stream) {
  if (d.rows == 0) return cudaMemsetAsync(dgamma, 0, (size_t)d.D * sizeof(float), stream);
  const BackwardArgs P{s,  dout,   gamma, ds, eps, dx, dgamma ? static_cast<float*>(workspace) : nullptr,
                       d.rows, d.D};
  return with_team(d.D, few_rows(d.rows), [&](auto tw, auto nv) {
    return d.dtype == SDM_BF16
               ? backward_as<__nv_bfloat16, decltype(tw)::value, decltype(nv)::value>(P, dgamma, stream)
               : backward_as<float, decltype(tw)::value, decltype(nv)::value>(P, dgamma, stream);
  });
}

}  // namespace sdm
