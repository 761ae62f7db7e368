// residual_norm.cu -- residual addition and RMS-Norm, forward (16-, 32- or
// 8-bit output with scales) and backward.
//
//   s = round(x + residual),  inv = 1 / sqrt(mean s^2 + eps),  n = s inv gamma;
//   8 bits: scale = max(max|n| / 448, 2^-126) of a row or a group of channels,
//   out = n / scale rounded to e4m3.
//   backward: w = dout gamma,  dx = ds + inv (w - s inv mean(w s inv)),
//   dgamma = sum over rows of dout s inv.
//
// Measured at 32768 x 1024 bf16: forward 39.9 us (the copy rate), backward 46.7 us
// (0.86); 8-bit output at 16384 x 3840, groups of 128, 75.1 us (0.88).
// All of it is bound by the bytes of the rows, each read and written once: a
// row is held in the registers of a team of warps (eight channels a thread and
// step, 16 bytes of a bf16 tensor) between the reduction and the output.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"

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
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __float22bfloat162_rn(f[i]);
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
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    f[0] = make_float2(lo.x, lo.y);
    f[1] = make_float2(lo.z, lo.w);
    f[2] = make_float2(hi.x, hi.y);
    f[3] = make_float2(hi.z, hi.w);
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    lo = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    hi = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = lo;
    reinterpret_cast<float4*>(p)[1] = hi;
  }
};

__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  uint16_t q;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(q) : "f"(v.y), "f"(v.x));
  return q;
}

// max / 448, rounded to nearest: a product with the constant's reciprocal is off
// by an ulp at most, and its remainder, which is exact, says by how much.  (What is
// infinite has no remainder.)
__device__ __forceinline__ float scale_of(float most) {
  constexpr float r = 1.f / kE4m3Max;
  const float q = most * r, exact = fmaf(fmaf(-kE4m3Max, q, most), r, q);
  return max_nan(most < INFINITY ? exact : most, 1.17549435e-38f);
}
// n / scale, rounded once: the reciprocal r and what it lacks, r (1 - scale r), are
// together good to 2^-46 of it, and n times their sum is rounded by one multiply-add.
// (Measured at 16384 x 3840, groups of 128: 1% more time than n r, which puts
// elements next to a tie of the 8-bit rounding on the wrong side.)
struct Reciprocal {
  float2 r, rest;
};
__device__ __forceinline__ Reciprocal reciprocal(float scale) {
  const float r = rcp(scale), lacks = fmaf(-scale, r, 1.f);
  return Reciprocal{both(r), both(scale < INFINITY ? r * lacks : 0.f)};
}
__device__ __forceinline__ float2 divided(float2 n, const Reciprocal& d) {
  return fma2(n, d.r, mul2(n, d.rest));
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

// The largest over a team of values that are not negative; NaN if one is.  As
// bit patterns: a NaN (its sign taken off) is above every number.
template <int TW>
__device__ __forceinline__ float team_max(float m, uint32_t* red, int team) {
  uint32_t v = __reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu);
  if (TW > 1) {
    if ((threadIdx.x & 31) == 0) red[(threadIdx.x >> 5) % TW] = v;
    named_bar_sync(1 + team, TW * 32);
#pragma unroll
    for (int k = 0; k < TW; ++k) v = max(v, red[k]);
  }
  return __uint_as_float(v);
}
__device__ __forceinline__ float largest(const float2 (&n)[4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_nan(m, max_nan(fabsf(n[i].x), fabsf(n[i].y)));
  return m;
}

struct ForwardArgs {
  const void* x;
  const void* residual;
  const float* gamma;
  float eps;
  void* s;
  void* out;
  int group;
  float* scale;
  int rows, D;
  float one_over_D;
};

template <typename T, int TW, int NV, int kOut>
__global__ void __launch_bounds__(kBlock<TW>) forward_kernel(const ForwardArgs P) {
  wait_for_stream();
  __shared__ float red[2][kTeams<TW>][TW][1];
  __shared__ uint32_t redmax[2][kTeams<TW>][TW];
  const int team = threadIdx.x / (TW * 32), lane = threadIdx.x % (TW * 32), D = P.D;
  const int group_log = 31 - __clz(P.group | 1);
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
    float2 ss2 = both(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        float2 f[4];
        s[j].get(f);
        if (P.residual) {
          float2 r[4];
          res[j].get(r);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = add2(f[i], r[i]);
          s[j].set(f);                     // rounds
          s[j].get(f);
        }
        if (P.s) s[j].store(static_cast<T*>(P.s) + base + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss2 = fma2(f[i], f[i], ss2);
      }
    }
    float ss[1] = {ss2.x + ss2.y};
    team_sum<TW, 1>(ss, red[flip][team], team);
    const float2 inv = both(rsqrtf(fmaf(ss[0], P.one_over_D, P.eps)));
    // n, kept where the scale of the 8-bit output has yet to be found.
    float2 n[NV][4];
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        s[j].get(n[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) n[j][i] = mul2(n[j][i], inv);
        if (P.gamma) {
          Eight<float> g;
          float2 gm[4];
          g.load(P.gamma + c);
          g.get(gm);
#pragma unroll
          for (int i = 0; i < 4; ++i) n[j][i] = mul2(n[j][i], gm[i]);
        }
        if (kOut == SDM_BF16) {
          Eight<__nv_bfloat16> o;
          o.set(n[j]);
          o.store(static_cast<__nv_bfloat16*>(P.out) + base + c);
        } else if (kOut == SDM_F32) {
          Eight<float> o;
          o.set(n[j]);
          o.store(static_cast<float*>(P.out) + base + c);
        } else if (P.group == 0) {
          most = max_nan(most, largest(n[j]));
        }
      }
    }
    if (kOut != SDM_E4M3) continue;
    if (P.group == 0) most = team_max<TW>(most, redmax[flip][team], team);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (P.group) {                       // 4, 8 or 16 neighbouring threads
        most = c < D ? largest(n[j]) : 0.f;
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
        if (P.group >= 64) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 4));
        if (P.group >= 128) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 8));
      }
      const float scale = scale_of(most);
      const Reciprocal by = reciprocal(scale);
      if (c < D) {
        uint2 q;
        q.x = e4m3x2(divided(n[j][0], by)) | e4m3x2(divided(n[j][1], by)) << 16;
        q.y = e4m3x2(divided(n[j][2], by)) | e4m3x2(divided(n[j][3], by)) << 16;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(P.out) + base + c) = q;
        if (P.group) {
          if ((c & (P.group - 1)) == 0)
            P.scale[(size_t)row * (D >> group_log) + (c >> group_log)] = scale;
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
  float one_over_D;
};

// Threads keep their channels from row to row, so that the gradient of gamma
// is summed in registers; the teams of a block are added in shared memory at
// the end, the blocks by column_sums_kernel.
template <typename T, int TW, int NV>
__global__ void __launch_bounds__(kBlock<TW>) backward_kernel(const BackwardArgs P) {
  wait_for_stream();
  __shared__ float red[2][kTeams<TW>][TW][2];
  extern __shared__ __align__(16) float teams[];   // [kTeams - 1][TW * NV * 256]
  const int team = threadIdx.x / (TW * 32), lane = threadIdx.x % (TW * 32), D = P.D;
  float2 acc[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.f);
  int flip = 0;
  const long long step = (long long)gridDim.x * kTeams<TW>;
  // The next row's loads are under way while a row is worked on (not with 64
  // or 128 bytes of a tensor a thread: the registers do not suffice).
  constexpr bool kAhead = NV * sizeof(T) <= 4;
  Eight<T> ahead_s[NV], ahead_d[NV], ahead_more[NV];
  auto ask = [&](long long row) {
    const size_t base = (size_t)row * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D && row < P.rows) {
        ahead_s[j].load(static_cast<const T*>(P.s) + base + c);
        ahead_d[j].load(static_cast<const T*>(P.dout) + base + c);
        if (P.ds) ahead_more[j].load(static_cast<const T*>(P.ds) + base + c);
      }
    }
  };
  long long row = (long long)blockIdx.x * kTeams<TW> + team;
  if (kAhead) ask(row);
  for (; row < P.rows; row += step, flip ^= 1) {
    const size_t base = (size_t)row * D;
    if (!kAhead) ask(row);
    Eight<T> s[NV], d[NV], more[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      s[j] = ahead_s[j];
      d[j] = ahead_d[j];
      more[j] = ahead_more[j];
    }
    if (kAhead) ask(row + step);
    float2 ss = both(0.f), ws = both(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        float2 fs[4], w[4];
        s[j].get(fs);
        d[j].get(w);
        if (P.gamma) {
          Eight<float> g;
          float2 gm[4];
          g.load(P.gamma + c);
          g.get(gm);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = mul2(w[i], gm[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss = fma2(fs[i], fs[i], ss);
          ws = fma2(w[i], fs[i], ws);
        }
      }
    }
    float v[2] = {ss.x + ss.y, ws.x + ws.y};
    team_sum<TW, 2>(v, red[flip][team], team);
    const float inv1 = rsqrtf(fmaf(v[0], P.one_over_D, P.eps));
    const float2 inv = both(inv1), mean = both(-v[1] * inv1 * P.one_over_D);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TW * 32 + lane) * kVec;
      if (c < D) {
        float2 fs[4], fd[4], w[4], dx[4];
        s[j].get(fs);
        d[j].get(fd);
        if (P.gamma) {
          Eight<float> g;
          float2 gm[4];
          g.load(P.gamma + c);
          g.get(gm);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = mul2(fd[i], gm[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = fd[i];
        }
        if (P.ds) {
          more[j].get(dx);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) dx[i] = both(0.f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 hat = mul2(fs[i], inv);
          acc[j][i] = fma2(fd[i], hat, acc[j][i]);
          dx[i] = fma2(inv, fma2(hat, mean, w[i]), dx[i]);
        }
        Eight<T> o;
        o.set(dx);
        o.store(static_cast<T*>(P.dx) + base + c);
      }
    }
  }
  if (!P.partial) return;
  constexpr int kRow = TW * NV * 256;
  if (kTeams<TW> > 1) {
    float2* const mine = reinterpret_cast<float2*>(teams) + lane * 4;
    if (team > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[((team - 1) * kRow + j * TW * 256) / 2 + i] = acc[j][i];
    }
    __syncthreads();
    if (team > 0) return;
    for (int k = 0; k < kTeams<TW> - 1; ++k)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[j][i] = add2(acc[j][i], mine[(k * kRow + j * TW * 256) / 2 + i]);
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
  wait_for_stream();
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

// Blocks of the backward kernel: what the GPU holds at once, so that gamma's
// gradient is summed in registers over as many rows as can be.
constexpr int kMostPerSm = 4;
int most_parts() { return kMostPerSm * device_limits().sms; }

template <class K>
int blocks_per_sm(K kernel, int threads, int smem, std::atomic<int>* cache) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1)
      n = 1;
    if (n > kMostPerSm) n = kMostPerSm;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <typename T, int TW, int NV>
cudaError_t forward_as(const ForwardArgs& P, int out_dtype, cudaStream_t stream) {
  const long long want = ((long long)P.rows + kTeams<TW> - 1) / kTeams<TW>;
  const long long most = 1 << 20;
  const unsigned blocks = (unsigned)(want < most ? want : most);
  const auto kernel = out_dtype == SDM_E4M3   ? forward_kernel<T, TW, NV, SDM_E4M3>
                      : out_dtype == SDM_BF16 ? forward_kernel<T, TW, NV, SDM_BF16>
                                              : forward_kernel<T, TW, NV, SDM_F32>;
  return launch_behind(kernel, blocks, kBlock<TW>, 0, stream, P);
}

template <typename T, int TW, int NV>
cudaError_t backward_as(const BackwardArgs& P, float* dgamma, cudaStream_t stream) {
  static std::atomic<int> cache[64];       // zeros
  const auto kernel = backward_kernel<T, TW, NV>;
  const int smem = (kTeams<TW> - 1) * TW * NV * 256 * (int)sizeof(float);
  const long long want = ((long long)P.rows + kTeams<TW> - 1) / kTeams<TW>;
  const int most = blocks_per_sm(kernel, kBlock<TW>, smem, cache) * device_limits().sms;
  const int blocks = (int)(want < most ? want : most);
  const cudaError_t e = launch_behind(kernel, blocks, kBlock<TW>, smem, stream, P);
  if (e != cudaSuccess || !dgamma) return e;
  return launch_behind(column_sums_kernel, (P.D + 31) / 32, 1024, 0, stream, P.partial, blocks, P.D,
                       dgamma);
}

// Calls f with the team for rows of D channels: a thread takes 32 bytes of a
// tensor's row, so a warp 512 channels of bf16 or 256 of float32, until the
// team has 16 warps.  Measured at 32768 x 1024 bf16, backward: 47 us, with 64
// bytes a thread 51 us, with 16 bytes 49 us; at 4999 x 1920 float32: 29 us, with
// 64 bytes 34 us.  Where there are too few rows to fill the GPU (few), 16 bytes
// of bf16: a row's latency is that of fewer steps per thread.
template <typename T, class F>
cudaError_t with_team(int D, bool few, F f) {
  using std::integral_constant;
#define SDM_TEAM(tw, nv) return f(integral_constant<int, tw>{}, integral_constant<int, nv>{})
  if (sizeof(T) == 4 || (few && D <= 4096)) {
    if (D <= 256) SDM_TEAM(1, 1);
    if (D <= 512) SDM_TEAM(2, 1);
    if (D <= 1024) SDM_TEAM(4, 1);
    if (D <= 2048) SDM_TEAM(8, 1);
    if (D <= 4096) SDM_TEAM(16, 1);
  } else {
    if (D <= 512) SDM_TEAM(1, 2);
    if (D <= 1024) SDM_TEAM(2, 2);
    if (D <= 2048) SDM_TEAM(4, 2);
    if (D <= 4096) SDM_TEAM(8, 2);
  }
  if (D <= 8192) SDM_TEAM(16, 2);
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
  const ForwardArgs P{x, residual, gamma, eps, s, out, group, scale, d.rows, d.D, 1.f / (float)d.D};
  const bool few = few_rows(d.rows);
  if (d.dtype == SDM_BF16)
    return with_team<__nv_bfloat16>(d.D, few, [&](auto tw, auto nv) {
      return forward_as<__nv_bfloat16, decltype(tw)::value, decltype(nv)::value>(P, out_dtype, stream);
    });
  return with_team<float>(d.D, few, [&](auto tw, auto nv) {
    return forward_as<float, decltype(tw)::value, decltype(nv)::value>(P, out_dtype, stream);
  });
}

cudaError_t launch_add_rmsnorm_backward(const NormDims& d, const void* s, const void* dout,
                                        const float* gamma, const void* ds, float eps, void* dx,
                                        float* dgamma, void* workspace, cudaStream_t stream) {
  if (d.rows == 0) return cudaMemsetAsync(dgamma, 0, (size_t)d.D * sizeof(float), stream);
  const BackwardArgs P{s,  dout,   gamma, ds, eps, dx, dgamma ? static_cast<float*>(workspace) : nullptr,
                       d.rows, d.D, 1.f / (float)d.D};
  const bool few = few_rows(d.rows);
  if (d.dtype == SDM_BF16)
    return with_team<__nv_bfloat16>(d.D, few, [&](auto tw, auto nv) {
      return backward_as<__nv_bfloat16, decltype(tw)::value, decltype(nv)::value>(P, dgamma, stream);
    });
  return with_team<float>(d.D, few, [&](auto tw, auto nv) {
    return backward_as<float, decltype(tw)::value, decltype(nv)::value>(P, dgamma, stream);
  });
}

}  // namespace sdm
