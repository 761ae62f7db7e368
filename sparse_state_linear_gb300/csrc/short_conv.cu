// short_conv.cu -- short causal convolution of every channel with its own taps
// over packed sequences: forward, backward and single-token step.
//
//   pre[t] = bias + sum_k w[taps-1-k] x[t-k],  y = pre or silu(pre),
// where rows before a sequence are its start x0.  Backward, with dpre = dy act'(pre):
//   dx[t] = sum_k w[taps-1-k] dpre[t+k],  dw[j] = sum_t dpre[t] x[t-(taps-1-j)],
//   dbias = sum dpre; rows before the sequence take part as rows of dx0, and the
//   gradient of the final rows xT is added to the rows that they are copies of.
//
// Bound by the bytes of x and y (x, dy and dx): a warp walks a run of rows of 128
// channels, four a lane, with the last rows in registers, so that every row is
// loaded once but for taps - 1 rows in front of (behind) a run.
#include <type_traits>

#include "common.cuh"
#include "gates.cuh"
#include "internal.h"
#include "launch.cuh"
#include "packing.cuh"
#include "rows.cuh"
#include "slots.cuh"

namespace sdm {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32, kWarpCols = 128;

struct ConvArgs {
  Packed packed;
  const void* x;
  const float* w;
  const float* bias;
  const void* x0;
  void* y;
  void* xT;
  // backward
  const void* dy;
  const void* dxT;
  void* dx;
  void* dx0;
  float* partial;      // [parts][taps + 1][D]
  long long ld, ld_grad;
  int D, col_tiles, run, runs;
  unsigned* status;
};

// Four channels as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void get(float2 (&f)[2]) const {
    f[0] = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
  __device__ __forceinline__ void zero() { w = make_uint2(0u, 0u); }
};
template <>
struct Raw<float> {
  float4 w;
  __device__ __forceinline__ void get(float2 (&f)[2]) const {
    f[0] = make_float2(w.x, w.y);
    f[1] = make_float2(w.z, w.w);
  }
  __device__ __forceinline__ void zero() { w = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <typename T>
__device__ __forceinline__ Raw<T> raw_at(const T* p) {
  return *reinterpret_cast<const Raw<T>*>(p);
}
template <typename T>
__device__ __forceinline__ void put_raw(T* p, Raw<T> v) {
  *reinterpret_cast<Raw<T>*>(p) = v;
}

// Taps of four channels: w[j] of [D][K] as pairs of channels.
template <int K>
struct Taps {
  float2 w[K][2], bias[2];
  __device__ __forceinline__ void load(const float* at, const float* b, int c, bool in) {
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        w[j][p] = both(0.f);
        if (in)
          w[j][p] = make_float2(__ldg(at + (size_t)(c + 2 * p) * K + j),
                                __ldg(at + (size_t)(c + 2 * p + 1) * K + j));
      }
    bias[0] = bias[1] = both(0.f);
    if (b && in) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(b + c));
      bias[0] = make_float2(v.x, v.y);
      bias[1] = make_float2(v.z, v.w);
    }
  }
};

// 1 / (1 + exp(-v)); where exp overflows it is 0.
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 z = mul2(v, both(-kLog2e));
  return make_float2(rcp(1.f + ex2(z.x)), rcp(1.f + ex2(z.y)));
}

// The first s in [0, n_seq] with begin(s) >= row (a whole warp calls it), or
// n_seq + 1.
__device__ __forceinline__ int first_from(const Packed& P, int row) {
  const int lane = threadIdx.x & 31;
  int lo = -1, hi = P.n_seq + 1;           // begin(lo) < row <= begin(hi), of the ends none is looked at
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, s = lo + (lane + 1) * step;
    const int n = __popc(__ballot_sync(0xffffffffu, s < hi && P.begin(s) < row));
    const int next = lo + (n + 1) * step;
    lo += n * step;
    hi = next < hi ? next : hi;
  }
  return hi;
}

// ------------------------------------------------------------------- forward
// Runs of P.run rows.  The first taps - 1 rows of a sequence belong to the run
// that its first row lies in, which therefore alone reads the sequence's start
// and may overwrite it with the final rows (xT = x0).
template <typename T, int K, bool kSilu>
__global__ void __launch_bounds__(kThreads) forward_kernel(const ConvArgs P) {
  wait_for_stream();
  if (!offsets_ok(P.packed)) {
    if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    return;
  }
  const int lane = threadIdx.x & 31, run = blockIdx.x / P.col_tiles * kWarps + (threadIdx.x >> 5);
  if (run >= P.runs) return;
  const int c = (blockIdx.x % P.col_tiles * 32 + lane) * 4, D = P.D;
  const bool in = c < D;
  const int r0 = run * P.run, r1 = min(r0 + P.run, P.packed.rows);
  const bool last_run = run == P.runs - 1;
  const T* const x = static_cast<const T*>(P.x) + c;
  const T* const x0 = static_cast<const T*>(P.x0) + c;
  T* const y = static_cast<T*>(P.y) + c;
  T* const xT = static_cast<T*>(P.xT) + c;
  Taps<K> taps;
  taps.load(P.w, P.bias, c, in);

  Raw<T> window[K - 1];                    // the rows before the next, oldest first
  auto rows = [&](int a, int e) {
    constexpr int kBatch = 32 / (int)sizeof(Raw<T>) * 2;      // 8 rows of bf16, 4 of float32
    for (int t = a; t < e; t += kBatch) {
      Raw<T> now[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (in && t + i < e) now[i] = raw_at(x + (size_t)(t + i) * P.ld);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (t + i >= e) break;
        float2 pre[2] = {taps.bias[0], taps.bias[1]}, f[2];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
          window[j].get(f);
          pre[0] = fma2(taps.w[j][0], f[0], pre[0]);
          pre[1] = fma2(taps.w[j][1], f[1], pre[1]);
        }
        now[i].get(f);
        pre[0] = fma2(taps.w[K - 1][0], f[0], pre[0]);
        pre[1] = fma2(taps.w[K - 1][1], f[1], pre[1]);
        if (kSilu) {
          pre[0] = mul2(pre[0], sigmoid2(pre[0]));
          pre[1] = mul2(pre[1], sigmoid2(pre[1]));
        }
        if (in) store_row(y + (size_t)(t + i) * D, pre[0], pre[1]);
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) window[j] = window[j + 1];
        window[K - 2] = now[i];
      }
    }
  };

  int s = first_from(P.packed, r0);
  // A sequence that began before the run.
  if (s > 0 && s <= P.packed.n_seq) {
    const int begin = P.packed.begin(s - 1), end = P.packed.begin(s);
    const int a = max(r0, begin + K - 1), e = min(end, r1);
    if (a < e) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        if (in) window[j] = raw_at(x + (size_t)(a - (K - 1) + j) * P.ld);
      rows(a, e);
    }
  }
  for (; s < P.packed.n_seq; ++s) {
    const int begin = P.packed.begin(s), end = P.packed.begin(s + 1);
    if (begin >= r1 && !(last_run && begin == r1)) break;
    Raw<T> last[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      window[j].zero();
      if (P.x0 && in) window[j] = raw_at(x0 + ((size_t)s * (K - 1) + j) * D);
    }
    if (P.xT) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int at = end - (K - 1) + j;
        last[j].zero();
        if (!in) continue;
        if (at >= begin) last[j] = raw_at(x + (size_t)at * P.ld);
        else if (P.x0) last[j] = raw_at(x0 + ((size_t)s * (K - 1) + (K - 1) + at - begin) * D);
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        if (in) put_raw(xT + ((size_t)s * (K - 1) + j) * D, last[j]);
    }
    rows(begin, min(end, max(r1, begin + K - 1)));
  }
}

// ------------------------------------------------------------------ backward
// A block takes 128 channels, its warps a run of rows each, every gridDim-th
// group of runs; the sums over rows stay in registers until the end.  A run's
// rows t are walked to taps - 1 rows behind its last one: dx of a row is whole
// once dpre of the taps - 1 rows behind it is known.
template <typename T, int K, bool kSilu>
__global__ void __launch_bounds__(kThreads) backward_kernel(const ConvArgs P) {
  wait_for_stream();
  if (!offsets_ok(P.packed)) {
    if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    return;
  }
  __shared__ float2 sums[kWarps - 1][K + 1][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = P.D;
  const int part = blockIdx.x / P.col_tiles, parts = gridDim.x / P.col_tiles;
  const int c = (blockIdx.x % P.col_tiles * 32 + lane) * 4;
  const bool in = c < D;
  const T* const x = static_cast<const T*>(P.x) + c;
  const T* const x0 = static_cast<const T*>(P.x0) + c;
  const T* const dy = static_cast<const T*>(P.dy) + c;
  const T* const dxT = static_cast<const T*>(P.dxT) + c;
  T* const dx = static_cast<T*>(P.dx) + c;
  T* const dx0 = static_cast<T*>(P.dx0) + c;
  Taps<K> taps;
  taps.load(P.w, P.bias, c, in);
  float2 dw[K][2], dbias[2] = {both(0.f), both(0.f)};
#pragma unroll
  for (int j = 0; j < K; ++j) dw[j][0] = dw[j][1] = both(0.f);

  // Rows a .. e - 1 of sequence s (rows begin .. end - 1).
  auto rows = [&](int s, int begin, int end, int a, int e) {
    Raw<T> window[K - 1];
    float2 acc[K][2];                      // of dx rows t, t - 1, .. as far as known
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int at = a - (K - 1) + j;
      window[j].zero();
      if (!in) continue;
      if (at >= begin) window[j] = raw_at(x + (size_t)at * P.ld);
      else if (P.x0) window[j] = raw_at(x0 + ((size_t)s * (K - 1) + (K - 1) + at - begin) * D);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k][0] = acc[k][1] = both(0.f);
    constexpr int kBatch = 4;
    const int stop = e + K - 1;            // dx of row t - (K - 1) leaves at t
    for (int t0 = a; t0 < stop; t0 += kBatch) {
      Raw<T> now[kBatch], grad[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        now[i].zero();
        grad[i].zero();
        if (in && t0 + i < stop && t0 + i < end) {
          now[i] = raw_at(x + (size_t)(t0 + i) * P.ld);
          grad[i] = raw_at(dy + (size_t)(t0 + i) * D);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = t0 + i;
        if (t >= stop) break;
        if (t < end) {
          float2 f[K][2], g[2], pre[2] = {taps.bias[0], taps.bias[1]};
          now[i].get(f[K - 1]);
          grad[i].get(g);
#pragma unroll
          for (int j = 0; j < K - 1; ++j) window[j].get(f[j]);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            if (kSilu) {
#pragma unroll
              for (int j = 0; j < K; ++j) pre[p] = fma2(taps.w[j][p], f[j][p], pre[p]);
              // silu' = sig (1 + pre (1 - sig)).
              const float2 sig = sigmoid2(pre[p]);
              g[p] = mul2(g[p], mul2(sig, fma2(pre[p], sub2(both(1.f), sig), both(1.f))));
            }
#pragma unroll
            for (int k = 0; k < K; ++k) acc[k][p] = fma2(taps.w[K - 1 - k][p], g[p], acc[k][p]);
            if (t < e) {
              dbias[p] = add2(dbias[p], g[p]);
#pragma unroll
              for (int j = 0; j < K; ++j) dw[j][p] = fma2(g[p], f[j][p], dw[j][p]);
            }
          }
#pragma unroll
          for (int j = 0; j + 1 < K - 1; ++j) window[j] = window[j + 1];
          window[K - 2] = now[i];
        }
        const int out = t - (K - 1);       // whole now
        if (in && (out >= a || (a == begin && P.dx0))) {
          if (P.dxT && out >= end - (K - 1)) {
            float2 f[2];
            raw_at(dxT + ((size_t)s * (K - 1) + out - (end - (K - 1))) * D).get(f);
            acc[K - 1][0] = add2(acc[K - 1][0], f[0]);
            acc[K - 1][1] = add2(acc[K - 1][1], f[1]);
          }
          T* const at = out >= a ? dx + (size_t)out * P.ld_grad
                                 : dx0 + ((size_t)s * (K - 1) + (K - 1) + out - begin) * D;
          store_row(at, acc[K - 1][0], acc[K - 1][1]);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int k = K - 1; k > 0; --k) acc[k][p] = acc[k - 1][p];
          acc[0][p] = both(0.f);
        }
      }
    }
  };

  for (int run = part * kWarps + warp; run < P.runs; run += parts * kWarps) {
    const int r0 = run * P.run, r1 = min(r0 + P.run, P.packed.rows);
    const bool last_run = run == P.runs - 1;
    int s = first_from(P.packed, r0);
    if (s > 0 && s <= P.packed.n_seq) {
      const int end = P.packed.begin(s);
      if (r0 < min(end, r1)) rows(s - 1, P.packed.begin(s - 1), end, r0, min(end, r1));
    }
    for (; s < P.packed.n_seq; ++s) {
      const int begin = P.packed.begin(s), end = P.packed.begin(s + 1);
      if (begin >= r1 && !(last_run && begin == r1)) break;
      rows(s, begin, end, begin, min(end, r1));
    }
  }
  if (!P.partial) return;
  if (warp > 0) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int j = 0; j < K; ++j) sums[warp - 1][j][p][lane] = dw[j][p];
      sums[warp - 1][K][p][lane] = dbias[p];
    }
  }
  __syncthreads();
  if (warp > 0 || !in) return;
  float* const to = P.partial + (size_t)part * (K + 1) * D + c;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    float2 v[2] = {j < K ? dw[j < K ? j : 0][0] : dbias[0], j < K ? dw[j < K ? j : 0][1] : dbias[1]};
#pragma unroll
    for (int q = 0; q < kWarps - 1; ++q) {
      v[0] = add2(v[0], sums[q][j][0][lane]);
      v[1] = add2(v[1], sums[q][j][1][lane]);
    }
    store_row(to + (size_t)j * D, v[0], v[1]);
  }
}

// Sums of [parts][taps + 1][D] over the parts, always in the same order: 32
// columns a block, each of 32 warps every 32nd part, then the warps.
__global__ void __launch_bounds__(1024)
    conv_sums_kernel(const Packed packed, const float* partial, int parts, int D, int K, float* dw,
                     float* dbias) {
  wait_for_stream();
  if (!offsets_ok(packed)) return;
  __shared__ float warps[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, width = (K + 1) * D;
  const int i = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (i < width) {
#pragma unroll 4
    for (int n = warp; n < parts; n += 32) a += __ldg(partial + (size_t)n * width + i);
  }
  warps[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || i >= width) return;
  float sum = 0.f;
  for (int w = 0; w < 32; ++w) sum += warps[w][lane];
  const int j = i / D, c = i % D;
  if (j == K) {
    if (dbias) dbias[c] = sum;
  } else if (dw) {
    dw[(size_t)c * K + j] = sum;
  }
}

// ----------------------------------------------------------------- one token
// A block takes kGroup tokens and all of their channels, four a thread.
template <typename T, int K, bool kSilu, int kGroup>
__global__ void __launch_bounds__(kThreads) step_kernel(const ConvArgs P, T* state, int n_slots,
                                                        const int32_t* slots) {
  wait_for_stream();
  __shared__ SlotTable<kGroup, kThreads> table;
  const int row0 = blockIdx.x * kGroup, n = min(kGroup, P.packed.rows - row0), D = P.D;
  table.find(slots, row0, n, n_slots, P.status);
  for (int c = threadIdx.x * 4; c < D; c += kThreads * 4) {
    Taps<K> taps;
    taps.load(P.w, P.bias, c, true);
    for (int i = 0; i < n; ++i) {
      const int slot = table.own[i];
      if (slot < 0) continue;
      const int row = row0 + i;
      T* const at = state + (size_t)slot * (K - 1) * D + c;
      Raw<T> window[K];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) window[j] = raw_at(at + (size_t)j * D);
      window[K - 1] = raw_at(static_cast<const T*>(P.x) + (size_t)row * P.ld + c);
      float2 pre[2] = {taps.bias[0], taps.bias[1]};
#pragma unroll
      for (int j = 0; j < K; ++j) {
        float2 f[2];
        window[j].get(f);
        pre[0] = fma2(taps.w[j][0], f[0], pre[0]);
        pre[1] = fma2(taps.w[j][1], f[1], pre[1]);
      }
      if (kSilu) {
        pre[0] = mul2(pre[0], sigmoid2(pre[0]));
        pre[1] = mul2(pre[1], sigmoid2(pre[1]));
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j) put_raw(at + (size_t)j * D, window[j + 1]);
      store_row(static_cast<T*>(P.y) + (size_t)row * D + c, pre[0], pre[1]);
    }
  }
}

int col_tiles_of(int D) { return (D + kWarpCols - 1) / kWarpCols; }

// Rows of a run: at most kMostRun, fewer where the GPU would not be filled.
constexpr int kMostRun = 32, kLeastRun = 8;
int run_of(int rows, int D) {
  const long long warps = (long long)device_limits().sms * 32;
  const long long run = (long long)rows * col_tiles_of(D) / warps;
  return run >= kMostRun ? kMostRun : run <= kLeastRun ? kLeastRun : (int)run;
}

// Parts of the sums over rows: at most what fills the GPU.
int most_parts(int D) { return 4 * device_limits().sms / col_tiles_of(D) + 1; }

ConvArgs args_of(const ConvDims& d, const ConvInputs& in, unsigned* status) {
  ConvArgs P{};
  P.packed = Packed{in.offsets, d.n_seq, d.rows};
  P.x = in.x;
  P.w = in.w;
  P.bias = in.bias;
  P.x0 = in.x0;
  P.ld = d.ld;
  P.ld_grad = d.ld_grad;
  P.D = d.D;
  P.col_tiles = col_tiles_of(d.D);
  P.run = run_of(d.rows, d.D);
  P.runs = d.rows > 0 ? (d.rows + P.run - 1) / P.run : 1;
  P.status = status;
  return P;
}

// f<T, K, kSilu>() of a call.
template <class F>
cudaError_t with_kind(const ConvDims& d, F f) {
  using std::integral_constant;
  auto act = [&](auto t, auto k) {
    return d.act == SDM_ACT_SILU ? f(t, k, integral_constant<bool, true>{})
                                 : f(t, k, integral_constant<bool, false>{});
  };
  auto taps = [&](auto t) {
    if (d.taps == 2) return act(t, integral_constant<int, 2>{});
    if (d.taps == 3) return act(t, integral_constant<int, 3>{});
    return act(t, integral_constant<int, 4>{});
  };
  return d.dtype == SDM_BF16 ? taps(__nv_bfloat16{}) : taps(float{});
}

}  // namespace

size_t short_conv_workspace_bytes(const ConvDims& d) {
  return (size_t)most_parts(d.D) * (d.taps + 1) * d.D * sizeof(float);
}

cudaError_t launch_short_conv_forward(const ConvDims& d, const ConvInputs& in, void* y, void* xT,
                                      unsigned* status, cudaStream_t stream) {
  ConvArgs P = args_of(d, in, status);
  P.y = y;
  P.xT = xT;
  const unsigned blocks = (unsigned)((P.runs + kWarps - 1) / kWarps) * P.col_tiles;
  return with_kind(d, [&](auto t, auto k, auto silu) {
    return launch_behind(forward_kernel<decltype(t), decltype(k)::value, decltype(silu)::value>,
                         blocks, kThreads, 0, stream, P);
  });
}

cudaError_t launch_short_conv_backward(const ConvDims& d, const ConvInputs& in, const void* dy,
                                       const void* dxT, void* dx, float* dw, float* dbias,
                                       void* dx0, void* workspace, unsigned* status,
                                       cudaStream_t stream) {
  if (d.n_seq == 0) {                      // sums over nothing
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemsetAsync(dw, 0, (size_t)d.D * d.taps * 4, stream);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)d.D * 4, stream);
    return e;
  }
  ConvArgs P = args_of(d, in, status);
  P.dy = dy;
  P.dxT = dxT;
  P.dx = dx;
  P.dx0 = dx0;
  P.partial = dw || dbias ? static_cast<float*>(workspace) : nullptr;
  const int most = most_parts(d.D), want = (P.runs + kWarps - 1) / kWarps;
  const int parts = want < most ? want : most;
  const cudaError_t e = with_kind(d, [&](auto t, auto k, auto silu) {
    return launch_behind(backward_kernel<decltype(t), decltype(k)::value, decltype(silu)::value>,
                         (unsigned)parts * P.col_tiles, kThreads, 0, stream, P);
  });
  if (e != cudaSuccess || !P.partial) return e;
  const unsigned blocks = (unsigned)(((d.taps + 1) * d.D + 31) / 32);
  return launch_behind(conv_sums_kernel, blocks, 1024, 0, stream, P.packed, (const float*)P.partial,
                       parts, d.D, d.taps, dw, dbias);
}

// Tokens from which on a block takes kMany of them (see SlotTable).
constexpr int kManyRows = 16384, kMany = 64;

cudaError_t launch_short_conv_step(const ConvDims& d, const ConvInputs& in, void* state,
                                   int n_slots, const int32_t* slots, void* y, unsigned* status,
                                   cudaStream_t stream) {
  ConvArgs P = args_of(d, in, status);
  P.y = y;
  const bool many = slots && d.rows >= kManyRows;
  return with_kind(d, [&](auto t, auto k, auto silu) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value;
    constexpr bool kSilu = decltype(silu)::value;
    if (many)
      return launch_behind(step_kernel<T, K, kSilu, kMany>, (unsigned)((d.rows + kMany - 1) / kMany),
                           kThreads, 0, stream, P, static_cast<T*>(state), n_slots, slots);
    return launch_behind(step_kernel<T, K, kSilu, 1>, (unsigned)d.rows, kThreads, 0, stream, P,
                         static_cast<T*>(state), n_slots, slots);
  });
}

}  // namespace sdm
