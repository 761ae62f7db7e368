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
// loaded once but for taps - 1 rows in front of (behind) a run.  Where sequences begin
// does not matter to the cutting, so that short ones cost no more than their rows.  Rows
// come through shared memory a few batches ahead: in registers there was room for one
// batch (32768 x 2048 bf16: backward 95 us, now 79; 3000 sequences of two rows, 1920
// channels: forward 39, now 33).
// Measured at 32768 x 2048 bf16: forward 47 us (0.84 of the copy rate), backward 79 us
// (0.75: latency at three warps a scheduler, issue slots 54% and fp32 units 51% busy); at
// 10007 x 1000 float32 11 and 24 us; 64 single tokens of 1920 channels 3.5 us, 4000 24 us.
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

// Blocks a multiprocessor of the forward and the backward pass.  Measured at 32768 x 2048
// bf16, us: forward with 4, 5, 6, 8 blocks 47, 49, 48, 48 (65535 sequences of four rows,
// 1024 channels, with starts, which wait for their first rows: 574, 492, 442, 411); backward
// with 2, 3, 4 76, 79, 82 (3000 sequences of two rows, 1920 channels: 91, 72, 67).
constexpr int kPerSm = 4, kBackPerSm = 3;
// Batches of rows in shared memory, one of them being worked on: what 48 KB hold of float32
// (backward).  Backward at 32768 x 2048 bf16 with 2, 3, 4, 6 batches of four rows 86, 80, 80,
// 81 us; batches of three and six rows 82 and 80.
constexpr int kBatch = 4, kRingBf16 = 4, kRingF32 = 3;
template <typename T>
constexpr int kRing = sizeof(T) == 2 ? kRingBf16 : kRingF32;
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
  __device__ __forceinline__ void get(Pair (&f)[2]) const {
    f[0] = bits2(make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u)));
    f[1] = bits2(make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)));
  }
  __device__ __forceinline__ void zero() { w = make_uint2(0u, 0u); }
};
template <>
struct Raw<float> {
  float4 w;
  __device__ __forceinline__ void get(Pair (&f)[2]) const {
    f[0] = bits2(make_float2(w.x, w.y));
    f[1] = bits2(make_float2(w.z, w.w));
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

// The same on its way to shared memory.
__device__ __forceinline__ void copy_raw(Raw<__nv_bfloat16>* to, const __nv_bfloat16* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_raw(Raw<float>* to, const float* from) { cp_async16(to, from); }

// Rounded to T: apart from the store, so that a condition covers that alone.
template <typename T>
__device__ __forceinline__ Raw<T> raw_of(const Pair (&f)[2]) {
  Raw<T> r;
  store_row(reinterpret_cast<T*>(&r), float2_of(f[0]), float2_of(f[1]));
  return r;
}
template <typename T>
__device__ __forceinline__ void put(T* p, const Pair (&f)[2]) {
  store_row(p, float2_of(f[0]), float2_of(f[1]));
}

// Taps of four channels: w[j] of [D][K] as pairs of channels; and constants of the
// activation, made out of the compiler's sight (see Constants).
template <int K>
struct Taps {
  Pair w[K][2], bias[2], minus_log2e, one;
  __device__ __forceinline__ void load(const float* at, const float* b, int c) {
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        w[j][p] = bits2(make_float2(__ldg(at + (size_t)(c + 2 * p) * K + j),
                                    __ldg(at + (size_t)(c + 2 * p + 1) * K + j)));
    bias[0] = bias[1] = 0;
    if (b) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(b + c));
      bias[0] = bits2(make_float2(v.x, v.y));
      bias[1] = bits2(make_float2(v.z, v.w));
    }
    minus_log2e = bits2(hidden(-kLog2e));
    one = bits2(hidden(1.f));
  }
  // 1 / (1 + exp(-v)); where exp overflows it is 0.
  __device__ __forceinline__ Pair sigmoid(Pair v) const {
    return rcp_pair(add2(one, ex2_pair(mul2(v, minus_log2e))));
  }
  // bias + sum w[j] row[j], of one pair of channels.
  template <class Rows>
  __device__ __forceinline__ Pair pre(const Rows& rows, Pair now, int p) const {
    Pair v = bias[p];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) v = fma2(w[j][p], rows[j][p], v);
    return fma2(w[K - 1][p], now, v);
  }
};
// A new row behind the others, the first one leaves.
template <int M>
__device__ __forceinline__ void shift(Pair (&rows)[M][2], const Pair (&now)[2]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int j = 0; j + 1 < M; ++j) rows[j][p] = rows[j + 1][p];
    rows[M - 1][p] = now[p];
  }
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
__global__ void __launch_bounds__(kThreads, kPerSm) forward_kernel(const ConvArgs P) {
  wait_for_stream();
  if (!offsets_ok(P.packed)) {
    if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    return;
  }
  // Rows of x on their way, every thread's own channels.
  __shared__ Raw<T> ring[kRing<T>][kBatch][kThreads];
  const int lane = threadIdx.x & 31, run = blockIdx.x / P.col_tiles * kWarps + (threadIdx.x >> 5);
  if (run >= P.runs) return;
  const int D = P.D, col = (blockIdx.x % P.col_tiles * 32 + lane) * 4;
  const bool in = col < D;
  const int c = min(col, D - 4);           // (lanes without channels go along with the last)
  const int r0 = run * P.run, r1 = min(r0 + P.run, P.packed.rows);
  const bool last_run = run == P.runs - 1;
  const T* const x = static_cast<const T*>(P.x) + c;
  const T* const x0 = static_cast<const T*>(P.x0) + c;
  T* const y = static_cast<T*>(P.y) + c;
  T* const xT = static_cast<T*>(P.xT) + c;
  Taps<K> taps;
  taps.load(P.w, P.bias, c);

  Pair window[K - 1][2];                   // the rows before the next, oldest first
  T* to;                                   // the next row of y
  auto row = [&](const Raw<T>& raw) {
    Pair now[2], out[2];
    raw.get(now);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      out[p] = taps.pre(window, now[p], p);
      if (kSilu) out[p] = mul2(out[p], taps.sigmoid(out[p]));
    }
    const Raw<T> o = raw_of<T>(out);
    if (in) put_raw(to, o);
    to += D;
    shift(window, now);
  };
  // Batches of rows, the next ones' copies on their way during one's arithmetic.
  auto rows = [&](int a, int e) {
    const T* from = x + (size_t)a * P.ld;  // (a product of 64 bits per row otherwise)
    to = y + (size_t)a * D;
    auto ask = [&](int t, int slot) {      // (a group of copies a batch, if an empty one)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (t + i < e) copy_raw(&ring[slot][i][threadIdx.x], from);
        from += P.ld;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing<T> - 1; ++i) ask(a + i * kBatch, i);
    int slot = 0, free = kRing<T> - 1;        // the batch's place, and the one of the batch before
    for (int t = a; t < e; t += kBatch) {
      cp_async_wait<kRing<T> - 2>();
      ask(t + (kRing<T> - 1) * kBatch, free);
      const auto& now = ring[slot];
      if (t + kBatch <= e) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) row(now[i][threadIdx.x]);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (t + i < e) row(now[i][threadIdx.x]);
      }
      free = slot;
      slot = slot + 1 == kRing<T> ? 0 : slot + 1;
    }
  };

  int s = first_from(P.packed, r0);
  // A sequence that began before the run.
  if (s > 0 && s <= P.packed.n_seq) {
    const int begin = P.packed.begin(s - 1), end = P.packed.begin(s);
    const int a = max(r0, begin + K - 1), e = min(end, r1);
    if (a < e) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) raw_at(x + (size_t)(a - (K - 1) + j) * P.ld).get(window[j]);
      rows(a, e);
    }
  }
  for (; s < P.packed.n_seq; ++s) {
    const int begin = P.packed.begin(s), end = P.packed.begin(s + 1);
    if (begin >= r1 && !(last_run && begin == r1)) break;
    Raw<T> last[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      Raw<T> w;
      w.zero();
      if (P.x0) w = raw_at(x0 + ((size_t)s * (K - 1) + j) * D);
      w.get(window[j]);
    }
    if (P.xT) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int at = end - (K - 1) + j;
        last[j].zero();
        if (at >= begin) last[j] = raw_at(x + (size_t)at * P.ld);
        else if (P.x0) last[j] = raw_at(x0 + ((size_t)s * (K - 1) + (K - 1) + at - begin) * D);
      }
      __syncwarp();                        // (lanes that go along have read it too)
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
__global__ void __launch_bounds__(kThreads, kBackPerSm) backward_kernel(const ConvArgs P) {
  wait_for_stream();
  if (!offsets_ok(P.packed)) {
    if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    return;
  }
  // Rows of x and dy on their way, every thread's own channels: a batch is worked on, the
  // others are under way.  At the end the sums of the warps.
  __shared__ union Smem {
    Raw<T> ring[kRing<T>][kBatch][2][kThreads];
    Pair sums[kWarps - 1][K + 1][2][32];
    __device__ Smem() {}
  } sh;
  static_assert(sizeof(sh) <= 48 * 1024, "");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = P.D;
  const int part = blockIdx.x / P.col_tiles, parts = gridDim.x / P.col_tiles;
  const int col = (blockIdx.x % P.col_tiles * 32 + lane) * 4;
  const bool in = col < D;
  const int c = min(col, D - 4);           // (lanes without channels go along with the last)
  const T* const x = static_cast<const T*>(P.x) + c;
  const T* const x0 = static_cast<const T*>(P.x0) + c;
  const T* const dy = static_cast<const T*>(P.dy) + c;
  const T* const dxT = static_cast<const T*>(P.dxT) + c;
  T* const dx = static_cast<T*>(P.dx) + c;
  T* const dx0 = static_cast<T*>(P.dx0) + c;
  Taps<K> taps;
  taps.load(P.w, P.bias, c);
  const Pair minus_one = bits2(hidden(-1.f));
  Pair dw[K][2], dbias[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < K; ++j) dw[j][0] = dw[j][1] = 0;

  // Rows a .. e - 1 of sequence s (rows begin .. end - 1).
  auto rows = [&](int s, int begin, int end, int a, int e) {
    Pair window[K - 1][2], dpre[K - 1][2]; // x and dpre of the rows before t, oldest first
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int at = a - (K - 1) + j;
      Raw<T> w;
      w.zero();
      if (at >= begin) w = raw_at(x + (size_t)at * P.ld);
      else if (P.x0) w = raw_at(x0 + ((size_t)s * (K - 1) + (K - 1) + at - begin) * D);
      w.get(window[j]);
      dpre[j][0] = dpre[j][1] = 0;
    }
    const int stop = e + K - 1;            // dx of row t - (K - 1) leaves at t
    const T* from_x = x + (size_t)a * P.ld;   // (products of 64 bits per row otherwise)
    const T* from_dy = dy + (size_t)a * D;
    T* to = dx + (a - (K - 1)) * P.ld_grad;
    const int known = min(stop, end);
    auto ask = [&](int t, int slot) {      // (a group of copies a batch, if an empty one)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (t + i < known) {
          copy_raw(&sh.ring[slot][i][0][threadIdx.x], from_x);
          copy_raw(&sh.ring[slot][i][1][threadIdx.x], from_dy);
        }
        from_x += P.ld;
        from_dy += D;
      }
      cp_async_commit();
    };
    // One row: kInside where it and the row that leaves are rows a .. e - 1.
    auto row = [&](int t, const Raw<T>& raw_x, const Raw<T>& raw_dy, auto inside) {
      constexpr bool kInside = decltype(inside)::value;
      Pair now[2] = {0, 0}, g[2] = {0, 0}, leaves[2];
      if (kInside || t < end) {
        raw_x.get(now);
        raw_dy.get(g);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (kSilu) {
            // silu' = sig (1 + pre (1 - sig)).
            const Pair pre = taps.pre(window, now[p], p), sig = taps.sigmoid(pre);
            const Pair rest = fma2(sig, minus_one, taps.one);
            g[p] = mul2(g[p], mul2(sig, fma2(pre, rest, taps.one)));
          }
          if (kInside || t < e) {
            dbias[p] = add2(dbias[p], g[p]);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) dw[j][p] = fma2(g[p], window[j][p], dw[j][p]);
            dw[K - 1][p] = fma2(g[p], now[p], dw[K - 1][p]);
          }
        }
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        leaves[p] = mul2(taps.w[0][p], g[p]);
#pragma unroll
        for (int j = K - 2; j >= 0; --j) leaves[p] = fma2(taps.w[K - 1 - j][p], dpre[j][p], leaves[p]);
      }
      shift(window, now);
      shift(dpre, g);
      const int out = t - (K - 1);
      if (kInside) {
        const Raw<T> o = raw_of<T>(leaves);
        if (in) put_raw(to, o);
      } else if (in && (out >= a || (a == begin && P.dx0))) {
        if (P.dxT && out >= end - (K - 1)) {
          Pair f[2];
          raw_at(dxT + ((size_t)s * (K - 1) + out - (end - (K - 1))) * D).get(f);
          leaves[0] = add2(leaves[0], f[0]);
          leaves[1] = add2(leaves[1], f[1]);
        }
        put(out >= a ? to : dx0 + ((size_t)s * (K - 1) + (K - 1) + out - begin) * D, leaves);
      }
      to += P.ld_grad;
    };
#pragma unroll
    for (int i = 0; i < kRing<T> - 1; ++i) ask(a + i * kBatch, i);
    int slot = 0, free = kRing<T> - 1;        // the batch's place, and the one of the batch before
    for (int t = a; t < stop; t += kBatch) {
      cp_async_wait<kRing<T> - 2>();
      ask(t + (kRing<T> - 1) * kBatch, free);
      const auto& now = sh.ring[slot];
      if (t > a && t + kBatch <= e) {      // (kBatch >= K - 1: what leaves is at least row a)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) row(t + i, now[i][0][threadIdx.x], now[i][1][threadIdx.x], std::true_type{});
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (t + i < stop) row(t + i, now[i][0][threadIdx.x], now[i][1][threadIdx.x], std::false_type{});
      }
      free = slot;
      slot = slot + 1 == kRing<T> ? 0 : slot + 1;
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
  cp_async_wait_all();
  __syncthreads();                         // the warps are done with the rows
  if (warp > 0) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int j = 0; j < K; ++j) sh.sums[warp - 1][j][p][lane] = dw[j][p];
      sh.sums[warp - 1][K][p][lane] = dbias[p];
    }
  }
  __syncthreads();
  if (warp > 0 || !in) return;
  float* const to = P.partial + (size_t)part * (K + 1) * D + c;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    Pair v[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      v[p] = j < K ? dw[j < K ? j : 0][p] : dbias[p];
#pragma unroll
      for (int q = 0; q < kWarps - 1; ++q) v[p] = add2(v[p], sh.sums[q][j][p][lane]);
    }
    put(to + (size_t)j * D, v);
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
// A block takes kGroup tokens by 512 channels, four a thread.  What does not depend on
// the slots is on its way while they are looked at.
template <typename T, int K, bool kSilu, int kGroup>
__global__ void __launch_bounds__(kThreads) step_kernel(const ConvArgs P, T* state, int n_slots,
                                                        const int32_t* slots, int parts) {
  wait_for_stream();
  __shared__ SlotTable<kGroup, kThreads> table;
  const int row0 = (int)(blockIdx.x / parts) * kGroup, n = min(kGroup, P.packed.rows - row0), D = P.D;
  const int col = ((int)(blockIdx.x % parts) * kThreads + threadIdx.x) * 4, c = min(col, D - 4);
  const T* const x = static_cast<const T*>(P.x) + (size_t)row0 * P.ld + c;
  Taps<K> taps;
  taps.load(P.w, P.bias, c);
  constexpr int kAhead = kGroup < 4 ? kGroup : 4;            // tokens at a time
  Raw<T> first = raw_at(x);
  table.find(slots, row0, n, n_slots, P.status);
  if (col >= D) return;
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    Raw<T> raw[kAhead][K];
    T* at[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int slot = i0 + i < n ? table.own[i0 + i] : -1;
      at[i] = slot < 0 ? nullptr : state + (size_t)slot * (K - 1) * D + c;
      if (slot < 0) continue;
#pragma unroll
      for (int j = 0; j < K - 1; ++j) raw[i][j] = raw_at(at[i] + (size_t)j * D);
      raw[i][K - 1] = kGroup == 1 ? first : raw_at(x + (size_t)(i0 + i) * P.ld);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!at[i]) continue;
      Pair window[K - 1][2], now[2], out[2];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) raw[i][j].get(window[j]);
      raw[i][K - 1].get(now);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        out[p] = taps.pre(window, now[p], p);
        if (kSilu) out[p] = mul2(out[p], taps.sigmoid(out[p]));
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j) put_raw(at[i] + (size_t)j * D, raw[i][j + 1]);
      put(static_cast<T*>(P.y) + (size_t)(row0 + i0 + i) * D + c, out);
    }
  }
}

int col_tiles_of(int D) { return (D + kWarpCols - 1) / kWarpCols; }

// Rows of a run, so that the runs' blocks of kWarps runs fill the GPU once with
// `per_sm` blocks a multiprocessor.
constexpr int kLeastRun = 8, kMostRun = 1 << 16;
int groups_of(int D, int per_sm) {
  const int n = per_sm * device_limits().sms / col_tiles_of(D);
  return n > 0 ? n : 1;
}
int run_of(int rows, int D, int per_sm) {
  const long long warps = (long long)groups_of(D, per_sm) * kWarps, run = (rows + warps - 1) / warps;
  return run >= kMostRun ? kMostRun : run <= kLeastRun ? kLeastRun : (int)run;
}

ConvArgs args_of(const ConvDims& d, const ConvInputs& in, int per_sm, unsigned* status) {
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
  P.run = run_of(d.rows, d.D, per_sm);
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
  return (size_t)groups_of(d.D, kBackPerSm) * (d.taps + 1) * d.D * sizeof(float);
}

cudaError_t launch_short_conv_forward(const ConvDims& d, const ConvInputs& in, void* y, void* xT,
                                      unsigned* status, cudaStream_t stream) {
  ConvArgs P = args_of(d, in, kPerSm, status);
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
  ConvArgs P = args_of(d, in, kBackPerSm, status);
  P.dy = dy;
  P.dxT = dxT;
  P.dx = dx;
  P.dx0 = dx0;
  P.partial = dw || dbias ? static_cast<float*>(workspace) : nullptr;
  const int most = groups_of(d.D, kBackPerSm), want = (P.runs + kWarps - 1) / kWarps;
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

cudaError_t launch_short_conv_step(const ConvDims& d, const ConvInputs& in, void* state,
                                   int n_slots, const int32_t* slots, void* y, unsigned* status,
                                   cudaStream_t stream) {
  ConvArgs P = args_of(d, in, 1, status);
  P.y = y;
  const int parts = (d.D / 4 + kThreads - 1) / kThreads;
  return with_kind(d, [&](auto t, auto k, auto silu) {
    using T = decltype(t);
    constexpr int K = decltype(k)::value;
    constexpr bool kSilu = decltype(silu)::value;
    return with_group(d.rows, (long long)d.rows * parts, 2048, [&](auto group) {
      constexpr int G = decltype(group)::value;
      return launch_behind(step_kernel<T, K, kSilu, G>, (unsigned)(((long long)d.rows + G - 1) / G * parts),
                           kThreads, 0, stream, P, static_cast<T*>(state), n_slots, slots, parts);
    });
  });
}

}  // namespace sdm
