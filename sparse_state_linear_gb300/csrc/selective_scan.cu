// selective_scan.cu -- selective state space scan over packed sequences:
// forward, backward and single-token step.
//
// Per channel c, state n and row t, with one B and C for the channels of a group:
//   delta = softplus(dt + bias),  a = exp(-A delta),  u = delta x,
//   h[t] = a h[t-1] + u B[n],  inner = sum_n C[n] h[t] + skip x,  y = inner silu(z).
// Backward, from the last row to the first, with dinner = dy silu(z):
//   g = dinner C[n] + r,  r = a g (r starts as the gradient of the final state),
//   p = r h[t-1],  du = sum_n g B[n],  ddelta = du x - sum_n A p,
//   dx = du delta + dinner skip,  ddt = ddelta sigmoid(dt + bias),  dz = dy inner silu'(z),
//   dB[n] = sum_c g u,  dC[n] = sum_c dinner h[t],  dA = -sum_t delta p,
//   dskip = sum_t dinner x,  dbias = sum_t ddt.
//
// Sequences are cut into chunks of L rows where the GPU would not be filled
// otherwise.  The state behind a chunk is S + exp(-A sum delta) h with S the state
// behind it from zeros: one kernel finds S and the sum of every chunk, one folds
// them along each sequence, and the third walks every chunk from the state in
// front of it (backward: behind it, from the last row to the first).
//
// Bound by latency at few warps: the warps of a block load, form delta and u, meet, run the
// rows and write out one after the other, and two to four warps a scheduler do not fill
// these stretches.  No unit is saturated (issue slots 55 to 61%, fp32 46 to 52%, 2^x 25 to
// 57%); by its 2^x (4 cycles a warp) and packed fp32 pairs (2) the work would take about half
// the time.  Measured, bf16, N = 16: 131072 x 1024 in one sequence 996 us (summary 395,
// forward 600; operations 560, bytes 159), 32768 x 1024 in eight sequences with its backward
// pass 985 us (summaries 117 and 126, forward 174, backward 541; operations 420, bytes 110),
// 64 single tokens of 1920 channels 5.2 us.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "gates.cuh"
#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"
#include "packing.cuh"
#include "park.cuh"
#include "rows.cuh"
#include "slots.cuh"

namespace sdm {
namespace {

constexpr int kStateRows = 16;             // rows between saved states

// Blocks of the forward pass and of the summaries: two warps, eight rows at a time.  A
// thread holds 16 neighbouring states (all 8 where N = 8) of CH channels, as pairs of
// states, so that what a row of B and C brings from shared memory serves CH channels
// and y is summed within a thread (over 2 or 4 lanes where N is 32 or 64).  (131072 x
// 1024 x 16: with four states of four channels 1204 us, with 16 of one 1062, so 1022; the
// forward kernel with 4, 8 and 16 rows at a time 628, 592 and 653.)
template <int N>
struct Wide {
  static constexpr int kWarps = 2, kRows = 8, kCols = 1024 / N;   // channels of a warp
  static constexpr int NT = N < 16 ? N : 16, CH = 32 / NT, NL = N / NT;
};
// Blocks of the backward pass: four warps, 16 rows at a time.  A thread holds four
// states of four channels, as pairs of channels, so that the sums over states and those
// over channels are both half done within it.  NL neighbouring lanes share channels, CL
// groups of them have channels of their own.
template <int N>
struct Square {
  static constexpr int kWarps = 4, kRows = 16, kCols = 512 / N;
  static constexpr int NL = N / 4, CL = 32 / NL;
  static constexpr int kNBits = NL == 2 ? 1 : NL == 4 ? 2 : NL == 8 ? 3 : 4, kCBits = 5 - kNBits;
};
// Blocks a multiprocessor that the registers leave room for.  Measured, us: scan of 131072
// x 1024 x 16 bf16 with 5, 6, 7, 8 forward blocks 1044, 1035, 1042, 1088; the backward
// pass of 32768 x 1024 with 2 blocks 570, and with 3 of half the rows at a time 577.
// (At 8 summary blocks the backward pass's summary of bf16, N = 16, spills 36 bytes.)  With
// N = 8 a block has 256 channels and shared memory allows fewer: summaries 7 blocks (float32
// 5), forward 5 (3), backward 1.
constexpr int kSummaryBlocks = 8, kForwardBlocks = 6, kBackBlocks = 2;
constexpr int kBlockStates = 2048;         // a block's states: its channels are 2048 / N
// How a warp goes through rows of its channels: four channels a lane and step.
template <class S>
struct Steps {
  static constexpr int kThreads = 32 * S::kWarps, QL = S::kCols / 4, kItems = S::kRows * QL / 32;
};

// From this many sequences on the offsets are checked by a kernel of their own, which
// leaves its finding in the workspace: looked through by every block they are most of the
// work (6000 rows in 3000 sequences, 1920 channels bf16: 888 us forward, 2438 without).
constexpr int kManySequences = 32;

struct ScanArgs {
  Packed packed;
  int* bad_offsets;      // of many sequences
  const void* x;
  const void* dt;
  const void* z;
  const void* B;
  const void* C;
  const float* A;
  const float* skip;
  const float* bias;
  long long ld, ld_z, ld_bc;
  int D, G, per;         // channels, groups, channels of a group
  int tiles, group_tiles;
  int L, chunks;         // rows of a chunk; of a sequence where all are equal
  unsigned indexes;      // chunks to look at, see Span
  float* carry;          // [numbers][D][N]: S, then the state in front of (behind) the chunk
  float* sums;           // [numbers][D]: sum of delta log2(e)
  bool split;            // whether there are chunks to be carried between
  const float* h0;       // (dhT)
  float* hT;             // (dh0)
  float* states;         // [numbers of kStateRows rows][D][N], see save_states
  void* y;
  // backward
  const void* dy;
  void* dx;
  void* ddt;
  void* dz;
  long long ld_grad, ld_z_grad;
  float* partial;        // [parts][D (N + 2)]: dA, dskip, dbias
  float* partial_bc;     // [rows][tiles][2 N]
  unsigned* status;
};

// A chunk of a sequence.
struct Span {
  int seq, number, row0, rows, begin;
  bool first, last;
};
// Whether the offsets are good (all threads of the block call it).
__device__ __forceinline__ bool offsets_good(const ScanArgs& P) {
  if (!P.packed.offsets || P.packed.n_seq < kManySequences) return offsets_ok(P.packed);
  return *P.bad_offsets == 0;
}
__global__ void __launch_bounds__(1024) check_offsets_kernel(const Packed P, int* bad) {
  wait_for_stream();
  const bool ok = offsets_ok(P);
  if (threadIdx.x == 0) *bad = !ok;
}

enum Found { kBad, kNone, kChunk };
// The chunk of an index: its number, or where sequences are equal the place among all
// of them.  All threads of the block call it; kBad: the offsets break their rules.  Up
// to 31 sequences every lane looks at one, so that there is one load's latency.
// kChecked: the offsets are known to be good.
template <bool kChecked>
__device__ __forceinline__ Found find_chunk(const ScanArgs& args, int index, Span& s) {
  const Packed& P = args.packed;
  const int lane = threadIdx.x & 31, L = args.L;
  int chunk, end;
  if (!P.offsets) {
    s.seq = index / args.chunks;
    chunk = index % args.chunks;
    s.begin = P.begin(s.seq);
    end = P.begin(s.seq + 1);
  } else if (P.n_seq < kManySequences) {   // at most 31
    const int o = __ldg(P.offsets + min(lane, P.n_seq)), before = __shfl_up_sync(0xffffffffu, o, 1);
    if (__any_sync(0xffffffffu, o < 0 || o > P.rows || (lane > 0 && o < before))) return kBad;
    s.seq = __popc(__ballot_sync(0xffffffffu, lane < P.n_seq && o / L + lane <= index)) - 1;
    if (s.seq < 0) return kNone;
    s.begin = __shfl_sync(0xffffffffu, o, s.seq);
    end = __shfl_sync(0xffffffffu, o, s.seq + 1);
    chunk = index - (s.begin / L + s.seq);
  } else {
    if (!kChecked && !offsets_good(args)) return kBad;
    s.seq = sequence_of(P, L, index);
    if (s.seq < 0) return kNone;
    s.begin = P.begin(s.seq);
    end = P.begin(s.seq + 1);
    chunk = index - (s.begin / L + s.seq);
  }
  const long long row0 = s.begin + (long long)chunk * L;
  if (chunk > 0 && row0 >= end) return kNone;
  s.row0 = (int)row0;
  s.rows = min(L, end - s.row0);
  s.number = s.begin / L + s.seq + chunk;
  s.first = chunk == 0;
  s.last = s.row0 + s.rows == end;
  return kChunk;
}

// Which channels a block's warps and threads work on.
template <int N, class S>
struct Place {
  int lane, warp, group, c0, c_end;        // c0: the warp's first channel; c_end: behind the group's last
  __device__ __forceinline__ Place(const ScanArgs& P, int tile) {
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    group = tile / P.group_tiles;
    c0 = group * P.per + tile % P.group_tiles * (kBlockStates / N) + warp * S::kCols;
    c_end = (group + 1) * P.per;
  }
  // The four channels and the rows that a thread takes from the inputs.
  __device__ __forceinline__ int quad() const { return lane % Steps<S>::QL * 4; }
  __device__ __forceinline__ int row(int i) const { return lane / Steps<S>::QL + i * (32 / Steps<S>::QL); }
};

// State registers: v[cp * 4 + n] holds state n of channels 2 cp and 2 cp + 1.
__device__ __forceinline__ void zero8(float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = both(0.f);
}
// From / to [D][N] at the thread's channels and states.
template <int N>
__device__ __forceinline__ void load_states(const float* p, float2 (&v)[8]) {
#pragma unroll
  for (int cp = 0; cp < 2; ++cp) {
    const float4 a = *reinterpret_cast<const float4*>(p + (2 * cp) * N);
    const float4 b = *reinterpret_cast<const float4*>(p + (2 * cp + 1) * N);
    v[cp * 4 + 0] = make_float2(a.x, b.x);
    v[cp * 4 + 1] = make_float2(a.y, b.y);
    v[cp * 4 + 2] = make_float2(a.z, b.z);
    v[cp * 4 + 3] = make_float2(a.w, b.w);
  }
}
template <int N>
__device__ __forceinline__ void store_states(float* p, const float2 (&v)[8]) {
#pragma unroll
  for (int cp = 0; cp < 2; ++cp) {
    const float2* w = v + cp * 4;
    *reinterpret_cast<float4*>(p + (2 * cp) * N) = make_float4(w[0].x, w[1].x, w[2].x, w[3].x);
    *reinterpret_cast<float4*>(p + (2 * cp + 1) * N) = make_float4(w[0].y, w[1].y, w[2].y, w[3].y);
  }
}

// Sums of V values over 2^kBits lanes, lane bits kBase on: each step a lane keeps
// half of the values and gives away the other.  In the end it has kLeft of them, from
// index() on, and one of the lanes that have the same ones is chosen().
template <int V, int kBits, int kBase>
struct Halving {
  static constexpr int kHalvings = V >= 8 ? (kBits < 3 ? kBits : 3) : V >= 4 ? (kBits < 2 ? kBits : 2) : 0;
  static constexpr int kLeft = V >> kHalvings;
  static __device__ __forceinline__ void sum(float (&v)[V], int lane) {
    int n = V;
#pragma unroll
    for (int b = kBits - 1; b >= 0; --b) {
      const int mask = 1 << (kBase + b);
      if (n > kLeft) {
        n /= 2;
        const bool upper = lane & mask;
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
          if (i < n) {
            const float keep = upper ? v[n + i] : v[i], give = upper ? v[i] : v[n + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, mask);
          }
      } else {
#pragma unroll
        for (int i = 0; i < kLeft; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], mask);
      }
    }
  }
  static __device__ __forceinline__ int index(int lane) {
    return (lane >> (kBase + kBits - kHalvings) & ((1 << kHalvings) - 1)) * kLeft;
  }
  static __device__ __forceinline__ bool chosen(int lane) {
    return (lane >> kBase & ((1 << (kBits - kHalvings)) - 1)) == 0;
  }
};

template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 w;
};
template <>
struct Raw4<float> {
  float4 w;
};
template <typename T>
__device__ __forceinline__ void get4(const Raw4<T>& r, float2 (&f)[2]) {
  load_row(reinterpret_cast<const T*>(&r), f[0], f[1]);
}
template <typename T>
__device__ __forceinline__ Raw4<T> raw4(const void* base, size_t i) {
  return *reinterpret_cast<const Raw4<T>*>(static_cast<const T*>(base) + i);
}
// The same, zeros where not `in`: a choice of what was loaded, not a branch, so that the
// arithmetic of a thread's items is interleaved.
template <typename T>
__device__ __forceinline__ void get4_if(bool in, const Raw4<T>& r, float2 (&f)[2]) {
  get4(r, f);
#pragma unroll
  for (int p = 0; p < 2; ++p) f[p] = in ? f[p] : both(0.f);
}
__device__ __forceinline__ void load_four(const float* p, bool in, float none, float2 (&f)[2]) {
  f[0] = f[1] = both(none);
  if (p && in) load_row(p, f[0], f[1]);
}

// sigmoid(v); 0 where exp(-v) overflows.
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 z = mul2(v, both(-kLog2e));
  return make_float2(rcp(1.f + ex2(z.x)), rcp(1.f + ex2(z.y)));
}

// Inputs are copied to shared memory one turn ahead, every thread what it will itself
// take from there: its items of the tensors of channels, and of B and C.
__device__ __forceinline__ void copy_item(void* to, const void* from, bool in, int bytes) {
  if (!in) return;
  if (bytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(to)), "l"(from) : "memory");
  else
    cp_async16(to, from);
}
template <typename T, int N, class S, int kTensors>
struct RawRows {
  static constexpr int kThreads = Steps<S>::kThreads, kItems = Steps<S>::kItems, kQuads = S::kRows * N / 4;
  static constexpr int kBC = (2 * kQuads + kThreads - 1) / kThreads;
  Raw4<T> rows[kTensors][kItems][kThreads];
  Raw4<T> bc[kBC][kThreads];

  // n rows from row0 on; kB, kC: which of B and C.
  template <bool kB, bool kC>
  __device__ __forceinline__ void ask(const ScanArgs& P, const Place<N, S>& at, bool in,
                                      const void* const (&from)[kTensors], const long long (&ld)[kTensors],
                                      int row0, int n) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int t = at.row(i);
#pragma unroll
      for (int k = 0; k < kTensors; ++k)
        if (from[k])
          copy_item(&rows[k][i][threadIdx.x],
                    static_cast<const T*>(from[k]) + (size_t)(row0 + t) * ld[k] + at.c0 + at.quad(), in && t < n,
                    sizeof(Raw4<T>));
    }
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int j = i * kThreads + threadIdx.x, t = j % kQuads / (N / 4), q = j % (N / 4) * 4;
      const bool c = j >= kQuads;
      const bool wanted = j < 2 * kQuads && t < n && (c ? kC : kB);
      copy_item(&bc[i][threadIdx.x],
                static_cast<const T*>(c ? P.C : P.B) + (size_t)(row0 + t) * P.ld_bc + (size_t)at.group * N + q,
                wanted, sizeof(Raw4<T>));
    }
    cp_async_commit();
  }
  // B and C to where all threads read them, zeros behind row n; as float2 every number
  // twice.
  template <bool kB, bool kC, class Out>
  __device__ __forceinline__ void spread(int n, Out (*B)[N], Out (*C)[N]) const {
#pragma unroll
    for (int i = 0; i < kBC; ++i) {
      const int j = i * kThreads + threadIdx.x, t = j % kQuads / (N / 4), q = j % (N / 4) * 4;
      const bool c = j >= kQuads;
      if (j >= 2 * kQuads || !(c ? kC : kB)) continue;
      float2 f[2] = {both(0.f), both(0.f)};
      if (t < n) get4(bc[i][threadIdx.x], f);
      float4* const to = reinterpret_cast<float4*>(&(c ? C : B)[t][q]);
      if (std::is_same<Out, float2>::value) {
        to[0] = make_float4(f[0].x, f[0].x, f[0].y, f[0].y);
        to[1] = make_float4(f[1].x, f[1].x, f[1].y, f[1].y);
      } else {
        to[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      }
    }
  }
};

// dinner = dy silu(z) of four channels; zeros where not `in`.
template <typename T>
__device__ __forceinline__ void dinner_of(bool in, const Raw4<T>& dy, const Raw4<T>& z, bool gated, float2 (&d)[2]) {
  get4_if(in, dy, d);
  if (!gated) return;
  float2 g[2];
  get4_if(in, z, g);
#pragma unroll
  for (int p = 0; p < 2; ++p) d[p] = mul2(d[p], mul2(g[p], sigmoid2(g[p])));
}

// ------------------------------------------------------------------ summaries
// Neighbouring numbers as pairs.
template <int V>
__device__ __forceinline__ void load_pairs(const float* p, float2 (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) load_row(p + 4 * i, v[2 * i], v[2 * i + 1]);
}
// A thread's states from or to [D][N]: NT of each of its CH channels.
template <int N>
__device__ __forceinline__ void load_wide(const float* p, float2 (&v)[16]) {
  using W = Wide<N>;
#pragma unroll
  for (int j = 0; j < W::CH; ++j)
#pragma unroll
    for (int k = 0; k < W::NT / 4; ++k)
      load_row(p + j * N + 4 * k, v[j * (W::NT / 2) + 2 * k], v[j * (W::NT / 2) + 2 * k + 1]);
}
template <int N>
__device__ __forceinline__ void store_wide(float* p, const float2 (&v)[16]) {
  using W = Wide<N>;
#pragma unroll
  for (int j = 0; j < W::CH; ++j)
#pragma unroll
    for (int k = 0; k < W::NT / 4; ++k)
      store_row(p + j * N + 4 * k, v[j * (W::NT / 2) + 2 * k], v[j * (W::NT / 2) + 2 * k + 1]);
}
template <int N>
__device__ __forceinline__ void load_rates(const float* p, bool in, float2 (&nA)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) nA[i] = both(0.f);
  if (in) load_wide<N>(p, nA);
#pragma unroll
  for (int i = 0; i < 16; ++i) nA[i] = make_float2(-nA[i].x, -nA[i].y);
}
// Saved states lie as the forward pass's threads hold them: of every warp's channels the
// first four states of all its threads with channels, then the next four, and so on, so
// that a warp's stores are whole lines.  Lanes with channels of a warp that begins at c0:
template <int N>
__device__ __forceinline__ int lanes_from(int c0, int c_end) {
  return min(32, max(0, c_end - c0) * Wide<N>::NL / Wide<N>::CH);
}
template <int N>
__device__ __forceinline__ void save_states(float* p, int lane, int lanes, const float2 (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) store_row(p + (i * lanes + lane) * 4, v[2 * i], v[2 * i + 1]);
}
// Where the backward pass finds four states, from 4 nl on, of channel c.
template <int N>
__device__ __forceinline__ int saved_at(int c, int tile_c0, int c_end, int nl) {
  using W = Wide<N>;
  const int c0 = tile_c0 + (c - tile_c0) / W::kCols * W::kCols, o = c - c0;
  const int lane = o / W::CH * W::NL + nl * 4 / W::NT, i = o % W::CH * (W::NT / 4) + nl * 4 % W::NT / 4;
  return c0 * N + (i * lanes_from<N>(c0, c_end) + lane) * 4;
}
// A thread's CH channels of a row of shared memory.
template <int CH>
__device__ __forceinline__ void load_channels(const float* p, float (&v)[CH]) {
  if (CH == 4) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x, v[1] = w.y, v[CH - 2] = w.z, v[CH - 1] = w.w;
  } else {
    const float2 w = *reinterpret_cast<const float2*>(p);
    v[0] = w.x, v[1] = w.y;
  }
}

template <typename T, int N>
struct SummarySmem {
  float v[2][Wide<N>::kRows][N];           // B, or C; of two times so many rows in turn
  struct {
    float sp[Wide<N>::kRows][Wide<N>::kCols], u[Wide<N>::kRows][Wide<N>::kCols];   // (dinner in the place of u)
  } warp[Wide<N>::kWarps];
  RawRows<T, N, Wide<N>, 3> raw;
};

// The state behind a chunk from zeros in front of it, and the sum of delta; with
// kBack the gradient of the state in front of it from zeros behind it.
template <typename T, int N, bool kBack>
__global__ void __launch_bounds__(Steps<Wide<N>>::kThreads, kSummaryBlocks) summary_kernel(const ScanArgs P) {
  using W = Wide<N>;
  using St = Steps<W>;
  constexpr int R = W::kRows;
  extern __shared__ __align__(16) char smem[];
  SummarySmem<T, N>& sh = *reinterpret_cast<SummarySmem<T, N>*>(smem);
  wait_for_stream();
  const Place<N, W> at(P, blockIdx.x % P.tiles);
  auto& mem = sh.warp[at.warp];
  const int nl = at.lane % W::NL, col = at.lane / W::NL * W::CH, cs = at.c0 + at.quad();
  const bool in = at.c0 + col < at.c_end, in_s = cs < at.c_end;
  const size_t state = (size_t)(at.c0 + col) * N + nl * W::NT;
  float2 nA[16], h[16];
  load_rates<N>(P.A + state, in, nA);
  float2 bias[2], sum[2] = {both(0.f), both(0.f)};
  load_four(P.bias ? P.bias + cs : nullptr, in_s, 0.f, bias);
  Span s;
  const Found found = find_chunk<false>(P, blockIdx.x / P.tiles, s);
  if (found == kBad && threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
  if (found != kChunk) return;
  if (kBack ? s.first : s.last) return;    // nobody needs it
  const void* const from[3] = {kBack ? P.dy : P.x, P.dt, kBack ? P.z : nullptr};
  const long long ld[3] = {kBack ? P.D : P.ld, P.ld, P.ld_z};
  // (What is left has rows.)
  const int last = (s.rows - 1) / R * R, step = kBack ? -R : R;
  int r = kBack ? last : 0;
  sh.raw.template ask<!kBack, kBack>(P, at, in_s, from, ld, s.row0 + r, min(R, s.rows - r));
  const Constants K = constants();
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = both(0.f);
  for (int turn = 0; r >= 0 && r <= last; r += step, turn ^= 1) {
    const int n = min(R, s.rows - r), next = r + step;
    cp_async_wait_all();
    sh.raw.template spread<!kBack, kBack>(n, sh.v[turn], sh.v[turn]);
#pragma unroll
    for (int i = 0; i < St::kItems; ++i) {
      const int t = at.row(i), q = at.quad();
      const bool valid = t < n && in_s;
      float2 sp[2], u[2], d[2];
      get4_if(valid, sh.raw.rows[1][i][threadIdx.x], d);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float2 unused, e;
        softplus_pair(K, d[p], bias[p], unused, e, sp[p]);
        sp[p] = valid ? sp[p] : both(0.f);
        sum[p] = add2(sum[p], sp[p]);
      }
      if (kBack) {
        dinner_of(valid, sh.raw.rows[0][i][threadIdx.x], sh.raw.rows[2][i][threadIdx.x], P.z != nullptr, u);
      } else {
        get4_if(valid, sh.raw.rows[0][i][threadIdx.x], d);
#pragma unroll
        for (int p = 0; p < 2; ++p) u[p] = mul2(mul2(sp[p], both(kLn2)), d[p]);
      }
      store_row(&mem.sp[t][q], sp[0], sp[1]);
      store_row(&mem.u[t][q], u[0], u[1]);
    }
    if (next >= 0 && next <= last)
      sh.raw.template ask<!kBack, kBack>(P, at, in_s, from, ld, s.row0 + next, min(R, s.rows - next));
    __syncthreads();                       // (v of the turn before is done with)
#pragma unroll 4
    for (int j = 0; j < R; ++j) {
      const int t = kBack ? R - 1 - j : j;
      float sp[W::CH], u[W::CH];
      float2 v[W::NT / 2];
      load_channels(&mem.sp[t][col], sp);
      load_channels(&mem.u[t][col], u);
      load_pairs(&sh.v[turn][t][nl * W::NT], v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int ch = i / (W::NT / 2), k = i % (W::NT / 2);
        const float2 a = ex2_pair(mul2(nA[i], both(sp[ch])));
        h[i] = kBack ? mul2(a, fma2(both(u[ch]), v[k], h[i])) : fma2(a, h[i], mul2(both(u[ch]), v[k]));
      }
    }
    __syncwarp();                          // the warp's rows are done with
  }
  if (in) store_wide<N>(P.carry + (size_t)s.number * P.D * N + state, h);
  float v[4] = {sum[0].x, sum[0].y, sum[1].x, sum[1].y};
#pragma unroll
  for (int o = St::QL; o < 32; o *= 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (at.lane < St::QL && in_s)
    store_row(P.sums + (size_t)s.number * P.D + cs, make_float2(v[0], v[1]), make_float2(v[2], v[3]));
}

// ------------------------------------------------------------------- forward
template <typename T, int N>
struct ForwardSmem {
  float B[2][Wide<N>::kRows][N], C[2][Wide<N>::kRows][N];   // of two times so many rows in turn
  struct {                                 // sp becomes y row by row
    float sp[Wide<N>::kRows][Wide<N>::kCols], u[Wide<N>::kRows][Wide<N>::kCols];
  } warp[Wide<N>::kWarps];
  RawRows<T, N, Wide<N>, 3> raw[2];
};

template <typename T, int N>
__global__ void __launch_bounds__(Steps<Wide<N>>::kThreads, kForwardBlocks) forward_kernel(const ScanArgs P) {
  using W = Wide<N>;
  using St = Steps<W>;
  constexpr int R = W::kRows;
  extern __shared__ __align__(16) char smem[];
  ForwardSmem<T, N>& sh = *reinterpret_cast<ForwardSmem<T, N>*>(smem);
  wait_for_stream();
  const Place<N, W> at(P, blockIdx.x % P.tiles);
  auto& mem = sh.warp[at.warp];
  const int nl = at.lane % W::NL, col = at.lane / W::NL * W::CH, cs = at.c0 + at.quad();
  const bool in = at.c0 + col < at.c_end, in_s = cs < at.c_end;
  const size_t state = (size_t)(at.c0 + col) * N + nl * W::NT, DN = (size_t)P.D * N;
  float2 nA[16], h[16], bias[2], skip[2];
  load_rates<N>(P.A + state, in, nA);
  load_four(P.bias ? P.bias + cs : nullptr, in_s, 0.f, bias);
  load_four(P.skip ? P.skip + cs : nullptr, in_s, 0.f, skip);
  Span s;
  const Found found = find_chunk<false>(P, blockIdx.x / P.tiles, s);
  if (found == kBad && threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
  if (found != kChunk) return;
  const void* const from[3] = {P.x, P.dt, P.z};
  const long long ld[3] = {P.ld, P.ld, P.ld_z};
  if (s.rows > 0) sh.raw[0].template ask<true, true>(P, at, in_s, from, ld, s.row0, min(R, s.rows));
  const Constants K = constants();
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = both(0.f);
  if (in) {
    if (P.split) load_wide<N>(P.carry + s.number * DN + state, h);
    else if (P.h0) load_wide<N>(P.h0 + s.seq * DN + state, h);
  }
  for (int r = 0, turn = 0; r < s.rows; r += R, turn ^= 1) {
    const int row0 = s.row0 + r, n = min(R, s.rows - r);
    auto& raw = sh.raw[turn];
    cp_async_wait_all();
    if (r + R < s.rows)
      sh.raw[turn ^ 1].template ask<true, true>(P, at, in_s, from, ld, row0 + R, min(R, s.rows - r - R));
    raw.template spread<true, true>(n, sh.B[turn], sh.C[turn]);
#pragma unroll
    for (int i = 0; i < St::kItems; ++i) {
      const int t = at.row(i), q = at.quad();
      const bool valid = t < n && in_s;
      float2 sp[2], u[2], f[2], d[2];
      get4_if(valid, raw.rows[0][i][threadIdx.x], f);
      get4_if(valid, raw.rows[1][i][threadIdx.x], d);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float2 unused, e;
        softplus_pair(K, d[p], bias[p], unused, e, sp[p]);
        sp[p] = valid ? sp[p] : both(0.f);
        u[p] = mul2(mul2(sp[p], both(kLn2)), f[p]);
      }
      store_row(&mem.sp[t][q], sp[0], sp[1]);
      store_row(&mem.u[t][q], u[0], u[1]);
    }
    __syncthreads();                       // (B and C of the turn before are done with)
    if (P.states && in && (row0 - s.begin) % kStateRows == 0)
      save_states<N>(P.states + ((size_t)(s.begin / kStateRows + s.seq) + (row0 - s.begin) / kStateRows) * DN +
                         (size_t)at.c0 * N, at.lane, lanes_from<N>(at.c0, at.c_end), h);
#pragma unroll 4
    for (int t = 0; t < R; ++t) {
      float sp[W::CH], u[W::CH], y[W::CH];
      float2 B[W::NT / 2], C[W::NT / 2];
      load_channels(&mem.sp[t][col], sp);
      load_channels(&mem.u[t][col], u);
      load_pairs(&sh.B[turn][t][nl * W::NT], B);
      load_pairs(&sh.C[turn][t][nl * W::NT], C);
#pragma unroll
      for (int j = 0; j < W::CH; ++j) {
        float2 sum = both(0.f);
#pragma unroll
        for (int k = 0; k < W::NT / 2; ++k) {
          const int i = j * (W::NT / 2) + k;
          h[i] = fma2(ex2_pair(mul2(nA[i], both(sp[j]))), h[i], mul2(both(u[j]), B[k]));
          sum = k ? fma2(C[k], h[i], sum) : mul2(C[k], h[i]);
        }
        y[j] = sum.x + sum.y;
#pragma unroll
        for (int m = 1; m < W::NL; m *= 2) y[j] += __shfl_xor_sync(0xffffffffu, y[j], m);
      }
      if (W::NL > 1) __syncwarp();         // row t of sp has been read
      if (nl == 0) {
        if (W::CH == 4) store_row(&mem.sp[t][col], make_float2(y[0], y[1]), make_float2(y[W::CH - 2], y[W::CH - 1]));
        else *reinterpret_cast<float2*>(&mem.sp[t][col]) = make_float2(y[0], y[1]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < St::kItems; ++i) {
      const int t = at.row(i);
      float2 y[2], f[2], g[2];
      load_row(&mem.sp[t][at.quad()], y[0], y[1]);
      get4(raw.rows[0][i][threadIdx.x], f);
      get4(raw.rows[2][i][threadIdx.x], g);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        y[p] = fma2(skip[p], f[p], y[p]);
        const float2 gated = mul2(y[p], mul2(g[p], sigmoid2(g[p])));
        y[p] = P.z ? gated : y[p];
      }
      if (t < n && in_s) store_row(static_cast<T*>(P.y) + (size_t)(row0 + t) * P.D + cs, y[0], y[1]);
    }
    __syncwarp();                          // the warp's rows are done with
  }
  if (P.hT && s.last && in) store_wide<N>(P.hT + (size_t)s.seq * DN + state, h);
}

// The state in front of every chunk from those behind the chunks before it; with
// kBack the gradient of the state behind every chunk.  Four states a thread; the loads of
// up to 16 chunks together, since the time is their latency.
constexpr int kFoldThreads = 128;
template <bool kBack>
__global__ void __launch_bounds__(kFoldThreads) fold_kernel(const ScanArgs P, int N, int blocks) {
  wait_for_stream();
  const int seq = blockIdx.x / blocks, i = ((int)(blockIdx.x % blocks) * kFoldThreads + threadIdx.x) * 4;
  const size_t DN = (size_t)P.D * N;
  const bool in = i < (long long)DN;
  float4 A, h = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in) A = *reinterpret_cast<const float4*>(P.A + i);
  if (in && P.h0) h = *reinterpret_cast<const float4*>(P.h0 + seq * DN + i);
  if (!offsets_good(P) || !in) return;
  const int begin = P.packed.begin(seq), end = P.packed.begin(seq + 1);
  const int chunks = max(1, (int)(((long long)end - begin + P.L - 1) / P.L));
  const size_t number = (size_t)(begin / P.L + seq) + (kBack ? chunks - 1 : 0);
  float* at = P.carry + number * DN + i;
  const float* sums = P.sums + number * P.D + i / N;
  const long long step = kBack ? -(long long)DN : (long long)DN, sums_step = kBack ? -P.D : P.D;
  // n of up to M chunks.
  auto some = [&](auto most, int n) {
    constexpr int M = decltype(most)::value;
    float4 S[M];
    float sum[M];
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (j < n) {
        S[j] = *reinterpret_cast<const float4*>(at + j * step);
        sum[j] = sums[j * sums_step];
      }
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (j < n) {
        *reinterpret_cast<float4*>(at + j * step) = h;
        h.x = fmaf(ex2(-A.x * sum[j]), h.x, S[j].x);
        h.y = fmaf(ex2(-A.y * sum[j]), h.y, S[j].y);
        h.z = fmaf(ex2(-A.z * sum[j]), h.z, S[j].z);
        h.w = fmaf(ex2(-A.w * sum[j]), h.w, S[j].w);
      }
    at += n * step;
    sums += n * sums_step;
  };
  int left = chunks - 1;                   // behind the last chunk nothing is needed
  for (; left >= 16; left -= 16) some(std::integral_constant<int, 16>{}, 16);
  for (; left > 0; left -= 8) some(std::integral_constant<int, 8>{}, min(left, 8));
  *reinterpret_cast<float4*>(at) = h;
}

// ------------------------------------------------------------------ backward
// (Held as float2 through the loops of the backward pass pairs are taken apart and put
// together again at every turn: 76 moves per row of 32 channels.)
__device__ __forceinline__ void load_pairs(const void* p, Pair& a, Pair& b) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  a = v.x;
  b = v.y;
}
// As park16 and ask16, the latter with its wait.
__device__ __forceinline__ void park_pairs(uint32_t taddr, const Pair (&v)[8]) {
  asm volatile(
      "{\n .reg .b32 a<16>;\n"
      " mov.b64 {a0, a1}, %1;\n mov.b64 {a2, a3}, %2;\n mov.b64 {a4, a5}, %3;\n mov.b64 {a6, a7}, %4;\n"
      " mov.b64 {a8, a9}, %5;\n mov.b64 {a10, a11}, %6;\n mov.b64 {a12, a13}, %7;\n mov.b64 {a14, a15}, %8;\n"
      " tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15};\n}\n" ::"r"(taddr),
      "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]), "l"(v[4]), "l"(v[5]), "l"(v[6]), "l"(v[7])
      : "memory");
}
__device__ __forceinline__ void fetch_pairs(uint32_t taddr, Pair (&v)[8]) {
  asm volatile(
      "{\n .reg .b32 a<16>;\n"
      " tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15}, [%8];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {a0, a1};\n mov.b64 %1, {a2, a3};\n mov.b64 %2, {a4, a5};\n mov.b64 %3, {a6, a7};\n"
      " mov.b64 %4, {a8, a9};\n mov.b64 %5, {a10, a11};\n mov.b64 %6, {a12, a13};\n mov.b64 %7, {a14, a15};\n}\n"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void pairs_of(const float2 (&v)[8], Pair (&p)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = bits2(v[i]);
}
__device__ __forceinline__ void floats_of(const Pair (&p)[8], float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = float2_of(p[i]);
}

template <typename T, int N>
struct BackwardSmem {
  float2 B[kStateRows][N], C[kStateRows][N];
  float bc[Square<N>::kWarps][kStateRows][2 * N];              // a warp's channels' shares of dB and dC
  struct {                                 // u becomes du row by row, d (where gated) inner
    float sp[kStateRows][Square<N>::kCols], u[kStateRows][Square<N>::kCols], d[kStateRows][Square<N>::kCols], dl[kStateRows][Square<N>::kCols];
  } warp[Square<N>::kWarps];
  RawRows<T, N, Square<N>, 4> raw[2];                 // of these and the next R rows
  uint32_t tmem;
};

// A block takes a tile of channels and every parts-th chunk, from its last rows to
// its first, R at a time: forward from the saved state with the state in front of
// every row parked in tensor memory, then back.
template <typename T, int N>
__global__ void __launch_bounds__(Steps<Square<N>>::kThreads, kBackBlocks) backward_kernel(const ScanArgs P) {
  using Sq = Square<N>;
  using St = Steps<Sq>;
  constexpr int R = Sq::kRows;
  static_assert(R == kStateRows, "");
  extern __shared__ __align__(16) char smem[];
  BackwardSmem<T, N>& sh = *reinterpret_cast<BackwardSmem<T, N>*>(smem);
  constexpr uint32_t kTmemCols = R * 16;
  static_assert(sizeof(BackwardSmem<T, N>) <= 227 * 1024, "shared memory of a block");
  // A block that holds tensor memory must not wait for a kernel in front of it.
  wait_for_stream();
  if (!offsets_good(P)) {
    if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    return;
  }
  const Place<N, Sq> at(P, blockIdx.x % P.tiles);
  const int nl = at.lane % Sq::NL, cl = at.lane / Sq::NL;
  if (at.warp == 0) tc::tmem_alloc(&sh.tmem, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t park = sh.tmem + ((uint32_t)at.warp << 21);
  auto& mem = sh.warp[at.warp];
  const Constants K = constants();
  const int c = at.c0 + cl * 4, cs = at.c0 + at.quad();
  const bool in = c < at.c_end, in_s = cs < at.c_end;
  const size_t state = (size_t)c * N + nl * 4, DN = (size_t)P.D * N;
  float2 some[8];                          // states on their way to or from memory
  int saved[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) saved[j] = saved_at<N>(c + j, at.c0 - at.warp * Sq::kCols, at.c_end, nl);
  Pair nA[8], dA[8];
  zero8(some);
  pairs_of(some, dA);
  if (in) load_states<N>(P.A + state, some);
#pragma unroll
  for (int i = 0; i < 8; ++i) nA[i] = bits2(make_float2(-some[i].x, -some[i].y));
  float2 bias[2], skip[2], dskip[2] = {both(0.f), both(0.f)}, dbias[2] = {both(0.f), both(0.f)};
  load_four(P.bias ? P.bias + cs : nullptr, in_s, 0.f, bias);
  load_four(P.skip ? P.skip + cs : nullptr, in_s, 0.f, skip);

  const void* const from[4] = {P.x, P.dt, P.dy, P.z};
  const long long ld[4] = {P.ld, P.ld, P.D, P.ld_z};
  int turn = 0;
  const unsigned parts = gridDim.x / P.tiles, part = blockIdx.x / P.tiles;
  for (unsigned index = part; index < P.indexes; index += parts) {
    Span s;
    if (find_chunk<true>(P, (int)index, s) != kChunk) continue;
    Pair r[8];
    zero8(some);
    if (in) {
      if (P.split) load_states<N>(P.carry + s.number * DN + state, some);
      else if (P.h0) load_states<N>(P.h0 + s.seq * DN + state, some);
    }
    pairs_of(some, r);
    const int last = s.rows > 0 ? (s.rows - 1) / R * R : -1;
    if (last >= 0) sh.raw[turn].template ask<true, true>(P, at, in_s, from, ld, s.row0 + last, s.rows - last);
    for (int r0 = last; r0 >= 0; r0 -= R, turn ^= 1) {
      const int row0 = s.row0 + r0, n = min(R, s.rows - r0);
      auto& raw = sh.raw[turn];
      zero8(some);
      if (in) {
        const float* const p = P.states + ((size_t)(s.begin / R + s.seq) + (row0 - s.begin) / R) * DN;
#pragma unroll
        for (int cp = 0; cp < 2; ++cp) {
          const float4 a = *reinterpret_cast<const float4*>(p + saved[2 * cp]);
          const float4 b = *reinterpret_cast<const float4*>(p + saved[2 * cp + 1]);
          some[cp * 4 + 0] = make_float2(a.x, b.x);
          some[cp * 4 + 1] = make_float2(a.y, b.y);
          some[cp * 4 + 2] = make_float2(a.z, b.z);
          some[cp * 4 + 3] = make_float2(a.w, b.w);
        }
      }
      cp_async_wait_all();
      if (r0 > 0) sh.raw[turn ^ 1].template ask<true, true>(P, at, in_s, from, ld, row0 - R, R);
      __syncthreads();                     // the rows behind are done with
      raw.template spread<true, true>(n, sh.B, sh.C);
#pragma unroll
      for (int i = 0; i < St::kItems; ++i) {
        const int t = at.row(i), q = at.quad();
        const bool valid = t < n && in_s;
        float2 sp[2], u[2], d[2], f[2], v[2];
        get4_if(valid, raw.rows[0][i][threadIdx.x], f);
        get4_if(valid, raw.rows[1][i][threadIdx.x], v);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float2 unused, e;
          softplus_pair(K, v[p], bias[p], unused, e, sp[p]);
          sp[p] = valid ? sp[p] : both(0.f);
          u[p] = mul2(mul2(sp[p], both(kLn2)), f[p]);
        }
        dinner_of(valid, raw.rows[2][i][threadIdx.x], raw.rows[3][i][threadIdx.x], P.z != nullptr, d);
        store_row(&mem.sp[t][q], sp[0], sp[1]);
        store_row(&mem.u[t][q], u[0], u[1]);
        store_row(&mem.d[t][q], d[0], d[1]);
      }
      __syncthreads();
      Pair h[8], other[8];
      pairs_of(some, h);
#pragma unroll 8
      for (int t = 0; t < R; ++t) {
        Pair sp[2], u[2], B[4];
        park_pairs(park + t * 16, h);
        load_pairs(&mem.sp[t][cl * 4], sp[0], sp[1]);
        load_pairs(&mem.u[t][cl * 4], u[0], u[1]);
        load_pairs(&sh.B[t][nl * 4], B[0], B[1]);
        load_pairs(&sh.B[t][nl * 4 + 2], B[2], B[3]);
#pragma unroll
        for (int cp = 0; cp < 2; ++cp)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = cp * 4 + k;
            h[i] = fma2(ex2_pair(mul2(nA[i], sp[cp])), h[i], mul2(u[cp], B[k]));
          }
      }
      parked();
      // A row's sums: over a thread's states of four channels (du, what delta gets by the
      // decay, inner), and over its channels of four states (dB, dC).
      struct Sums {
        float du[4], dl[4], y[4], bc[8];
      };
      // Row t: h is the state behind it, and the state in front of it comes to `before`.
      // (A row that does not exist changes r by nothing, but a state or gradient that is not
      // finite times its delta of 0 must not go into dA.)
      auto back = [&](int t, Pair (&before)[8], const Pair (&h)[8], Sums& out, bool exists = true) {
        Pair sp[2], u[2], d[2], B[4], C[4], du[2], dl[2], y[2], dB[4], dC[4];
        load_pairs(&mem.sp[t][cl * 4], sp[0], sp[1]);
        load_pairs(&mem.u[t][cl * 4], u[0], u[1]);
        load_pairs(&mem.d[t][cl * 4], d[0], d[1]);
        load_pairs(&sh.B[t][nl * 4], B[0], B[1]);
        load_pairs(&sh.B[t][nl * 4 + 2], B[2], B[3]);
        load_pairs(&sh.C[t][nl * 4], C[0], C[1]);
        load_pairs(&sh.C[t][nl * 4 + 2], C[2], C[3]);
        fetch_pairs(park + t * 16, before);
#pragma unroll
        for (int cp = 0; cp < 2; ++cp)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = cp * 4 + k;
            const Pair g = fma2(d[cp], C[k], r[i]);
            r[i] = mul2(g, ex2_pair(mul2(nA[i], sp[cp])));
            const Pair p = mul2(r[i], before[i]);
            if (exists) dA[i] = fma2(p, sp[cp], dA[i]);
            du[cp] = k ? fma2(g, B[k], du[cp]) : mul2(g, B[k]);
            dl[cp] = k ? fma2(p, nA[i], dl[cp]) : mul2(p, nA[i]);
            y[cp] = k ? fma2(C[k], h[i], y[cp]) : mul2(C[k], h[i]);
            dB[k] = cp ? fma2(g, u[cp], dB[k]) : mul2(g, u[cp]);
            dC[k] = cp ? fma2(d[cp], h[i], dC[k]) : mul2(d[cp], h[i]);
          }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 b = float2_of(dB[k]), c = float2_of(dC[k]);
          out.bc[k] = b.x + b.y;
          out.bc[4 + k] = c.x + c.y;
          const float2 e = float2_of(du[k / 2]), f = float2_of(dl[k / 2]), g = float2_of(y[k / 2]);
          out.du[k] = k % 2 ? e.y : e.x;
          out.dl[k] = k % 2 ? f.y : f.x;
          out.y[k] = k % 2 ? g.y : g.x;
        }
      };
      // The sums over the lanes, one row later: between their steps there is the next row's
      // arithmetic.
      auto finish = [&](int t, Sums& v) {
        using Sum = Halving<4, Sq::kNBits, 0>;
        using Over = Halving<8, Sq::kCBits, Sq::kNBits>;
        Over::sum(v.bc, at.lane);
        Sum::sum(v.du, at.lane);
        Sum::sum(v.dl, at.lane);
        Sum::sum(v.y, at.lane);
        if (Sum::chosen(at.lane)) {        // (all lanes have read row t of u and d)
          const int to = cl * 4 + Sum::index(at.lane);
#pragma unroll
          for (int j = 0; j < Sum::kLeft; ++j) {
            mem.u[t][to + j] = v.du[j];
            mem.dl[t][to + j] = v.dl[j];
            if (P.z) mem.d[t][to + j] = v.y[j];
          }
        }
        if (Over::chosen(at.lane)) {
#pragma unroll
          for (int j = 0; j < Over::kLeft; ++j) {
            const int to = Over::index(at.lane) + j;
            sh.bc[at.warp][t][(to >> 2) * N + nl * 4 + (to & 3)] = v.bc[j];
          }
        }
      };
      const int top = (n - 1) | 1;         // rows in pairs: the last one, or the one behind it
      Sums even, odd;
      back(top, other, h, odd, top < n);
#pragma unroll 1
      for (int t = top - 1; t > 0; t -= 2) {
        __syncwarp();                      // row t + 1 has been read
        back(t, h, other, even);
        finish(t + 1, odd);
        __syncwarp();
        back(t - 1, other, h, odd);
        finish(t, even);
      }
      back(0, h, other, even);
      __syncwarp();
      finish(1, odd);
      finish(0, even);
      __syncthreads();
      for (int i = threadIdx.x; i < n * 2 * N; i += St::kThreads) {
        const int t = i / (2 * N), k = i % (2 * N);
        float v = sh.bc[0][t][k];
#pragma unroll
        for (int w = 1; w < Sq::kWarps; ++w) v += sh.bc[w][t][k];
        P.partial_bc[((size_t)(row0 + t) * P.tiles + blockIdx.x % P.tiles) * (2 * N) + k] = v;
      }
#pragma unroll
      for (int i = 0; i < St::kItems; ++i) {
        const int t = at.row(i), q = at.quad();
        const bool valid = t < n && in_s;
        const size_t row = row0 + t;
        float2 x[2], dt[2], d[2], sp[2], du[2], dl[2], dx[2], ddt[2], dz[2];
        get4_if(valid, raw.rows[0][i][threadIdx.x], x);
        get4_if(valid, raw.rows[1][i][threadIdx.x], dt);
        load_row(&mem.sp[t][q], sp[0], sp[1]);
        load_row(&mem.u[t][q], du[0], du[1]);
        load_row(&mem.dl[t][q], dl[0], dl[1]);
        load_row(&mem.d[t][q], d[0], d[1]);
        if (P.z) {
          float2 z[2], dy[2];
          get4_if(valid, raw.rows[2][i][threadIdx.x], dy);
          get4_if(valid, raw.rows[3][i][threadIdx.x], z);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 sig = sigmoid2(z[p]), inner = fma2(skip[p], x[p], d[p]);
            d[p] = mul2(dy[p], mul2(z[p], sig));
            // silu' = sig (1 + z (1 - sig)).
            dz[p] = mul2(mul2(dy[p], inner), mul2(sig, fma2(z[p], sub2(both(1.f), sig), both(1.f))));
          }
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          dx[p] = fma2(du[p], mul2(sp[p], both(kLn2)), mul2(d[p], skip[p]));
          ddt[p] = mul2(fma2(du[p], x[p], dl[p]), sigmoid2(add2(dt[p], bias[p])));
          dskip[p] = fma2(d[p], x[p], dskip[p]);
          dbias[p] = valid ? add2(dbias[p], ddt[p]) : dbias[p];
        }
        if (valid) {
          store_row(static_cast<T*>(P.dx) + row * P.ld_grad + cs, dx[0], dx[1]);
          store_row(static_cast<T*>(P.ddt) + row * P.ld_grad + cs, ddt[0], ddt[1]);
          if (P.z) store_row(static_cast<T*>(P.dz) + row * P.ld_z_grad + cs, dz[0], dz[1]);
        }
      }
    }
    floats_of(r, some);
    if (P.hT && s.first && in) store_states<N>(P.hT + s.seq * DN + state, some);
  }
  // The chunks' sums.  dA = -sum delta p, and sp is delta log2(e).
  float* const to = P.partial + (size_t)part * P.D * (N + 2);
  floats_of(dA, some);
#pragma unroll
  for (int i = 0; i < 8; ++i) some[i] = mul2(some[i], both(-kLn2));
  if (in) store_states<N>(to + state, some);
  float v[8] = {dskip[0].x, dskip[0].y, dskip[1].x, dskip[1].y, dbias[0].x, dbias[0].y, dbias[1].x, dbias[1].y};
#pragma unroll
  for (int o = Sq::CL; o < 32; o *= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (at.lane < Sq::CL && in_s) {
    store_row(to + DN + cs, make_float2(v[0], v[1]), make_float2(v[2], v[3]));
    store_row(to + DN + P.D + cs, make_float2(v[4], v[5]), make_float2(v[6], v[7]));
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (at.warp == 0) tc::tmem_dealloc(sh.tmem, kTmemCols);
}

// dB and dC of every row of a sequence: the tiles' shares of a group, in their order.
template <typename T>
__global__ void __launch_bounds__(256)
    bc_sums_kernel(const ScanArgs P, int N, T* dB, T* dC, long long ld) {
  wait_for_stream();
  if (!offsets_good(P)) return;
  const int width = P.G * 2 * N;
  const long long first = P.packed.begin(0), n = (long long)(P.packed.begin(P.packed.n_seq) - first) * width;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long row = first + i / width;
    const int k = (int)(i % width), g = k / (2 * N), j = k % (2 * N);
    const float* at = P.partial_bc + ((size_t)row * P.tiles + (size_t)g * P.group_tiles) * (2 * N) + j;
    float v = 0.f;
    for (int t = 0; t < P.group_tiles; ++t) v += __ldg(at + (size_t)t * (2 * N));
    T* const to = j < N ? dB : dC;
    to[(size_t)row * ld + (size_t)g * N + j % N] = (T)v;
  }
}

// Sums of [parts][D (N + 2)] over the parts, always in the same order: 32 columns a
// block, each of 32 warps every 32nd part, then the warps.
__global__ void __launch_bounds__(1024)
    scan_sums_kernel(const ScanArgs P, int parts, int N, float* dA, float* dskip, float* dbias) {
  wait_for_stream();
  if (!offsets_good(P)) return;
  const float* const partial = P.partial;
  const long long D = P.D;
  __shared__ float warps[32][33];
  const long long width = D * (N + 2), i = (long long)blockIdx.x * 32 + (threadIdx.x & 31);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float a = 0.f;
  if (i < width) {
#pragma unroll 4
    for (int n = warp; n < parts; n += 32) a += __ldg(partial + n * width + i);
  }
  warps[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || i >= width) return;
  float sum = 0.f;
  for (int w = 0; w < 32; ++w) sum += warps[w][lane];
  if (i < D * N) {
    if (dA) dA[i] = sum;
  } else if (i < D * (N + 1)) {
    if (dskip) dskip[i - D * N] = sum;
  } else if (dbias) {
    dbias[i - D * (N + 1)] = sum;
  }
}

// ----------------------------------------------------------------- one token
// A block takes kGroup tokens by a tile of channels, with the lanes of the backward pass.
template <typename T, int N, int kGroup>
__global__ void __launch_bounds__(Steps<Square<N>>::kThreads) step_kernel(const ScanArgs P, float* pool, int n_slots,
                                                        const int32_t* slots) {
  using Sq = Square<N>;
  wait_for_stream();
  __shared__ SlotTable<kGroup, Steps<Sq>::kThreads> table;
  const int row0 = (int)(blockIdx.x / P.tiles) * kGroup, rows = min(kGroup, P.packed.rows - row0);
  const Place<N, Sq> at(P, blockIdx.x % P.tiles);
  const int nl = at.lane % Sq::NL;
  table.find(slots, row0, rows, n_slots, P.status);
  const Constants K = constants();
  const int c = at.c0 + at.lane / Sq::NL * 4;
  const unsigned lanes = __ballot_sync(0xffffffffu, c < at.c_end);   // whole groups of NL lanes
  if (c >= at.c_end) return;
  const size_t state = (size_t)c * N + nl * 4;
  float2 nA[8], bias[2], skip[2];
  load_states<N>(P.A + state, nA);
#pragma unroll
  for (int i = 0; i < 8; ++i) nA[i] = make_float2(-nA[i].x, -nA[i].y);
  load_four(P.bias ? P.bias + c : nullptr, true, 0.f, bias);
  load_four(P.skip ? P.skip + c : nullptr, true, 0.f, skip);
  constexpr int kAhead = kGroup == 1 ? 1 : 2;                // tokens at a time
  for (int j0 = 0; j0 < rows; j0 += kAhead) {
    float2 h[kAhead][8];
    float* at_pool[kAhead];
    Raw4<T> raw_x[kAhead], raw_dt[kAhead], raw_z[kAhead], raw_B[kAhead], raw_C[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int slot = j0 + j < rows ? table.own[j0 + j] : -1;
      at_pool[j] = slot < 0 ? nullptr : pool + (size_t)slot * P.D * N + state;
      if (slot < 0) continue;
      const size_t row = row0 + j0 + j;
      load_states<N>(at_pool[j], h[j]);
      raw_x[j] = raw4<T>(P.x, row * P.ld + c);
      raw_dt[j] = raw4<T>(P.dt, row * P.ld + c);
      raw_B[j] = raw4<T>(P.B, row * P.ld_bc + (size_t)at.group * N + nl * 4);
      raw_C[j] = raw4<T>(P.C, row * P.ld_bc + (size_t)at.group * N + nl * 4);
      if (P.z) raw_z[j] = raw4<T>(P.z, row * P.ld_z + c);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!at_pool[j]) continue;           // (the whole block has the same tokens)
      float2 x[2], dt[2], z[2], B[2], C[2], y[2];
      get4(raw_x[j], x);
      get4(raw_dt[j], dt);
      get4(raw_B[j], B);
      get4(raw_C[j], C);
      if (P.z) get4(raw_z[j], z);
      const float b[4] = {B[0].x, B[0].y, B[1].x, B[1].y}, o[4] = {C[0].x, C[0].y, C[1].x, C[1].y};
#pragma unroll
      for (int cp = 0; cp < 2; ++cp) {
        float2 unused, e, sp;
        softplus_pair(K, dt[cp], bias[cp], unused, e, sp);
        const float2 u = mul2(mul2(sp, both(kLn2)), x[cp]);
        y[cp] = both(0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = cp * 4 + k;
          h[j][i] = fma2(ex2_pair(mul2(nA[i], sp)), h[j][i], mul2(u, both(b[k])));
          y[cp] = fma2(both(o[k]), h[j][i], y[cp]);
        }
      }
      store_states<N>(at_pool[j], h[j]);
      float v[4] = {y[0].x, y[0].y, y[1].x, y[1].y};
#pragma unroll
      for (int m = 1; m < Sq::NL; m *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(lanes, v[i], m);
      if (nl == 0) {
        y[0] = make_float2(v[0], v[1]);
        y[1] = make_float2(v[2], v[3]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          y[q] = fma2(skip[q], x[q], y[q]);
          if (P.z) y[q] = mul2(y[q], mul2(z[q], sigmoid2(z[q])));
        }
        store_row(static_cast<T*>(P.y) + (size_t)(row0 + j0 + j) * P.D + c, y[0], y[1]);
      }
    }
  }
}

// ---------------------------------------------------------------- host side
size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

int tile_cols(int N) { return kBlockStates / N; }
int group_tiles_of(const SelectiveDims& d) {
  return (d.D / d.groups + tile_cols(d.N) - 1) / tile_cols(d.N);
}

// How the sequences are cut: rows of a chunk, a multiple of kStateRows, and whether any
// sequence has more than one.  A chunk more costs its block's start and end and a step of
// the fold, a chunk less leaves multiprocessors idle at the end: there are as many as make
// kFillEqual (where lengths are on the device kFillPacked) blocks a multiprocessor.
// Measured with 6, 12, 24, 36: scan of 131072 x 1024 x 16 in one sequence 1025, 1022, 1041
// and 1098 us, training of 32768 x 1024 in eight 1039, 1035, 1026 and 1020; packed, with 8,
// 16, 32, 48: training of 5003 x 960 x 32 338, 328, 335 and 355.  Chunks go down to 16 rows:
// 600 rows of 16 sequences take 28 us with them, 39 with 64 rows, 50 without any cut.
struct Cut {
  int L;
  bool split;
};
constexpr int kFillEqual = 12, kFillPacked = 16;
// (In the backward pass a block takes several chunks, which more of them spread evenly.)
constexpr int kFillEqualBack = 36;
constexpr int kLeastChunk = 16, kMostChunk = 1 << 20;
Cut cut_of(const SelectiveDims& d, bool equal, bool back) {
  const long long tiles = (long long)group_tiles_of(d) * d.groups;
  const long long slots = (long long)(!equal ? kFillPacked : back ? kFillEqualBack : kFillEqual) * device_limits().sms / tiles;
  const int longest = equal && d.n_seq > 0 ? d.rows / d.n_seq : d.rows;
  long long chunks = equal && d.n_seq > 0 ? slots / d.n_seq : slots;   // of `longest` rows
  if (chunks < 1) chunks = 1;
  long long L = (longest + chunks - 1) / chunks;
  L = (L + kStateRows - 1) / kStateRows * kStateRows;
  if (L > kMostChunk) L = kMostChunk;
  if (L < kLeastChunk) L = kLeastChunk;
  return Cut{(int)L, longest > L};
}
constexpr size_t kHeaderBytes = 256;       // of the workspace, in front of the carry
size_t numbers_of(const SelectiveDims& d, int L) { return (size_t)chunk_numbers(d.rows, d.n_seq, L); }
size_t carry_bytes(const SelectiveDims& d, const Cut& cut) {
  if (!cut.split) return 0;
  return round256(numbers_of(d, cut.L) * d.D * d.N * 4) + round256(numbers_of(d, cut.L) * d.D * 4);
}
// Parts of the sums over rows: at most what fills the GPU.
size_t most_parts(const SelectiveDims& d) {
  const size_t tiles = (size_t)group_tiles_of(d) * d.groups, fill = kBackBlocks * (size_t)device_limits().sms;
  return fill > tiles ? fill / tiles : 1;
}

ScanArgs args_of(const SelectiveDims& d, const SelectiveInputs& in, const Cut& cut, void* workspace,
                 unsigned* status) {
  ScanArgs P{};
  P.packed = Packed{in.offsets, d.n_seq, d.rows};
  P.x = in.x;
  P.dt = in.dt;
  P.z = in.z;
  P.B = in.B;
  P.C = in.C;
  P.A = in.A;
  P.skip = in.skip;
  P.bias = in.bias;
  P.ld = d.ld;
  P.ld_z = d.ld_z;
  P.ld_bc = d.ld_bc;
  P.D = d.D;
  P.G = d.groups;
  P.per = d.D / d.groups;
  P.group_tiles = group_tiles_of(d);
  P.tiles = P.group_tiles * d.groups;
  P.L = cut.L;
  P.split = cut.split;
  P.chunks = 1;
  if (in.offsets || d.n_seq == 0) {
    P.indexes = (unsigned)numbers_of(d, cut.L);
  } else {
    const int len = d.rows / d.n_seq;
    P.chunks = len > cut.L ? (int)(((long long)len + cut.L - 1) / cut.L) : 1;
    P.indexes = (unsigned)P.chunks * d.n_seq;
  }
  P.bad_offsets = static_cast<int*>(workspace);
  if (cut.split) {
    char* w = static_cast<char*>(workspace) + kHeaderBytes;
    P.carry = reinterpret_cast<float*>(w);
    P.sums = reinterpret_cast<float*>(w + round256(numbers_of(d, cut.L) * d.D * d.N * 4));
  }
  P.status = status;
  return P;
}

// Dynamic shared memory of a kernel, allowed once per device.
template <class K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t f = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (f == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return f;
}
template <class K>
cudaError_t launch_with(K kernel, std::atomic<bool>* allowed, unsigned blocks, int threads, size_t smem,
                        cudaStream_t stream, const ScanArgs& P) {
  const cudaError_t e = allow_smem(kernel, (int)smem, allowed);
  return e != cudaSuccess ? e : launch_behind(kernel, blocks, threads, smem, stream, P);
}

template <class F>
cudaError_t with_kind(const SelectiveDims& d, F f) {
  using std::integral_constant;
  auto states = [&](auto t) {
    if (d.N == 8) return f(t, integral_constant<int, 8>{});
    if (d.N == 16) return f(t, integral_constant<int, 16>{});
    if (d.N == 32) return f(t, integral_constant<int, 32>{});
    return f(t, integral_constant<int, 64>{});
  };
  return d.dtype == SDM_BF16 ? states(__nv_bfloat16{}) : states(float{});
}

cudaError_t check_offsets(const ScanArgs& P, cudaStream_t stream) {
  if (!P.packed.offsets || P.packed.n_seq < kManySequences) return cudaSuccess;
  return launch_behind(check_offsets_kernel, 1, 1024, 0, stream, P.packed, P.bad_offsets);
}

template <bool kBack>
cudaError_t launch_fold(const SelectiveDims& d, const ScanArgs& P, cudaStream_t stream) {
  const int blocks = (int)(((long long)d.D * d.N / 4 + kFoldThreads - 1) / kFoldThreads);
  return launch_behind(fold_kernel<kBack>, (unsigned)blocks * d.n_seq, kFoldThreads, 0, stream, P, d.N, blocks);
}

}  // namespace

int selective_scan_tiles(const SelectiveDims& d) { return group_tiles_of(d) * d.groups; }

namespace {
// Whatever the sequences' lengths may be given as.
size_t most_carry_bytes(const SelectiveDims& d, bool back) {
  const size_t a = carry_bytes(d, cut_of(d, false, back));
  const size_t b = d.n_seq > 0 && d.rows % d.n_seq == 0 ? carry_bytes(d, cut_of(d, true, back)) : 0;
  return a > b ? a : b;
}
}  // namespace

size_t selective_scan_workspace_bytes(const SelectiveDims& d) { return kHeaderBytes + most_carry_bytes(d, false); }
size_t selective_scan_backward_workspace_bytes(const SelectiveDims& d) {
  const size_t tiles = (size_t)group_tiles_of(d) * d.groups;
  return kHeaderBytes + most_carry_bytes(d, true) + round256(most_parts(d) * d.D * (d.N + 2) * 4) +
         (size_t)d.rows * tiles * 2 * d.N * 4;
}

size_t selective_scan_states_bytes(const SelectiveDims& d) {
  return numbers_of(d, kStateRows) * d.D * d.N * sizeof(float);
}

cudaError_t launch_selective_scan_forward(const SelectiveDims& d, const SelectiveInputs& in,
                                          const float* h0, void* y, float* hT, float* states,
                                          void* workspace, unsigned* status, cudaStream_t stream) {
  const Cut cut = cut_of(d, !in.offsets, false);
  ScanArgs P = args_of(d, in, cut, workspace, status);
  P.h0 = h0;
  P.hT = hT;
  P.y = y;
  P.states = states;
  return with_kind(d, [&](auto t, auto n) {
    using T = decltype(t);
    constexpr int N = decltype(n)::value;
    static std::atomic<bool> allowed[2][64];
    const unsigned blocks = P.indexes * P.tiles;
    cudaError_t e = check_offsets(P, stream);
    if (e == cudaSuccess && cut.split) {
      e = launch_with(summary_kernel<T, N, false>, allowed[0], blocks, Steps<Wide<N>>::kThreads, sizeof(SummarySmem<T, N>), stream, P);
      if (e == cudaSuccess) e = launch_fold<false>(d, P, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_with(forward_kernel<T, N>, allowed[1], blocks, Steps<Wide<N>>::kThreads, sizeof(ForwardSmem<T, N>), stream, P);
  });
}

cudaError_t launch_selective_scan_backward(const SelectiveDims& d, const SelectiveInputs& in,
                                           const float* states, const void* dy, const float* dhT,
                                           const SelectiveGrads& out, void* workspace,
                                           unsigned* status, cudaStream_t stream) {
  if (d.n_seq == 0) {                      // sums over nothing
    cudaError_t e = cudaSuccess;
    if (out.dA) e = cudaMemsetAsync(out.dA, 0, (size_t)d.D * d.N * 4, stream);
    if (e == cudaSuccess && out.dskip) e = cudaMemsetAsync(out.dskip, 0, (size_t)d.D * 4, stream);
    if (e == cudaSuccess && out.dbias) e = cudaMemsetAsync(out.dbias, 0, (size_t)d.D * 4, stream);
    return e;
  }
  const Cut cut = cut_of(d, !in.offsets, true);
  ScanArgs P = args_of(d, in, cut, workspace, status);
  char* w = static_cast<char*>(workspace) + kHeaderBytes + carry_bytes(d, cut);
  P.partial = reinterpret_cast<float*>(w);
  P.partial_bc = reinterpret_cast<float*>(w + round256(most_parts(d) * d.D * (d.N + 2) * 4));
  P.h0 = dhT;
  P.hT = out.dh0;
  P.states = const_cast<float*>(states);
  P.dy = dy;
  P.dx = out.dx;
  P.ddt = out.ddt;
  P.dz = out.dz;
  P.ld_grad = d.ld_grad;
  P.ld_z_grad = d.ld_z_grad;
  const unsigned parts = (unsigned)(P.indexes < most_parts(d) ? P.indexes : most_parts(d));
  cudaError_t e = with_kind(d, [&](auto t, auto n) {
    using T = decltype(t);
    constexpr int N = decltype(n)::value;
    static std::atomic<bool> allowed[2][64];
    cudaError_t e = check_offsets(P, stream);
    if (e == cudaSuccess && cut.split) {
      e = launch_with(summary_kernel<T, N, true>, allowed[0], P.indexes * P.tiles, Steps<Wide<N>>::kThreads, sizeof(SummarySmem<T, N>), stream, P);
      if (e == cudaSuccess) e = launch_fold<true>(d, P, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_with(backward_kernel<T, N>, allowed[1], parts * P.tiles, Steps<Square<N>>::kThreads, sizeof(BackwardSmem<T, N>), stream, P);
  });
  if (e == cudaSuccess && d.rows > 0) {
    const long long want = ((long long)d.rows * d.groups * 2 * d.N + 255) / 256, most = 16ll * device_limits().sms;
    const unsigned blocks = (unsigned)(want < most ? want : most);
    e = d.dtype == SDM_BF16
            ? launch_behind(bc_sums_kernel<__nv_bfloat16>, blocks, 256, 0, stream, P, d.N,
                            static_cast<__nv_bfloat16*>(out.dB), static_cast<__nv_bfloat16*>(out.dC), d.ld_bc_grad)
            : launch_behind(bc_sums_kernel<float>, blocks, 256, 0, stream, P, d.N,
                            static_cast<float*>(out.dB), static_cast<float*>(out.dC), d.ld_bc_grad);
  }
  if (e != cudaSuccess || (!out.dA && !out.dskip && !out.dbias)) return e;
  const unsigned blocks = (unsigned)(((long long)d.D * (d.N + 2) + 31) / 32);
  return launch_behind(scan_sums_kernel, blocks, 1024, 0, stream, P, (int)parts, d.N, out.dA, out.dskip,
                       out.dbias);
}

cudaError_t launch_selective_scan_step(const SelectiveDims& d, const SelectiveInputs& in,
                                       float* state, int n_slots, const int32_t* slots, void* y,
                                       unsigned* status, cudaStream_t stream) {
  ScanArgs P = args_of(d, in, Cut{kStateRows, false}, nullptr, status);
  P.y = y;
  return with_kind(d, [&](auto t, auto n) {
    using T = decltype(t);
    constexpr int N = decltype(n)::value;
    return with_group(d.rows, (long long)d.rows * P.tiles, 16384, [&](auto group) {
      constexpr int G = decltype(group)::value;
      return launch_behind(step_kernel<T, N, G>, (unsigned)(((long long)d.rows + G - 1) / G * P.tiles),
                           Steps<Square<N>>::kThreads, 0, stream, P, state, n_slots, slots);
    });
  });
}

}  // namespace sdm
