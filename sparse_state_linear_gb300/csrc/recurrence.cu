// recurrence.cu -- gated delta recurrence over packed sequences: forward,
// backward and single-token step.
//
// [SDM notes] "Sparse Delta Memory：中文精读笔记", 2.4: the gates
//   alpha = exp(-A softplus(z + b)),  beta = sigmoid(z)
// and Eq. (3)-(4) with one slot of weight 1 per channel:
//   h[t] = (1 - beta) alpha h[t-1] + beta v.
// With a = (1 - beta) alpha the backward pass is, from the last row to the
// first, g = dy + r, r = a g (r starts as the gradient of the final state):
//   dv = beta g,  dzb = g (v - alpha h[t-1]) beta (1 - beta),
//   dl = g a h[t-1] (gradient of ln alpha),
//   dza = -A sigmoid(za + b) dl,  dA = sum -softplus(za + b) dl,  db = sum dza.
#include <cuda.h>   // CUtensorMap and its enums; the encoder comes through the runtime

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "packed.cuh"
#include "tcgen05.cuh"

namespace sdm {
namespace {

// ------------------------------------------------------------------- gates
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
// One row of one channel: the state behind it.
__device__ __forceinline__ float step_one(float h, float za, float zb, float v, float A,
                                          float bias) {
  const float x = za + bias, e = ex2(-fabsf(x) * kLog2e);
  const float sp = fmaxf(x, 0.f) * kLog2e + log2p1_unit(e);
  const float z = zb * kLog2e, beta = rcp(1.f + ex2(-z));                    // see decay_pair
  const float a = fmaxf(beta, 1.f - beta) * ex2(-fmaf(A, sp, fmaxf(z, 0.f)));
  return fmaf(a, h, beta * v);
}

__device__ __forceinline__ float4 load4(const void* base, size_t i, int dt) {
  if (dt == SDM_F32) return __ldg(reinterpret_cast<const float4*>(base) + i);
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(base) + i);
  return make_float4(bf16_bits_to_float(w.x & 0xffffu), __uint_as_float(w.x & 0xffff0000u),
                     bf16_bits_to_float(w.y & 0xffffu), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(void* base, size_t i, int dt, float4 v) {
  if (dt == SDM_F32) {
    reinterpret_cast<float4*>(base)[i] = v;
    return;
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.z, v.w);
  reinterpret_cast<uint2*>(base)[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                 *reinterpret_cast<const uint32_t*>(&b));
}

// ------------------------------------------------------------- pairs of floats
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

// beta = sigmoid(zb) = 1 / (1 + 2^-z) with z = zb log2(e) (2^-z may be infinite:
// beta is 0), and a = (1 - beta) alpha.  1 - beta is r 2^-max(z, 0) with
// r = 1 / (1 + 2^-|z|) = max(beta, 1 - beta), so that a is r 2^-(max(z, 0) + A softplus).
// Where the gate is closed (z < 0) the exponent is A softplus alone: a z in the sum
// would round off the slow decay of a state that is held for long (at zb = -80 and
// 65536 rows the state was 19% off, now 0.5%, as with every step apart in float32).
__device__ __forceinline__ void sigmoid_pair(const Constants& K, float2 zb, float2& z, float2& eb,
                                             float2& beta) {
  z = mul2(zb, K.log2e);
  eb = make_float2(ex2(-z.x), ex2(-z.y));
  const float2 d = add2(eb, K.one);
  beta = make_float2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ float2 decay_pair(const Constants& K, float2 A, float2 sp, float2 z,
                                             float2 beta, float2& r) {
  const float2 closed = sub2(K.one, beta);
  r = make_float2(fmaxf(beta.x, closed.x), fmaxf(beta.y, closed.y));
  const float2 l = fma2(A, sp, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
  return mul2(r, make_float2(ex2(-l.x), ex2(-l.y)));
}

// a and b = beta v of two channels.
__device__ __forceinline__ void gate_pair(const Constants& K, float2 za, float2 zb, float2 v,
                                          float2 A, float2 bias, float2& a, float2& b) {
  float2 x, e, sp, z, eb, beta, r;
  softplus_pair(K, za, bias, x, e, sp);
  sigmoid_pair(K, zb, z, eb, beta);
  a = decay_pair(K, A, sp, z, beta, r);
  b = mul2(beta, v);
}

// ------------------------------------------------------------------ packing
// A tile is L rows of one sequence by 64 channels.  Chunk c (of L rows) of
// sequence s whose first row is o has number o / L + s + c: distinct for all
// chunks of all sequences, below rows / L + n_seq, and growing with s and c.
constexpr int kCols = 64;

__host__ __device__ inline long long chunk_numbers(int rows, int n_seq, int L) {
  return (long long)rows / L + n_seq;
}

struct Packed {
  const int32_t* offsets;
  int n_seq, rows;
  __device__ int begin(int s) const {
    return offsets ? __ldg(offsets + s) : (int)((long long)rows / n_seq * s);
  }
};

// Whether the offsets stay within [0, rows] and never decrease (all threads
// of the block call it).
__device__ bool offsets_ok(const Packed& P) {
  if (!P.offsets) return true;
  bool bad = false;
  for (int s = threadIdx.x; s <= P.n_seq; s += blockDim.x) {
    const int o = P.begin(s);
    bad |= o < 0 || o > P.rows || (s > 0 && o < P.begin(s - 1));
  }
  return !__syncthreads_or(bad);
}

// Rows between saved states = rows of a backward tile.
template <typename T>
constexpr int kStateRows = 128 / (int)sizeof(T);

// --------------------------------------------------------------------- scan
// A (or ones) and bias (or zeros) of a tile's channels, brought to shared memory
// by the warp that fetches it, two channels a lane.
struct Rates {
  float2 A, bias;
};
__device__ __forceinline__ Rates rates_of(const float* A, const float* bias, int c, int D) {
  Rates r{both(1.f), both(0.f)};
  if (A && c < D) r.A = __ldg(reinterpret_cast<const float2*>(A + c));
  if (bias && c < D) r.bias = __ldg(reinterpret_cast<const float2*>(bias + c));
  return r;
}

// What a block has to know of a tile, found out by the warp that fetches it.
struct __align__(16) Tile {
  int rows;      // valid rows, 1..L; 0: no tile is left
  int row0;      // first row
  int seq, chunk;
  int number;    // of the chunk, indexes what chunks publish
  int back;      // number - back is the chunk before along the chain
  int col0;      // first channel
  int pos;       // along the chain: chunks before it (after it, in the backward pass)
  int last;      // the chain's last chunk
};

// Workspace of one call, cleared to all ones by clear_kernel: a header (ticket
// counter, from 2^32 - 1 on; abort word, 0 once a block has given up) and a pair
// (P, S) of floats per chunk and channel.
struct Chain {
  unsigned* ticket;
  unsigned* abort;
  float* pairs;       // [numbers][D][2]
};

// What a block's warps share about giving up, in shared memory: whether one has,
// and the limit of the waits for other blocks in us.  (Waits within the block have
// a fixed one: with a limit to look up, every one of them, the forward pass takes
// 2% longer and the float32 backward pass 4%.)
struct GiveUp {
  int done;
  unsigned limit_us;
};

__device__ __forceinline__ unsigned next_ticket(const Chain& c) {
  return atomicAdd(c.ticket, 1u) + 1u;
}

// Chunks per group, see fold_before.  Measured, forward at 131072 x 2048 bf16 and
// backward at 10007 x 1000 float32: 409 and 98 us with 6, 412 and 93 with 8, 431
// and 115 with 12, 440 and 109 with 16 (a fold waits for and reads more).
constexpr int kGroup = 8;
constexpr unsigned long long kWaitNs = 4000000000ull;         // limit of waits within a block

__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Pairs are published word by word: a word of all ones (a NaN that no result
// keeps, see publish) is one that is not there yet, any other is its value.
// So there is no flag, no fence, and no order that the words have to keep.
constexpr unsigned kUnset = 0xffffffffu;
__device__ __forceinline__ uint4 load_pairs(const float* p) {
  uint4 v;
  asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ unsigned largest(uint4 v) { return max(max(v.x, v.y), max(v.z, v.w)); }
__device__ __forceinline__ unsigned word(float x) { return x != x ? 0x7fffffffu : __float_as_uint(x); }
// The pairs of two channels.
__device__ __forceinline__ void publish(float* p, float2 P, float2 S) {
  asm volatile("st.relaxed.gpu.global.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"l"(p), "r"(word(P.x)),
               "r"(word(S.x)), "r"(word(P.y)), "r"(word(S.y))
               : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// Test of an mbarrier phase that may let the thread sleep for a while until it
// completes (a warp that spins takes issue slots from the arithmetic).
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for an mbarrier phase (a whole warp calls it); false once the limit has
// passed or another warp of the block has given up (which the first to do so
// marks).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, unsigned parity, volatile GiveUp* give_up) {
  for (uint64_t t0 = 0; !__all_sync(0xffffffffu, mbar_sleep_wait(bar, parity));) {
    const uint64_t now = global_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(0xffffffffu, give_up->done || now - t0 > kWaitNs)) {
      give_up->done = 1;
      return false;
    }
  }
  return true;
}
// Arrive from one lane, without a branch.
__device__ __forceinline__ void mbar_arrive_if(bool p, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n"
      " @p mbarrier.arrive.shared::cta.b64 _, [%1];\n}\n" ::"r"((uint32_t)p),
      "r"(smem_u32(bar))
      : "memory");
}
// x: first channel (a multiple of 64, so 16-byte aligned), y: first row; what
// lies outside the tensor arrives as zeros.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// The sequence a chunk number belongs to (a whole warp calls it): the last s
// with base(s) = begin(s) / L + s <= number, or -1.
template <int L>
__device__ int sequence_of(const Packed& P, int number) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = P.n_seq;
  if (P.begin(0) / L > number) return -1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, s = lo + lane * step;
    const bool below = s < hi && P.begin(s) / L + s <= number;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    const int next = lo + n * step;
    lo += (n - 1) * step;
    hi = next < hi ? next : hi;
  }
  return lo;
}

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
// The same to global memory where `p` holds, without a branch.
__device__ __forceinline__ void store_row_if(bool p, float* at, float2 lo, float2 hi) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n"
      " @p st.global.v4.f32 [%1], {%2, %3, %4, %5};\n}\n" ::"r"((uint32_t)p),
      "l"(at), "f"(lo.x), "f"(lo.y), "f"(hi.x), "f"(hi.y)
      : "memory");
}
__device__ __forceinline__ void store_row_if(bool p, __nv_bfloat16* at, float2 lo, float2 hi) {
  const __nv_bfloat162 a = __float22bfloat162_rn(lo), b = __float22bfloat162_rn(hi);
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n"
      " @p st.global.v2.b32 [%1], {%2, %3};\n}\n" ::"r"((uint32_t)p),
      "l"(at), "r"(*reinterpret_cast<const uint32_t*>(&a)),
      "r"(*reinterpret_cast<const uint32_t*>(&b))
      : "memory");
}
__device__ __forceinline__ float2 shfl_xor2(float2 a, int m) {
  return make_float2(__shfl_xor_sync(0xffffffffu, a.x, m), __shfl_xor_sync(0xffffffffu, a.y, m));
}

struct ForwardArgs {
  CUtensorMap za, zb, v;
  Packed packed;
  const float* A;
  const float* bias;
  const float* h0;
  void* y;
  float* hT;
  float* states;
  Chain chain;
  int D, col_tiles;
  unsigned tiles;
  unsigned limit_us;
  unsigned* status;
};

// The order in which chunks of packed sequences are handed out.  Taken as they
// are numbered, the chunks in flight would be neighbours of one sequence, each
// waiting for the one before.  So the numbers are cut into kParts parts, where
// sequences begin, of about equal length, and handed out in turn, one of each
// part; parts that run out drop out.  A chunk still comes after its predecessor.
// Measured, forward and backward at 10007 x 1000 float32 in 11 sequences: 144 us
// in one part, 123 in four.
constexpr int kParts = 4;
struct Order {
  int begin[kParts];       // of the parts, sorted by length
  int length[kParts];
};

template <int L>
__device__ Order order_of(const Packed& P, int numbers, bool many) {
  int at[kParts + 1];
  at[0] = 0;
  at[kParts] = numbers;
  if (!many) {             // all in flight within two rounds: one part
    Order o;
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
      o.begin[j] = 0;
      o.length[j] = j == kParts - 1 ? numbers : 0;
    }
    return o;
  }
#pragma unroll
  for (int j = 1; j < kParts; ++j) {
    const int aim = (int)((long long)numbers * j / kParts), s = sequence_of<L>(P, aim);
    const int lo = s < 0 ? 0 : P.begin(s) / L + s, hi = s < 0 ? P.begin(0) / L : P.begin(s + 1) / L + s + 1;
    at[j] = aim - lo < hi - aim ? lo : min(hi, numbers);
  }
  Order o;
#pragma unroll
  for (int j = 0; j < kParts; ++j) {
    o.begin[j] = at[j];
    o.length[j] = at[j + 1] - at[j];
  }
#pragma unroll
  for (int i = 0; i < kParts - 1; ++i)
#pragma unroll
    for (int j = 0; j < kParts - 1 - i; ++j)
      if (o.length[j] > o.length[j + 1]) {
        const int b = o.begin[j], l = o.length[j];
        o.begin[j] = o.begin[j + 1];
        o.length[j] = o.length[j + 1];
        o.begin[j + 1] = b;
        o.length[j + 1] = l;
      }
  return o;
}

// The number that is handed out q-th; backwards through each part if kReverse.
template <bool kReverse>
__device__ __forceinline__ int number_at(const Order& o, int q) {
  int done = 0, number = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const int parts = kParts - i, count = (o.length[i] - done) * parts;
    if (!found && q < count) {
      found = true;
      const int round = q / parts, j = i + q - round * parts;
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        if (k == j)
          number = kReverse ? o.begin[k] + o.length[k] - 1 - done - round : o.begin[k] + done + round;
    }
    q -= count;
    done = o.length[i];
  }
  return number;
}

// The next tile that has rows (a whole warp calls it): takes tickets until one
// does; false when there is none left.  `ticket` (lane 0) was taken earlier and
// is replaced by a new one, so that its latency lies behind other work.
// `skip` is called for a number without rows: of a sequence without any (its
// chunk 0), or of no chunk at all (seq < 0).
template <int L, bool kReverse, class Skip>
__device__ __forceinline__ bool fetch(const Packed& packed, const Order& order, const Chain& chain,
                                      unsigned tiles, int col_tiles, unsigned& ticket, Tile& t,
                                      Skip skip) {
  const int lane = threadIdx.x & 31;
  while (true) {
    const unsigned k = __shfl_sync(0xffffffffu, ticket, 0);
    if (k >= tiles) {
      t.rows = 0;
      return false;
    }
    if (lane == 0) ticket = next_ticket(chain);
    const int q = (int)(k / (unsigned)col_tiles);
    t.col0 = (int)(k - (unsigned)q * (unsigned)col_tiles) * kCols;
    int o = 0, len = 0;
    t.chunk = 0;
    if (packed.offsets) {
      t.number = number_at<kReverse>(order, q);
      t.seq = sequence_of<L>(packed, t.number);
      if (t.seq >= 0) {
        o = packed.begin(t.seq);
        len = packed.begin(t.seq + 1) - o;
        t.chunk = t.number - (o / L + t.seq);
      }
      t.back = 1;
    } else {
      // Equal lengths: chunk c of every sequence before chunk c + 1 of any, so
      // that a chunk's predecessor is as far back as can be.
      t.number = kReverse ? (int)(tiles / (unsigned)col_tiles) - 1 - q : q;
      t.chunk = t.number / packed.n_seq;
      t.seq = t.number - t.chunk * packed.n_seq;
      len = packed.rows / packed.n_seq;
      o = len * t.seq;
      t.back = packed.n_seq;
    }
    t.row0 = o + t.chunk * L;
    t.rows = len - t.chunk * L;
    if (t.rows <= 0) {
      if (t.chunk > 0) t.seq = -1;
      skip(t);
      continue;
    }
    if (kReverse) {
      t.pos = (t.rows - 1) / L;
      t.last = t.chunk == 0;
      t.back = -t.back;
    } else {
      t.pos = t.chunk;
      t.last = t.rows <= L;
    }
    if (t.rows > L) t.rows = L;
    return true;
  }
}

// Whether a chunk publishes the state behind it (with P = 0), known only after
// the fold, not its pair: the last of a group, and a sequence's first.  The
// first's would be known at once, but this way its block's read of h0 has
// happened when the chunks behind go on, and the last may overwrite h0 (hT = h0).
__device__ __forceinline__ bool publishes_state(int pos) {
  return pos % kGroup == kGroup - 1 || pos == 0;
}

// The state in front of a tile from what the chunks before it published (a
// whole warp; each lane two channels).  Chunks are in groups of kGroup: the
// last of a group publishes the state behind it, the others the pair (P, S)
// with which a state h in front of them becomes P h + S behind them (the first
// chunk of a sequence has its initial state in S and P = 0).  So a tile needs
// the state behind the group before and the pairs of its own group, and the
// serial chain through the grid has one link per kGroup chunks, not one per
// chunk.  The pairs, there early, are put together first; a link is then one
// wait, one multiply-add and one store.  Always in the same order: results do
// not depend on timing.  Returns false if the wait ran out or another block
// gave up.
__device__ __forceinline__ bool keep_waiting(const Chain& ch, const volatile GiveUp* give_up,
                                             int& spin, uint64_t& t0) {
  if ((++spin & 63) != 1) return true;
  const unsigned limit_us = give_up->limit_us;
  const uint64_t now = global_ns();
  if (t0 == 0) t0 = now;
  return __all_sync(0xffffffffu, now - t0 < limit_us * 1000ull && load_acquire(ch.abort) != 0);
}

__device__ __forceinline__ bool fold_before(const Chain& ch, const Tile& t, int D,
                                            const volatile GiveUp* give_up, float2& h) {
  const int lane = threadIdx.x & 31, c = t.col0 + lane * 2;
  const int n = t.pos % kGroup;            // pairs of its own group
  const bool in = c < D, grouped = t.pos >= kGroup;
  const ptrdiff_t step = (ptrdiff_t)t.back * D * 2;
  const float* near = ch.pairs + ((size_t)t.number * D + c) * 2 - step;   // the chunk before
  const float* state = near - n * step;                                   // the group before
  int spin = 0;
  uint64_t t0 = 0;
  uint4 q[kGroup - 1], from = make_uint4(0u, 0u, 0u, 0u);
  while (true) {
    // Everything at once: mostly it is there, and costs one way to L2.
    unsigned most = 0;
    const float* f = near;
#pragma unroll
    for (int k = 0; k < kGroup - 1; ++k, f -= step) {
      q[k] = make_uint4(0x3f800000u, 0u, 0x3f800000u, 0u);                // changes nothing
      if (k < n && in) q[k] = load_pairs(f);
    }
    if (grouped && in) from = load_pairs(state);
#pragma unroll
    for (int k = 0; k < kGroup - 1; ++k) most = max(most, largest(q[k]));
    if (__all_sync(0xffffffffu, most != kUnset)) break;
    // If not, mostly the nearest is the last to arrive.
    while (!__all_sync(0xffffffffu, !in || largest(load_pairs(near)) != kUnset)) {
      __nanosleep(20);
      if (!keep_waiting(ch, give_up, spin, t0)) return false;
    }
    if (!keep_waiting(ch, give_up, spin, t0)) return false;
  }
  float2 P = both(1.f), S = both(0.f);
#pragma unroll
  for (int k = kGroup - 2; k >= 0; --k) {
    const float2 p = make_float2(__uint_as_float(q[k].x), __uint_as_float(q[k].z));
    S = fma2(p, S, make_float2(__uint_as_float(q[k].y), __uint_as_float(q[k].w)));
    P = mul2(p, P);
  }
  h = S;
  if (!grouped) return true;               // the sequence's first chunk has P = 0
  while (!__all_sync(0xffffffffu, largest(from) != kUnset)) {
    if (!keep_waiting(ch, give_up, spin, t0)) return false;
    if (in) from = load_pairs(state);
  }
  h = fma2(P, make_float2(__uint_as_float(from.y), __uint_as_float(from.w)), S);
  return true;
}

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

// A block is eight warps for the arithmetic (a half-warp takes R rows by 64
// channels, four channels a thread) and four more: one fetches tiles, one
// publishes their pairs, two (even and odd tiles) fold what the chunks before
// published into the state in front of them.
//
// That state comes from other blocks, a microsecond or two after a tile's pair
// is out.  So the arithmetic warps do not wait for it: they form a tile's
// gates, put a and b aside in tensor memory (which nothing else here uses),
// go on to the next tile, and only then come back to finish the one before.
//
// Measured at 131072 x 2048 bf16: 384 us, 2.15 GB once = 0.84 of the copy rate;
// at 9001 x 1920 float32 in 13 sequences 50 us, 0.82.  With every gate left out
// (a = za + zb, b = v) the first takes 336 us: what bounds it is the arithmetic,
// about 19 instructions of every element's 36, on 60% of the issue slots.  A first
// form in which the block waited for each tile's state took 791 us.
//
// Inputs come in units of one tensor's tile (16 KB), in a ring of kUnits.
// Barriers, all in shared memory: a tile's description is there (known), its
// units are (full) and have been read (empty); its warps' pairs are there
// (paired) and have been summed up (summed), the state in front of it is
// (folded), both have been read (taken).
constexpr int kWarps = 8;
constexpr int kUnits = 5;
constexpr int kSlots = 2;    // tiles between gates and outputs
constexpr int kInfo = 8;     // ring of descriptions: longer than any tile's life
constexpr int kThreads = (kWarps + 4) * 32;

template <typename T>
struct ForwardShape {
  static constexpr int R = 16 / sizeof(T);                              // rows per thread
  static constexpr int L = 2 * kWarps * R;                              // rows per tile
  static constexpr int kUnitBytes = L * kCols * (int)sizeof(T);
  static constexpr int kSmem = kUnits * kUnitBytes + 128;               // + alignment
  static constexpr int kParkCols = 8 * R;                               // per thread and tile
  static constexpr int kSlotCols = kWarps / 4 * kParkCols;
  static constexpr int kTmemCols = kSlots * kSlotCols;                  // a power of two
  static_assert(kStateRows<T> % R == 0, "states fall on a thread's first row");
};

// The pairs of a tile's warps become those of all rows in front of each warp;
// `whole` gets the whole tile's before anything is written (two channels per
// lane).
template <class Whole>
__device__ __forceinline__ void running_pairs(float (*total)[2][kCols], int lane, Whole whole) {
  float2 p[kWarps], s[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    p[w] = *reinterpret_cast<const float2*>(&total[w][0][lane * 2]);
    s[w] = *reinterpret_cast<const float2*>(&total[w][1][lane * 2]);
  }
  float2 P = both(1.f), S = both(0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float2 wp = p[w], ws = s[w];
    p[w] = P;
    s[w] = S;
    S = fma2(wp, S, ws);
    P = mul2(wp, P);
  }
  whole(P, S);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    *reinterpret_cast<float2*>(&total[w][0][lane * 2]) = p[w];
    *reinterpret_cast<float2*>(&total[w][1][lane * 2]) = s[w];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) forward_kernel(const __grid_constant__ ForwardArgs P) {
  using Sh = ForwardShape<T>;
  constexpr int L = Sh::L, R = Sh::R, W = kWarps;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((128 - (smem_u32(raw) & 127)) & 127);
  __shared__ uint64_t full[2], empty[2], known[kInfo], paired[kSlots], summed[kSlots],
      folded[kSlots], taken[kSlots];
  __shared__ Tile tiles[kInfo];
  __shared__ __align__(16) float total[kSlots][W][2][kCols];   // (P, S) of each warp's rows,
                                                               // then of all rows in front of it
  __shared__ __align__(16) float lower[kSlots][W][2][kCols];   // and of its lower half-warp's
  __shared__ __align__(16) float whole[kSlots][2][kCols];      // the tile's
  __shared__ __align__(16) float carry[kSlots][kCols];         // the state in front of the tile
  __shared__ __align__(16) float rates[2][2][kCols];           // A, bias
  __shared__ uint32_t tmem_base;
  __shared__ GiveUp quit;
  volatile GiveUp* give_up = &quit;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // First of all: a block that holds tensor memory must not wait for a kernel in
  // front of it, which may want it.
  wait_for_stream();
  if (warp == W + 1) tc::tmem_alloc(&tmem_base, Sh::kTmemCols);
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&full[s], 2);              // copies asked for, rates there
      mbar_init(&empty[s], W);
    }
    for (int s = 0; s < kInfo; ++s) mbar_init(&known[s], 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&paired[s], W);
      mbar_init(&summed[s], 1);
      mbar_init(&folded[s], 1);
      mbar_init(&taken[s], W);
    }
    quit = GiveUp{0, P.limit_us};
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (!offsets_ok(P.packed)) {
    if (tid == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    if (warp == W + 1) tc::tmem_dealloc(tmem_base, Sh::kTmemCols);
    return;
  }

  if (warp == W) {                         // fetches
    unsigned ticket = 0;
    if (lane == 0) ticket = next_ticket(P.chain);
    Order order;
    if (P.packed.offsets)
      order = order_of<L>(P.packed, (int)(P.tiles / (unsigned)P.col_tiles), P.tiles > 2 * gridDim.x);
    bool more = true;
    int n = 0, unit = 0;                   // tiles asked for; place of the next unit
    for (; more; ++n) {
      Tile t{};
      more = fetch<L, false>(P.packed, order, P.chain, P.tiles, P.col_tiles, ticket, t,
                      [&](const Tile& e) {               // a sequence without rows
                        const int c = e.col0 + lane * 2;
                        if (P.hT && e.seq >= 0 && c < P.D) {
                          const size_t i = (size_t)e.seq * P.D + c;
                          *reinterpret_cast<float2*>(P.hT + i) =
                              P.h0 ? *reinterpret_cast<const float2*>(P.h0 + i)
                                   : make_float2(0.f, 0.f);
                        }
                      });
      const Rates rt = rates_of(P.A, P.bias, more ? t.col0 + lane * 2 : P.D, P.D);
      // The places of the first two units held the last two of the tile two
      // before, that of the third the first of the tile before.
      if (n >= 2 && !wait_phase(&empty[n & 1], ((n >> 1) - 1) & 1, give_up)) break;
      if (lane == 0) {
        tiles[n % kInfo] = t;
        mbar_arrive(&known[n % kInfo]);
        if (more)
          mbar_expect(&full[n & 1], 3 * Sh::kUnitBytes);
        else
          mbar_arrive(&full[n & 1]);
      }
      __syncwarp();
      bool there = true;
      for (int j = 0; j < 3 && more; ++j) {
        if (j == 2 && n >= 1)
          there = wait_phase(&empty[(n - 1) & 1], ((n - 1) >> 1) & 1, give_up);
        // Where the block gives up (its results are void then), the copy is made
        // all the same, so that the barrier completes.
        if (lane == 0)
          tma_load(smem + unit * Sh::kUnitBytes, j == 0 ? &P.za : j == 1 ? &P.zb : &P.v, t.col0,
                   t.row0, &full[n & 1]);
        if (++unit == kUnits) unit = 0;
      }
      *reinterpret_cast<float2*>(&rates[n & 1][0][lane * 2]) = rt.A;
      *reinterpret_cast<float2*>(&rates[n & 1][1][lane * 2]) = rt.bias;
      __syncwarp();
      mbar_arrive_if(lane == 0, &full[n & 1]);
      if (!there) {
        ++n;
        break;
      }
    }
    // Stay until every copy has arrived, also when the block gives up.
    for (int x = n > 2 ? n - 2 : 0; x < n; ++x)
      mbar_wait_bounded(&full[x & 1], (x >> 1) & 1, kWaitNs);
  } else if (warp == W + 1) {              // publishes
    for (int it = 0;; ++it) {
      const int slot = it % kSlots;
      if (!wait_phase(&known[it % kInfo], (it / kInfo) & 1, give_up)) break;
      const Tile t = tiles[it % kInfo];
      if (t.rows == 0) break;
      if (!wait_phase(&paired[slot], (it / kSlots) & 1, give_up)) break;
      const int c = t.col0 + lane * 2;
      running_pairs(total[slot], lane, [&](float2 p, float2 s) {
        if (t.last) return;
        if (publishes_state(t.pos)) {      // left to the fold
          *reinterpret_cast<float2*>(&whole[slot][0][lane * 2]) = p;
          *reinterpret_cast<float2*>(&whole[slot][1][lane * 2]) = s;
        } else if (c < P.D) {
          publish(P.chain.pairs + ((size_t)t.number * P.D + c) * 2, p, s);
        }
      });
      __syncwarp();
      mbar_arrive_if(lane == 0, &summed[slot]);
    }
  } else if (warp > W + 1) {               // folds
    for (int it = warp - (W + 2);; it += 2) {
      const int slot = it % kSlots;
      // The end may come before this warp's next tile.
      if (it > 0) {
        if (!wait_phase(&known[(it - 1) % kInfo], ((it - 1) / kInfo) & 1, give_up)) break;
        if (tiles[(it - 1) % kInfo].rows == 0) break;
      }
      if (!wait_phase(&known[it % kInfo], (it / kInfo) & 1, give_up)) break;
      const Tile t = tiles[it % kInfo];
      if (t.rows == 0) break;
      const int c = t.col0 + lane * 2;
      float2 h = make_float2(0.f, 0.f);
      if (t.chunk == 0) {
        if (P.h0 && c < P.D) h = *reinterpret_cast<const float2*>(P.h0 + (size_t)t.seq * P.D + c);
      } else if (!fold_before(P.chain, t, P.D, give_up, h)) {
        give_up->done = 1;
        break;
      }
      // (Which also means that the tile two before has been finished: its state
      // may be overwritten.)
      if (!wait_phase(&summed[slot], (it / kSlots) & 1, give_up)) break;
      *reinterpret_cast<float2*>(&carry[slot][lane * 2]) = h;
      if (!t.last && publishes_state(t.pos)) {
        const float2 p = *reinterpret_cast<const float2*>(&whole[slot][0][lane * 2]);
        const float2 s = *reinterpret_cast<const float2*>(&whole[slot][1][lane * 2]);
        if (c < P.D)
          publish(P.chain.pairs + ((size_t)t.number * P.D + c) * 2, both(0.f), fma2(p, h, s));
      }
      __syncwarp();
      mbar_arrive_if(lane == 0, &folded[slot]);
    }
  } else {                                 // gates and outputs
    const int c4 = (lane & 15) * 4, first = (tid >> 4) * R;   // first row in the tile
    const uint32_t park = tmem_base + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * Sh::kParkCols;
    const uint32_t from = (uint32_t)((first * kCols + c4) * sizeof(T));
    const Constants K = constants();
    int unit = 0;                          // place of the tile's first unit
    int end = 0x7fffffff;                  // number of this block's tiles, once known
    for (int it = 0; it - 1 < end; ++it) {
      if (it < end) {
        const int slot = it & 1;
        if (!wait_phase(&full[it & 1], (it >> 1) & 1, give_up)) break;
        const Tile t = tiles[it % kInfo];
        if (t.rows == 0) {
          end = it;
        } else {
          float2 A[2], bias[2];
          load_row(&rates[it & 1][0][c4], A[0], A[1]);
          load_row(&rates[it & 1][1][c4], bias[0], bias[1]);
          const int u1 = unit + 1 < kUnits ? unit + 1 : 0, u2 = u1 + 1 < kUnits ? u1 + 1 : 0;
          const T* bza = reinterpret_cast<const T*>(smem + unit * Sh::kUnitBytes + from);
          const T* bzb = reinterpret_cast<const T*>(smem + u1 * Sh::kUnitBytes + from);
          const T* bv = reinterpret_cast<const T*>(smem + u2 * Sh::kUnitBytes + from);
          unit = u2 + 1 < kUnits ? u2 + 1 : 0;
          // Four rows at a time: gates, the pair of all rows so far, aside.
          float2 p[2] = {both(1.f), both(1.f)}, s[2] = {both(0.f), both(0.f)};
#pragma unroll
          for (int r4 = 0; r4 < R; r4 += 4) {
            float2 a[8], b[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float2 za[2], zb[2], v[2];
              load_row(bza + (r4 + r) * kCols, za[0], za[1]);
              load_row(bzb + (r4 + r) * kCols, zb[0], zb[1]);
              load_row(bv + (r4 + r) * kCols, v[0], v[1]);
              gate_pair(K, za[0], zb[0], v[0], A[0], bias[0], a[2 * r], b[2 * r]);
              gate_pair(K, za[1], zb[1], v[1], A[1], bias[1], a[2 * r + 1], b[2 * r + 1]);
            }
            if (t.rows < L) {              // rows behind the sequence change nothing
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (first + r4 + r >= t.rows) {
                  a[2 * r] = a[2 * r + 1] = both(1.f);
                  b[2 * r] = b[2 * r + 1] = both(0.f);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                s[k] = fma2(a[2 * r + k], s[k], b[2 * r + k]);
                p[k] = mul2(a[2 * r + k], p[k]);
              }
            }
            park16(park + slot * Sh::kSlotCols + r4 * 8, a);
            park16(park + slot * Sh::kSlotCols + r4 * 8 + 16, b);
          }
          __syncwarp();
          mbar_arrive_if(lane == 0, &empty[it & 1]);
          // The warp's pair (the lower half-warp's rows come first).
          float2 pl[2], sl[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            pl[k] = shfl_xor2(p[k], 16);
            sl[k] = shfl_xor2(s[k], 16);
          }
          if (it >= kSlots && !wait_phase(&taken[slot], ((it >> 1) - 1) & 1, give_up)) break;
          if (lane >= 16) {
            store_row(&total[slot][warp][0][c4], mul2(p[0], pl[0]), mul2(p[1], pl[1]));
            store_row(&total[slot][warp][1][c4], fma2(p[0], sl[0], s[0]), fma2(p[1], sl[1], s[1]));
          } else {
            store_row(&lower[slot][warp][0][c4], p[0], p[1]);
            store_row(&lower[slot][warp][1][c4], s[0], s[1]);
          }
          parked();
          __syncwarp();
          mbar_arrive_if(lane == 0, &paired[slot]);
        }
      }
      const int out = it - 1;              // the tile to finish
      if (out < 0) continue;
      const int slot = out & 1;
      const Tile t = tiles[out % kInfo];
      const int c = t.col0 + c4;
      if (!wait_phase(&folded[slot], (out >> 1) & 1, give_up)) break;
      float2 h[2];
      load_row(&carry[slot][c4], h[0], h[1]);
      float2 wp[2], ws[2];
      load_row(&total[slot][warp][0][c4], wp[0], wp[1]);
      load_row(&total[slot][warp][1][c4], ws[0], ws[1]);
      h[0] = fma2(wp[0], h[0], ws[0]);
      h[1] = fma2(wp[1], h[1], ws[1]);
      if (lane >= 16) {
        load_row(&lower[slot][warp][0][c4], wp[0], wp[1]);
        load_row(&lower[slot][warp][1][c4], ws[0], ws[1]);
        h[0] = fma2(wp[0], h[0], ws[0]);
        h[1] = fma2(wp[1], h[1], ws[1]);
      }
      __syncwarp();
      mbar_arrive_if(lane == 0, &taken[slot]);
      const int row = t.chunk * L + first;                     // in the sequence
      if (P.states && row % kStateRows<T> == 0 && first < t.rows && c < P.D) {
        const int begin = t.row0 - t.chunk * L;
        const size_t n = (size_t)(begin / kStateRows<T> + t.seq + row / kStateRows<T>);
        store_row(P.states + n * P.D + c, h[0], h[1]);
      }
      T* y = reinterpret_cast<T*>(P.y) + (size_t)(t.row0 + first) * P.D + c;
      int left = c < P.D ? t.rows - first : 0;                 // rows to store
#pragma unroll
      for (int r4 = 0; r4 < R; r4 += 4) {
        float2 a[8], b[8];
        ask16(park + slot * Sh::kSlotCols + r4 * 8, a);
        ask16(park + slot * Sh::kSlotCols + r4 * 8 + 16, b);
        asked();
        here(a);
        here(b);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          h[0] = fma2(a[2 * r], h[0], b[2 * r]);
          h[1] = fma2(a[2 * r + 1], h[1], b[2 * r + 1]);
          store_row_if(r < left, y + (size_t)r * P.D, h[0], h[1]);
        }
        left -= 4;
        y += (size_t)4 * P.D;
      }
      if (P.hT && t.last && first < t.rows && t.rows <= first + R && c < P.D)
        store_row(P.hT + (size_t)t.seq * P.D + c, h[0], h[1]);
    }
    parked();    // where the block gives up: nothing is on its way when the columns are freed
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == W + 1) tc::tmem_dealloc(tmem_base, Sh::kTmemCols);
  if (quit.done && tid == 0) {             // tell the other blocks
    record_status(P.status, SDM_ERR_TIMEOUT);
    atomicExch(P.chain.abort, 0u);
  }
}

// ----------------------------------------------------------------- backward
// The gates of two channels again, all that the gradients need of them: a,
// beta, 1 - beta, softplus (times log2 e) and sigmoid of za + bias.
struct Gates2 {
  float2 a, beta, keep, sp, sig;
};
__device__ __forceinline__ Gates2 gates_pair(const Constants& K, float2 za, float2 zb, float2 A,
                                             float2 bias) {
  Gates2 g;
  float2 x, e, z, eb, r;
  softplus_pair(K, za, bias, x, e, g.sp);
  const float2 f = add2(e, K.one);
  g.sig = mul2(make_float2(x.x >= 0.f ? 1.f : e.x, x.y >= 0.f ? 1.f : e.y),
               make_float2(rcp(f.x), rcp(f.y)));
  sigmoid_pair(K, zb, z, eb, g.beta);
  g.a = decay_pair(K, A, g.sp, z, g.beta, r);
  g.keep = mul2(make_float2(fminf(eb.x, 1.f), fminf(eb.y, 1.f)), r);
  return g;
}

// A row's a (four channels) in the place of its za and zb in shared memory,
// which are as many bytes (twice as many for float32).
__device__ __forceinline__ void keep_a(float* za, float*, float2 lo, float2 hi) { store_row(za, lo, hi); }
__device__ __forceinline__ void take_a(const float* za, const float*, float2& lo, float2& hi) {
  load_row(za, lo, hi);
}
__device__ __forceinline__ void keep_a(__nv_bfloat16* za, __nv_bfloat16* zb, float2 lo, float2 hi) {
  *reinterpret_cast<float2*>(za) = lo;
  *reinterpret_cast<float2*>(zb) = hi;
}
__device__ __forceinline__ void take_a(const __nv_bfloat16* za, const __nv_bfloat16* zb, float2& lo,
                                       float2& hi) {
  lo = *reinterpret_cast<const float2*>(za);
  hi = *reinterpret_cast<const float2*>(zb);
}
struct BackwardArgs {
  CUtensorMap za, zb, v, dy;
  Packed packed;
  const float* A;
  const float* bias;
  const float* states;
  const float* dhT;
  void* dza;
  void* dzb;
  void* dv;
  float* dh0;
  float* partial;     // [numbers][2][D]
  Chain chain;
  int D, col_tiles;
  long long ld_grad;
  unsigned tiles;
  unsigned limit_us;
  unsigned* status;
};

// The chain runs from the last chunk to the first; what it carries is r, the
// gradient of the state in front of a chunk (r[t] = a[t] (dy[t] + r[t+1])), and
// what a chunk publishes is the pair (P, Q) with r_front = P r_behind + Q.  The
// states inside a tile come from the saved one in front of it without a wait.
//
// A block is four warps for the arithmetic (a half-warp takes R rows) and
// three more: one fetches tiles, one sums up the half-warps' pairs and
// publishes, one folds.  Of a tile's gates, a goes into shared memory, in the
// place of za and zb, and the rest into tensor memory.
//
// kLag: a tile is finished after the next one's gates, as in the forward pass,
// so that a fold has a tile's time to come; otherwise at once, which takes less
// memory and, in float32, leaves room for three blocks (75 us with two, 68 with
// three at 10007 x 1000; bf16, 32768 x 1024: 109 with two and 113 with three, which
// are short of registers).  See lags.
constexpr int kBackWarps = 4;
constexpr int kHalves = 2 * kBackWarps;
constexpr int kBackThreads = (kBackWarps + 3) * 32;

template <typename T, bool kLag>
struct BackwardShape {
  static constexpr int R = 16 / sizeof(T);
  static constexpr int L = kHalves * R;
  static constexpr int kBlocks = kLag || sizeof(T) == 2 ? 2 : 3;        // per SM
  static constexpr int kUnits = kLag ? 11 : 8;   // places for tensors' tiles, four of a tile
  static constexpr int kRing = kLag ? 4 : 2;     // barriers of tiles' copies
  static constexpr int kOpen = kLag ? 2 : 1;     // tiles between gates and gradients
  static constexpr int kUnitBytes = L * kCols * (int)sizeof(T);
  static constexpr int kSmem = kUnits * kUnitBytes + 128;
  static constexpr int kOpenCols = 16 * R;
  static constexpr int kTmemCols = kOpen * kOpenCols;
  static_assert(L == kStateRows<T>, "a saved state in front of every tile");
};

template <typename T, bool kLag>
__global__ void __launch_bounds__(kBackThreads, BackwardShape<T, kLag>::kBlocks)
    backward_kernel(const __grid_constant__ BackwardArgs P) {
  using Sh = BackwardShape<T, kLag>;
  constexpr int L = Sh::L, R = Sh::R, W = kBackWarps, kRing = Sh::kRing, kOpen = Sh::kOpen;
  // (With a lag, 32768 x 1024 bf16: 119 us rolled, 120 by two.)
  constexpr int kUnroll = sizeof(T) == 2 && !kLag ? 2 : 1;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((128 - (smem_u32(raw) & 127)) & 127);
  __shared__ uint64_t full[kRing], empty[kRing], known[kInfo], paired[kOpen], summed[2],
      folded[2], taken[2];
  __shared__ Tile tiles[kInfo];
  // Of each half-warp's rows P, S (of the states) and Q (of the gradients); then
  // P of the rows behind them, the state in front of them, Q of the rows behind.
  __shared__ __align__(16) float half[kOpen][kHalves][3][kCols];
  __shared__ __align__(16) float whole[kOpen][2][kCols];
  __shared__ __align__(16) float carry[2][kCols];
  __shared__ __align__(16) float sums[kOpen][W][2][kCols];     // of the gradients of A and bias
  __shared__ __align__(16) float rates[kRing][2][kCols];       // A, bias
  __shared__ uint32_t tmem_base;
  __shared__ GiveUp quit;
  volatile GiveUp* give_up = &quit;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // First of all: a block that holds tensor memory must not wait for a kernel in
  // front of it, which may want it.
  wait_for_stream();
  if (warp == W + 1) tc::tmem_alloc(&tmem_base, Sh::kTmemCols);
  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&full[s], 2);              // copies asked for, rates there
      mbar_init(&empty[s], W);
    }
    for (int s = 0; s < kInfo; ++s) mbar_init(&known[s], 1);
    for (int s = 0; s < kOpen; ++s) mbar_init(&paired[s], W);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&summed[s], 1);
      mbar_init(&folded[s], 1);
      mbar_init(&taken[s], W);
    }
    quit = GiveUp{0, P.limit_us};
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (!offsets_ok(P.packed)) {
    if (tid == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    if (warp == W + 1) tc::tmem_dealloc(tmem_base, Sh::kTmemCols);
    return;
  }

  if (warp == W) {                         // fetches
    unsigned ticket = 0;
    if (lane == 0) ticket = next_ticket(P.chain);
    Order order;
    if (P.packed.offsets)
      order = order_of<L>(P.packed, (int)(P.tiles / (unsigned)P.col_tiles), P.tiles > 2 * gridDim.x);
    bool more = true;
    int n = 0, unit = 0;                   // tiles asked for; place of the next unit
    for (; more; ++n) {
      Tile t{};
      more = fetch<L, true>(
          P.packed, order, P.chain, P.tiles, P.col_tiles, ticket, t, [&](const Tile& e) {
            const int c = e.col0 + lane * 2;
            if (c >= P.D) return;
            float* part = P.partial + (size_t)e.number * 2 * P.D + c;
            *reinterpret_cast<float2*>(part) = make_float2(0.f, 0.f);
            *reinterpret_cast<float2*>(part + P.D) = make_float2(0.f, 0.f);
            if (P.dh0 && e.seq >= 0) {
              const size_t i = (size_t)e.seq * P.D + c;
              *reinterpret_cast<float2*>(P.dh0 + i) =
                  P.dhT ? *reinterpret_cast<const float2*>(P.dhT + i) : make_float2(0.f, 0.f);
            }
          });
      const Rates rt = rates_of(P.A, P.bias, more ? t.col0 + lane * 2 : P.D, P.D);
      // With a lag, the places of the first three units held the last three of
      // the tile three before, that of the fourth the first of the tile two
      // before; up to three tiles' copies are under way, so full is a ring of
      // four: its barrier of the tile four before has been waited for.
      constexpr int kBehind = kLag ? 3 : 2;
      if (n >= kBehind &&
          !wait_phase(&empty[(n - kBehind) % kRing], ((n - kBehind) / kRing) & 1, give_up))
        break;
      if (lane == 0) {
        tiles[n % kInfo] = t;
        mbar_arrive(&known[n % kInfo]);
        if (more)
          mbar_expect(&full[n % kRing], 4 * Sh::kUnitBytes);
        else
          mbar_arrive(&full[n % kRing]);
      }
      __syncwarp();
      bool there = true;
      for (int j = 0; j < 4 && more; ++j) {
        if (kLag && j == 3 && n >= 2)
          there = wait_phase(&empty[(n - 2) % kRing], ((n - 2) / kRing) & 1, give_up);
        // Where the block gives up (its results are void then), the copy is made
        // all the same, so that the barrier completes.
        if (lane == 0)
          tma_load(smem + unit * Sh::kUnitBytes,
                   j == 0 ? &P.za : j == 1 ? &P.zb : j == 2 ? &P.v : &P.dy, t.col0, t.row0,
                   &full[n % kRing]);
        if (++unit == Sh::kUnits) unit = 0;
      }
      *reinterpret_cast<float2*>(&rates[n % kRing][0][lane * 2]) = rt.A;
      *reinterpret_cast<float2*>(&rates[n % kRing][1][lane * 2]) = rt.bias;
      __syncwarp();
      mbar_arrive_if(lane == 0, &full[n % kRing]);
      if (!there) {
        ++n;
        break;
      }
    }
    // Stay until every copy has arrived, also when the block gives up.
    for (int x = n > kRing ? n - kRing : 0; x < n; ++x)
      mbar_wait_bounded(&full[x % kRing], (x / kRing) & 1, kWaitNs);
  } else if (warp == W + 1) {              // sums up and publishes
    Tile before{}, earlier{};              // the tile before this one, and before that
    auto add_up = [&](int slot, float2& sa, float2& sb) {
      sa = sb = both(0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        sa = add2(sa, *reinterpret_cast<const float2*>(&sums[slot][w][0][lane * 2]));
        sb = add2(sb, *reinterpret_cast<const float2*>(&sums[slot][w][1][lane * 2]));
      }
    };
    auto write_sums = [&](const Tile& t, float2 sa, float2 sb) {
      const int c = t.col0 + lane * 2;
      if (c < P.D) {
        float* part = P.partial + (size_t)t.number * 2 * P.D + c;
        *reinterpret_cast<float2*>(part) = sa;
        *reinterpret_cast<float2*>(part + P.D) = sb;
      }
    };
    for (int it = 0;; ++it) {
      const int slot = it % kOpen;
      if (!wait_phase(&known[it % kInfo], (it / kInfo) & 1, give_up)) break;
      const Tile t = tiles[it % kInfo];
      const int c = t.col0 + lane * 2;
      float2 h = make_float2(0.f, 0.f);
      if (t.rows > 0 && c < P.D) {
        const int begin = t.row0 - t.chunk * L;
        h = __ldg(reinterpret_cast<const float2*>(
            P.states + (size_t)(begin / L + t.seq + t.chunk) * P.D + c));
      }
      if (!wait_phase(&paired[slot], (it / kOpen) & 1, give_up)) break;
      if (t.rows > 0) {
        // What others wait for goes out first.
        float2 wp[kHalves], wq[kHalves];
#pragma unroll
        for (int w = 0; w < kHalves; ++w) {
          wp[w] = *reinterpret_cast<const float2*>(&half[slot][w][0][lane * 2]);
          wq[w] = *reinterpret_cast<const float2*>(&half[slot][w][2][lane * 2]);
        }
        float2 p = both(1.f), q = both(0.f);
#pragma unroll
        for (int w = kHalves - 1; w >= 0; --w) {
          q = fma2(wp[w], q, wq[w]);
          p = mul2(wp[w], p);
        }
        if (!t.last) {
          if (publishes_state(t.pos)) {    // left to the fold
            *reinterpret_cast<float2*>(&whole[slot][0][lane * 2]) = p;
            *reinterpret_cast<float2*>(&whole[slot][1][lane * 2]) = q;
          } else if (c < P.D) {
            publish(P.chain.pairs + ((size_t)t.number * P.D + c) * 2, p, q);
          }
        }
#pragma unroll
        for (int w = 0; w < kHalves; ++w) {
          float2* const ws = reinterpret_cast<float2*>(&half[slot][w][1][lane * 2]);
          const float2 s = *ws;
          *ws = h;
          h = fma2(wp[w], h, s);
        }
        p = both(1.f);
        q = both(0.f);
#pragma unroll
        for (int w = kHalves - 1; w >= 0; --w) {
          *reinterpret_cast<float2*>(&half[slot][w][0][lane * 2]) = p;
          *reinterpret_cast<float2*>(&half[slot][w][2][lane * 2]) = q;
          q = fma2(wp[w], q, wq[w]);
          p = mul2(wp[w], p);
        }
      }
      // The arithmetic warps have finished the tile kOpen before, and write its
      // slot again only after this one has been summed up.
      float2 sa, sb;
      add_up(slot, sa, sb);
      if (t.rows > 0) {
        __syncwarp();
        mbar_arrive_if(lane == 0, &summed[it & 1]);
      }
      if (it >= kOpen) write_sums(kLag ? earlier : before, sa, sb);
      if (t.rows == 0) {
        if (kLag && it > 0) {
          add_up(slot ^ 1, sa, sb);
          write_sums(before, sa, sb);
        }
        break;
      }
      earlier = before;
      before = t;
    }
  } else if (warp == W + 2) {              // folds
    for (int it = 0;; ++it) {
      const int slot = it % kOpen;
      if (!wait_phase(&known[it % kInfo], (it / kInfo) & 1, give_up)) break;
      const Tile t = tiles[it % kInfo];
      if (t.rows == 0) break;
      const int c = t.col0 + lane * 2;
      float2 r = make_float2(0.f, 0.f);
      if (t.pos == 0) {
        if (P.dhT && c < P.D)
          r = *reinterpret_cast<const float2*>(P.dhT + (size_t)t.seq * P.D + c);
      } else if (!fold_before(P.chain, t, P.D, give_up, r)) {
        give_up->done = 1;
        break;
      }
      // The tile that last used this carry has been finished.
      const int past = kLag ? it : it - 1;
      if (past >= 0 && !wait_phase(&summed[past & 1], (past >> 1) & 1, give_up)) break;
      *reinterpret_cast<float2*>(&carry[it & 1][lane * 2]) = r;
      if (!t.last && publishes_state(t.pos)) {
        if (!kLag && !wait_phase(&summed[it & 1], (it >> 1) & 1, give_up)) break;
        const float2 p = *reinterpret_cast<const float2*>(&whole[slot][0][lane * 2]);
        const float2 q = *reinterpret_cast<const float2*>(&whole[slot][1][lane * 2]);
        if (c < P.D)
          publish(P.chain.pairs + ((size_t)t.number * P.D + c) * 2, both(0.f), fma2(p, r, q));
      }
      __syncwarp();
      mbar_arrive_if(lane == 0, &folded[it & 1]);
    }
  } else {                                 // gates and gradients
    const Constants K = constants();
    const int c4 = (lane & 15) * 4, hw = tid >> 4, first = hw * R;
    const uint32_t park = tmem_base + ((uint32_t)warp << 21);
    // This half-warp's first row in the place of tensor j of the tile whose first
    // unit is u (without a lag a tile never wraps around).
    auto place = [&](int u, int j) {
      if (kLag && u + j >= Sh::kUnits) u -= Sh::kUnits;
      return reinterpret_cast<T*>(smem + u * Sh::kUnitBytes) + first * kCols + c4 +
             j * (L * kCols);
    };
    int unit = 0, unit_before = 0;         // places of a tile's first unit
    int end = 0x7fffffff;                  // number of this block's tiles, once known
    int it = 0;
    for (; it - (kOpen - 1) < end; ++it) {
      const int finished = kLag ? unit_before : unit;
      unit_before = unit;
      if (it < end) {
        const int slot = it % kOpen;
        if (!wait_phase(&full[it % kRing], (it / kRing) & 1, give_up)) break;
        const Tile t = tiles[it % kInfo];
        if (t.rows == 0) {
          end = it;
        } else {
          float2 A[2], bias[2];
          load_row(&rates[it % kRing][0][c4], A[0], A[1]);
          load_row(&rates[it % kRing][1][c4], bias[0], bias[1]);
          T *const bza = place(unit, 0), *const bzb = place(unit, 1), *const bv = place(unit, 2),
                  *const bdy = place(unit, 3);
          unit = unit + 4 < Sh::kUnits ? unit + 4 : unit + 4 - Sh::kUnits;
          // Gates, set aside, and the pairs of this half-warp's rows: (p, s) of
          // the states, (p, q) of the gradients.
          float2 p[2] = {both(1.f), both(1.f)}, s[2] = {both(0.f), both(0.f)},
                 q[2] = {both(0.f), both(0.f)};
#pragma unroll kUnroll
          for (int r = 0; r < R; ++r) {
            float2 za[2], zb[2], v[2], dy[2];
            load_row(bza + r * kCols, za[0], za[1]);
            load_row(bzb + r * kCols, zb[0], zb[1]);
            load_row(bv + r * kCols, v[0], v[1]);
            load_row(bdy + r * kCols, dy[0], dy[1]);
            Gates2 g[2];
            g[0] = gates_pair(K, za[0], zb[0], A[0], bias[0]);
            g[1] = gates_pair(K, za[1], zb[1], A[1], bias[1]);
            if (first + r >= t.rows) {     // a row behind the sequence changes nothing
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                g[k].a = both(1.f);
                g[k].beta = g[k].keep = g[k].sp = g[k].sig = v[k] = dy[k] = both(0.f);
              }
              store_row(bv + r * kCols, v[0], v[1]);
              store_row(bdy + r * kCols, dy[0], dy[1]);
            }
            float2 aside[8] = {g[0].beta, g[1].beta, g[0].keep, g[1].keep,
                               g[0].sp,   g[1].sp,   g[0].sig,  g[1].sig};
            park16(park + slot * Sh::kOpenCols + r * 16, aside);
            keep_a(bza + r * kCols, bzb + r * kCols, g[0].a, g[1].a);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              s[k] = fma2(g[k].a, s[k], mul2(g[k].beta, v[k]));
              p[k] = mul2(g[k].a, p[k]);
              q[k] = fma2(p[k], dy[k], q[k]);
            }
          }
          if (kLag && it >= 2 && !wait_phase(&taken[it & 1], ((it >> 1) - 1) & 1, give_up)) break;
          store_row(&half[slot][hw][0][c4], p[0], p[1]);
          store_row(&half[slot][hw][1][c4], s[0], s[1]);
          store_row(&half[slot][hw][2][c4], q[0], q[1]);
          parked();
          __syncwarp();
          mbar_arrive_if(lane == 0, &paired[slot]);
        }
      }
      const int out = it - (kOpen - 1);    // the tile to finish
      if (out < 0 || out >= end) continue;
      const int slot = out % kOpen;
      const Tile t = tiles[out % kInfo];
      const int c = t.col0 + c4;
      const bool in = c < P.D;
      const uint32_t at_park = park + slot * Sh::kOpenCols;
      T *const bza = place(finished, 0), *const bzb = place(finished, 1),
              *const bv = place(finished, 2), *const bdy = place(finished, 3);
      if (!wait_phase(&summed[out & 1], (out >> 1) & 1, give_up)) break;
      // w[r] = a h[r-1], the decayed state in front of each row.
      float2 h[2], w[R][2];
      load_row(&half[slot][hw][1][c4], h[0], h[1]);
#pragma unroll
      for (int r4 = 0; r4 < R; r4 += 4) {
        float2 beta[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) ask4(at_park + (r4 + r) * 16, beta[2 * r], beta[2 * r + 1]);
        asked();
        here(beta);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float2 a[2], v[2];
          take_a(bza + (r4 + r) * kCols, bzb + (r4 + r) * kCols, a[0], a[1]);
          load_row(bv + (r4 + r) * kCols, v[0], v[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            w[r4 + r][k] = mul2(a[k], h[k]);
            h[k] = fma2(beta[2 * r + k], v[k], w[r4 + r][k]);
          }
        }
      }
      float2 rr[2], bp[2], bq[2];
      load_row(&half[slot][hw][0][c4], bp[0], bp[1]);
      load_row(&half[slot][hw][2][c4], bq[0], bq[1]);
      if (!wait_phase(&folded[out & 1], (out >> 1) & 1, give_up)) break;
      load_row(&carry[out & 1][c4], rr[0], rr[1]);
      rr[0] = fma2(bp[0], rr[0], bq[0]);
      rr[1] = fma2(bp[1], rr[1], bq[1]);
      if (kLag) {
        __syncwarp();
        mbar_arrive_if(lane == 0, &taken[out & 1]);
      }
      float2 A[2];
      load_row(&rates[out % kRing][0][c4], A[0], A[1]);
      A[0] = sub2(both(0.f), A[0]);
      A[1] = sub2(both(0.f), A[1]);
      float2 sa[2] = {both(0.f), both(0.f)}, sb[2] = {both(0.f), both(0.f)};
      const size_t o = (size_t)(t.row0 + first) * P.ld_grad + c;
      const int left = in ? t.rows - first : 0;
      float2 ahead[8];                     // the next row's gates are on their way
      ask16(at_park + (R - 1) * 16, ahead);
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        float2 a[2], v[2], dy[2], m[8];
        asked();
        here(ahead);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = ahead[i];
        if (r > 0) ask16(at_park + (r - 1) * 16, ahead);
        take_a(bza + r * kCols, bzb + r * kCols, a[0], a[1]);
        load_row(bv + r * kCols, v[0], v[1]);
        load_row(bdy + r * kCols, dy[0], dy[1]);
        float2 dza[2], dzb[2], dv[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 beta = m[k], keep = m[2 + k], sp = m[4 + k], sig = m[6 + k];
          const float2 g = add2(dy[k], rr[k]);
          dv[k] = mul2(beta, g);
          // v - alpha h times 1 - beta is keep v - a h.
          dzb[k] = mul2(dv[k], sub2(mul2(keep, v[k]), w[r][k]));
          const float2 dlog = mul2(g, w[r][k]);
          sa[k] = fma2(sp, dlog, sa[k]);
          dza[k] = mul2(A[k], mul2(sig, dlog));
          sb[k] = add2(sb[k], dza[k]);
          rr[k] = mul2(a[k], g);
        }
        const size_t at = o + (size_t)r * P.ld_grad;
        store_row_if(r < left, reinterpret_cast<T*>(P.dza) + at, dza[0], dza[1]);
        store_row_if(r < left, reinterpret_cast<T*>(P.dzb) + at, dzb[0], dzb[1]);
        store_row_if(r < left, reinterpret_cast<T*>(P.dv) + at, dv[0], dv[1]);
      }
      if (P.dh0 && t.last && hw == 0 && in)
        store_row(P.dh0 + (size_t)t.seq * P.D + c, rr[0], rr[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        sa[k] = mul2(add2(sa[k], shfl_xor2(sa[k], 16)), both(-kLn2));
        sb[k] = add2(sb[k], shfl_xor2(sb[k], 16));
      }
      if (lane < 16) {
        store_row(&sums[slot][warp][0][c4], sa[0], sa[1]);
        store_row(&sums[slot][warp][1][c4], sb[0], sb[1]);
      }
      // This tile's places were written to: order that before the copies that
      // come next.
      tc::fence_smem_to_async();
      __syncwarp();
      mbar_arrive_if(lane == 0, &empty[out % kRing]);
    }
    parked();    // where the block gives up: nothing is on its way when the columns are freed
    __syncwarp();                          // lets the last sums be written
    mbar_arrive_if(lane == 0 && it - (kOpen - 1) >= end, &paired[end % kOpen]);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == W + 1) tc::tmem_dealloc(tmem_base, Sh::kTmemCols);
  if (quit.done && tid == 0) {             // tell the other blocks
    record_status(P.status, SDM_ERR_TIMEOUT);
    atomicExch(P.chain.abort, 0u);
  }
}

// The workspace of a call, all ones.  (A memset would do, but the kernels behind
// it could then not be launched before it has ended.)
constexpr int kClearThreads = 256;
__global__ void __launch_bounds__(kClearThreads) clear_kernel(uint4* p, size_t n) {
  wait_for_stream();
  for (size_t i = (size_t)blockIdx.x * kClearThreads + threadIdx.x; i < n;
       i += (size_t)gridDim.x * kClearThreads)
    p[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
}

// Sums of the tiles' gradients of A and bias, always in the same order: 32
// channels a block, each of 32 warps every 32nd chunk, then the warps.
__global__ void __launch_bounds__(1024)
    column_sums_kernel(const Packed packed, const float* partial, int numbers, int D, float* dA,
                       float* dbias) {
  __shared__ float warps[2][32][33];
  wait_for_stream();
  if (!offsets_ok(packed)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f, b = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int n = warp; n < numbers; n += 32) {
      a += __ldg(partial + (size_t)n * 2 * D + c);
      b += __ldg(partial + (size_t)n * 2 * D + D + c);
    }
  }
  warps[0][warp][lane] = a;
  warps[1][warp][lane] = b;
  __syncthreads();
  if (warp < 2 && c < D) {
    float* out = warp == 0 ? dA : dbias;
    float sum = 0.f;
    for (int w = 0; w < 32; ++w) sum += warps[warp][w][lane];
    if (out) out[c] = sum;
  }
}

struct Args {
  RecurrenceDims d;
  RecurrenceInputs in;
  void* y;
  unsigned* status;
};

// ---------------------------------------------------------------- one token
// Four channels per thread (8 or 16 bytes of each input, 16 of the state), a
// block of 128 threads per 512 channels of a row.  The inputs and the state
// are on their way while the block looks for its slot among the earlier rows'.
// Bound by the bytes: 1024 x 3840 float32 on a pool of 1500 rows in 16.5 us (0.86 of
// the copy rate); 64 x 1920 bf16 is one launch's latency, 2.2 us.
constexpr int kStepThreads = 128;

__global__ void __launch_bounds__(kStepThreads) step_kernel(const Args P, float* state,
                                                            int n_slots, const int32_t* slots,
                                                            int parts) {
  wait_for_stream();
  const int D = P.d.D, dt = P.d.dtype;
  const long long blocks = (long long)P.d.rows * parts;
  for (long long w = blockIdx.x; w < blocks; w += gridDim.x) {
    const int row = (int)(w / parts), c = ((int)(w % parts) * kStepThreads + threadIdx.x) * 4;
    const int slot = slots ? __ldg(slots + row) : row;
    if (slot < 0) continue;
    if (slot >= n_slots) {
      if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
      continue;
    }
    const bool in = c < D;
    const size_t i = ((size_t)row * P.d.ld + c) >> 2, o = ((size_t)row * D + c) >> 2;
    float4* hp = reinterpret_cast<float4*>(state) + (((size_t)slot * D + c) >> 2);
    float4 za, zb, v, h, A = make_float4(1.f, 1.f, 1.f, 1.f), bias = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      za = load4(P.in.za, i, dt);
      zb = load4(P.in.zb, i, dt);
      v = load4(P.in.v, i, dt);
      h = *hp;
      if (P.in.A) A = __ldg(reinterpret_cast<const float4*>(P.in.A) + (c >> 2));
      if (P.in.bias) bias = __ldg(reinterpret_cast<const float4*>(P.in.bias) + (c >> 2));
    }
    if (slots) {
      bool twice = false;
      const int4* s4 = reinterpret_cast<const int4*>(slots);
      for (int k = threadIdx.x; k < row >> 2; k += kStepThreads) {
        const int4 q = __ldg(s4 + k);
        twice |= q.x == slot || q.y == slot || q.z == slot || q.w == slot;
      }
      if (threadIdx.x < (row & 3)) twice |= __ldg(slots + (row & ~3) + threadIdx.x) == slot;
      if (__syncthreads_or(twice)) {
        if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DUPLICATE_SLOT);
        continue;
      }
    }
    if (!in) continue;
    const float4 y = make_float4(step_one(h.x, za.x, zb.x, v.x, A.x, bias.x),
                                 step_one(h.y, za.y, zb.y, v.y, A.y, bias.y),
                                 step_one(h.z, za.z, zb.z, v.z, A.z, bias.z),
                                 step_one(h.w, za.w, zb.w, v.w, A.w, bias.w));
    *hp = y;
    store4(P.y, o, dt, y);
  }
}

// The same for many rows with slots, where looking through all earlier slots row
// by row would be most of the work: a block takes kManyGroup rows by 512 channels,
// puts the group's slots into a hash table in shared memory and looks all earlier
// ones up in it once.  Its kManyLanes groups of 128 threads then take a row each,
// two at a time, their loads on the way together.
// From kStepMany blocks of step_kernel on.  Measured, step_kernel and this one, us:
// bf16, 1920 channels: 2048 rows 17.9 and 24.5, 4096 33.5 and 30.6, 16384 138 and 122,
// 70000 1468 and 594 (without slots 441); bf16, 256 channels: 8192 rows 13.8 and 20.0,
// 16384 32.2 and 32.9, 70000 336 and 157 (74).  With 128 rows a group 24 us at least, and
// 559 and 154 in the last; four rows at a time are short of registers.
constexpr int kStepMany = 16384;
constexpr int kManyGroup = 64, kManyLanes = 4, kManyThreads = kManyLanes * kStepThreads;
constexpr int kManyTable = 512, kManyAhead = 2;

__device__ __forceinline__ int place_of(int slot) {
  return (int)((unsigned)slot * 2654435769u >> 23);          // golden ratio, 9 bits
}

__global__ void __launch_bounds__(kManyThreads) step_many_kernel(const Args P, float* state,
                                                                 int n_slots, const int32_t* slots,
                                                                 int parts) {
  static_assert(kManyTable == 512 && kManyGroup < kManyTable, "place_of gives 9 bits");
  wait_for_stream();
  __shared__ int key[kManyTable], first[kManyTable], seen[kManyTable], group[kManyGroup];
  const int D = P.d.D, dt = P.d.dtype, tid = threadIdx.x, lane = tid / kStepThreads;
  const long long blocks = ((long long)P.d.rows + kManyGroup - 1) / kManyGroup * parts;
  for (long long w = blockIdx.x; w < blocks; w += gridDim.x) {
    const int row0 = (int)(w / parts) * kManyGroup, n = min(kManyGroup, P.d.rows - row0);
    const int c = ((int)(w % parts) * kStepThreads + tid % kStepThreads) * 4;
    for (int i = tid; i < kManyTable; i += kManyThreads) {
      key[i] = -1;
      first[i] = kManyGroup;
      seen[i] = 0;
    }
    __syncthreads();
    int slot = tid < n ? __ldg(slots + row0 + tid) : -1, at = 0;
    if (slot >= n_slots) {
      record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
      slot = -1;
    }
    if (slot >= 0) {                       // ends: the table has more places than the group rows
      at = place_of(slot);
      for (int k; (k = atomicCAS(&key[at], -1, slot)) != -1 && k != slot;) at = (at + 1) % kManyTable;
      atomicMin(&first[at], tid);
    }
    __syncthreads();
    const int4* s4 = reinterpret_cast<const int4*>(slots);
#pragma unroll 4
    for (int k = tid; k < row0 / 4; k += kManyThreads) {
      const int4 q = __ldg(s4 + k);
      const int e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        int p = place_of(e[j]), there;
        while ((there = key[p]) != -1 && there != e[j]) p = (p + 1) % kManyTable;
        if (there != -1) seen[p] = 1;      // (a negative slot, were it -1, finds an empty place)
      }
    }
    __syncthreads();
    if (slot >= 0 && (seen[at] || first[at] != tid)) {
      record_status(P.status, SDM_ERR_DUPLICATE_SLOT);
      slot = -1;
    }
    if (tid < kManyGroup) group[tid] = slot;
    __syncthreads();
    if (c < D) {
      float4 A = make_float4(1.f, 1.f, 1.f, 1.f), bias = make_float4(0.f, 0.f, 0.f, 0.f);
      if (P.in.A) A = __ldg(reinterpret_cast<const float4*>(P.in.A) + (c >> 2));
      if (P.in.bias) bias = __ldg(reinterpret_cast<const float4*>(P.in.bias) + (c >> 2));
      for (int i0 = lane; i0 < n; i0 += kManyLanes * kManyAhead) {
        float4 za[kManyAhead], zb[kManyAhead], v[kManyAhead], h[kManyAhead];
        float4* hp[kManyAhead];
#pragma unroll
        for (int j = 0; j < kManyAhead; ++j) {
          const int r = i0 + j * kManyLanes, s = r < n ? group[r] : -1;
          hp[j] = s < 0 ? nullptr : reinterpret_cast<float4*>(state) + (((size_t)s * D + c) >> 2);
          if (s < 0) continue;
          const size_t i = ((size_t)(row0 + r) * P.d.ld + c) >> 2;
          za[j] = load4(P.in.za, i, dt);
          zb[j] = load4(P.in.zb, i, dt);
          v[j] = load4(P.in.v, i, dt);
          h[j] = *hp[j];
        }
#pragma unroll
        for (int j = 0; j < kManyAhead; ++j) {
          if (!hp[j]) continue;
          const float4 y = make_float4(step_one(h[j].x, za[j].x, zb[j].x, v[j].x, A.x, bias.x),
                                       step_one(h[j].y, za[j].y, zb[j].y, v[j].y, A.y, bias.y),
                                       step_one(h[j].z, za[j].z, zb[j].z, v[j].z, A.z, bias.z),
                                       step_one(h[j].w, za[j].w, zb[j].w, v[j].w, A.w, bias.w));
          *hp[j] = y;
          store4(P.y, ((size_t)(row0 + i0 + j * kManyLanes) * D + c) >> 2, dt, y);
        }
      }
    }
    __syncthreads();                       // the tables are filled again
  }
}

}  // namespace

namespace {

constexpr size_t kHeaderBytes = 256;

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
int col_tiles_of(int D) { return (D + kCols - 1) / kCols; }

// Bytes of a call whose chunks have L rows: the header, then the pairs.
size_t chain_bytes(const RecurrenceDims& d, int L) {
  return kHeaderBytes + round256((size_t)chunk_numbers(d.rows, d.n_seq, L) * d.D * 8);
}

Chain chain_in(void* workspace) {
  char* w = static_cast<char*>(workspace);
  return Chain{reinterpret_cast<unsigned*>(w), reinterpret_cast<unsigned*>(w + 128),
               reinterpret_cast<float*>(w + kHeaderBytes)};
}

cudaError_t clear_chain(void* workspace, const RecurrenceDims& d, int L, cudaStream_t stream) {
  const size_t n = chain_bytes(d, L) / 16;
  const size_t most = (size_t)8 * device_limits().sms, want = (n + kClearThreads - 1) / kClearThreads;
  return launch_behind(clear_kernel, (unsigned)(want < most ? want : most), kClearThreads, 0, stream,
                       static_cast<uint4*>(workspace), n);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Map of a [rows, D] tensor with rows `ld` elements apart, in boxes of
// box_rows x 64 channels.
bool make_map(CUtensorMap* map, const void* base, int dtype, int rows, int D, long long ld,
              int box_rows) {
  const EncodeTiled f = encoder();
  if (!f) return false;
  const cuuint64_t e = dtype == SDM_BF16 ? 2 : 4;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * e};
  const cuuint32_t box[2] = {(cuuint32_t)kCols, (cuuint32_t)box_rows}, one[2] = {1, 1};
  return f(map, dtype == SDM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
           2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiles of a call: all chunk numbers where the lengths are on the device,
// else the chunks there are.
unsigned tiles_of(const RecurrenceDims& d, bool offsets, int L) {
  long long n = chunk_numbers(d.rows, d.n_seq, L);
  if (!offsets) {
    const long long per = (d.rows / d.n_seq + L - 1) / L;
    n = (per > 0 ? per : 1) * d.n_seq;
  }
  return (unsigned)(n * col_tiles_of(d.D));
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

template <typename T>
cudaError_t forward_as(const RecurrenceDims& d, const RecurrenceInputs& in, const float* h0,
                       void* y, float* hT, float* states, void* workspace, unsigned* status,
                       cudaStream_t stream) {
  using Sh = ForwardShape<T>;
  constexpr int L = Sh::L;
  ForwardArgs P;
  if (d.rows > 0 && (!make_map(&P.za, in.za, d.dtype, d.rows, d.D, d.ld, L) ||
                     !make_map(&P.zb, in.zb, d.dtype, d.rows, d.D, d.ld, L) ||
                     !make_map(&P.v, in.v, d.dtype, d.rows, d.D, d.ld, L)))
    return cudaErrorInvalidValue;
  P.packed = Packed{in.offsets, d.n_seq, d.rows};
  P.A = in.A;
  P.bias = in.bias;
  P.h0 = h0;
  P.y = y;
  P.hT = hT;
  P.states = states;
  P.chain = chain_in(workspace);
  P.D = d.D;
  P.col_tiles = col_tiles_of(d.D);
  P.tiles = tiles_of(d, in.offsets != nullptr, L);
  P.status = status;
  P.limit_us = api_recurrence_wait_us();
  const auto kernel = forward_kernel<T>;
  static std::atomic<bool> allowed[64];   // false
  cudaError_t e = allow_smem(kernel, Sh::kSmem, allowed);
  if (e == cudaSuccess) e = clear_chain(workspace, d, L, stream);
  if (e != cudaSuccess) return e;
  const unsigned most = (unsigned)(2 * device_limits().sms);
  return launch_behind(kernel, P.tiles < most ? P.tiles : most, kThreads, Sh::kSmem, stream, P);
}

}  // namespace

size_t recurrence_workspace_bytes(const RecurrenceDims& d) {
  const bool b16 = d.dtype == SDM_BF16;
  const size_t fwd = chain_bytes(d, b16 ? ForwardShape<__nv_bfloat16>::L : ForwardShape<float>::L);
  const int L = b16 ? kStateRows<__nv_bfloat16> : kStateRows<float>;
  const size_t back = chain_bytes(d, L) + (size_t)chunk_numbers(d.rows, d.n_seq, L) * 2 * d.D * 4;
  return back > fwd ? back : fwd;
}

size_t recurrence_states_bytes(const RecurrenceDims& d) {
  const int L = d.dtype == SDM_BF16 ? kStateRows<__nv_bfloat16> : kStateRows<float>;
  return (size_t)chunk_numbers(d.rows, d.n_seq, L) * d.D * sizeof(float);
}

cudaError_t launch_recurrence_forward(const RecurrenceDims& d, const RecurrenceInputs& in,
                                      const float* h0, void* y, float* hT, float* states,
                                      void* workspace, unsigned* status, cudaStream_t stream) {
  if (d.dtype == SDM_BF16)
    return forward_as<__nv_bfloat16>(d, in, h0, y, hT, states, workspace, status, stream);
  return forward_as<float>(d, in, h0, y, hT, states, workspace, status, stream);
}

namespace {

// Whether the backward pass finishes a tile one tile later.  A chain is a
// sequence's 64 channels; with few of them many of the tiles at work are of one
// chain and wait for folds, with many the lag only takes room.  Measured, at once
// and later, 65536 x 512 bf16: 8 chains 206 and 124 us, 32 150 and 122, 64 125 and
// 122, 128 110 and 123; 32768 x 1024 float32: 16 chains 261 and 186, 64 187 and
// 183, 128 167 and 183.  (Sequences' lengths are not known here: one long one among
// many short ones is taken for many chains.)
bool lags(const RecurrenceDims& d) {
  return 2 * (long long)d.n_seq * col_tiles_of(d.D) <= device_limits().sms;
}

template <typename T, bool kLag>
cudaError_t backward_as(const RecurrenceDims& d, const RecurrenceInputs& in, const float* states,
                        const void* dy, const float* dhT, void* dza, void* dzb, void* dv,
                        float* dA, float* dbias, float* dh0, void* workspace, unsigned* status,
                        cudaStream_t stream) {
  using Sh = BackwardShape<T, kLag>;
  constexpr int L = Sh::L;
  BackwardArgs P;
  if (d.rows > 0 && (!make_map(&P.za, in.za, d.dtype, d.rows, d.D, d.ld, L) ||
                     !make_map(&P.zb, in.zb, d.dtype, d.rows, d.D, d.ld, L) ||
                     !make_map(&P.v, in.v, d.dtype, d.rows, d.D, d.ld, L) ||
                     !make_map(&P.dy, dy, d.dtype, d.rows, d.D, d.D, L)))
    return cudaErrorInvalidValue;
  P.packed = Packed{in.offsets, d.n_seq, d.rows};
  P.A = in.A;
  P.bias = in.bias;
  P.states = states;
  P.dhT = dhT;
  P.dza = dza;
  P.dzb = dzb;
  P.dv = dv;
  P.dh0 = dh0;
  P.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + chain_bytes(d, L));
  P.chain = chain_in(workspace);
  P.D = d.D;
  P.col_tiles = col_tiles_of(d.D);
  P.ld_grad = d.ld_grad;
  P.tiles = tiles_of(d, in.offsets != nullptr, L);
  P.status = status;
  P.limit_us = api_recurrence_wait_us();
  const auto kernel = backward_kernel<T, kLag>;
  static std::atomic<bool> allowed[64];   // false
  cudaError_t e = allow_smem(kernel, Sh::kSmem, allowed);
  if (e == cudaSuccess) e = clear_chain(workspace, d, L, stream);
  if (e != cudaSuccess) return e;
  const unsigned most = (unsigned)(Sh::kBlocks * device_limits().sms);
  e = launch_behind(kernel, P.tiles < most ? P.tiles : most, kBackThreads, Sh::kSmem, stream, P);
  if (e != cudaSuccess || (!dA && !dbias)) return e;
  return launch_behind(column_sums_kernel, (unsigned)(d.D + 31) / 32, 1024, 0, stream, P.packed,
                       (const float*)P.partial, (int)(P.tiles / P.col_tiles), d.D, dA, dbias);
}

}  // namespace

cudaError_t launch_recurrence_backward(const RecurrenceDims& d, const RecurrenceInputs& in,
                                       const float* states, const void* dy, const float* dhT,
                                       void* dza, void* dzb, void* dv, float* dA, float* dbias,
                                       float* dh0, void* workspace, unsigned* status,
                                       cudaStream_t stream) {
  if (d.n_seq == 0) {                      // sums over nothing
    cudaError_t e = cudaSuccess;
    if (dA) e = cudaMemsetAsync(dA, 0, (size_t)d.D * 4, stream);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)d.D * 4, stream);
    return e;
  }
  const bool b16 = d.dtype == SDM_BF16;
  const auto run = lags(d) ? (b16 ? backward_as<__nv_bfloat16, true> : backward_as<float, true>)
                           : (b16 ? backward_as<__nv_bfloat16, false> : backward_as<float, false>);
  return run(d, in, states, dy, dhT, dza, dzb, dv, dA, dbias, dh0, workspace, status, stream);
}

cudaError_t launch_recurrence_step(const RecurrenceDims& d, const RecurrenceInputs& in,
                                   float* state, int n_slots, const int32_t* slots, void* y,
                                   unsigned* status, cudaStream_t stream) {
  Args P{};
  P.d = d;
  P.in = in;
  P.y = y;
  P.status = status;
  const int parts = (d.D / 4 + kStepThreads - 1) / kStepThreads;
  const long long rows = (long long)d.rows * parts;           // by 512 channels
  const bool many = slots && rows >= kStepMany;
  const long long want = many ? ((long long)d.rows + kManyGroup - 1) / kManyGroup * parts : rows;
  const unsigned blocks = (unsigned)(want < (1 << 20) ? want : (1 << 20));
  if (many)
    return launch_behind(step_many_kernel, blocks, kManyThreads, 0, stream, P, state, n_slots, slots, parts);
  return launch_behind(step_kernel, blocks, kStepThreads, 0, stream, P, state, n_slots, slots, parts);
}

}  // namespace sdm
