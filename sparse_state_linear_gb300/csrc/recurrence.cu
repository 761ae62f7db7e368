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
#include "common.cuh"
#include "internal.h"

namespace sdm {
namespace {

constexpr int kChunk = 128;   // rows between saved states

// ------------------------------------------------------------------- gates
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

constexpr float kLog2e = 1.4426950408889634f;

// ln(1 + e) for e in [0, 1]: e times the degree-9 polynomial that interpolates
// ln(1 + e) / e at the Chebyshev points of [0, 1].  Relative error 1.3e-7 for
// every e, which the logarithm instruction (an absolute bound) does not give
// where the gate hardly decays.
__device__ __forceinline__ float log1p_unit(float e) {
  float p = -0.00317605701f;
  p = fmaf(p, e, 0.0195425265f);
  p = fmaf(p, e, -0.0563736111f);
  p = fmaf(p, e, 0.105436236f);
  p = fmaf(p, e, -0.152696669f);
  p = fmaf(p, e, 0.196632743f);
  p = fmaf(p, e, -0.249516159f);
  p = fmaf(p, e, 0.333297104f);
  p = fmaf(p, e, -0.499998927f);
  p = fmaf(p, e, 1.f);
  return p * e;
}

struct Gate {
  float sp;      // softplus(za + bias)
  float sig;     // sigmoid(za + bias)
  float alpha;   // exp(-A sp)
  float beta;    // sigmoid(zb)
  float keep;    // 1 - beta, to full relative precision
};

__device__ __forceinline__ Gate make_gate(float za, float zb, float A, float bias) {
  Gate g;
  const float x = za + bias;
  const float e = ex2(-fabsf(x) * kLog2e);
  g.sp = fmaxf(x, 0.f) + log1p_unit(e);
  g.alpha = ex2(-A * kLog2e * g.sp);
  const float r = rcp(1.f + e);
  g.sig = x >= 0.f ? r : e * r;
  const float eb = ex2(-fabsf(zb) * kLog2e);
  const float rb = rcp(1.f + eb);
  g.beta = zb >= 0.f ? rb : eb * rb;
  g.keep = zb >= 0.f ? eb * rb : rb;
  return g;
}

__device__ __forceinline__ void store_scalar(void* base, size_t i, int dt, float x) {
  if (dt == SDM_F32)
    reinterpret_cast<float*>(base)[i] = x;
  else
    reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(x);
}

__device__ __forceinline__ float step_one(float h, float za, float zb, float v, float A,
                                          float bias) {
  const Gate g = make_gate(za, zb, A, bias);
  return fmaf(g.keep * g.alpha, h, g.beta * v);
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

// ------------------------------------------------------------------ packing
// Chunk c of sequence s (first row o) has number o / kChunk + s + c: distinct
// for all chunks of all sequences, below rows / kChunk + n_seq, and growing
// with s and c.
__host__ __device__ inline int chunk_numbers(int rows, int n_seq) { return rows / kChunk + n_seq; }

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

struct Args {
  RecurrenceDims d;
  RecurrenceInputs in;
  Packed packed;
  const float* h0;
  void* y;
  float* hT;
  float* states;
  const void* dy;
  const float* dhT;
  void* dza;
  void* dzb;
  void* dv;
  float* dh0;
  float* partial;
  unsigned* status;
};

// One thread per channel and sequence, one row after the other.
__global__ void __launch_bounds__(128) forward_kernel(const Args P) {
  if (!offsets_ok(P.packed)) {
    if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    return;
  }
  const int c = blockIdx.x * blockDim.x + threadIdx.x, s = blockIdx.y, D = P.d.D, dt = P.d.dtype;
  if (c >= D) return;
  const float A = P.in.A ? P.in.A[c] : 1.f, bias = P.in.bias ? P.in.bias[c] : 0.f;
  const int t0 = P.packed.begin(s), t1 = P.packed.begin(s + 1);
  float h = P.h0 ? P.h0[(size_t)s * D + c] : 0.f;
  for (int t = t0; t < t1; ++t) {
    if (P.states && (t - t0) % kChunk == 0)
      P.states[(size_t)(t0 / kChunk + s + (t - t0) / kChunk) * D + c] = h;
    const size_t i = (size_t)t * P.d.ld + c;
    const Gate g = make_gate(load_scalar(P.in.za, i, dt), load_scalar(P.in.zb, i, dt), A, bias);
    h = fmaf(g.keep * g.alpha, h, g.beta * load_scalar(P.in.v, i, dt));
    store_scalar(P.y, (size_t)t * D + c, dt, h);
  }
  if (P.hT) P.hT[(size_t)s * D + c] = h;
}

// As above from the last chunk to the first: the states before the chunk's
// rows again from the saved one, then the gradients.
__global__ void __launch_bounds__(32) backward_kernel(const Args P) {
  __shared__ float hs[kChunk][32];
  if (!offsets_ok(P.packed)) {
    if (threadIdx.x == 0) record_status(P.status, SDM_ERR_DEVICE_BOUNDS);
    return;
  }
  const int c = blockIdx.x * 32 + threadIdx.x, s = blockIdx.y, D = P.d.D, dt = P.d.dtype;
  if (c >= D) return;
  const float A = P.in.A ? P.in.A[c] : 1.f, bias = P.in.bias ? P.in.bias[c] : 0.f;
  const int t0 = P.packed.begin(s), t1 = P.packed.begin(s + 1);
  float r = P.dhT ? P.dhT[(size_t)s * D + c] : 0.f, dA = 0.f, db = 0.f;
  for (int k = (t1 - t0 + kChunk - 1) / kChunk - 1; k >= 0; --k) {
    const int b = t0 + k * kChunk, e = b + kChunk < t1 ? b + kChunk : t1;
    float h = P.states[(size_t)(t0 / kChunk + s + k) * D + c];
    for (int t = b; t < e; ++t) {
      hs[t - b][threadIdx.x] = h;
      const size_t i = (size_t)t * P.d.ld + c;
      const Gate g = make_gate(load_scalar(P.in.za, i, dt), load_scalar(P.in.zb, i, dt), A, bias);
      h = fmaf(g.keep * g.alpha, h, g.beta * load_scalar(P.in.v, i, dt));
    }
    for (int t = e - 1; t >= b; --t) {
      const size_t i = (size_t)t * P.d.ld + c, o = (size_t)t * P.d.ld_grad + c;
      const Gate g = make_gate(load_scalar(P.in.za, i, dt), load_scalar(P.in.zb, i, dt), A, bias);
      const float before = hs[t - b][threadIdx.x];
      const float gr = load_scalar(P.dy, (size_t)t * D + c, dt) + r;
      const float dlog = gr * g.keep * g.alpha * before;
      const float dza = -A * g.sig * dlog;
      r = g.keep * g.alpha * gr;
      dA -= g.sp * dlog;
      db += dza;
      store_scalar(P.dza, o, dt, dza);
      store_scalar(P.dzb, o, dt,
                   gr * (load_scalar(P.in.v, i, dt) - g.alpha * before) * g.beta * g.keep);
      store_scalar(P.dv, o, dt, g.beta * gr);
    }
  }
  if (P.dh0) P.dh0[(size_t)s * D + c] = r;
  P.partial[(size_t)s * 2 * D + c] = dA;
  P.partial[(size_t)s * 2 * D + D + c] = db;
}

__global__ void reduce_kernel(const Args P, float* dA, float* dbias) {
  if (!offsets_ok(P.packed)) return;
  const int c = blockIdx.x * blockDim.x + threadIdx.x, D = P.d.D;
  if (c >= D) return;
  float a = 0.f, b = 0.f;
  for (int s = 0; s < P.d.n_seq; ++s) {
    a += P.partial[(size_t)s * 2 * D + c];
    b += P.partial[(size_t)s * 2 * D + D + c];
  }
  if (dA) dA[c] = a;
  if (dbias) dbias[c] = b;
}

// ---------------------------------------------------------------- one token
// Four channels per thread (8 or 16 bytes of each input, 16 of the state), a
// block of 128 threads per 512 channels of a row.  The inputs and the state
// are on their way while the block looks for its slot among the earlier rows'.
constexpr int kStepThreads = 128;

__global__ void __launch_bounds__(kStepThreads) step_kernel(const Args P, float* state,
                                                            int n_slots, const int32_t* slots,
                                                            int parts) {
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

}  // namespace

size_t recurrence_workspace_bytes(const RecurrenceDims& d) {
  return (size_t)(d.n_seq + 1) * 2 * d.D * sizeof(float);
}

size_t recurrence_states_bytes(const RecurrenceDims& d) {
  return (size_t)chunk_numbers(d.rows, d.n_seq) * d.D * sizeof(float);
}

cudaError_t launch_recurrence_forward(const RecurrenceDims& d, const RecurrenceInputs& in,
                                      const float* h0, void* y, float* hT, float* states,
                                      void* workspace, unsigned* status, cudaStream_t stream) {
  (void)workspace;
  Args P{};
  P.d = d;
  P.in = in;
  P.packed = Packed{in.offsets, d.n_seq, d.rows};
  P.h0 = h0;
  P.y = y;
  P.hT = hT;
  P.states = states;
  P.status = status;
  forward_kernel<<<dim3((d.D + 127) / 128, d.n_seq), 128, 0, stream>>>(P);
  return cudaGetLastError();
}

cudaError_t launch_recurrence_backward(const RecurrenceDims& d, const RecurrenceInputs& in,
                                       const float* states, const void* dy, const float* dhT,
                                       void* dza, void* dzb, void* dv, float* dA, float* dbias,
                                       float* dh0, void* workspace, unsigned* status,
                                       cudaStream_t stream) {
  Args P{};
  P.d = d;
  P.in = in;
  P.packed = Packed{in.offsets, d.n_seq, d.rows};
  P.states = const_cast<float*>(states);
  P.dy = dy;
  P.dhT = dhT;
  P.dza = dza;
  P.dzb = dzb;
  P.dv = dv;
  P.dh0 = dh0;
  P.partial = static_cast<float*>(workspace);
  P.status = status;
  if (d.n_seq > 0) backward_kernel<<<dim3((d.D + 31) / 32, d.n_seq), 32, 0, stream>>>(P);
  if (d.n_seq == 0) P.packed.offsets = nullptr;
  if (dA || dbias) reduce_kernel<<<(d.D + 127) / 128, 128, 0, stream>>>(P, dA, dbias);
  return cudaGetLastError();
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
  const long long want = (long long)d.rows * parts;
  const unsigned blocks = (unsigned)(want < (1 << 20) ? want : (1 << 20));
  step_kernel<<<blocks, kStepThreads, 0, stream>>>(P, state, n_slots, slots, parts);
  return cudaGetLastError();
}

}  // namespace sdm
