// packing.cuh -- sequences packed into the rows of one tensor, and the chunks of
// L rows that they are cut into.
//
// Chunk c (of L rows) of sequence s whose first row is o has number
// o / L + s + c: distinct for all chunks of all sequences, below
// rows / L + n_seq, and growing with s and c.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace sdm {

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
__device__ inline bool offsets_ok(const Packed& P) {
  if (!P.offsets) return true;
  bool bad = false;
  for (int s = threadIdx.x; s <= P.n_seq; s += blockDim.x) {
    const int o = P.begin(s);
    bad |= o < 0 || o > P.rows || (s > 0 && o < P.begin(s - 1));
  }
  return !__syncthreads_or(bad);
}

// The sequence a chunk number belongs to (a whole warp calls it): the last s
// with base(s) = begin(s) / L + s <= number, or -1.
__device__ __forceinline__ int sequence_of(const Packed& P, int L, int number) {
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

}  // namespace sdm
