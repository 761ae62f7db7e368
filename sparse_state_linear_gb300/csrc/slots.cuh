// slots.cuh -- the rows of a pool of states that a batch of single tokens steps:
// which of a block's tokens step their slot.
//
// A negative slot is padding, one at or beyond n_slots is out of bounds, and of
// the tokens that name one slot only the first steps it; what is skipped for the
// last two reasons is recorded.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace sdm {

// kGroup tokens from row0 on (n of them valid).  `own[i]` is token i's slot or -1.
// All threads of the block call it; it ends with a barrier.  A group is looked up
// in a hash table of its slots, by all earlier slots once; a single token compares
// its own with them.
template <int kGroup, int kThreads>
struct SlotTable {
  static constexpr int kPlaces = kGroup == 1 ? 1 : 8 * kGroup;
  int own[kGroup];
  int key[kPlaces], first[kPlaces], seen[kPlaces];

  static __device__ __forceinline__ int place_of(int slot) {
    return (int)(((unsigned)slot * 2654435769u >> 16) & (unsigned)(kPlaces - 1));   // golden ratio
  }

  __device__ __forceinline__ void find(const int32_t* slots, int row0, int n, int n_slots,
                                       unsigned* status) {
    static_assert((kPlaces & (kPlaces - 1)) == 0 && kGroup <= kThreads, "");
    const int tid = threadIdx.x;
    const int4* s4 = reinterpret_cast<const int4*>(slots);
    int slot = -1;
    if (tid < n) {
      slot = slots ? __ldg(slots + row0 + tid) : row0 + tid;
      if (slot >= n_slots) {
        record_status(status, SDM_ERR_DEVICE_BOUNDS);
        slot = -1;
      }
    }
    if (!slots) {
      if (tid < kGroup) own[tid] = slot;
      __syncthreads();
      return;
    }
    if constexpr (kGroup == 1) {
      const int mine = __ldg(slots + row0);
      bool twice = false;
      if (mine >= 0) {
        for (int k = tid; k < row0 >> 2; k += kThreads) {
          const int4 q = __ldg(s4 + k);
          twice |= q.x == mine || q.y == mine || q.z == mine || q.w == mine;
        }
        if (tid < (row0 & 3)) twice |= __ldg(slots + (row0 & ~3) + tid) == mine;
      }
      twice = __syncthreads_or(twice);
      if (tid == 0) {
        if (twice && slot >= 0) record_status(status, SDM_ERR_DUPLICATE_SLOT);
        own[0] = twice ? -1 : slot;
      }
      __syncthreads();
    } else {
      for (int i = tid; i < kPlaces; i += kThreads) {
        key[i] = -1;
        first[i] = kGroup;
        seen[i] = 0;
      }
      __syncthreads();
      int at = 0;
      if (slot >= 0) {                       // ends: there are more places than tokens
        at = place_of(slot);
        for (int k; (k = atomicCAS(&key[at], -1, slot)) != -1 && k != slot;) at = (at + 1) % kPlaces;
        atomicMin(&first[at], tid);
      }
      __syncthreads();
#pragma unroll 4
      for (int k = tid; k < row0 / 4; k += kThreads) {          // row0 is a multiple of kGroup
        const int4 q = __ldg(s4 + k);
        const int e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          int p = place_of(e[j]), there;
          while ((there = key[p]) != -1 && there != e[j]) p = (p + 1) % kPlaces;
          if (there != -1) seen[p] = 1;      // (a negative slot finds an empty place)
        }
      }
      __syncthreads();
      if (slot >= 0 && (seen[at] || first[at] != tid)) {
        record_status(status, SDM_ERR_DUPLICATE_SLOT);
        slot = -1;
      }
      if (tid < kGroup) own[tid] = slot;
      __syncthreads();
    }
  }
};

// Tokens a block takes, f(group): one up to `most` blocks of one token each, then 16, and
// 64 where looking through all earlier slots is much of the work.  Measured, bf16, 1920
// channels, us with one and with 16 (64) tokens a block: convolution, 512 rows 12.3 and
// 6.8, 4000 67 and 24, 16384 304 and 107 (128 with 16); scan of 16 states, 256 rows 12.1
// and 14.2, 1024 50 and 50, 4360 209 and 192, 16400 865 and 711.  For the scan the switch
// (16384 blocks) is where both take the same; for the convolution (2048 blocks, 512 rows of
// 1920 channels) 16 tokens are well ahead there, and from where on they are was not measured.
template <class F>
cudaError_t with_group(int rows, long long blocks, int most, F f) {
  if (blocks < most && rows < 4096) return f(std::integral_constant<int, 1>{});
  if (rows < 16384) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 64>{});
}

}  // namespace sdm
