// Keys of the top-1 searches (lowbit_argmax, lowbit_logits_process) and their
// reduction over a work-group of 256 threads.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lowbit {

// argmax: key(v, i) = (ordered bits of v) << 32 | (2^32 - 1 - i), so the
// largest key is the largest value and, among equal values, the lowest
// index.  The ordered bits map the IEEE order onto unsigned order (negative:
// all bits flipped, positive: sign bit set); a NaN with a clear sign bit
// sorts above +inf, so NaN wins as it does for numpy's and torch's argmax.

__device__ __forceinline__ uint32_t ordered_bits(float v) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  if (__builtin_isnan(v)) u = 0x7FC00000u;  // every NaN the same, above +inf
  if (v == 0.0f) u = 0u;                    // -0 and +0 are equal values
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint64_t argmax_pack(uint32_t ordered, int64_t i) {
  return ((uint64_t)ordered << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)i);
}

__device__ __forceinline__ uint64_t argmax_key(float v, int64_t i) {
  return argmax_pack(ordered_bits(v), i);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t k) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor(k, off, 64);
    k = o > k ? o : k;
  }
  return k;
}

// block-wide maximum of one key per thread (256 threads)
__device__ __forceinline__ uint64_t block_max(uint64_t k, uint64_t* red) {
  k = wave_max(k);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = k;
  __syncthreads();
  uint64_t m = red[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) m = red[w] > m ? red[w] : m;
  __syncthreads();
  return m;
}

}  // namespace lowbit
