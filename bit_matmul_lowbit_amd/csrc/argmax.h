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

// One step of wave_max: the larger of the own key and the one that the DPP
// control brings from another lane (0, below every key, where it brings none).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_max(uint64_t k) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)k, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(k >> 32), CTRL, ROWS, 0xF, false);
  const uint64_t o = ((uint64_t)hi << 32) | lo;
  return o > k ? o : k;
}

// largest key of the wave, in every lane
__device__ __forceinline__ uint64_t wave_max(uint64_t k) {
  k = dpp_max<0x111, 0xF>(k);  // row_shr:1
  k = dpp_max<0x112, 0xF>(k);  // row_shr:2
  k = dpp_max<0x114, 0xF>(k);  // row_shr:4
  k = dpp_max<0x118, 0xF>(k);  // row_shr:8: lane 15 of each row of 16 has the row's
  k = dpp_max<0x142, 0xA>(k);  // row_bcast:15 into rows 1 and 3
  k = dpp_max<0x143, 0xC>(k);  // row_bcast:31 into rows 2 and 3: lane 63 has the wave's
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k >> 32), 63);
  return ((uint64_t)hi << 32) | lo;
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
