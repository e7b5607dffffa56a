// The 4-bit cache as the kernels see it (layout in include/lowbit.h): a page
// holds `page` tokens of every head, and of each head its K codes, K params, V
// codes and V params, one after another.
#pragma once
#include "common.h"

namespace lowbit {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// byte offsets inside the part of a page that belongs to one head
struct KvHead {
  int code_bytes;   // K codes; as many V codes
  int param_bytes;  // K params; as many V params
  __host__ __device__ constexpr KvHead(int page, int d) : code_bytes(page * d / 2), param_bytes(page * d / 8) {}
  __host__ __device__ constexpr int k_params() const { return code_bytes; }
  __host__ __device__ constexpr int v_codes() const { return code_bytes + param_bytes; }
  __host__ __device__ constexpr int v_params() const { return 2 * code_bytes + param_bytes; }
  __host__ __device__ constexpr int bytes() const { return 2 * (code_bytes + param_bytes); }
};

// The byte of a V dword (one pair of values of four tokens) that token t of
// the four has: 0, 2, 1, 3, so that the two halves of the dword hold tokens
// that become neighbours when nibbles are spread over FP16 pairs.
__device__ __forceinline__ int v_byte(int t) { return ((t & 1) << 1) | (t >> 1); }

// Nibbles N and N + 4 of w as the FP16 pair 1 + code / 16: the code is put at
// the top of the mantissa of 1.0 (no conversion and no subtraction).  `ones` is a
// pair of 1.0 in a register (ones_of), which makes mask and insertion one
// instruction: it takes one constant from outside the vector registers, not two.
__device__ __forceinline__ uint32_t ones_of() {
  uint32_t ones;
  __asm__("v_mov_b32 %0, 0x3c003c00" : "=v"(ones));
  return ones;
}
template <int N>
__device__ __forceinline__ f16x2 nibbles(uint32_t w, uint32_t ones) {
  constexpr int kShift = 6 - 4 * N;  // to bits 6..9 of both halves
  const uint32_t s = kShift >= 0 ? w << (kShift & 31) : w >> (-kShift & 31);
  return __builtin_bit_cast(f16x2, (s & 0x03C003C0u) | ones);
}

__device__ __forceinline__ f16x2 fma2(f16x2 x, f16x2 a, f16x2 b) { return __builtin_elementwise_fma(x, a, b); }

}  // namespace lowbit
