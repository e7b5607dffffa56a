// Eight neighbouring elements of a row of FP32, FP16 or BF16: loaded as they
// lie in memory, widened, stored.
#pragma once
#include "common.h"

namespace lowbit {

// 8 elements as they lie in memory, S bytes each
template <int S>
struct Raw8 {
  uint32_t d[2 * S];
};

// Eight elements from p[at] on: 16-byte loads at any element alignment
template <int S>
__device__ __forceinline__ Raw8<S> load8(const void* p, int64_t at) {
  Raw8<S> r;
  __builtin_memcpy(&r, static_cast<const char*>(p) + at * S, sizeof(r));
  return r;
}

template <int S>
__device__ __forceinline__ void widen(const Raw8<S>& r, int type, float (&v)[8]) {
  if constexpr (S == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_bit_cast(float, r.d[j]);
  } else if (type == 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.d[j >> 1] >> ((j & 1) * 16)));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = __builtin_bit_cast(float, (j & 1) ? r.d[j >> 1] & 0xFFFF0000u : r.d[j >> 1] << 16);
  }
}

// all eight, or those from `skip` on
template <typename T>
__device__ __forceinline__ void store8_as(void* p, int64_t at, int skip, const float (&v)[8]) {
  T o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = (T)v[j];
  T* out = static_cast<T*>(p) + at;
  if (skip == 0) {
    __builtin_memcpy(out, o, sizeof(o));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= skip) out[j] = o[j];
  }
}

__device__ __forceinline__ void store8(void* p, int type, int64_t at, int skip, const float (&v)[8]) {
  if (type == 1) store8_as<float>(p, at, skip, v);
  else if (type == 2) store8_as<_Float16>(p, at, skip, v);
  else store8_as<bf16_t>(p, at, skip, v);
}

}  // namespace lowbit
