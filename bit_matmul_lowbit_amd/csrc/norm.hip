// The norms around a block, its gate and the residual add, in one launch:
//   u = post(y),  r' = r + scale * gate * u,  x = pre(r')
// with post and pre a root-mean-square or a layer norm, or none.
//
// [P2] 7minutos.es, "PrismML lanza Bonsai 27B ...", "Como funciona la
//      compresion": the projections of a block are low-bit; the norms and the
//      residual stream between them are not.
//
// A row of y and r is read once and held in registers (8 elements per thread
// and step, raw, as they were loaded) while its sums are formed: the
// deviations of a layer norm are summed in a second sweep over the registers,
// which keeps a small variance beside a large mean.  A row belongs to one
// work-group, or to one wave where rows are short and many; rows longer than the
// registers of a work-group hold are read again for every sum.
//
// What bounds it: memory.  16384 x 5120, everything BF16, a norm on both sides:
// 125 us for 671 MB (5.4 TB/s; a large copy of torch's reaches 4.8); 4096 x 4096
// 28 us (4.8); 11886 x 1621, FP16, gated, 46 us for 154 MB (3.3).  Small calls
// are a launch and two or three latencies: 1 x 2048 2.3 us, 8 x 5120 with a gate
// 4.5 us, 777 x 1283 with layer norms 6.2 us.
#include "common.h"

namespace lowbit {
namespace {

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

// from FP32 vector p, or `none` everywhere where it is not given
__device__ __forceinline__ void vector8(const float* p, float none, int at, float (&v)[8]) {
  if (p) {
    widen<4>(load8<4>(p, at), 1, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = none;
  }
}

// Sum over the wave in every lane: DPP adds within 16 lanes and across the
// halves (no LDS round trip), the same order for every row.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS,
                                                                   0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr:1
  v = dpp_add<0x112, 0xF>(v);  // row_shr:2
  v = dpp_add<0x114, 0xF>(v);  // row_shr:4
  v = dpp_add<0x118, 0xF>(v);  // row_shr:8: lane 15 of each row holds the row's sum
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sum over the threads that share a row.  Consecutive sums of a work-group
// use the two halves of `red` in turn, so that one barrier each is enough; the
// places of waves that the work-group does not have hold zeros (row_sum_init).
__device__ __forceinline__ void row_sum_init(float (*red)[16]) {
  if (threadIdx.x < 32 && (threadIdx.x & 15) >= (blockDim.x >> 6)) red[threadIdx.x >> 4][threadIdx.x & 15] = 0.0f;
}
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int& turn) {
  v = wave_sum(v);
  if constexpr (WAVE) return v;
  if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
  __syncthreads();
  float4 w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const float4*>(&red[turn][q * 4]);
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) s += (w[q].x + w[q].y) + (w[q].z + w[q].w);
  turn ^= 1;
  return s;
}

// Rows of up to threads * NV * 8 elements in registers.  SY, SR: bytes per
// element of y and r.  MODE:
//   kLate : weights and gate are fetched when they are needed, which leaves
//           registers for rows of several steps
//   kExact: the same for rows of whole eights: no masks but one a step, no
//           short stores (16384 x 5120: 143 -> 125 us, 8192 x 7000 107 -> 90)
//   kAhead: they are fetched with the row, which takes two memory latencies off
//           a small call
//   kHeld : a work-group takes every gridDim.x-th row, keeps the weights (and a
//           gate that all rows share), and has the next row on its way while it
//           works on one (11886 x 1621, FP16, a norm on both sides, gated: 78 ->
//           46 us)
// A thread's elements in step n are the eight from c on.  Where fewer are left
// it holds the row's last eight (k >= 8) and passes over the first `skip` of
// them, which are another thread's: no load has a short form.
enum { kLate, kExact, kAhead, kHeld };
template <bool WAVE, int SY, int SR, int NV, int MODE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(NormArgs a) {
  __shared__ __align__(16) float red[2][16];
  if constexpr (!WAVE) row_sum_init(red);
  const int threads = WAVE ? 64 : (int)blockDim.x;
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  int64_t i = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  const int64_t step = WAVE ? (int64_t)gridDim.x * 4 : (int64_t)gridDim.x;
  if (WAVE && i >= a.m) return;
  const int k = (int)a.k;
  const float inv_k = 1.0f / (float)k;
  int turn = 0;

  constexpr bool kLater = MODE == kLate || MODE == kExact;
  int at[NV], skip[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c = (n * threads + t) * 8;
    at[n] = c < k - 8 ? c : k - 8;
    skip[n] = MODE == kExact ? (c < k ? 0 : 8) : c - at[n];
  }
  // sums over this thread's elements of step n
  auto sum8 = [&](const float (&w)[8], int n) __attribute__((always_inline)) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += MODE == kExact || j >= skip[n] ? w[j] : 0.0f;
    return MODE == kExact && skip[n] != 0 ? 0.0f : s;
  };
  auto square8 = [&](const float (&w)[8], float mean, int n) __attribute__((always_inline)) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = MODE == kExact || j >= skip[n] ? w[j] - mean : 0.0f;
      s += d * d;
    }
    return MODE == kExact && skip[n] != 0 ? 0.0f : s;
  };
  Raw8<SY> yr[NV], yn[NV];
  Raw8<SR> rr[NV], rn[NV];
  auto load_row = [&](Raw8<SY> (&y)[NV], Raw8<SR> (&r)[NV], int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (a.y) y[n] = load8<SY>(a.y, row * a.ldy + at[n]);
      r[n] = load8<SR>(a.r, row * a.ldr + at[n]);
    }
  };
  load_row(yr, rr, i);
  float post_w[NV][8], post_b[NV][8], gate[NV][8], pre_w[NV][8], pre_b[NV][8];
  auto gate8 = [&](int n, int64_t row) __attribute__((always_inline)) {
    if (a.gate_type == 1) widen<4>(load8<4>(a.gate, row * a.ldg + at[n]), 1, gate[n]);
    else widen<2>(load8<2>(a.gate, row * a.ldg + at[n]), a.gate_type, gate[n]);
  };
  if constexpr (!kLater) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if (a.post != 0) {
        vector8(a.post_w, 1.0f, at[n], post_w[n]);
        vector8(a.post_b, 0.0f, at[n], post_b[n]);
      }
      if (a.pre != 0) {
        vector8(a.pre_w, 1.0f, at[n], pre_w[n]);
        vector8(a.pre_b, 0.0f, at[n], pre_b[n]);
      }
      if (a.gate) gate8(n, i);
    }
  }
  for (;;) {
    const int64_t next = i + step;
    const bool more = MODE == kHeld && next < a.m;
    if (more) load_row(yn, rn, next);
    float v[NV][8];
    if (a.y) {
      float u[NV][8];
#pragma unroll
      for (int n = 0; n < NV; ++n) widen<SY>(yr[n], a.y_type, u[n]);
      float mean = 0.0f, rs = 1.0f;
      if (a.post == 2) {
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) s += sum8(u[n], n);
        mean = row_sum<WAVE>(s, red, turn) * inv_k;
      }
      if (a.post != 0) {
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) s += square8(u[n], mean, n);
        rs = 1.0f / sqrtf(row_sum<WAVE>(s, red, turn) * inv_k + a.eps);
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (skip[n] < 8) {
          if (a.post != 0) {
            if constexpr (kLater) {
              vector8(a.post_w, 1.0f, at[n], post_w[n]);
              vector8(a.post_b, 0.0f, at[n], post_b[n]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) u[n][j] = (u[n][j] - mean) * rs * post_w[n][j] + post_b[n][j];
          }
          if (a.gate) {
            if constexpr (kLater) gate8(n, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[n][j] *= gate[n][j];
            if (more && a.ldg != 0) gate8(n, next);
          }
        }
        widen<SR>(rr[n], a.r_type, v[n]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[n][j] += a.scale * u[n][j];
      }
    } else {
#pragma unroll
      for (int n = 0; n < NV; ++n) widen<SR>(rr[n], a.r_type, v[n]);
    }
    if (a.r_out) {
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (skip[n] < 8) store8(a.r_out, a.r_type, i * a.ldro + at[n], MODE == kExact ? 0 : skip[n], v[n]);
      }
    }
    if (a.x_out) {
      float mean = 0.0f, rs = 1.0f;
      if (a.pre == 2) {
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) s += sum8(v[n], n);
        mean = row_sum<WAVE>(s, red, turn) * inv_k;
      }
      if (a.pre != 0) {
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) s += square8(v[n], mean, n);
        rs = 1.0f / sqrtf(row_sum<WAVE>(s, red, turn) * inv_k + a.eps);
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        if (skip[n] >= 8) continue;
        if (a.pre != 0) {
          if constexpr (kLater) {
            vector8(a.pre_w, 1.0f, at[n], pre_w[n]);
            vector8(a.pre_b, 0.0f, at[n], pre_b[n]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) v[n][j] = (v[n][j] - mean) * rs * pre_w[n][j] + pre_b[n][j];
        }
        store8(a.x_out, a.x_type, i * a.ldx + at[n], MODE == kExact ? 0 : skip[n], v[n]);
      }
    }
    if (!more) return;
    i = next;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      yr[n] = yn[n];
      rr[n] = rn[n];
    }
  }
}

template <int TYPE>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return (float)static_cast<const typename Elem<TYPE>::type*>(p)[i];
}

__device__ __forceinline__ float load_any(const void* p, int type, int64_t i) {
  return type == 1 ? load1<1>(p, i) : type == 2 ? load1<2>(p, i) : load1<3>(p, i);
}

__device__ __forceinline__ void store_any(void* p, int type, int64_t i, float v) {
  if (type == 1) static_cast<float*>(p)[i] = v;
  else if (type == 2) static_cast<_Float16*>(p)[i] = (_Float16)v;
  else static_cast<bf16_t*>(p)[i] = (bf16_t)v;
}

// Rows longer than a work-group's registers, or shorter than 8: nothing is
// kept, each sum reads the row again (a row of 2^22 would not fit a compute unit
// in any form).
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
  __shared__ __align__(16) float red[2][16];
  row_sum_init(red);
  int turn = 0;
  const int64_t i = blockIdx.x;
  const float inv_k = 1.0f / (float)a.k;
  const int64_t iy = i * a.ldy, ir = i * a.ldr, ig = i * a.ldg;

  float mean_y = 0.0f, rs_y = 1.0f;
  if (a.post != 0) {
    if (a.post == 2) {
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < a.k; c += blockDim.x) s += load_any(a.y, a.y_type, iy + c);
      mean_y = row_sum<false>(s, red, turn) * inv_k;
    }
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.k; c += blockDim.x) {
      const float d = load_any(a.y, a.y_type, iy + c) - mean_y;
      s += d * d;
    }
    rs_y = 1.0f / sqrtf(row_sum<false>(s, red, turn) * inv_k + a.eps);
  }
  auto residual = [&](int64_t c) {
    float v = load_any(a.r, a.r_type, ir + c);
    if (a.y) {
      float u = load_any(a.y, a.y_type, iy + c);
      if (a.post != 0) {
        u = (u - mean_y) * rs_y;
        if (a.post_w) u *= a.post_w[c];
        if (a.post_b) u += a.post_b[c];
      }
      if (a.gate) u *= load_any(a.gate, a.gate_type, ig + c);
      v += a.scale * u;
    }
    return v;
  };
  float mean_r = 0.0f, rs_r = 1.0f;
  if (a.pre != 0) {
    if (a.pre == 2) {
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < a.k; c += blockDim.x) s += residual(c);
      mean_r = row_sum<false>(s, red, turn) * inv_k;
    }
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.k; c += blockDim.x) {
      const float d = residual(c) - mean_r;
      s += d * d;
    }
    rs_r = 1.0f / sqrtf(row_sum<false>(s, red, turn) * inv_k + a.eps);
  }
  for (int64_t c = threadIdx.x; c < a.k; c += blockDim.x) {
    const float v = residual(c);
    if (a.r_out) store_any(a.r_out, a.r_type, i * a.ldro + c, v);
    if (a.x_out) {
      float x = v;
      if (a.pre != 0) {
        x = (v - mean_r) * rs_r;
        if (a.pre_w) x *= a.pre_w[c];
        if (a.pre_b) x += a.pre_b[c];
      }
      store_any(a.x_out, a.x_type, i * a.ldx + c, x);
    }
  }
}

template <bool WAVE, int NV, int MODE>
hipError_t launch_as(const NormArgs& a, dim3 grid, dim3 block, hipStream_t st) {
  const bool y4 = a.y_type == 1, r4 = a.r_type == 1;
  if (y4 && r4) hipLaunchKernelGGL((norm_kernel<WAVE, 4, 4, NV, MODE>), grid, block, 0, st, a);
  else if (y4) hipLaunchKernelGGL((norm_kernel<WAVE, 4, 2, NV, MODE>), grid, block, 0, st, a);
  else if (r4) hipLaunchKernelGGL((norm_kernel<WAVE, 2, 4, NV, MODE>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((norm_kernel<WAVE, 2, 2, NV, MODE>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_residual(const NormArgs& a, hipStream_t st) {
  const int64_t chunks = (a.k + 7) / 8;
  const dim3 grid((unsigned)a.m);
  if (a.k < 8) {
    hipLaunchKernelGGL(norm_long_kernel, grid, dim3(64), 0, st, a);
    return hipGetLastError();
  }
  const bool many = a.m >= 1024;
  const bool exact = a.k % 8 == 0;
  // Many rows: those of whole eights need nothing else to come near the memory's
  // rate; of others the weights are kept where a row would read at least as much
  // of them as of itself (11886 x 1621, FP16, four of them: 78 us read again, 46
  // kept).  Rows of FP32 on both sides, which take more registers, need more of
  // them (4096 x 2048, two: 28 and 30; four: 83 and 81).
  const int vectors = !!a.post_w + !!a.post_b + !!a.pre_w + !!a.pre_b + (a.gate && a.ldg == 0);
  const int bytes = (a.y ? (a.y_type == 1 ? 4 : 2) : 0) + (a.r_type == 1 ? 4 : 2);
  const bool keep = !exact && 4 * vectors >= (bytes == 8 ? 12 : bytes);
  // As many work-groups of `waves` waves as run at once, `simd` waves to a SIMD, each
  // with as many of the rows.  Four run with up to 128 registers; two steps of one
  // wave take 163 to 165 with a 16-bit y (three), 171 to 173 with an FP32 one (two):
  // 40000 x 601, FP16, four weights and a gate 75.6 -> 65.8 us, 5000 x 1001, FP32 24.3
  // -> 20.0 against four; 16384 x 1001, BF16 y, FP32 r 55.6 -> 58.1.
  const auto running = [](int64_t waves, int64_t simd) { return 256 * 4 * simd / waves; };
  const auto held = [&](int64_t rows, int64_t waves, int64_t simd) {
    const int64_t each = (rows + running(waves, simd) - 1) / running(waves, simd);
    return dim3((unsigned)((rows + each - 1) / each));
  };
  // short rows, many of them: one wave each, no barriers (12030 x 128, one weight
  // and a gate per row: 8.6 us kept, 12.8 read again)
  if (chunks <= 64 && many) return launch_as<true, 1, kHeld>(a, held((a.m + 3) / 4, 4, 4), dim3(256), st);
  if (chunks <= 128 && many) {
    if (keep) return launch_as<true, 2, kHeld>(a, held((a.m + 3) / 4, 4, a.y_type == 1 ? 2 : 3), dim3(256), st);
    const dim3 g((unsigned)((a.m + 3) / 4));
    return exact ? launch_as<true, 2, kExact>(a, g, dim3(256), st) : launch_as<true, 2, kLate>(a, g, dim3(256), st);
  }
  auto block = [&](int64_t nv) { return dim3((unsigned)((chunks + nv * 64 - 1) / (nv * 64) * 64)); };
  // Many long rows: 16 elements a thread, so that more work-groups of fewer
  // waves share a compute unit (16384 x 5120 BF16: 125 us, with 8 elements 137).
  if (chunks <= 1024 && !(many && chunks > 512)) {
    const int64_t waves = (chunks + 63) / 64;
    if (many && !keep)
      return exact ? launch_as<false, 1, kExact>(a, grid, block(1), st)
                   : launch_as<false, 1, kLate>(a, grid, block(1), st);
    if (many && a.m >= 2 * running(waves, 4)) return launch_as<false, 1, kHeld>(a, held(a.m, waves, 4), block(1), st);
    return launch_as<false, 1, kAhead>(a, grid, block(1), st);
  }
  // Above 12288 a work-group of 16 elements a thread no longer has a second one
  // beside it, unless y and r are FP32 with its fewer conversions (4096 x 16384,
  // BF16: 32 elements 109 us, 16 117; 2048 x 16384, FP32: 100 and 95).
  const bool whole = many && exact;
  if (chunks <= (whole && bytes < 8 ? 1536 : 2048))
    return whole ? launch_as<false, 2, kExact>(a, grid, block(2), st)
                 : launch_as<false, 2, kLate>(a, grid, block(2), st);
  if (chunks <= 4096)
    return whole ? launch_as<false, 4, kExact>(a, grid, block(4), st)
                 : launch_as<false, 4, kLate>(a, grid, block(4), st);
  hipLaunchKernelGGL(norm_long_kernel, grid, dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace lowbit
