// The norms around a block, its gate and the residual add, in one launch:
//   u = post(y),  r' = r + scale * gate * u,  x = pre(r')
// with post and pre a root-mean-square or a layer norm, or none.
//
// [P2] 7minutos.es, "PrismML lanza Bonsai 27B ...", "Como funciona la
//      compresion": the projections of a block are low-bit; the norms and the
//      residual stream between them are not.
#include "common.h"

namespace lowbit {
namespace {

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

// sum over the work-group, the same in every thread; `red` holds one float
// per wave and is free again when the call returns
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += red[w];
  __syncthreads();
  return s;
}

// One work-group per row, any k, stride and alignment: nothing of the row is
// kept, each pass over it reads it again.
__global__ __launch_bounds__(256) void norm_rows_kernel(NormArgs a) {
  __shared__ float red[4];
  const int64_t i = blockIdx.x;
  const float inv_k = 1.0f / (float)a.k;
  const int64_t iy = i * a.ldy, ir = i * a.ldr, ig = i * a.ldg;

  float mean_y = 0.0f, rs_y = 1.0f;
  if (a.post != 0) {
    if (a.post == 2) {
      float s = 0.0f;
      for (int64_t c = threadIdx.x; c < a.k; c += 256) s += load_any(a.y, a.y_type, iy + c);
      mean_y = block_sum(s, red) * inv_k;
    }
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.k; c += 256) {
      const float d = load_any(a.y, a.y_type, iy + c) - mean_y;
      s += d * d;
    }
    rs_y = 1.0f / sqrtf(block_sum(s, red) * inv_k + a.eps);
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
      for (int64_t c = threadIdx.x; c < a.k; c += 256) s += residual(c);
      mean_r = block_sum(s, red) * inv_k;
    }
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.k; c += 256) {
      const float d = residual(c) - mean_r;
      s += d * d;
    }
    rs_r = 1.0f / sqrtf(block_sum(s, red) * inv_k + a.eps);
  }
  for (int64_t c = threadIdx.x; c < a.k; c += 256) {
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

}  // namespace

hipError_t launch_norm_residual(const NormArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(norm_rows_kernel, dim3((unsigned)a.m), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace lowbit
