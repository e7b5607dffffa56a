// Low-rank adapters of many requests beside a shared low-bit projection:
//   v[i][j]  = scale[s] * sum_k A[s][j][k] x[i][k],  s = ids[i], j < rank[s]
//   y[i][o] += sum_j B[s][o][j] v[i][j]
// The first product ("shrink") leaves v in the workspace as FP32, the second
// ("expand") adds to y in place.  No atomics: every v and every y element has
// one writer.
//
// [P2] 7minutos.es, "PrismML lanza Bonsai 27B ...", "Como funciona la
//      compresion": every projection of the model is a frozen low-bit matrix;
//      what is learned on top of it lives in such adapters.
#include "common.h"

namespace lowbit {
namespace {

__device__ __forceinline__ int rank_of(const LoraArgs& a, int64_t s) {
  if (!a.ranks) return (int)a.r;
  const int v = a.ranks[s];
  return v < 0 ? 0 : (v > (int)a.r ? (int)a.r : v);
}

// one wave per (row, j)
template <int XT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs a, float* __restrict__ v) {
  typedef typename Elem<XT>::type T;
  const int64_t i = blockIdx.x;
  const int64_t s = a.ids[i];
  if (s < 0 || s >= a.slots) return;
  const int rank = rank_of(a, s);
  const T* x = static_cast<const T*>(a.x) + i * a.ldx;
  const int lane = threadIdx.x & 63;
  for (int j = threadIdx.x >> 6; j < rank; j += 4) {
    const T* w = static_cast<const T*>(a.a) + (s * a.r + j) * a.k;
    float acc = 0.0f;
    for (int64_t c = lane; c < a.k; c += 64) acc += (float)w[c] * (float)x[c];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) acc += __shfl_xor(acc, off, 64);
    if (lane == 0) v[i * a.r + j] = a.scales ? acc * a.scales[s] : acc;
  }
}

// one thread per (row, output), the outputs of a row over gridDim.y work-groups
template <int XT, int YT>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a, const float* __restrict__ v) {
  typedef typename Elem<XT>::type T;
  typedef typename Elem<YT>::type Y;
  const int64_t i = blockIdx.x;
  const int64_t s = a.ids[i];
  if (s < 0 || s >= a.slots) return;
  const int rank = rank_of(a, s);
  if (rank == 0) return;
  Y* y = static_cast<Y*>(a.y) + i * a.ldy;
  for (int64_t o = (int64_t)blockIdx.y * 256 + threadIdx.x; o < a.n; o += (int64_t)gridDim.y * 256) {
    const T* w = static_cast<const T*>(a.b) + (s * a.n + o) * a.r;
    float acc = 0.0f;
    for (int j = 0; j < rank; ++j) acc += (float)w[j] * v[i * a.r + j];
    y[o] = (Y)((float)y[o] + acc);
  }
}

}  // namespace

size_t lora_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t r, int64_t slots) {
  (void)n;
  (void)k;
  (void)slots;
  return (size_t)((m * r * 4 + 255) / 256 * 256);
}

hipError_t launch_lora_accumulate(const LoraArgs& a, void* ws, hipStream_t st) {
  float* v = static_cast<float*>(ws);
  const int64_t tiles = (a.n + 255) / 256;
  const dim3 gs((unsigned)a.m), ge((unsigned)a.m, (unsigned)(tiles < 1024 ? tiles : 1024));
  if (a.x_type == 2)
    hipLaunchKernelGGL(lora_shrink_kernel<2>, gs, dim3(256), 0, st, a, v);
  else
    hipLaunchKernelGGL(lora_shrink_kernel<3>, gs, dim3(256), 0, st, a, v);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.x_type == 2)
    hipLaunchKernelGGL((lora_expand_kernel<2, 1>), ge, dim3(256), 0, st, a, v);
  else if (a.y_type == 1)
    hipLaunchKernelGGL((lora_expand_kernel<3, 1>), ge, dim3(256), 0, st, a, v);
  else
    hipLaunchKernelGGL((lora_expand_kernel<3, 3>), ge, dim3(256), 0, st, a, v);
  return hipGetLastError();
}

}  // namespace lowbit
