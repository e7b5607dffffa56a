// Logits on their way to a token: biases, penalties for repeated tokens and a
// grammar's mask applied in one pass over the logits, with the top-1 of the
// result.
//
// [P5] openclawradar.com, "Bonsai 1.7B Modelo Ternario ...", "Detalles
//      tecnicos": decode is checked by top-1 token match.
//
// A work-group takes one part of the vocabulary of one row.  It counts the
// row's tokens that fall into its part in LDS (integer adds: no order
// matters), adds up the biases there, then reads its logits once.
#include "argmax.h"
#include "common.h"

namespace lowbit {
namespace {

constexpr int kPart = 4096;             // tokens of the vocabulary per work-group
constexpr uint32_t kSeen = 0x80000000u;  // the token stands in the prompt; below: its count after it

__device__ __forceinline__ int64_t clamp_len(const int32_t* len, int64_t i, int64_t none, int64_t cap) {
  const int64_t v = len ? (int64_t)len[i] : none;
  return v < 0 ? 0 : (v > cap ? cap : v);
}

// One logit through the rules, each operation rounded to FP32 (no fused
// multiply-add): the same inputs give the same bits wherever a token sits.
__device__ __forceinline__ float process(float v, float bias, uint32_t cnt, float p, float f, float q) {
#pragma clang fp contract(off)
  v = v + bias;
  if (cnt != 0) v = v > 0.0f ? v / p : v * p;
  const uint32_t c = cnt & ~kSeen;
  if (c != 0) {
    v = v - f * (float)c;
    v = v - q;
  }
  return v;
}

template <int TYPE>
__global__ __launch_bounds__(256) void logits_kernel(LogitsArgs a, uint64_t* __restrict__ part) {
  __shared__ uint32_t cnt[kPart];
  __shared__ float bias[kPart];
  __shared__ uint64_t red[4];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y;
  const int64_t lo = (int64_t)blockIdx.x * kPart;
  const int64_t hi = lo + kPart < a.n ? lo + kPart : a.n;
  for (int c = tid; c < kPart; c += 256) {
    cnt[c] = 0u;
    bias[c] = 0.0f;
  }
  __syncthreads();
  if (a.tokens) {
    const int32_t* t = a.tokens + row * a.ldt;
    const int64_t total = clamp_len(a.total_len, row, a.tcap, a.tcap);
    const int64_t prompt = clamp_len(a.prompt_len, row, 0, total);
    for (int64_t j = tid; j < total; j += 256) {
      const int64_t id = t[j];
      if (id < lo || id >= hi) continue;
      if (j < prompt) atomicOr(&cnt[id - lo], kSeen);
      else atomicAdd(&cnt[id - lo], 1u);
    }
  }
  if (a.bias_ids && tid == 0) {  // one thread: repeated ids add up in the list's order
    const int64_t len = clamp_len(a.bias_len, row, a.bcap, a.bcap);
    for (int64_t j = 0; j < len; ++j) {
      const int64_t id = a.bias_ids[row * a.ldb + j];
      if (id >= lo && id < hi) bias[id - lo] += a.bias_vals[row * a.ldb + j];
    }
  }
  __syncthreads();
  const float p = a.repetition ? a.repetition[row] : 1.0f;
  const float f = a.frequency ? a.frequency[row] : 0.0f;
  const float q = a.presence ? a.presence[row] : 0.0f;
  const int32_t* mask = nullptr;
  bool none = false;  // a mask row past the last: nothing is allowed
  if (a.mask) {
    const int64_t mr = a.mask_row ? (int64_t)a.mask_row[row] : row;
    none = mr >= a.mask_rows;
    if (mr >= 0 && !none) mask = a.mask + mr * a.ldm;
  }
  const typename Elem<TYPE>::type* y = static_cast<const typename Elem<TYPE>::type*>(a.y) + row * a.ldy;
  uint64_t best = 0;
  for (int64_t i = lo + tid; i < hi; i += 256) {
    const bool ok = !none && (!mask || ((mask[i >> 5] >> (i & 31)) & 1));
    float v = process((float)y[i], bias[i - lo], cnt[i - lo], p, f, q);
    if (!ok) v = -__builtin_inff();
    if (a.out) a.out[row * a.ldo + i] = v;
    if (ok) {
      const uint64_t key = argmax_key(v, i);
      best = key > best ? key : best;
    }
  }
  if (part) {
    best = block_max(best, red);
    if (tid == 0) part[row * gridDim.x + blockIdx.x] = best;
  }
}

// The row's best key: key 0 is that of no allowed token.
__global__ __launch_bounds__(256) void logits_top1_kernel(const uint64_t* __restrict__ part, int nparts,
                                                          int32_t* __restrict__ idx, float* __restrict__ val) {
  __shared__ uint64_t red[4];
  const int64_t row = blockIdx.x;
  uint64_t best = 0;
  for (int i = threadIdx.x; i < nparts; i += 256) {
    const uint64_t k = part[row * nparts + i];
    best = k > best ? k : best;
  }
  best = block_max(best, red);
  if (threadIdx.x == 0) {
    const uint32_t u = (uint32_t)(best >> 32);
    idx[row] = best == 0 ? -1 : (int32_t)(0xFFFFFFFFu - (uint32_t)best);
    if (val)
      val[row] = best == 0 ? -__builtin_inff()
                           : __builtin_bit_cast(float, (u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
  }
}

int64_t parts_of(int64_t n) { return (n + kPart - 1) / kPart; }

}  // namespace

size_t logits_workspace_bytes(int64_t n, int64_t b) {
  return (size_t)((b * parts_of(n) * 8 + 255) / 256 * 256);
}

hipError_t launch_logits_process(const LogitsArgs& a, void* ws, hipStream_t st) {
  const int64_t parts = parts_of(a.n);
  uint64_t* part = a.idx ? static_cast<uint64_t*>(ws) : nullptr;
  const dim3 grid((unsigned)parts, (unsigned)a.b);
  if (a.y_type == 1)
    hipLaunchKernelGGL(logits_kernel<1>, grid, dim3(256), 0, st, a, part);
  else if (a.y_type == 2)
    hipLaunchKernelGGL(logits_kernel<2>, grid, dim3(256), 0, st, a, part);
  else
    hipLaunchKernelGGL(logits_kernel<3>, grid, dim3(256), 0, st, a, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.idx) return e;
  hipLaunchKernelGGL(logits_top1_kernel, dim3((unsigned)a.b), dim3(256), 0, st, part, (int)parts, a.idx,
                     a.val);
  return hipGetLastError();
}

}  // namespace lowbit
