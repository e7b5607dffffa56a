// Logits on their way to a token: biases, penalties for repeated tokens and a
// grammar's mask applied in one pass over the logits, with the top-1 of the
// result.
//
// [P5] openclawradar.com, "Bonsai 1.7B Modelo Ternario ...", "Detalles
//      tecnicos": decode is checked by top-1 token match.
//
// A work-group takes one part of the vocabulary of one row.  It counts the
// row's tokens that fall into its part in LDS (integer adds: no order
// matters), then reads its logits once, four tokens to a thread.  The counts
// need no state between calls and no table in memory; the price is that every
// part reads the row's tokens, which come from the cache.  The few tokens
// with a bias are left out of that pass and taken one by one after it, so
// that the pass itself holds no table of biases.
#include "argmax.h"
#include "common.h"

namespace lowbit {
namespace {

// what is known of a token: it stands in the prompt; it has a bias; the rest:
// its count after the prompt (lists are shorter than 2^30)
constexpr uint32_t kSeen = 0x80000000u;
constexpr uint32_t kBias = 0x40000000u;
constexpr int kBiasCap = 1024;  // biases of one part that are held in LDS

__device__ __forceinline__ int64_t clamp_len(const int32_t* len, int64_t i, int64_t none, int64_t cap) {
  const int64_t v = len ? (int64_t)len[i] : none;
  return v < 0 ? 0 : (v > cap ? cap : v);
}

// Penalties of a logit, each operation rounded to FP32 (no fused
// multiply-add): the same inputs give the same bits wherever a token sits.
__device__ __forceinline__ float penalise(float v, uint32_t cnt, float p, float f, float q) {
#pragma clang fp contract(off)
  if ((cnt & ~kBias) != 0) v = v > 0.0f ? v / p : v * p;
  const uint32_t c = cnt & ~(kSeen | kBias);
  if (c != 0) {
    v = v - f * (float)c;
    v = v - q;
  }
  return v;
}

template <int TYPE>
struct Row4 {
  typename Elem<TYPE>::type e[4];
};

template <int TYPE, int R>
__global__ __launch_bounds__(256) void logits_kernel(LogitsArgs a, uint64_t* __restrict__ part) {
  typedef typename Elem<TYPE>::type Y;
  constexpr int kSteps = R / 1024;             // steps of four tokens a thread
  constexpr int G = kSteps < 4 ? kSteps : 4;   // steps whose loads are in flight together
  __shared__ __align__(16) uint32_t cnt[R];
  __shared__ int bias_at[kBiasCap];
  __shared__ float bias_val[kBiasCap];
  __shared__ int bias_n;
  __shared__ uint64_t red[4];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y;
  const int64_t lo = (int64_t)blockIdx.x * R;
  const int size = a.n - lo < R ? (int)(a.n - lo) : R;
  const Y* y = static_cast<const Y*>(a.y) + row * a.ldy + lo;

  Row4<TYPE> in[G];
  auto load = [&](int g0) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c = (g0 + g) * 1024 + tid * 4;
      if (c + 4 <= size) {
        __builtin_memcpy(&in[g], y + c, sizeof(in[g]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) in[g].e[e] = c + e < size ? y[c + e] : (Y)0.0f;
      }
    }
  };
  load(0);  // on their way while the tokens are counted

#pragma unroll
  for (int s = 0; s < kSteps; ++s) reinterpret_cast<uint4*>(cnt)[s * 256 + tid] = make_uint4(0, 0, 0, 0);
  if (tid == 0) bias_n = 0;
  if (a.tokens || a.bias_ids) {
    __syncthreads();
    if (a.bias_ids && tid < 64) {  // one wave: the list's order is kept
      const int64_t len = clamp_len(a.bias_len, row, a.bcap, a.bcap);
      int n = 0;
      for (int64_t j0 = 0; j0 < len; j0 += 64) {
        const int64_t j = j0 + tid;
        const int64_t off = j < len ? (int64_t)a.bias_ids[row * a.ldb + j] - lo : -1;
        const bool mine = off >= 0 && off < size;
        const uint64_t all = __ballot(mine);
        if (mine) {
          const int at = n + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32),
                                                            __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0u));
          if (at < kBiasCap) {
            bias_at[at] = (int)off;
            bias_val[at] = a.bias_vals[row * a.ldb + j];
          }
          atomicOr(&cnt[off], kBias);
        }
        n += __popcll(all);
      }
      if (tid == 0) bias_n = n;
    }
    if (a.tokens) {
      const int32_t* t = a.tokens + row * a.ldt;
      const int64_t total = clamp_len(a.total_len, row, a.tcap, a.tcap);
      const int64_t prompt = clamp_len(a.prompt_len, row, 0, total);
      auto count = [&](int64_t j, int32_t id) __attribute__((always_inline)) {
        const int64_t off = (int64_t)id - lo;
        if (off >= 0 && off < size) {
          if (j < prompt) atomicOr(&cnt[off], kSeen);
          else atomicAdd(&cnt[off], 1u);
        }
      };
      constexpr int U = 4;
      int64_t j0 = 0;
      for (; j0 + U * 1024 <= total; j0 += U * 1024) {
        int id[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) __builtin_memcpy(id[u], t + j0 + u * 1024 + tid * 4, 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) count(j0 + u * 1024 + tid * 4 + e, id[u][e]);
      }
      for (int64_t j = j0 + tid; j < total; j += 256) count(j, t[j]);
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
    if (mr >= 0 && !none) mask = a.mask + mr * a.ldm + (lo >> 5);
  }
  float* out = a.out ? a.out + row * a.ldo + lo : nullptr;

  uint32_t best_u = 0;  // ordered bits of the best value (0: no allowed token yet) and its place
  int best_c = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < kSteps; g0 += G) {
    if (g0) load(g0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c = (g0 + g) * 1024 + tid * 4;
      if (c >= size) continue;
      const uint4 k4 = *reinterpret_cast<const uint4*>(cnt + c);
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
      const uint32_t any = k4.x | k4.y | k4.z | k4.w;
      const uint32_t ok = none ? 0u : (mask ? (uint32_t)mask[c >> 5] >> (c & 31) : 0xFu);
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (float)in[g].e[e];
      if (any) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = penalise(v[e], k[e], p, f, q);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool on = ((ok >> e) & 1u) && c + e < size;
        v[e] = on ? v[e] : -__builtin_inff();
        const uint32_t u = on && !(k[e] & kBias) ? ordered_bits(v[e]) : 0u;
        if (u > best_u) {
          best_u = u;
          best_c = c + e;
        }
      }
      if (out) {
        if (c + 4 <= size && !(any & kBias)) {
          __builtin_memcpy(out + c, v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < size && !(k[e] & kBias)) out[c + e] = v[e];
        }
      }
    }
  }
  uint64_t best = best_u ? argmax_pack(best_u, lo + best_c) : 0;

  // the tokens with a bias, by their first entry: its value and those of the
  // later ones with the same id, added in the list's order
  auto biased = [&](int off, float bias) __attribute__((always_inline)) {
    float v = penalise((float)y[off] + bias, cnt[off], p, f, q);
    if (none || (mask && !((mask[off >> 5] >> (off & 31)) & 1))) {
      v = -__builtin_inff();
    } else {
      const uint64_t key = argmax_key(v, lo + off);
      best = key > best ? key : best;
    }
    if (out) out[off] = v;
  };
  const int nb = bias_n;
  if (nb <= kBiasCap) {
    for (int i = tid; i < nb; i += 256) {
      const int off = bias_at[i];
      bool first = true;
      for (int j = 0; j < i; ++j) first = first && bias_at[j] != off;
      if (!first) continue;
      float bias = bias_val[i];
      for (int j = i + 1; j < nb; ++j)
        if (bias_at[j] == off) bias += bias_val[j];
      biased(off, bias);
    }
  } else {  // more than LDS holds: the same from the list itself
    const int64_t len = clamp_len(a.bias_len, row, a.bcap, a.bcap);
    const int32_t* ids = a.bias_ids + row * a.ldb;
    const float* vals = a.bias_vals + row * a.ldb;
    for (int64_t i = tid; i < len; i += 256) {
      const int32_t id = ids[i];
      if (id < lo || id >= lo + size) continue;
      bool first = true;
      for (int64_t j = 0; first && j < i; ++j) first = ids[j] != id;
      if (!first) continue;
      float bias = vals[i];
      for (int64_t j = i + 1; j < len; ++j)
        if (ids[j] == id) bias += vals[j];
      biased((int)(id - lo), bias);
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

// Tokens of a part: large ones read the row's list of tokens less often,
// small ones give a small call enough work-groups to fill the chip.
int part_size(int64_t n, int64_t b) {
  for (int r = 8192; r > 1024; r /= 2)
    if ((n + r - 1) / r * b >= 512) return r;
  return 1024;
}

int64_t parts_of(int64_t n, int64_t b) {
  const int r = part_size(n, b);
  return (n + r - 1) / r;
}

template <int TYPE>
void launch_part(const LogitsArgs& a, uint64_t* part, dim3 grid, hipStream_t st) {
  switch (part_size(a.n, a.b)) {
    case 8192: hipLaunchKernelGGL((logits_kernel<TYPE, 8192>), grid, dim3(256), 0, st, a, part); break;
    case 4096: hipLaunchKernelGGL((logits_kernel<TYPE, 4096>), grid, dim3(256), 0, st, a, part); break;
    case 2048: hipLaunchKernelGGL((logits_kernel<TYPE, 2048>), grid, dim3(256), 0, st, a, part); break;
    default: hipLaunchKernelGGL((logits_kernel<TYPE, 1024>), grid, dim3(256), 0, st, a, part); break;
  }
}

}  // namespace

size_t logits_workspace_bytes(int64_t n, int64_t b) {
  return (size_t)((b * parts_of(n, b) * 8 + 255) / 256 * 256);
}

hipError_t launch_logits_process(const LogitsArgs& a, void* ws, hipStream_t st) {
  const int64_t parts = parts_of(a.n, a.b);
  uint64_t* part = a.idx ? static_cast<uint64_t*>(ws) : nullptr;
  const dim3 grid((unsigned)parts, (unsigned)a.b);
  if (a.y_type == 1) launch_part<1>(a, part, grid, st);
  else if (a.y_type == 2) launch_part<2>(a, part, grid, st);
  else launch_part<3>(a, part, grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.idx) return e;
  hipLaunchKernelGGL(logits_top1_kernel, dim3((unsigned)a.b), dim3(256), 0, st, part, (int)parts, a.idx,
                     a.val);
  return hipGetLastError();
}

}  // namespace lowbit
