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
//
// What bounds it.  Large calls: the logits read and written, and the tokens,
// read once by every part.  64 x 151936 with lists of up to 32768, 300 biases, a
// mask, logits written: 28 us and 4 to 5 for the rows' ends (86 MB of logits,
// mask and lists; counting the tokens is some 10 of them, the biases 3).  Small calls:
// a launch and the latencies of lengths, tokens and logits: 1 x 151936, the token
// alone, 4.5 + 1.6 us; 8 x 151936 with everything 8 to 9.6 + 1.5 to 3.9 us.
#include "argmax.h"
#include "common.h"

namespace lowbit {
namespace {

// what is known of a token: it stands in the prompt; it has a bias; the rest:
// its count after the prompt (lists are shorter than 2^30)
constexpr uint32_t kSeen = 0x80000000u;
constexpr uint32_t kBias = 0x40000000u;
constexpr int kBiasCap = 256;  // biases of one part that are held in LDS

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

// Work-group id -> (row, part) so that the parts of a row run on one die (ids
// go round the eight dies): its tokens are then read into one L2, not eight.
// The last b % 8 rows are dealt out part by part.
__device__ __forceinline__ void place(int64_t b, int parts, int64_t* row, int* part) {
  const int64_t id = blockIdx.x, whole = b / 8 * 8;
  if (id < whole * parts) {
    const int64_t turn = id / 8;
    *row = turn / parts * 8 + id % 8;
    *part = (int)(turn % parts);
  } else {
    *row = id / parts;
    *part = (int)(id % parts);
  }
}

template <int TYPE, int THREADS, int R>
__global__ __launch_bounds__(THREADS, THREADS == 1024 ? 8 : 1) void logits_kernel(LogitsArgs a, int parts, uint64_t* __restrict__ part) {
  typedef typename Elem<TYPE>::type Y;
  constexpr int kStep = 4 * THREADS;
  constexpr int G = (R + kStep - 1) / kStep;   // steps of four tokens a thread, all in flight together
  constexpr int kWaves = THREADS / 64;
  __shared__ __align__(16) uint32_t cnt[R];
  __shared__ __align__(16) int bias_at[kBiasCap + 4];
  __shared__ float bias_val[kBiasCap];
  __shared__ int wave_n[kWaves];
  __shared__ uint64_t red[kWaves];
  const int tid = threadIdx.x;
  int64_t row;
  int pt;
  place(a.b, parts, &row, &pt);
  const int64_t lo = (int64_t)pt * R;
  const int size = a.n - lo < R ? (int)(a.n - lo) : R;
  const Y* y = static_cast<const Y*>(a.y) + row * a.ldy + lo;

  // The list of biases: entry j of the first THREADS stays with thread j, which
  // also fetches that token's logit; all in-range entries are gathered in LDS
  // in the list's order.
  const int nlist = a.bias_ids ? (int)clamp_len(a.bias_len, row, a.bcap, a.bcap) : 0;
  const int32_t* ids = a.bias_ids + row * a.ldb;
  const float* vals = a.bias_vals + row * a.ldb;
  uint32_t my_off = ~0u;
  float my_val = 0.0f;
  if (tid < nlist) {
    my_off = (uint32_t)ids[tid] - (uint32_t)lo;
    my_val = vals[tid];
  }

  Row4<TYPE> in[G];  // on their way while the tokens are counted
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c = g * kStep + tid * 4;
    if (c + 4 <= size) {
      __builtin_memcpy(&in[g], y + c, sizeof(in[g]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) in[g].e[e] = c + e < size ? y[c + e] : (Y)0.0f;
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
    if (R % kStep == 0 || g * kStep + tid * 4 < R)
      reinterpret_cast<uint4*>(cnt)[g * THREADS + tid] = make_uint4(0, 0, 0, 0);

  if (a.tokens) {
    const int32_t* t = a.tokens + row * a.ldt;
    const int total = (int)clamp_len(a.total_len, row, a.tcap, a.tcap);
    const int prompt = (int)clamp_len(a.prompt_len, row, 0, total);
    // Tokens j0 .. j1: U steps of four to a thread are in flight together.  Ids
    // below lo, negative ones among them, wrap to offsets past any part.
    auto scan = [&](int j0, int j1, auto hit) __attribute__((always_inline)) {
      constexpr int U = 4;
      for (; j0 + U * kStep <= j1; j0 += U * kStep) {
        uint32_t id[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) __builtin_memcpy(id[u], t + j0 + u * kStep + tid * 4, 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (id[u][e] - (uint32_t)lo < (uint32_t)size) hit(id[u][e] - (uint32_t)lo);
      }
      for (; j0 < j1; j0 += kStep) {
        uint32_t id[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + e * THREADS + tid;
          id[e] = j < j1 ? (uint32_t)t[j] : ~0u;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (id[e] - (uint32_t)lo < (uint32_t)size) hit(id[e] - (uint32_t)lo);
      }
    };
    __syncthreads();
    // the prompt first: plain stores of one value, whichever lane's stands
    scan(0, prompt, [&](uint32_t off) __attribute__((always_inline)) { cnt[off] = kSeen; });
    __syncthreads();
    scan(prompt, total, [&](uint32_t off) __attribute__((always_inline)) { atomicAdd(&cnt[off], 1u); });
  }
  int nb = 0, nkept = 0, my_at = 0;  // biases in this part, of them with a thread; this thread's place
  float my_y = 0.0f;
  if (nlist > 0) {
    if (!a.tokens) __syncthreads();
    for (int j0 = 0; j0 < nlist; j0 += THREADS) {
      const int j = j0 + tid;
      const uint32_t off = j0 == 0 ? my_off : (j < nlist ? (uint32_t)ids[j] - (uint32_t)lo : ~0u);
      const bool mine = off < (uint32_t)size;
      const uint64_t all = __ballot(mine);
      if ((tid & 63) == 0) wave_n[tid >> 6] = __popcll(all);
      __syncthreads();
      int at = nb + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32),
                                                   __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0u));
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        at += w < (tid >> 6) ? wave_n[w] : 0;
        nb += wave_n[w];
      }
      if (mine) {
        const float val = j0 == 0 ? my_val : vals[j];
        if (at < kBiasCap) {
          bias_at[at] = (int)off;
          bias_val[at] = val;
        }
        atomicOr(&cnt[off], kBias);
        if (j0 == 0) {
          my_at = at;
          my_y = (float)y[off];
        }
      }
      if (j0 == 0) nkept = nb;
      if (tid < 4 && nb <= kBiasCap) bias_at[nb + tid] = -1;
      if (j0 + THREADS < nlist) __syncthreads();
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
#pragma unroll
  for (int g = 0; g < G; ++g) {
    int t4 = tid * 4;
    // (made anew: kept since the loads, the places are more than 64 registers hold)
    if constexpr (THREADS == 1024) __asm__ volatile("" : "+v"(t4));
    const int c = g * kStep + t4;
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
  uint64_t best = best_u ? argmax_pack(best_u, lo + best_c) : 0;

  // the tokens with a bias, by their first entry: its value and those of the
  // later ones with the same id, added in the list's order
  auto biased = [&](int off, float yv, float bias) __attribute__((always_inline)) {
    float v = penalise(yv + bias, cnt[off], p, f, q);
    if (none || (mask && !((mask[off >> 5] >> (off & 31)) & 1))) {
      v = -__builtin_inff();
    } else {
      const uint64_t key = argmax_key(v, lo + off);
      best = key > best ? key : best;
    }
    if (out) out[off] = v;
  };
  if (nb <= kBiasCap) {
    auto entry = [&](int i, int off, float bias, float yv) __attribute__((always_inline)) {
      bool first = true;
      for (int j = 0; j < nb; j += 4) {  // places past nb hold no offset
        const int4 o = *reinterpret_cast<const int4*>(&bias_at[j]);
        const int at[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at[e] == off) {
            if (j + e < i) first = false;
            if (j + e > i) bias += bias_val[j + e];
          }
      }
      if (first) biased(off, yv, bias);
    };
    if (my_off < (uint32_t)size) entry(my_at, (int)my_off, my_val, my_y);
    for (int i = nkept + tid; i < nb; i += THREADS) entry(i, bias_at[i], bias_val[i], (float)y[bias_at[i]]);
  } else {
    // More than LDS holds: a wave takes 256 tokens at a time, four to a lane in
    // registers, and walks the list once for them; its entries are added one by
    // one, in the list's order.  64 x 151936 with 16384 biases a row: 0.45 ms
    // (127 with a walk for each entry); all of one id 1.0 ms (2.5).
    const int lane = tid & 63;
    for (int base = (tid >> 6) * 256; base < size; base += 4 * THREADS) {
      bool mine[4];
      float sum[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int off = base + e * 64 + lane;
        mine[e] = off < size && (cnt[off] & kBias);
        sum[e] = -0.0f;  // the first entry added to it keeps its bits
      }
      if (!__ballot(mine[0] || mine[1] || mine[2] || mine[3])) continue;
      constexpr int U = 4;
      for (int j0 = 0; j0 < nlist; j0 += U * 64) {
        uint32_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * 64 + lane;
          at[u] = j < nlist ? (uint32_t)ids[j] - (uint32_t)lo - (uint32_t)base : ~0u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint64_t hit = __ballot(at[u] < 256u);  // (places past the part's end are nobody's)
          if (!hit) continue;
          const float val = at[u] < 256u ? vals[j0 + u * 64 + lane] : 0.0f;
          while (hit) {
            const int l = __builtin_ctzll(hit);
            hit &= hit - 1;
            const int place = __builtin_amdgcn_readlane((int)at[u], l);
            const float v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, val), l));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (place == e * 64 + lane) sum[e] += v;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int off = base + e * 64 + lane;
        if (mine[e]) biased(off, (float)y[off], sum[e]);
      }
    }
  }
  if (part) {
    best = wave_max(best);
    if ((tid & 63) == 0) red[tid >> 6] = best;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) best = red[w] > best ? red[w] : best;
      part[row * parts + pt] = best;
    }
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

// Tokens of a part: large ones read the row's list of tokens less often, small
// ones give a call enough work-groups to fill the chip.  The largest (two
// work-groups of 1024 threads to a compute unit) pays where lists are long:
// 64 x 151936 with lists of 32768 takes 27 us against 32 with parts of 8192, of
// 4096 25.2 against 25.3, and 256 x 151936 with lists of 4096 85 against 74.
// Threads: 512 for parts of 4096 (45 x 44490, lists of 23821: 15.4 us against
// 18.5 with 256; 64 x 32000, lists of 2048: 11.7 against 13.6), 256 for 2048 (8 x
// 151936, lists of 4096: 10.1 against 10.4 with 512), 512 for 8192 (64 x 128000,
// lists of 4096: 24.9 against 27.3 with 1024).
constexpr int kLargePart = 19456;
int part_size(int64_t n, int64_t b, int64_t tcap) {
  auto enough = [&](int r) { return (n + r - 1) / r * b >= 384; };
  if (tcap >= 16384 && enough(kLargePart)) return kLargePart;
  for (int r : {8192, 4096, 2048})
    if (enough(r)) return r;
  return 1024;
}

int64_t parts_of(int64_t n, int64_t b, int64_t tcap) {
  const int r = part_size(n, b, tcap);
  return (n + r - 1) / r;
}

template <int TYPE>
void launch_part(const LogitsArgs& a, int parts, uint64_t* part, hipStream_t st) {
  const dim3 grid((unsigned)(parts * a.b));
  switch (part_size(a.n, a.b, a.tcap)) {
    case kLargePart:
      hipLaunchKernelGGL((logits_kernel<TYPE, 1024, kLargePart>), grid, dim3(1024), 0, st, a, parts, part);
      break;
    case 8192: hipLaunchKernelGGL((logits_kernel<TYPE, 512, 8192>), grid, dim3(512), 0, st, a, parts, part); break;
    case 4096: hipLaunchKernelGGL((logits_kernel<TYPE, 512, 4096>), grid, dim3(512), 0, st, a, parts, part); break;
    case 2048: hipLaunchKernelGGL((logits_kernel<TYPE, 256, 2048>), grid, dim3(256), 0, st, a, parts, part); break;
    default: hipLaunchKernelGGL((logits_kernel<TYPE, 256, 1024>), grid, dim3(256), 0, st, a, parts, part); break;
  }
}

}  // namespace

// (long lists never make more parts)
size_t logits_workspace_bytes(int64_t n, int64_t b) {
  return (size_t)((b * parts_of(n, b, 0) * 8 + 255) / 256 * 256);
}

hipError_t launch_logits_process(const LogitsArgs& a, void* ws, hipStream_t st) {
  const int64_t parts = parts_of(a.n, a.b, a.tcap);
  uint64_t* part = a.idx ? static_cast<uint64_t*>(ws) : nullptr;
  if (a.y_type == 1) launch_part<1>(a, (int)parts, part, st);
  else if (a.y_type == 2) launch_part<2>(a, (int)parts, part, st);
  else launch_part<3>(a, (int)parts, part, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.idx) return e;
  hipLaunchKernelGGL(logits_top1_kernel, dim3((unsigned)a.b), dim3(256), 0, st, part, (int)parts, a.idx,
                     a.val);
  return hipGetLastError();
}

}  // namespace lowbit
