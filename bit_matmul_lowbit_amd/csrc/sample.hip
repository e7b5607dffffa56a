// A token drawn from each row of logits, with temperature, top-k, top-p and
// min-p, from one given random number a row.
//
// [P1] 7minutos.es, "Un tutorial de codificacion ...", "9 Chat" and "10
//      Parametros de muestreo": temperature 0.5, top-p 0.85, top-k 20.
//
//   w_t = exp((y_t - max y) / T).  Sorted by value (ties by number), the filters
//   keep a first part of the row; in the order of their numbers, the token is the
//   first kept one at which the running sum of w passes u times their sum.
//
// The first launch cuts rows into parts of 4096 logits that stay in registers:
// the part's maximum, its weights relative to 2^ceil of that maximum, sums of their number
// and mass up to each quarter of an octave (a bin), and the part's tokens in the order of
// their bins.  Bins are places on one scale for all parts, so parts are added without being
// read again.  The second launch, a work-group a row, adds the sums and finds the bin in which
// each filter ends.  Where few tokens come before that (kList), they are gathered into LDS,
// each part's from where its order has them.  A filter's last token is found by narrowing an
// interval of (value, number) by 256 at a time, over the list or over the bin, until a
// wave can order the 64 that are left; nothing is sorted.  The draw goes by parts, blocks of 64
// tokens and tokens, or, where the kept tokens are many, by the parts' sums and one part of the
// row.
//
// What bounds it: the steps of the second launch, one after another (sums, a filter's end, its
// list, its narrowing, the draw: one to four microseconds each for their loads and barriers);
// a work-group reads 30 GB/s, so it must not read a row.  Measured, 151936 FP32 logits: one row
// with top-k 20 and top-p 0.85 4.4 and 14.4 us, 64 rows of mixed settings 21 us (1.9 TB/s: FP64
// weights and LDS atomics) and 52, most for those that keep 20000 tokens.
//
// Weights are made to 2^-40 relative (FP64, which runs at the rate of FP32 here) and rounded to whole
// numbers of 2^-51 of a part's base.  Where a row's are added they are cut to 2^-49 of its base, or to
// what leaves room for n of them in 62 bits (2^-44 for 151936; a weight below that counts nothing).
// So sums have no order: LDS atomics may come as they like, equal inputs give equal bits, and a
// draw among 150000 tokens finds the token that 64-bit arithmetic finds unless it is that close.
#include "pieces.h"

namespace lowbit {
namespace {

constexpr int kPart = 4096;      // logits of a part
constexpr int kPartThreads = kPart / 8;
constexpr int kBins = 256;       // quarters of an octave; the last one: everything below
constexpr int kRowThreads = 1024;
// parts whose sums a thread has on their way early (of 163840 logits; one row with top-k 20: 151936
// 18.7 us, 163841 19.2, 262144 21.1)
constexpr int kEarly = 10;
constexpr int kMostParts = 256;
static_assert((int64_t)kMostParts * kPart >= kSampleMost, "a row's parts have their places in LDS");
constexpr int kList = 8192;      // tokens that are held in LDS (64 mixed rows 80 us, 84 with 2048)
constexpr int kUnit = 51;        // a part's weights are whole numbers of 2^-51: 4096 of them stay below 2^64

// Order of values as whole numbers: NaN above all, both zeros alike
__device__ __forceinline__ uint32_t key_of(float y) {
  uint32_t u = __builtin_bit_cast(uint32_t, y);
  if (y != y) return 0xFFFFFFFFu;
  if (y == 0.0f) u = 0;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, (key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu, kKeyInf = 0xFF800000u;

// 2^x for x <= 0, off by less than 2^-41 relative; 0 below 2^-1000
__device__ __forceinline__ double exp2_of(double x) {
  if (!(x > -1000.0)) return 0.0;
  const double n = __builtin_rint(x), r = x - n;
  // sum of (r ln 2)^k / k!, |r| <= 1/2: the first term left out is below 2^-41
  double p = 7.0549116208011233e-9;
  p = __builtin_fma(p, r, 1.0178086009239699e-7);
  p = __builtin_fma(p, r, 1.3215486790144309e-6);
  p = __builtin_fma(p, r, 1.5252733804059841e-5);
  p = __builtin_fma(p, r, 1.5403530393381610e-4);
  p = __builtin_fma(p, r, 1.3333558146428443e-3);
  p = __builtin_fma(p, r, 9.6181291076284772e-3);
  p = __builtin_fma(p, r, 5.5504108664821580e-2);
  p = __builtin_fma(p, r, 2.4022650695910072e-1);
  p = __builtin_fma(p, r, 6.9314718055994531e-1);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}
// w in [0, 1] as a whole number of 2^-51: the mantissa of 2 + w
__device__ __forceinline__ uint64_t fixed_of(double w) {
  return __builtin_bit_cast(uint64_t, 2.0 + w) - 0x4000000000000000ull;
}

// Greedy: no temperature to speak of
__device__ __forceinline__ float temperature_of(const SampleArgs& a, int64_t row) {
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  return t >= 0x1p-20f ? t : 0.0f;
}
// (not 0 where the temperature is infinite: a masked logit, -inf, has to stay that; and no
// less than what leaves 2^-149 times it above FP64's smallest)
__device__ __forceinline__ double octaves(float t) { return fmax(1.4426950408889634074 / (double)t, 0x1p-400); }
// A value in octaves, c of them to one.  Rounded before a base is taken off: bases are rounded
// likewise, and at 1e38 an exact product less a rounded one is no small number.
__device__ __forceinline__ double in_octaves(float y, double c) {
#pragma clang fp contract(off)
  return (double)y * c;
}

// what the first launch leaves of a part
struct Parts {
  double* base;      // [rows][parts]: weights are relative to 2^base
  uint32_t* top;     // [rows][parts]: the largest key
  uint64_t* mass;    // [rows][parts][kBins]: up to and with the bin
  uint16_t* count;   // [rows][parts][kBins]: likewise
  uint16_t* order;   // [rows][parts][kPart]: the part's tokens by their bins
};
__host__ __device__ inline size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
inline size_t parts_layout(int64_t rows, int64_t parts, void* ws, Parts* p) {
  char* at = static_cast<char*>(ws);
  const size_t n = (size_t)(rows * parts);
  const size_t mass = align_up(n * kBins * 8), count = align_up(n * kBins * 2), base = align_up(n * 8), top = align_up(n * 4);
  const size_t order = align_up(n * kPart * 2);
  if (p) {
    p->mass = reinterpret_cast<uint64_t*>(at);
    p->count = reinterpret_cast<uint16_t*>(at + mass);
    p->base = reinterpret_cast<double*>(at + mass + count);
    p->top = reinterpret_cast<uint32_t*>(at + mass + count + base);
    p->order = reinterpret_cast<uint16_t*>(at + mass + count + base + top);
  }
  return mass + count + base + top + order;
}

// the quarter octave of v2 = y log2(e) / T on the scale of all parts
__device__ __forceinline__ double quarter(double v2) { return __builtin_floor(v2 * 4.0); }
// Quarters from the base down.  A base is a whole number of octaves that no value of its parts
// passes; one that lies on it is in bin 0, alone.  4 base - q is exact whatever the size, so a
// part's bin and the octaves from the row's base down to the part's add up to the row's bin.
__device__ __forceinline__ int bin_of(double q, double base) {
  const double b = base * 4.0 - q;
  return b >= kBins - 1 ? kBins - 1 : (int)b;
}

template <int S>
__device__ __forceinline__ void load_logits(const void* y, int type, int64_t at, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    widen<S>(load8<S>(y, at), type, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = -INFINITY;
      if (j < left) {
        if constexpr (S == 4) v[j] = static_cast<const float*>(y)[at + j];
        else if (type == 2) v[j] = (float)static_cast<const _Float16*>(y)[at + j];
        else v[j] = (float)static_cast<const bf16_t*>(y)[at + j];
      }
    }
  }
}

// The lanes' sums up to and with each, by DPP (no LDS round trips)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_add64(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
  return v + (((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
  v = dpp_add64<0x111, 0xF>(v);  // row_shr:1
  v = dpp_add64<0x112, 0xF>(v);
  v = dpp_add64<0x114, 0xF>(v);
  v = dpp_add64<0x118, 0xF>(v);
  v = dpp_add64<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add64<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Sums of v over the threads before this one; total: over all (1024 threads).
template <int N>
__device__ __forceinline__ void scan64(const uint64_t (&v)[N], uint64_t (&before)[N], uint64_t (&total)[N],
                                       uint64_t (*red)[16]) {
  const int t = threadIdx.x;
  uint64_t sum[N];
#pragma unroll
  for (int n = 0; n < N; ++n) sum[n] = wave_scan64(v[n]);
  __syncthreads();
  if ((t & 63) == 63)
#pragma unroll
    for (int n = 0; n < N; ++n) red[n][t >> 6] = sum[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint64_t b = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kRowThreads / 64; ++w) {
      const uint64_t r = red[n][w];
      if (w < (t >> 6)) b += r;
      all += r;
    }
    before[n] = b + sum[n] - v[n];
    total[n] = all;
  }
}
__device__ __forceinline__ uint64_t scan64(uint64_t v, uint64_t (*red)[16], uint64_t* total) {
  const uint64_t in[1] = {v};
  uint64_t before[1], all[1];
  scan64<1>(in, before, all, red);
  *total = all[0];
  return before[0];
}

// Where top-k keeps no more than the list has room for, no sums of mass are needed (64 mixed rows
// 80 us, 84 with them)
__device__ __forceinline__ int64_t top_k_of(const SampleArgs& a, int64_t row) {
  const int64_t k = a.top_k ? a.top_k[row] : 0;
  return k <= 0 || k > a.n ? a.n : k;
}
__device__ __forceinline__ bool without_mass(const SampleArgs& a, int64_t k) { return k < a.n && k <= kList; }

template <int S>
__global__ __launch_bounds__(kPartThreads) void sample_parts_kernel(SampleArgs a, Parts out) {
  __shared__ unsigned long long mass[kBins];
  __shared__ uint32_t count[kBins], before[kBins];
  __shared__ uint32_t tops[kPartThreads / 64], waves[kBins / 64];
  __shared__ unsigned long long wave_mass[kBins / 64];
  __shared__ __align__(16) uint16_t order[kPart];
  const int64_t row = blockIdx.y, part = blockIdx.x, slot = row * gridDim.x + part;
  const int t = threadIdx.x;
  const int64_t at = part * kPart + t * 8;
  float v[8];
  load_logits<S>(a.y, a.y_type, row * a.ldy + at, a.n - at, v);
  const float temp = temperature_of(a, row);
  const bool only_count = without_mass(a, top_k_of(a, row));
  if (t < kBins) {
    mass[t] = 0;
    count[t] = 0;
  }
  uint32_t top = kKeyNegInf;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, key_of(v[j]));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if ((t & 63) == 0) tops[t >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPartThreads / 64; ++w) top = max(top, tops[w]);
  if (t == 0) out.top[slot] = top;
  // greedy rows, and rows with NaN or infinity, go by the maximum alone
  const bool plain = temp != 0.0f && top < kKeyInf && top > kKeyNegInf;
  if (temp == 0.0f || top >= kKeyInf) return;
  const double c = octaves(temp);
  const double base = plain ? __builtin_ceil(in_octaves(value_of(top), c)) : -1e300;
  if (t == 0) out.base[slot] = base;
  int bin[8];
  uint32_t place[8];
  if (plain) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double v2 = in_octaves(v[j], c);
      bin[j] = bin_of(quarter(v2), base);
      if (bin[j] < kBins - 1) {  // what is below counts nothing
        place[j] = atomicAdd(&count[bin[j]], 1u);
        if (!only_count) atomicAdd(&mass[bin[j]], (unsigned long long)fixed_of(exp2_of(v2 - base)));
      }
    }
  }
  __syncthreads();
  // sums up to and with each bin
  uint32_t n = 0;
  uint64_t m = 0;
  if (t < kBins) {
    n = (uint32_t)wave_scan64(count[t]);
    m = wave_scan64(mass[t]);
    if ((t & 63) == 63) {
      waves[t >> 6] = n;
      wave_mass[t >> 6] = m;
    }
  }
  __syncthreads();
  if (t < kBins) {
    for (int w = 0; w < (t >> 6); ++w) {
      n += waves[w];
      m += wave_mass[w];
    }
    before[t] = n - count[t];
    out.count[slot * kBins + t] = (uint16_t)n;
    if (!only_count) out.mass[slot * kBins + t] = m;
  }
  __syncthreads();
  if (!plain) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (bin[j] < kBins - 1) order[before[bin[j]] + place[j]] = (uint16_t)(t * 8 + j);
  __syncthreads();
  if ((uint32_t)t * 8 < before[kBins - 1])
    *reinterpret_cast<uint4*>(out.order + slot * kPart + t * 8) = *reinterpret_cast<const uint4*>(order + t * 8);
}

// A token's place in the order: value first, then its number
__device__ __forceinline__ uint64_t place_of(uint32_t key, int token) {
  return ((uint64_t)key << 32) | (uint32_t)~token;
}

struct RowShared {
  double base[kMostParts];          // of the parts
  uint32_t top[kMostParts];
  int down[kMostParts];             // octaves from the row's base down to the part's
  int first[kMostParts], until[kMostParts];  // of the parts' tokens in a walk: in their order, and summed up
  unsigned long long kept[kMostParts];  // mass of a part's kept tokens
  unsigned long long mass[kBins];   // in the row's unit, up to and with the bin
  uint32_t count[kBins];
  unsigned long long sub_mass[kBins];
  uint32_t sub_count[kBins];
  uint64_t red[2][16];
  uint64_t list[kList], list_mass[kList], few[64], few_mass[64];
  uint64_t out[4];
  uint32_t fill, found;
  int pick;
};

template <int S>
__device__ __forceinline__ float one_logit(const SampleArgs& a, int64_t row, int64_t at) {
  const int64_t o = row * a.ldy + at;
  if constexpr (S == 4) return static_cast<const float*>(a.y)[o];
  else if (a.y_type == 2) return (float)static_cast<const _Float16*>(a.y)[o];
  else return (float)static_cast<const bf16_t*>(a.y)[o];
}

// u in [0, 1) of w, rounded down
__device__ __forceinline__ uint64_t share_of(uint64_t w, float u) {
  const float x = u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
  return __umul64hi(w, (uint64_t)((double)x * 0x1p64));
}

// ---------------------------------------------------------------------------
// a row's draw

template <int S>
__global__ __launch_bounds__(kRowThreads) void sample_rows_kernel(SampleArgs a, Parts in, int parts, int unit) {
  __shared__ RowShared s;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63;

  // the parts' maxima and bases, and the row's
  const float temp = temperature_of(a, row);
  const int64_t k = top_k_of(a, row);
  const float top_p = a.top_p ? a.top_p[row] : 1.0f, min_p = a.min_p ? a.min_p[row] : 0.0f, u = a.u[row];
  for (int p = t; p < parts; p += kRowThreads) {
    s.top[p] = in.top[row * parts + p];
    s.base[p] = in.base[row * parts + p];
    s.kept[p] = 0;
  }
  // Four threads a bin have a part's sums on their way before it is known where they belong (one
  // row 16.0 us, 14.7 with them; garbage where the row goes by its maximum)
  const bool only_count = without_mass(a, k);
  const int own_bin = t & (kBins - 1), part0 = t / kBins;
  uint32_t early_n[kEarly];
  uint64_t early_m[kEarly];
#pragma unroll
  for (int e = 0; e < kEarly; ++e) {
    const int p = min(part0 + e * (kRowThreads / kBins), parts - 1);
    early_n[e] = in.count[(row * parts + p) * kBins + own_bin];
  }
  if (!only_count)
#pragma unroll
    for (int e = 0; e < kEarly; ++e) {
      const int p = min(part0 + e * (kRowThreads / kBins), parts - 1);
      early_m[e] = in.mass[(row * parts + p) * kBins + own_bin];
    }
  if (t < kBins) {
    s.mass[t] = 0;
    s.count[t] = 0;
  }
  if (t == 0) s.found = 0xFFFFFFFFu;
  __syncthreads();
  uint32_t top = kKeyNegInf;
  double base = -1e300;
  for (int p = lane; p < parts; p += 64) {
    top = max(top, s.top[p]);
    base = fmax(base, s.base[p]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    top = max(top, (uint32_t)__shfl_xor((int)top, d));
    base = fmax(base, __shfl_xor(base, d));
  }
  if (temp == 0.0f || top >= kKeyInf || top == kKeyNegInf) {
    // the lowest token of the largest value, in the first part that has it
    if (top > kKeyNegInf) {
      int p = 0;
      while (s.top[p] != top) ++p;
      for (int64_t at = (int64_t)p * kPart + t; at < (int64_t)(p + 1) * kPart && at < a.n; at += kRowThreads)
        if (key_of(one_logit<S>(a, row, at)) == top) atomicMin(&s.found, (uint32_t)at);
    }
    __syncthreads();
    if (t == 0) {
      a.idx[row] = (int32_t)s.found;
      if (a.prob) a.prob[row] = s.found == 0xFFFFFFFFu ? 0.0f : 1.0f;
    }
    return;
  }

  const double c = octaves(temp);
  const int up = kUnit - unit;  // from the row's unit to a part's, at the same base
  // a token's weight in the unit of its part, and a part's mass in the row's
  auto weigh = [&](int p, float y) { return fixed_of(exp2_of(in_octaves(y, c) - s.base[p])); };
  auto to_row = [&](int p, uint64_t w) { return s.down[p] + up < 64 ? w >> (s.down[p] + up) : 0; };
  // of a place in the list
  auto token_of = [](uint64_t place) { return (int)~(uint32_t)place; };
  auto logit_of = [](uint64_t place) { return value_of((uint32_t)(place >> 32)); };
  auto mass_of = [&](uint64_t place) {
    const int p = token_of(place) / kPart;
    return to_row(p, weigh(p, logit_of(place)));
  };
  for (int p = t; p < parts; p += kRowThreads) {
    const double d = base - s.base[p];
    s.down[p] = d < 1000.0 ? (int)d : 1000;
  }
  __syncthreads();
  // the row's sums up to and with each bin; in the last bin there are the other tokens, without
  // mass
  const bool by_k = k < a.n, by_p = top_p < 1.0f, by_min = min_p > 0.0f;
  auto add_part = [&](int p, uint32_t n, uint64_t m) {
    const int down = s.down[p], r = own_bin + 4 * down;
    if (r >= kBins - 1) return;
    if (n) atomicAdd(&s.count[r], n);
    if (m) atomicAdd(&s.mass[r], (unsigned long long)to_row(p, m));
  };
#pragma unroll
  for (int e = 0; e < kEarly; ++e) {
    const int p = part0 + e * (kRowThreads / kBins);
    if (p < parts) add_part(p, early_n[e], only_count ? 0 : early_m[e]);
  }
  for (int p = part0 + kEarly * (kRowThreads / kBins); p < parts; p += kRowThreads / kBins) {
    const int64_t at = (row * parts + p) * kBins + own_bin;
    add_part(p, in.count[at], only_count ? 0 : in.mass[at]);
  }
  if (t == kBins - 1) s.count[t] = (uint32_t)a.n;
  __syncthreads();
  const uint64_t full = s.mass[kBins - 2];

  const double v2_top = in_octaves(value_of(top), c);
  const double least = by_min ? v2_top + log2((double)fminf(min_p, 1.0f)) : -1e308;  // of v2
  const int bin_min = by_min ? bin_of(quarter(least), base) : kBins - 1;

  // the smallest value that lies in `bin` or above; all values are in the last bin or above
  auto lowest = [&](int bin) {
    if (bin >= kBins - 1) return -INFINITY;
    if (bin < 0) return INFINITY;
    const double least2 = (base * 4.0 - bin) * 0.25;  // of v2
    const double guess = fmin(fmax(least2 / c, -3.4028234e38), 3.4028234e38);
    uint32_t key = key_of((float)guess);
    // the guess is off by a step at most (two where a zero of either sign lies there)
    for (int i = 0; i < 4 && key < kKeyInf && !(in_octaves(value_of(key), c) >= least2); ++i) ++key;
    for (int i = 0; i < 4 && key > kKeyNegInf + 1 && in_octaves(value_of(key - 1), c) >= least2; ++i) --key;
    return value_of(key);
  };
  // first bin at which a sum (which never falls) reaches what is wanted, or the last
  auto first_bin = [&](auto reaches) {
    if (t == 0) s.pick = kBins - 1;
    __syncthreads();
    if (t < kBins - 1 && reaches(t) && (t == 0 || !reaches(t - 1))) s.pick = t;
    __syncthreads();
    const int bin = s.pick;
    __syncthreads();
    return bin;
  };
  auto bin_at_count = [&](uint64_t want) { return first_bin([&](int b) { return s.count[b] >= want; }); };
  auto bin_at_mass = [&](uint64_t want) { return first_bin([&](int b) { return s.mass[b] >= want; }); };
  // kept: a token with less mass before it than this, top-p's share of w rounded up
  auto mass_wanted = [&](uint64_t w) {
    const uint64_t p = top_p > 0.0f ? (uint64_t)((double)top_p * 0x1p64) : 0;
    const uint64_t want = (uint64_t)__umul64hi(w, p) + (w * p != 0 ? 1 : 0);
    return want ? want : 1;
  };

  // Tokens of the bins from b0 to b1: where each part has its own, and how many there are
  auto set_walk = [&](int b0, int b1) {
    uint64_t n = 0;
    if (t < parts) {
      const int64_t at = (row * parts + t) * kBins;
      const int j0 = b0 - 4 * s.down[t] - 1, j1 = b1 - 4 * s.down[t];
      const int first = j0 >= 0 ? in.count[at + j0] : 0;
      n = j1 >= 0 ? in.count[at + j1] - first : 0;
      s.first[t] = first;
    }
    uint64_t all;
    const uint64_t before = scan64(n, s.red, &all);
    if (t < parts) {
      s.first[t] -= (int)before;
      s.until[t] = (int)(before + n);
    }
    __syncthreads();
    return (int)all;
  };
  // the i-th of them
  auto token_at = [&](int i) {
    int p = 0;
    for (int step = kMostParts / 2; step; step >>= 1)
      if (p + step <= parts - 1 && s.until[p + step - 1] <= i) p += step;
    return p * kPart + in.order[(row * parts + p) * kPart + s.first[p] + i];
  };
  auto walk_bins = [&](int n, auto f) {
    for (int i = t; i < n; i += kRowThreads) {
      const int token = token_at(i);
      f(i, token, one_logit<S>(a, row, token));
    }
  };
  // into the list, which has room
  auto gather_bins = [&](int b0, int b1) {
    const int n = set_walk(b0, b1);
    walk_bins(min(n, kList), [&](int i, int token, float y) { s.list[i] = place_of(key_of(y), token); });
    __syncthreads();
    return min(n, kList);
  };

  int bin_last = kBins - 1;
  if (by_k) bin_last = bin_at_count((uint64_t)k);
  if (by_p && !by_k) bin_last = bin_at_mass(mass_wanted(full));
  if (!by_p || !by_k) bin_last = min(bin_last, bin_min);
  bin_last = min(bin_last, kBins - 2);  // what is below weighs nothing
  bool few = s.count[bin_last] <= kList;  // all that may be kept is in the list
  int have = 0;                           // tokens there
  uint32_t key_lo = 0;
  if (few) {
    key_lo = key_of(lowest(bin_last));
    have = gather_bins(0, bin_last);
  }

  // the masses of the list
  auto weigh_list = [&]() {
    for (int i = t; i < have; i += kRowThreads) s.list_mass[i] = mass_of(s.list[i]);
  };
  weigh_list();

  // Places of the last tokens that top-k and top-p keep, the earlier of them in `cut` (0:
  // everything that weighs), and the mass of what is kept.
  uint64_t cut = 0, mass = full;
  int cut_bin = kBins - 1;
  int list_bin = -1;    // whose tokens the list has, where it has not all
  bool ranked = false;  // the list is few enough to be in s.few, with its sums
#pragma unroll 1
  for (int filter = 0; filter < 2; ++filter) {
    const bool by_count = filter == 0;
    if (!(by_count ? by_k : by_p)) continue;
    if (few && by_count && k >= have) continue;  // all that weighs
    if (few && !by_count && by_k && !ranked) {  // of the tokens of the list that top-k keeps
      uint64_t sum = 0;
      for (int i = t; i < have; i += kRowThreads) sum += s.list[i] >= cut ? s.list_mass[i] : 0;
      scan64(sum, s.red, &mass);
    }
    const uint64_t want = by_count ? (uint64_t)k : mass_wanted(mass);
    // the interval of places from lo to hi, and the tokens there and before it
    uint64_t inside = have, n_before = 0, m_before = 0;
    uint64_t lo = (uint64_t)key_lo << 32, hi = ((uint64_t)top << 32) | 0xFFFFFFFFu;
    if (!few) {
      const int bin = cut_bin = by_count ? bin_at_count(want) : bin_at_mass(want);
      if (bin == kBins - 1) continue;  // only what weighs nothing is cut off
      n_before = bin ? s.count[bin - 1] : 0;
      m_before = bin ? s.mass[bin - 1] : 0;
      inside = s.count[bin] - n_before;
      if (inside > kList) {
        set_walk(bin, bin);
      } else {
        have = gather_bins(bin, bin);
        weigh_list();
        list_bin = bin;
      }
      lo = (uint64_t)key_of(lowest(bin)) << 32;
      hi = ((uint64_t)(key_of(lowest(bin - 1)) - 1) << 32) | 0xFFFFFFFFu;
    }
    const bool in_list = inside <= kList;
    const int in_bin = (int)inside;
    // narrower by 256 at a time, until a wave can order the few that are left
    while (!ranked) {
      const bool order = inside <= 64;
      // numbers go no further than n; where the key is known, they alone differ
      if ((lo >> 32) == (hi >> 32)) {
        const uint64_t last_place = place_of((uint32_t)(hi >> 32), (int)(a.n - 1));
        lo = lo > last_place ? lo : last_place;
      }
      const int shift = hi - lo < kBins ? 0 : 64 - 8 - __builtin_clzll(hi - lo);
      __syncthreads();
      if (t < kBins) {
        s.sub_mass[t] = 0;
        s.sub_count[t] = 0;
      }
      if (t == 0) {
        s.found = 0xFFFFFFFFu;
        s.pick = 0;
        s.fill = 0;
      }
      __syncthreads();
      auto add = [&](uint64_t place, uint64_t w) {
        if (place < lo || place > hi) return;
        if (order) {
          const uint32_t at = atomicAdd(&s.fill, 1u);
          if (at < 64) {
            s.few[at] = place;
            s.few_mass[at] = w;
          }
        } else {
          const uint32_t j = (uint32_t)((hi - place) >> shift);
          atomicAdd(&s.sub_count[j], 1u);
          if (w) atomicAdd(&s.sub_mass[j], (unsigned long long)w);
        }
      };
      if (in_list) {
        for (int i = t; i < have; i += kRowThreads) add(s.list[i], s.list_mass[i]);
      } else {
        walk_bins(in_bin, [&](int, int token, float y) {
          const int p = token / kPart;
          add(place_of(key_of(y), token), to_row(p, weigh(p, y)));
        });
      }
      __syncthreads();
      if (order) break;
      // the first that reaches it, or the last that has any
      const uint64_t nm[2] = {t < kBins ? s.sub_count[t] : 0, t < kBins ? s.sub_mass[t] : 0};
      uint64_t before[2], ignored[2];
      scan64<2>(nm, before, ignored, s.red);
      const uint64_t n = n_before + before[0], m = m_before + before[1];
      if (nm[0] && (by_count ? n + nm[0] >= want : m + nm[1] >= want)) atomicMin(&s.found, (uint32_t)t);
      if (nm[0]) atomicMax(&s.pick, t);
      __syncthreads();
      const uint32_t found = s.found != 0xFFFFFFFFu ? s.found : (uint32_t)s.pick;
      if (t == (int)found) {
        s.out[0] = nm[0];
        s.out[1] = n;
        s.out[2] = m;
      }
      __syncthreads();
      inside = s.out[0];
      n_before = s.out[1];
      m_before = s.out[2];
      hi -= (uint64_t)found << shift;
      const uint64_t span = ((uint64_t)1 << shift) - 1;
      lo = hi - lo > span ? hi - span : lo;
    }
    // each of the few against four of them a wave
    const int left = min((int)s.fill, 64);
    const uint64_t place = lane < left ? s.few[lane] : 0;
    if (!ranked) {
      uint32_t up_to = 0;
      uint64_t mass_up_to = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = (t >> 6) * 4 + e;
        const bool first = i < left && s.few[i] >= place;
        up_to += first ? 1 : 0;
        mass_up_to += first ? s.few_mass[i] : 0;
      }
      if (lane < left && up_to) {
        atomicAdd(&s.sub_count[lane], up_to);
        atomicAdd(&s.sub_mass[lane], (unsigned long long)mass_up_to);
      }
      ranked = few && have <= 64;
    }
    __syncthreads();
    if (t < 64) {
      const uint64_t n = n_before + s.sub_count[t], m = m_before + s.sub_mass[t];
      // the first in their order that reaches it, else the last
      const bool reaches = t < left && (by_count ? n >= want : m >= want);
      const int reaching = __builtin_popcountll(__builtin_amdgcn_ballot_w64(reaches));
      if (t < left && (int)s.sub_count[t] == left - (reaching ? reaching - 1 : 0)) {
        s.out[0] = place;
        s.out[1] = m;
      }
    }
    __syncthreads();
    cut = s.out[0] > cut ? s.out[0] : cut;
    if (by_count) mass = s.out[1];
    if (!few && only_count) {  // what top-k keeps: there was no room for all of its last bin
      if (t == 0) s.fill = 0;
      const int n = set_walk(0, cut_bin);
      walk_bins(n, [&](int, int token, float y) {
        const uint64_t place = place_of(key_of(y), token);
        if (place < cut) return;
        const uint32_t at = atomicAdd(&s.fill, 1u);
        if (at < kList) s.list[at] = place;
      });
      __syncthreads();
      have = min((int)s.fill, kList);
      few = true;
      key_lo = (uint32_t)(cut >> 32);
      weigh_list();
      __syncthreads();
    }
  }

  if (few) {
    // the kept tokens' masses: of parts, of the drawn part's blocks of 64, of its tokens
    for (int i = t; i < have; i += kRowThreads) {
      const uint64_t place = s.list[i], w = s.list_mass[i];
      const bool keep = place >= cut && (!by_min || in_octaves(logit_of(place), c) >= least ||
                                         (uint32_t)(place >> 32) == top);
      if (!keep) s.list_mass[i] = 0;
      else if (w) atomicAdd(&s.kept[token_of(place) / kPart], (unsigned long long)w);
    }
    if (t < 64) {
      s.sub_mass[t] = 0;
      s.few_mass[t] = 0;
    }
    __syncthreads();
    uint64_t total;
    const uint64_t m = t < parts ? s.kept[t] : 0, before = scan64(m, s.red, &total);
    const uint64_t target = share_of(total, u);
    if (target >= before && target < before + m) {
      s.pick = t;
      s.out[2] = target - before;
    }
    __syncthreads();
    const int part = s.pick;
    for (int i = t; i < have; i += kRowThreads) {
      const int token = token_of(s.list[i]);
      if (token / kPart == part) atomicAdd(&s.sub_mass[token % kPart / 64], (unsigned long long)s.list_mass[i]);
    }
    __syncthreads();
    if (t < 64) {
      const uint64_t m = s.sub_mass[t], sum = wave_scan64(m), rest = s.out[2];
      if (rest >= sum - m && rest < sum) {
        s.found = (uint32_t)t;
        s.out[3] = rest - (sum - m);
      }
    }
    __syncthreads();
    const int block = part * (kPart / 64) + (int)s.found;
    for (int i = t; i < have; i += kRowThreads) {
      const int token = token_of(s.list[i]);
      if (token / 64 == block) s.few_mass[token % 64] = s.list_mass[i];
    }
    __syncthreads();
    if (t < 64) {
      const uint64_t m = s.few_mass[t], sum = wave_scan64(m), rest = s.out[3];
      if (rest >= sum - m && rest < sum) {
        const int token = block * 64 + t;
        a.idx[row] = token;
        if (a.prob)
          a.prob[row] = (float)(exp2_of(in_octaves(one_logit<S>(a, row, token), c) - base) /
                                __builtin_ldexp((double)total, -unit));
      }
    }
    return;
  }

  // Many tokens.
  const int bin_cut = cut ? bin_of(quarter(in_octaves(logit_of(cut), c)), base) : kBins;
  // kept: the bins before `last`, and in it what both the cut and min-p leave
  const int last = min(bin_cut, by_min ? bin_min : kBins);
  const float last_lo = lowest(min(last, kBins - 2)), last_hi = lowest(last - 1);
  auto kept = [&](int token, float y) {
    if (!(y >= last_lo)) return false;
    if (y >= last_hi || last > kBins - 2) return true;
    if (place_of(key_of(y), token) < cut) return false;
    return !by_min || in_octaves(y, c) >= least || key_of(y) == top;
  };
  // the bins before the last one, in the part's own unit
  if (t < parts) {
    const int b = min(last, kBins - 1) - 1 - 4 * s.down[t];
    s.kept[t] = b >= 0 ? in.mass[(row * parts + t) * kBins + b] : 0;
  }
  __syncthreads();
  if (last < kBins - 1) {
    auto add = [&](int token, float y) {
      if (kept(token, y)) atomicAdd(&s.kept[token / kPart], (unsigned long long)weigh(token / kPart, y));
    };
    if (last == list_bin) {
      for (int i = t; i < have; i += kRowThreads) add(token_of(s.list[i]), logit_of(s.list[i]));
    } else {
      walk_bins(set_walk(last, last), [&](int, int token, float y) { add(token, y); });
    }
  }
  __syncthreads();
  // the part that the draw falls into, and what is left of it there
  uint64_t total;
  const uint64_t m = t < parts ? to_row(t, s.kept[t]) : 0, before = scan64(m, s.red, &total);
  const uint64_t target = share_of(total, u);
  if (target >= before && target < before + m) {
    s.pick = t;
    s.out[2] = (target - before) << (s.down[t] + up);
  }
  __syncthreads();
  const int part = s.pick;
  const uint64_t rest = s.out[2];
  const int64_t at = (int64_t)part * kPart + t * 4;
  uint64_t x[4], sum = 0, ignored;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = 0;
    if (at + e < a.n) {
      const float y = one_logit<S>(a, row, at + e);
      if (kept((int)(at + e), y) && bin_of(quarter(in_octaves(y, c)), s.base[part]) < kBins - 1) x[e] = weigh(part, y);
    }
    sum += x[e];
  }
  uint64_t run = scan64(sum, s.red, &ignored);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (rest >= run && rest < run + x[e]) {
      a.idx[row] = (int32_t)(at + e);
      if (a.prob)
        a.prob[row] = (float)(exp2_of(in_octaves(one_logit<S>(a, row, at + e), c) - base) /
                              __builtin_ldexp((double)total, -unit));
    }
    run += x[e];
  }
}

int parts_of(int64_t n) { return (int)((n + kPart - 1) / kPart); }

}  // namespace

size_t sample_workspace_bytes(int64_t n, int64_t b) { return parts_layout(b, parts_of(n), nullptr, nullptr); }

hipError_t launch_sample(const SampleArgs& a, void* ws, hipStream_t st) {
  const int parts = parts_of(a.n);
  // the row's unit: as fine as leaves room for n weights in 62 bits
  int bits = 0;
  while (((int64_t)1 << bits) < a.n) ++bits;
  const int unit = min(kUnit - 2, 62 - bits);
  Parts p;
  parts_layout(a.b, parts, ws, &p);
  const dim3 grid((unsigned)parts, (unsigned)a.b);
  if (a.y_type == 1) {
    sample_parts_kernel<4><<<grid, kPartThreads, 0, st>>>(a, p);
    sample_rows_kernel<4><<<(unsigned)a.b, kRowThreads, 0, st>>>(a, p, parts, unit);
  } else {
    sample_parts_kernel<2><<<grid, kPartThreads, 0, st>>>(a, p);
    sample_rows_kernel<2><<<(unsigned)a.b, kRowThreads, 0, st>>>(a, p, parts, unit);
  }
  return hipGetLastError();
}

}  // namespace lowbit
