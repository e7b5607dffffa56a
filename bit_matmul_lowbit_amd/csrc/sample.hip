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
// the part's maximum, its weights relative to 2^ceil of that maximum, and
// a histogram of them by quarters of an octave (count and mass).  Bins are places
// on one scale for all parts, so parts are added without being read again.  The second
// launch, a work-group a row, adds the histograms and finds the bin in which
// each filter ends.  Where few tokens come before that (kList), they are
// gathered, sorted and drawn from in LDS.  Otherwise the bin is narrowed by the
// bits of its values until its end is one token, the kept mass of every part
// is known, and only the part in which the draw falls is walked.
//
// Weights are exact to 2^-40 (FP64, which runs at the rate of FP32 here) and
// masses are 64-bit whole numbers, so that sums have no order: LDS atomics may come as
// they like, equal inputs give equal bits, and a draw among 150000 tokens finds the
// token that 64-bit arithmetic finds.
#include "pieces.h"

namespace lowbit {
namespace {

constexpr int kPart = 4096;      // logits of a part
constexpr int kPartThreads = 256;
constexpr int kBins = 256;       // quarters of an octave; the last one: everything below
constexpr int kRowThreads = 1024;
constexpr int kMostParts = 256;
constexpr int kList = 2048;      // tokens that are sorted in LDS
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
__device__ __forceinline__ double octaves(float t) { return 1.4426950408889634074 / (double)t; }

// what the first launch leaves of a part
struct Parts {
  double* base;      // [rows][parts]: weights are relative to 2^base
  uint32_t* top;     // [rows][parts]: the largest key
  uint64_t* mass;    // [rows][parts][kBins]
  uint16_t* count;   // [rows][parts][kBins]
};
__host__ __device__ inline size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
inline size_t parts_layout(int64_t rows, int64_t parts, void* ws, Parts* p) {
  char* at = static_cast<char*>(ws);
  const size_t n = (size_t)(rows * parts);
  const size_t mass = align_up(n * kBins * 8), count = align_up(n * kBins * 2), base = align_up(n * 8), top = align_up(n * 4);
  if (p) {
    p->mass = reinterpret_cast<uint64_t*>(at);
    p->count = reinterpret_cast<uint16_t*>(at + mass);
    p->base = reinterpret_cast<double*>(at + mass + count);
    p->top = reinterpret_cast<uint32_t*>(at + mass + count + base);
  }
  return mass + count + base + top;
}

// the quarter octave of v2 = y log2(e) / T on the scale of all parts
__device__ __forceinline__ double quarter(double v2) { return __builtin_floor(v2 * 4.0); }
__device__ __forceinline__ int bin_of(double q, double base) {
  const double b = base * 4.0 - 1.0 - q;
  return b < 0.0 ? 0 : b >= kBins - 1 ? kBins - 1 : (int)b;
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

template <int S>
__global__ __launch_bounds__(kPartThreads) void sample_parts_kernel(SampleArgs a, Parts out) {
  __shared__ unsigned long long mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ uint32_t top4[4];
  const int64_t row = blockIdx.y, part = blockIdx.x, slot = row * gridDim.x + part;
  const int64_t from = part * kPart;
  const int t = threadIdx.x;
  mass[t] = 0;
  count[t] = 0;
  float v[2][8];
  uint32_t top = kKeyNegInf;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = from + (h * kPartThreads + t) * 8;
    load_logits<S>(a.y, a.y_type, row * a.ldy + at, a.n - at, v[h]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, key_of(v[h][j]));
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if ((t & 63) == 0) top4[t >> 6] = top;
  __syncthreads();
  top = max(max(top4[0], top4[1]), max(top4[2], top4[3]));
  const float temp = temperature_of(a, row);
  // greedy rows, and rows with NaN or infinity, go by the maximum alone
  const bool plain = temp != 0.0f && top < kKeyInf && top > kKeyNegInf;
  const double c = plain ? octaves(temp) : 0.0;
  const double base = plain ? __builtin_ceil((double)value_of(top) * c) : -1e300;
  if (plain) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double v2 = (double)v[h][j] * c;
        const int bin = bin_of(quarter(v2), base);
        if (bin < kBins - 1) {  // what is below counts nothing, and is counted from the others
          atomicAdd(&count[bin], 1u);
          atomicAdd(&mass[bin], (unsigned long long)fixed_of(exp2_of(v2 - base)));
        }
      }
  }
  __syncthreads();
  out.mass[slot * kBins + t] = mass[t];
  out.count[slot * kBins + t] = (uint16_t)count[t];
  if (t == 0) {
    out.base[slot] = base;
    out.top[slot] = top;
  }
}

// ---------------------------------------------------------------------------
// one work-group a row

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int d) { return (uint64_t)__shfl_up((unsigned long long)v, d); }

// Sum of v over the threads before this one; *total: over all (1024 threads).
__device__ __forceinline__ uint64_t scan64(uint64_t v, uint64_t* red, uint64_t* total) {
  const int t = threadIdx.x;
  uint64_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = shfl_up64(s, d);
    if ((t & 63) >= d) s += o;
  }
  __syncthreads();
  if ((t & 63) == 63) red[t >> 6] = s;
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRowThreads / 64; ++w) {
    if (w < (t >> 6)) before += red[w];
    all += red[w];
  }
  *total = all;
  return before + s - v;
}

// Descending (or ascending) order of size = a power of two entries in LDS
template <typename T, bool DESCENDING>
__device__ __forceinline__ void sort_lds(T* v, int size) {
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kRowThreads) {
        const int lo = 2 * j * (i / j) + i % j, hi = lo + j;
        const bool up = ((lo & k) == 0) != DESCENDING;
        const T x = v[lo], y = v[hi];
        if ((x > y) == up) {
          v[lo] = y;
          v[hi] = x;
        }
      }
      __syncthreads();
    }
}

// A token's place in the order: value first, then its number
__device__ __forceinline__ uint64_t place_of(uint32_t key, int token) {
  return ((uint64_t)key << 32) | (uint32_t)~token;
}

struct RowShared {
  double base[kMostParts];          // of the parts
  uint64_t kept[kMostParts];        // mass of a part's kept tokens, in its own unit
  int down[kMostParts];             // octaves from the row's base down to the part's
  unsigned long long mass[kBins];   // in the row's unit
  uint32_t count[kBins];
  uint64_t red[16];
  uint64_t list[kList], weight[kList];
  uint32_t order[kList];
  uint32_t fill;
  uint32_t found;
  uint64_t found64;
  int pick;
};

// Calls f(part, token, value) for the tokens of the parts that use(part) names
template <int S, class U, class F>
__device__ __forceinline__ void walk_row(const SampleArgs& a, int64_t row, int parts, U use, F f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int p = wave; p < parts; p += kRowThreads / 64) {
    if (!use(p)) continue;
    for (int i = 0; i < kPart / 512; ++i) {
      const int64_t at = (int64_t)p * kPart + i * 512 + lane * 8;
      if (at >= a.n) break;
      float v[8];
      load_logits<S>(a.y, a.y_type, row * a.ldy + at, a.n - at, v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < a.n) f(p, (int)at + j, v[j]);
    }
  }
}

// u in [0, 1) of w, rounded down
__device__ __forceinline__ uint64_t share_of(uint64_t w, float u) {
  const float x = u > 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
  return __umul64hi(w, (uint64_t)((double)x * 0x1p64));
}

// The last token that a filter keeps: `place` within `bin`.  Tokens up to and with
// it have the mass `mass` and the number `count`.
struct Cut {
  int bin;
  uint64_t place, mass;
};

template <int S>
__global__ __launch_bounds__(kRowThreads) void sample_rows_kernel(SampleArgs a, Parts in, int parts, int unit) {
  __shared__ RowShared s;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  const uint32_t* tops = in.top + row * parts;
  const double* bases = in.base + row * parts;

  // the row's maximum and base
  uint32_t top = kKeyNegInf;
  double base = -1e300;
  for (int p = t & 63; p < parts; p += 64) {
    top = max(top, tops[p]);
    base = fmax(base, bases[p]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    top = max(top, (uint32_t)__shfl_xor((int)top, d));
    base = fmax(base, __shfl_xor(base, d));
  }
  const float temp = temperature_of(a, row);
  if (temp == 0.0f || top >= kKeyInf || top == kKeyNegInf) {
    // the lowest token of the largest value
    if (t == 0) s.found = 0xFFFFFFFFu;
    __syncthreads();
    if (top != kKeyNegInf)
      walk_row<S>(a, row, parts, [&](int p) { return tops[p] == top; },
                  [&](int, int token, float y) {
                    if (key_of(y) == top) atomicMin(&s.found, (uint32_t)token);
                  });
    __syncthreads();
    if (t == 0) {
      a.idx[row] = (int32_t)s.found;
      if (a.prob) a.prob[row] = s.found == 0xFFFFFFFFu ? 0.0f : 1.0f;
    }
    return;
  }

  const double c = octaves(temp);
  const int up = kUnit - unit;  // from the row's unit to a part's, at the same base
  for (int p = t; p < parts; p += kRowThreads) {
    const double d = base - bases[p];
    s.base[p] = bases[p];
    s.down[p] = d < 1000.0 ? (int)d : 1000;
  }
  if (t < kBins) {
    s.mass[t] = 0;
    s.count[t] = 0;
  }
  __syncthreads();
  // the row's histogram: four threads a bin
  {
    const int r = t & (kBins - 1);
    uint64_t m = 0;
    uint32_t n = 0;
    if (r < kBins - 1)
      for (int p = t / kBins; p < parts; p += kRowThreads / kBins) {
        const int j = r - 4 * s.down[p];
        if (j < 0) continue;
        const int64_t at = (row * parts + p) * kBins + j;
        m += s.down[p] + up < 64 ? in.mass[at] >> (s.down[p] + up) : 0;
        n += in.count[at];
      }
    if (n) atomicAdd(&s.count[r], n);
    if (m) atomicAdd(&s.mass[r], (unsigned long long)m);
  }
  __syncthreads();
  // sums up to and with each bin (the last bin has the rest of the tokens, and no mass)
  uint64_t all_mass;
  {
    const uint64_t m = t < kBins ? s.mass[t] : 0, n = t < kBins ? s.count[t] : 0;
    const uint64_t bm = scan64(m, s.red, &all_mass);
    uint64_t dummy;
    const uint64_t bn = scan64(n, s.red, &dummy);
    __syncthreads();
    if (t < kBins) {
      s.mass[t] = bm + m;
      s.count[t] = t == kBins - 1 ? (uint32_t)a.n : (uint32_t)(bn + n);
    }
    __syncthreads();
  }
  const uint64_t full = all_mass;

  int64_t k = a.top_k ? a.top_k[row] : 0;
  if (k <= 0 || k > a.n) k = a.n;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f;
  const bool by_p = top_p < 1.0f;
  const float min_p = a.min_p ? a.min_p[row] : 0.0f;
  const bool by_min = min_p > 0.0f;
  const double v2_top = (double)value_of(top) * c;
  const double least = by_min ? v2_top + log2((double)fminf(min_p, 1.0f)) : -1e308;  // of v2
  const int bin_min = by_min ? bin_of(quarter(least), base) : kBins - 1;

  // first bin at which a sum (which never falls) reaches what is wanted, or the last
  auto first_bin = [&](auto reaches) {
    __syncthreads();
    if (t == 0) s.pick = kBins - 1;
    __syncthreads();
    if (t < kBins - 1 && reaches(t) && (t == 0 || !reaches(t - 1))) s.pick = t;
    __syncthreads();
    return s.pick;
  };
  auto bin_at_count = [&](uint64_t want) { return first_bin([&](int b) { return s.count[b] >= want; }); };
  auto bin_at_mass = [&](uint64_t want) { return first_bin([&](int b) { return s.mass[b] >= want; }); };
  // kept: a token with less mass before it than this, top-p's share of w rounded up
  auto mass_wanted = [&](uint64_t w) {
    const uint64_t p = top_p > 0.0f ? (uint64_t)((double)top_p * 0x1p64) : 0;
    return max((uint64_t)1, __umul64hi(w, p) + (w * p != 0 ? 1 : 0));
  };

  int bin_k = kBins - 1, bin_last = kBins - 1;
  if (k < a.n) bin_k = bin_last = bin_at_count((uint64_t)k);
  if (by_p && k == a.n) bin_last = bin_at_mass(mass_wanted(full));
  if (!by_p || k == a.n) bin_last = min(bin_last, bin_min);

  if (s.count[bin_last] <= kList) {
    // few tokens: in LDS
    if (t == 0) s.fill = 0;
    __syncthreads();
    walk_row<S>(a, row, parts, [&](int p) { return bin_of(quarter((double)value_of(tops[p]) * c), base) <= bin_last; },
                [&](int, int token, float y) {
                  if (bin_of(quarter((double)y * c), base) <= bin_last) {
                    const uint32_t at = atomicAdd(&s.fill, 1u);
                    if (at < kList) s.list[at] = place_of(key_of(y), token);
                  }
                });
    __syncthreads();
    const int have = min((int)s.fill, kList);
    int size = 2;
    while (size < have) size <<= 1;
    for (int i = have + t; i < size; i += kRowThreads) s.list[i] = 0;
    __syncthreads();
    sort_lds<uint64_t, true>(s.list, size);
    // two neighbours a thread, weights in units of 2^-51 of the row's base
    uint64_t w[2], sum = 0, before, ignored;
    double v2[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * t + e;
      v2[e] = i < have ? (double)value_of((uint32_t)(s.list[i] >> 32)) * c : -1e308;
      w[e] = i < have && i < k ? fixed_of(exp2_of(v2[e] - base)) : 0;
      sum += w[e];
    }
    uint64_t total;
    before = scan64(sum, s.red, &total);
    uint64_t want = mass_wanted(k < a.n ? total : full);
    if (k == a.n) want = want >> (63 - up) ? UINT64_MAX : want << up;
    uint64_t kept_sum = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * t + e;
      const bool keep = i < have && i < k && (i == 0 || ((!by_p || before < want) && (!by_min || v2[e] >= least)));
      before += w[e];
      if (!keep) w[e] = 0;
      kept_sum += w[e];
      if (i < kList) {
        s.weight[i] = w[e];
        // by number: those that are not kept weigh nothing wherever they are
        if (i < size) s.order[i] = i < have ? ((~(uint32_t)s.list[i]) << 11) | (uint32_t)i : 0xFFFFFFFFu;
      }
    }
    uint64_t kept;
    scan64(kept_sum, s.red, &kept);
    __syncthreads();
    sort_lds<uint32_t, false>(s.order, size);
    uint64_t x[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * t + e;
      if (i < have) x[e] = s.weight[s.order[i] & 2047u];
    }
    uint64_t at = scan64(x[0] + x[1], s.red, &ignored);
    const uint64_t target = share_of(kept, a.u[row]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * t + e;
      if (i < have && target >= at && target < at + x[e]) {
        a.idx[row] = (int32_t)(s.order[i] >> 11);
        if (a.prob) a.prob[row] = (float)((double)x[e] / (double)kept);
      }
      at += x[e];
    }
    return;
  }

  // many tokens: the place of the last kept one
  auto in_bin = [&](int bin, float y) { return bin_of(quarter((double)y * c), base) == bin; };
  auto part_has = [&](int bin, int p) {
    const int j = bin - 4 * s.down[p];
    return j >= 0 && in.count[(row * parts + p) * kBins + j] != 0;
  };
  // a token's weight in the unit of its part
  auto weigh = [&](int p, float y) { return fixed_of(exp2_of((double)y * c - s.base[p])); };
  auto to_row = [&](int p, uint64_t w) { return s.down[p] + up < 64 ? w >> (s.down[p] + up) : 0; };
  // by_count: the want-th token in order; else the first at which the mass reaches want
  auto cut_at = [&](bool by_count, uint64_t want) {
    Cut r;
    r.bin = by_count ? bin_at_count(want) : bin_at_mass(want);
    if (r.bin == kBins - 1) {  // only what weighs nothing is cut off
      r.place = 0;
      r.mass = full;
      return r;
    }
    uint64_t n_before = r.bin ? s.count[r.bin - 1] : 0, m_before = r.bin ? s.mass[r.bin - 1] : 0;
    uint32_t hi = 0xFFFFFFFFu, lo = 0;  // keys of the bin
    {
      // the values of the bin, and a little more on both sides
      const double q = base * 4.0 - 1.0 - r.bin;
      lo = key_of((float)(q * 0.25 / c));
      if (r.bin > 0) hi = key_of((float)((q + 1.0) * 0.25 / c));
      lo = lo > 4 ? lo - 4 : 0;
      hi = hi < 0xFFFFFFFBu ? hi + 4 : 0xFFFFFFFFu;
    }
    uint64_t inside = s.count[r.bin] - n_before;
    unsigned long long* sub_mass = reinterpret_cast<unsigned long long*>(s.weight);
    uint32_t* sub_count = s.order;
    while (inside > kList && hi > lo) {
      int shift = 0;
      while (((hi - lo) >> shift) >= kBins) ++shift;
      __syncthreads();
      if (t < kBins) {
        sub_mass[t] = 0;
        sub_count[t] = 0;
      }
      __syncthreads();
      walk_row<S>(a, row, parts, [&](int p) { return part_has(r.bin, p); },
                  [&](int p, int, float y) {
                    const uint32_t key = key_of(y);
                    if (key > hi || key < lo || !in_bin(r.bin, y)) return;
                    const uint32_t j = (hi - key) >> shift;
                    atomicAdd(&sub_count[j], 1u);
                    atomicAdd(&sub_mass[j], (unsigned long long)to_row(p, weigh(p, y)));
                  });
      __syncthreads();
      // the first that reaches it, or the last that has any
      uint64_t ignored;
      const uint64_t n0 = t < kBins ? sub_count[t] : 0, m0 = t < kBins ? sub_mass[t] : 0;
      const uint64_t n = n_before + scan64(n0, s.red, &ignored), m = m_before + scan64(m0, s.red, &ignored);
      if (t == 0) {
        s.found = 0xFFFFFFFFu;
        s.fill = 0;
      }
      __syncthreads();
      if (n0 && (by_count ? n + n0 >= want : m + m0 >= want)) atomicMin(&s.found, (uint32_t)t);
      if (n0) atomicMax(&s.fill, (uint32_t)t);
      __syncthreads();
      const uint32_t found = s.found != 0xFFFFFFFFu ? s.found : s.fill;
      if (t == (int)found) {
        s.red[0] = n0;
        s.red[1] = n;
        s.red[2] = m;
      }
      __syncthreads();
      inside = s.red[0];
      n_before = s.red[1];
      m_before = s.red[2];
      const uint32_t top_key = hi - (found << shift);
      const uint32_t span = ((uint32_t)1 << shift) - 1;
      lo = top_key - lo > span ? top_key - span : lo;
      hi = top_key;
    }
    __syncthreads();
    if (inside <= kList) {
      if (t == 0) {
        s.fill = 0;
        s.found = 0xFFFFFFFFu;
      }
      __syncthreads();
      walk_row<S>(a, row, parts, [&](int p) { return part_has(r.bin, p); },
                  [&](int, int token, float y) {
                    const uint32_t key = key_of(y);
                    if (key > hi || key < lo || !in_bin(r.bin, y)) return;
                    const uint32_t at = atomicAdd(&s.fill, 1u);
                    if (at < kList) s.list[at] = place_of(key, token);
                  });
      __syncthreads();
      const int have = min((int)s.fill, kList);
      int size = 2;
      while (size < have) size <<= 1;
      for (int i = have + t; i < size; i += kRowThreads) s.list[i] = 0;
      __syncthreads();
      sort_lds<uint64_t, true>(s.list, size);
      uint64_t w[2], total;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * t + e;
        w[e] = 0;
        if (i < have) {
          const int token = (int)~(uint32_t)s.list[i];
          w[e] = to_row(token / kPart, weigh(token / kPart, value_of((uint32_t)(s.list[i] >> 32))));
        }
      }
      uint64_t m = m_before + scan64(w[0] + w[1], s.red, &total);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * t + e;
        m += w[e];
        if (i < have && (by_count ? n_before + i + 1 >= want : m >= want)) atomicMin(&s.found, (uint32_t)i);
        if (i < have) s.weight[i] = m;
      }
      __syncthreads();
      const int at = s.found != 0xFFFFFFFFu ? (int)s.found : have - 1;
      r.place = s.list[at];
      r.mass = s.weight[at];
    } else {
      // one value that very many tokens have: the one of them that is wanted, by number
      if (t < kMostParts) s.order[t] = 0;
      __syncthreads();
      walk_row<S>(a, row, parts, [&](int p) { return part_has(r.bin, p); },
                  [&](int p, int, float y) {
                    if (key_of(y) == hi) atomicAdd(&s.order[p], 1u);
                  });
      __syncthreads();
      uint64_t left = by_count ? want - n_before : 0, m = m_before;
      int part = 0;
      uint32_t nth = 0;  // from 0, within the part
      for (int p = 0; p < parts; ++p) {
        const uint32_t n = s.order[p];
        if (n == 0) continue;
        const uint64_t w = to_row(p, weigh(p, value_of(hi)));
        part = p;
        if (by_count) {
          nth = (uint32_t)(left < n ? left : n) - 1;
          if (left <= n) {
            m += w * (nth + 1);
            break;
          }
          left -= n;
        } else {
          const uint64_t need = m >= want ? 1 : w ? (want - m + w - 1) / w : (uint64_t)n + 1;
          nth = (uint32_t)(need < n ? need : n) - 1;
          if (need <= n) {
            m += w * (nth + 1);
            break;
          }
        }
        m += w * n;
      }
      // its number: counted through the part, four tokens a thread
      const int64_t at = (int64_t)part * kPart + t * 4;
      uint32_t mine = 0;
      uint64_t ignored;
      bool is[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = 0.0f;
        const bool there = at + e < a.n;
        if (there) {
          const int64_t o = row * a.ldy + at + e;
          if constexpr (S == 4) y = static_cast<const float*>(a.y)[o];
          else if (a.y_type == 2) y = (float)static_cast<const _Float16*>(a.y)[o];
          else y = (float)static_cast<const bf16_t*>(a.y)[o];
        }
        is[e] = there && key_of(y) == hi;
        mine += is[e];
      }
      uint64_t n = scan64(mine, s.red, &ignored);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (is[e] && n == nth) s.found64 = place_of(hi, (int)(at + e));
        n += is[e];
      }
      __syncthreads();
      r.place = s.found64;
      r.mass = m;
    }
    __syncthreads();
    return r;
  };

  Cut cut = {kBins, 0, full};  // everything
  if (k < a.n) cut = cut_at(true, (uint64_t)k);
  if (by_p) {
    const Cut p = cut_at(false, mass_wanted(cut.mass));
    if (p.bin < cut.bin || (p.bin == cut.bin && p.place > cut.place)) cut = p;
  }
  // kept: the bins before `last`, and in it what both the cut and min-p leave
  const int last = min(cut.bin, by_min ? bin_min : kBins);
  auto kept = [&](int token, float y) {
    const double v2 = (double)y * c;
    const int b = bin_of(quarter(v2), base);
    if (b == kBins - 1) return false;  // weighs nothing
    if (b != last) return b < last;
    if (b == cut.bin && place_of(key_of(y), token) < cut.place) return false;
    return !by_min || v2 >= least || key_of(y) == top;
  };
  for (int p = t; p < parts; p += kRowThreads) s.kept[p] = 0;
  __syncthreads();
  // a wave a part: the bins before the last one
  for (int p = t >> 6; p < parts; p += kRowThreads / 64) {
    uint64_t m = 0;
    for (int j = t & 63; j < kBins; j += 64)
      if (j + 4 * s.down[p] < last) m += in.mass[(row * parts + p) * kBins + j];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m += (uint64_t)__shfl_xor((unsigned long long)m, d);
    if ((t & 63) == 0) s.kept[p] = m;
  }
  __syncthreads();
  if (last < kBins - 1)
    walk_row<S>(a, row, parts, [&](int p) { return part_has(last, p); },
                [&](int p, int token, float y) {
                  if (in_bin(last, y) && kept(token, y))
                    atomicAdd(reinterpret_cast<unsigned long long*>(&s.kept[p]), (unsigned long long)weigh(p, y));
                });
  __syncthreads();
  // the part that the draw falls into, and what is left of it there
  uint64_t w = t < parts ? to_row(t, s.kept[t]) : 0, total;
  uint64_t before = scan64(w, s.red, &total);
  const uint64_t target = share_of(total, a.u[row]);
  if (t < parts && target >= before && target < before + w) {
    s.pick = t;
    s.found64 = (target - before) << (s.down[t] + up);
  }
  __syncthreads();
  const int part = s.pick;
  const uint64_t rest = s.found64;
  const int64_t at = (int64_t)part * kPart + t * 4;
  uint64_t x[4], sum = 0, ignored;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = 0;
    if (at + e < a.n) {
      const int64_t o = row * a.ldy + at + e;
      float y;
      if constexpr (S == 4) y = static_cast<const float*>(a.y)[o];
      else if (a.y_type == 2) y = (float)static_cast<const _Float16*>(a.y)[o];
      else y = (float)static_cast<const bf16_t*>(a.y)[o];
      if (kept((int)(at + e), y) && bin_of(quarter((double)y * c), s.base[part]) < kBins - 1) x[e] = weigh(part, y);
    }
    sum += x[e];
  }
  uint64_t run = scan64(sum, s.red, &ignored);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (rest >= run && rest < run + x[e]) {
      a.idx[row] = (int32_t)(at + e);
      if (a.prob) a.prob[row] = (float)(__builtin_ldexp((double)x[e], -(s.down[part] + up)) / (double)total);
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
