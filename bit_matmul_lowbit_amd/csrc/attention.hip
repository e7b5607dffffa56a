// Attention of the queries of many sequences over a paged cache held in 4 bits.
//
//   o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q.k_t - m),   t <= last(q)
//
// in one pass over the cache: the running maximum m, the sum of p and the
// unnormalised o stay in registers, FP32.
//
// Rows.  The queries of a KV head's `group` query heads read the same keys: a
// tile is TT tokens (a power of two) by the group, up to RT = 16 NR or 64 NR rows.
//
// Products.  Both are v_mfma_f32_16x16x32_f16 with the cache as the A operand
// straight from memory, never through LDS:
//   S^T = K Q^T : a lane holds, of one token, the quarter of the head that its
//     16 lanes belong to -- d / 8 neighbouring bytes; Q is put in the order of
//     the nibbles once.
//   O^T = V^T P^T : the cache keeps four tokens of a pair of values in a
//     dword, so a lane has four tokens of d / 16 values in one load, and the
//     tokens that it needs of P are those that S^T gave it: P is rounded to FP16
//     and used where it is.
// A code becomes FP16(a (1 + c / 16) + b) with a shift, a mask and half a packed
// FMA: it is put into the mantissa of 1.0.  Keys and values of the cache are FP16
// numbers by definition, so nothing is lost there; BF16 queries are scaled by a power
// of two a row, which is exact.  The sum of p is a product with ones, of the same
// rounded p.
//
// The maximum is raised only where a score passes it by 2^8 (p stays far
// inside FP16), so most steps neither exchange lanes nor rescale o.
//
// Work.  All (sequence, KV head, tile) items are cut into units of kUnit
// tokens, and the units of all items, one after another, are shared out evenly
// over the work-groups from the lengths on the device: a work-group may end one item and
// begin others.  An item that does not end where it began leaves its parts (m,
// sum, o) in the workspace, and a second launch joins them in the order of their
// work-groups.  No atomics; equal inputs give equal bits.
#include "kv4.h"

namespace lowbit {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr float kEmpty = -1e30f;   // a maximum of nothing
constexpr float kRaise = 8.0f;     // log2 of what p may reach

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// over the four groups of 16 lanes
__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ float max_groups(float v) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  u = __builtin_bit_cast(uint32_t, fmaxf(as_float(r[0]), as_float(r[1])));
  auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(as_float(s[0]), as_float(s[1]));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)v) | ((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32));
}

// How rows and tokens are cut; made on the host.
struct Shape {
  int group;        // query heads of a KV head
  int part;         // of them in a tile
  int parts;        // tiles beside each other for all of them
  int tok_shift;    // a tile's tokens: 1 << tok_shift
  int unit_shift;   // log2(tokens of a unit / tokens of a tile)
  int page_shift;
};

// sum of ceil(y / r) for y = 1..x, r = 1 << shift
__device__ __forceinline__ int64_t units_up_to(int64_t x, int shift) {
  const int64_t a = x >> shift, b = x & (((int64_t)1 << shift) - 1);
  return ((a * (a + 1) / 2) << shift) + b * (a + 1);
}

// one sequence of the call
struct Seq {
  int q0, nq;        // its rows of q
  int off;           // token that the first of them sees last
  int len;
  int before;        // tiles' worth of tokens before the queries
  int64_t per;       // units of all tiles of a KV head and part
  int64_t units;
};
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, const Shape& s, int i) {
  Seq q;
  int64_t q0 = i, q1 = i + 1;
  if (a.q_start) {
    q0 = min(max((int64_t)a.q_start[i], (int64_t)0), a.m);
    q1 = min(max((int64_t)a.q_start[i + 1], q0), a.m);
  }
  q.q0 = (int)q0;
  q.nq = (int)(q1 - q0);
  q.len = min(max(a.lengths[i], 0), (int)a.tcap << s.page_shift);
  q.off = q.len - q.nq;
  const int tt = 1 << s.tok_shift;
  q.before = (max(q.off, 0) + tt - 1) >> s.tok_shift;
  const int tiles = (q.nq + tt - 1) >> s.tok_shift;
  q.per = units_up_to(q.before + tiles, s.unit_shift) - units_up_to(q.before, s.unit_shift);
  q.units = q.per * a.heads * s.parts;
  return q;
}

// Which work-group does what, found by every work-group for itself.
struct Walk {
  int seq;          // of the first unit of this work-group
  int64_t base;     // first unit of that sequence
  int64_t total;
};

// Sum of all units, and the sequence that unit `share(total)` is of: the threads
// take neighbouring sequences each, and add up.
template <class F>
__device__ __forceinline__ Walk find_walk(const AttnArgs& a, const Shape& s, int64_t* red, F share) {
  const int t = threadIdx.x, n = (int)a.b;
  const int chunk = (n + kThreads - 1) / kThreads, lo = min(n, t * chunk), hi = min(n, lo + chunk);
  int64_t mine = 0;
  for (int i = lo; i < hi; ++i) mine += seq_of(a, s, i).units;
  // within the wave, then over the four waves
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(sum, d);
    if ((t & 63) >= d) sum += o;
  }
  if ((t & 63) == 63) red[t >> 6] = sum;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < (t >> 6)) before += red[w];
    total += red[w];
  }
  int64_t at = before + sum - mine;
  const int64_t want = share(total);
  if (want >= at && want < at + mine) {
    for (int i = lo; i < hi; ++i) {
      const int64_t u = seq_of(a, s, i).units;
      if (want < at + u) {
        red[4] = i;
        red[5] = at;
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  return {uniform((int)red[4]), uniform64(red[5]), uniform64(total)};
}

__device__ __forceinline__ int64_t share_of(int64_t total, int64_t i, int64_t n) { return total * i / n; }

// one item: a tile of a KV head of a sequence
struct Item {
  int head, part, tile;
  int64_t first, units;  // its units, from the start of the sequence's
};
__device__ __forceinline__ Item item_of(const Seq& q, const Shape& s, int64_t unit) {
  Item it;
  const int64_t which = unit / q.per, rest = unit - which * q.per;
  it.head = (int)(which / s.parts);
  it.part = (int)(which - (int64_t)it.head * s.parts);
  // the tile that unit `rest` is of: the last one whose units begin at or before it
  const int64_t zero = units_up_to(q.before, s.unit_shift);
  int lo = 0, hi = (q.nq + (1 << s.tok_shift) - 1) >> s.tok_shift;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (units_up_to(q.before + mid, s.unit_shift) - zero <= rest) lo = mid;
    else hi = mid;
  }
  it.tile = lo;
  const int64_t begin = units_up_to(q.before + lo, s.unit_shift) - zero;
  it.units = units_up_to(q.before + lo + 1, s.unit_shift) - zero - begin;
  it.first = which * q.per + begin;
  return it;
}

// Codes and params of 32 tokens as a lane needs them
template <int D>
struct Raw {
  static constexpr int kW = D / 32;               // dwords of a lane
  static constexpr int kP = D / 32 >= 8 ? 2 : 1;  // groups of 32 values that a lane's K falls into
  uint32_t k[2][kW], kp[2][kP], v[2][kW];
  uint4 vp[2];
};

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&out)[W], const uint8_t* p) {
  if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    out[0] = x.x, out[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[i];
      out[4 * i] = x.x, out[4 * i + 1] = x.y, out[4 * i + 2] = x.z, out[4 * i + 3] = x.w;
    }
  }
}

// where 16 tokens lie, or that they do not (then somewhere that can be read)
struct Place {
  const uint8_t* head;
  int in;
  bool there;
};
__device__ __forceinline__ Place place16(const AttnArgs& a, const Shape& s, const int32_t* table, int len, int t,
                                         int head, int head_bytes, int64_t page_bytes) {
  Place p;
  int id = -1;
  if (t < len) id = table[t >> s.page_shift];
  id = uniform(id);
  p.there = id >= 0 && id < a.n_pages;
  p.head = a.pages + (p.there ? id : 0) * page_bytes + (int64_t)head * head_bytes;
  p.in = t & ((1 << s.page_shift) - 1);
  return p;
}

template <int D>
__device__ __forceinline__ void load_raw(Raw<D>& r, int h, const Place& p, const KvHead& lay, int lane) {
  const int m = lane & 15, g = lane >> 4;
  load_words(r.k[h], p.head + (p.in + m) * (D / 2) + g * (D / 8));
  const uint32_t* kp = reinterpret_cast<const uint32_t*>(p.head + lay.k_params()) + (p.in + m) * (D / 32);
  if constexpr (Raw<D>::kP == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(kp + 2 * g);
    r.kp[h][0] = x.x, r.kp[h][1] = x.y;
  } else {
    r.kp[h][0] = kp[D == 64 ? g >> 1 : g];
  }
  const int quad = (p.in >> 2) + g;
  load_words(r.v[h], p.head + lay.v_codes() + quad * (D * 2) + m * (D / 8));
  r.vp[h] = reinterpret_cast<const uint4*>(p.head + lay.v_params())[quad * (D / 32) + m * D / 512];
}

__device__ __forceinline__ f16x2 splat_lo(uint32_t w) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w, w, 0x01000100u));
}
__device__ __forceinline__ f16x2 splat_hi(uint32_t w) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w, w, 0x03020302u));
}
__device__ __forceinline__ f16x8 join(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
  return (f16x8){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The running state of NR tiles of 16 rows: a lane belongs to row lane % 16
template <int D, int NR>
struct State {
  static constexpr int kM = D / 16;
  f32x4 o[NR][kM], l[NR];  // l: the sum of p, the same in all four
  float m[NR];
};

// `p` of 32 tokens joins the state.  mask (the same in the whole wave): tokens
// past the row's last one, or past the end, or not there, are passed over.
template <int D, int NR>
__device__ __forceinline__ void step(State<D, NR>& st, const Raw<D>& r, const f16x8 (&q)[NR][D / 32],
                                     const float (&c)[NR], const int (&last)[NR], bool mask, int t0, int len,
                                     bool there0, bool there1, int lane) {
  const int g = lane >> 4;
  f32x4 s[NR][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int n = 0; n < NR; ++n) s[n][h] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t ab = r.kp[h][Raw<D>::kP == 2 ? w / 4 : 0];
      const f16x2 a = splat_lo(ab), b = splat_hi(ab);
      const uint32_t x = r.k[h][w];
      const f16x8 key = join(fma2(nibbles<0>(x), a, b), fma2(nibbles<1>(x), a, b), fma2(nibbles<2>(x), a, b),
                             fma2(nibbles<3>(x), a, b));
#pragma unroll
      for (int n = 0; n < NR; ++n) s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[n][w], s[n][h], 0, 0, 0);
    }
  }
  f16x8 p[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[n][e >> 2][e & 3] * c[n];
    if (mask) {
      const int see0 = there0 ? last[n] - (t0 + 4 * g) : -1, see1 = there1 ? last[n] - (t0 + 16 + 4 * g) : -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (e & 3) <= (e < 4 ? see0 : see1) ? x[e] : -INFINITY;
    }
    float most = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    if (__builtin_amdgcn_ballot_w64(most > st.m[n] + kRaise) != 0) {
      const float m = fmaxf(st.m[n], max_groups(most));
      const float f = exp2_fast(st.m[n] - m);
      st.m[n] = m;
      st.l[n] *= f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) st.o[n][i] *= f;
    }
    f16x2 pk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      auto two = __builtin_amdgcn_cvt_pkrtz(exp2_fast(x[2 * e] - st.m[n]), exp2_fast(x[2 * e + 1] - st.m[n]));
      pk[e] = __builtin_bit_cast(f16x2, two);
    }
    p[n] = join(pk[0], pk[1], pk[2], pk[3]);
    const _Float16 one = (_Float16)1.0f;
    st.l[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16((f16x8){one, one, one, one, one, one, one, one}, p[n], st.l[n], 0, 0,
                                                     0);
  }
  f16x2 a[2][2], b[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 w = r.vp[h];
    if (mask) {
      // what is not there counts 0 times p = 0, whatever its bits say
      const int have = (h ? there1 : there0) ? len - (t0 + 16 * h + 4 * g) : 0;
      const uint32_t m01 = have >= 2 ? 0xFFFFFFFFu : have == 1 ? 0x0000FFFFu : 0u;
      const uint32_t m23 = have >= 4 ? 0xFFFFFFFFu : have == 3 ? 0x0000FFFFu : 0u;
      w = make_uint4(w.x & m01, w.y & m23, w.z & m01, w.w & m23);
    }
    a[h][0] = __builtin_bit_cast(f16x2, w.x);
    a[h][1] = __builtin_bit_cast(f16x2, w.y);
    b[h][0] = __builtin_bit_cast(f16x2, w.z);
    b[h][1] = __builtin_bit_cast(f16x2, w.w);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    const uint32_t x = r.v[0][e], y = r.v[1][e];
    const f16x8 even = join(fma2(nibbles<0>(x), a[0][0], b[0][0]), fma2(nibbles<2>(x), a[0][1], b[0][1]),
                            fma2(nibbles<0>(y), a[1][0], b[1][0]), fma2(nibbles<2>(y), a[1][1], b[1][1]));
    const f16x8 odd = join(fma2(nibbles<1>(x), a[0][0], b[0][0]), fma2(nibbles<3>(x), a[0][1], b[0][1]),
                           fma2(nibbles<1>(y), a[1][0], b[1][0]), fma2(nibbles<3>(y), a[1][1], b[1][1]));
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      st.o[n][2 * e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(even, p[n], st.o[n][2 * e], 0, 0, 0);
      st.o[n][2 * e + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(odd, p[n], st.o[n][2 * e + 1], 0, 0, 0);
    }
  }
}

// Floats of a part in the workspace: o as the lanes hold it, then m and the sum
// of each row
template <int D, int ROWS>
constexpr int kPartFloats = ROWS * (D + 2);

__device__ __forceinline__ void store_out(void* out, int type, int64_t at, float v) {
  if (type == 1) static_cast<float*>(out)[at] = v;
  else if (type == 2) static_cast<_Float16*>(out)[at] = (_Float16)v;
  else static_cast<bf16_t*>(out)[at] = (bf16_t)v;
}
template <int N>
__device__ __forceinline__ void store_row(void* out, int type, int64_t at, const float (&v)[N]) {
  if (type == 1) {
    __builtin_memcpy(static_cast<float*>(out) + at, v, sizeof(v));
  } else if (type == 2) {
    _Float16 h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = (_Float16)v[i];
    __builtin_memcpy(static_cast<_Float16*>(out) + at, h, sizeof(h));
  } else {
    bf16_t h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = (bf16_t)v[i];
    __builtin_memcpy(static_cast<bf16_t*>(out) + at, h, sizeof(h));
  }
}

// row `row` of an item: its row of q and its head; false if it has none
__device__ __forceinline__ bool row_of(const Seq& q, const Item& it, const Shape& s, int row, int* token, int* head) {
  const int t = row / s.part, h = row - t * s.part;
  const int tok = (it.tile << s.tok_shift) + t;
  const int in = it.part * s.part + h;
  *token = q.q0 + tok;
  *head = it.head * s.group + in;
  return t < (1 << s.tok_shift) && tok < q.nq && in < s.group;
}

// SPLIT: the four waves take a unit's tokens in turn for the same rows and are
// joined through LDS; otherwise each has rows of its own.
template <int D, int NR, bool SPLIT>
__global__ __launch_bounds__(kThreads, NR == 1 ? 2 : 1) void attn_kernel(AttnArgs a, Shape s, float* parts) {
  constexpr int kM = D / 16;
  constexpr int kRows = SPLIT ? 16 * NR : 64 * NR;
  __shared__ int64_t red[6];
  __shared__ f32x4 swap[SPLIT ? 2 * NR * kM * 64 : 1];
  __shared__ float stat[SPLIT ? 4 * 2 * 16 * NR : 1];
  const int64_t wg = blockIdx.x, wgs = gridDim.x;
  Walk walk = find_walk(a, s, red, [&](int64_t total) { return share_of(total, wg, wgs); });
  const int64_t end = share_of(walk.total, wg + 1, wgs);
  int64_t at = share_of(walk.total, wg, wgs);
  if (at >= end) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4;
  const KvHead lay(1 << s.page_shift, D);
  const int64_t page_bytes = a.heads * lay.bytes();
  const int unit_tokens_shift = s.unit_shift + s.tok_shift;
  int i = walk.seq;
  int64_t base = walk.base;
  bool first = true;
  while (at < end) {
    Seq q = seq_of(a, s, i);
    if (at >= base + q.units) {
      base += q.units;
      ++i;
      continue;
    }
    const Item it = item_of(q, s, at - base);
    const int u0 = uniform((int)(at - base - it.first)), u1 = uniform((int)min(end - base - it.first, it.units));
    // its rows
    const int tile_end = uniform(min(q.len, q.off + ((it.tile + 1) << s.tok_shift)));  // tokens that any of them sees
    f16x8 qf[NR][D / 32];
    float c[NR];
    int last[NR];
    State<D, NR> st;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = (SPLIT ? 0 : wave * 16 * NR) + n * 16 + (lane & 15);
      int token, head;
      const bool have = row_of(q, it, s, row, &token, &head);
      last[n] = have ? q.off + (token - q.q0) : -1;
      const int64_t from = have ? token * a.ldq + head * a.ldqh + g * (D / 4) : 0;
      uint32_t w[D / 8];
#pragma unroll
      for (int j = 0; j < D / 8; ++j) w[j] = 0;
      if (have) __builtin_memcpy(w, static_cast<const uint16_t*>(a.q) + from, sizeof(w));
      c[n] = a.scale * 1.44269504088896340736f;
      if (a.q_type == 3) {
        // BF16: times the power of two that puts the row's largest near 2^14
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) big = max(big, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
        const int e = (int)(__builtin_bit_cast(uint32_t, max_groups(__builtin_bit_cast(float, big << 16))) >> 23);
        const int up = min(127 + 14 - e, 126);
        const float f = __builtin_bit_cast(float, (uint32_t)(127 + max(up, -126)) << 23);
        const float back = __builtin_bit_cast(float, (uint32_t)(127 - max(up, -126)) << 23);
        c[n] *= back;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float lo = __builtin_bit_cast(float, w[j] << 16) * f, hi = __builtin_bit_cast(float, w[j] & 0xFFFF0000u) * f;
          w[j] = __builtin_bit_cast(uint32_t, (f16x2){(_Float16)lo, (_Float16)hi});
        }
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const f16x2 x = __builtin_bit_cast(f16x2, w[4 * j]), y = __builtin_bit_cast(f16x2, w[4 * j + 1]),
                    z = __builtin_bit_cast(f16x2, w[4 * j + 2]), u = __builtin_bit_cast(f16x2, w[4 * j + 3]);
        qf[n][j] = (f16x8){x.x, z.x, x.y, z.y, y.x, u.x, y.y, u.y};  // 0 4 1 5 2 6 3 7
      }
      st.m[n] = kEmpty;
      st.l[n] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kM; ++j) st.o[n][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    // the token up to which every row that there is sees everything; rows that
    // are not there may count what they like
    const int open = uniform(min(q.len, q.off + (it.tile << s.tok_shift) + 1));
    const int32_t* table = a.table + (int64_t)i * a.ldt;
    const int t_end = (int)min((int64_t)tile_end, (int64_t)u1 << unit_tokens_shift);
    constexpr int kStep = SPLIT ? 128 : 32;
    int t = (u0 << unit_tokens_shift) + (SPLIT ? wave * 32 : 0);
    Raw<D> cur, next;
    bool c0 = false, c1 = false, n0 = false, n1 = false;
    auto fetch = [&](Raw<D>& r, int from, bool& h0, bool& h1) __attribute__((always_inline)) {
      const Place p0 = place16(a, s, table, q.len, from, it.head, lay.bytes(), page_bytes);
      const Place p1 = place16(a, s, table, q.len, from + 16, it.head, lay.bytes(), page_bytes);
      h0 = p0.there;
      h1 = p1.there;
      load_raw(r, 0, p0, lay, lane);
      load_raw(r, 1, p1, lay, lane);
    };
    if (t < t_end) fetch(cur, t, c0, c1);
    while (t < t_end) {
      const int then = t + kStep;
      if (then < t_end) fetch(next, then, n0, n1);
      step<D, NR>(st, cur, qf, c, last, t + 32 > open || !c0 || !c1, t, q.len, c0, c1, lane);
      cur = next;
      c0 = n0;
      c1 = n1;
      t = then;
    }
    if constexpr (SPLIT) {
      // one maximum for the four waves, then their sums
      __syncthreads();
      if (g == 0)
#pragma unroll
        for (int n = 0; n < NR; ++n) stat[wave * 16 * NR + n * 16 + lane] = st.m[n];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float m = st.m[n];
#pragma unroll
        for (int w = 0; w < 4; ++w) m = fmaxf(m, stat[w * 16 * NR + n * 16 + (lane & 15)]);
        const float f = exp2_fast(st.m[n] - m);
        st.m[n] = m;
        st.l[n] *= f;
#pragma unroll
        for (int j = 0; j < kM; ++j) st.o[n][j] *= f;
        if (g == 0) stat[64 * NR + wave * 16 * NR + n * 16 + lane] = st.l[n][0];
      }
      // waves 2 and 3 hand over to 0 and 1, then 1 to 0
#pragma unroll
      for (int half = 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int j = 0; j < kM; ++j) swap[(((wave - half) * NR + n) * kM + j) * 64 + lane] = st.o[n][j];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int j = 0; j < kM; ++j) st.o[n][j] += swap[((wave * NR + n) * kM + j) * 64 + lane];
        }
        __syncthreads();
      }
      if (wave == 0) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float l = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) l += stat[64 * NR + w * 16 * NR + n * 16 + (lane & 15)];
          st.l[n][0] = l;
        }
      }
    }
    if (!SPLIT || wave == 0) {
      const int row0 = SPLIT ? 0 : wave * 16 * NR;
      if (u0 == 0 && u1 == it.units) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          int token, head;
          if (!row_of(q, it, s, row0 + n * 16 + (lane & 15), &token, &head)) continue;
          const float l = st.l[n][0], f = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;  // NaN stays NaN
          const int64_t to = token * a.ldo + head * a.ldoh + g * (D / 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v[kM];
#pragma unroll
            for (int j = 0; j < kM; ++j) v[j] = st.o[n][j][e] * f;
            store_row(a.out, a.out_type, to + e * kM, v);
          }
          if (a.lse && g == 0)
            a.lse[token * a.hq + head] = l == 0.0f ? -INFINITY : 0.69314718055994530942f * (st.m[n] + __log2f(l));
        }
      } else {
        float* part = parts + (wg * 2 + (first ? 0 : 1)) * kPartFloats<D, kRows>;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
          for (int j = 0; j < kM; ++j)
            reinterpret_cast<f32x4*>(part)[((row0 / 16 + n) * kM + j) * 64 + lane] = st.o[n][j];
          if (g == 0) {
            part[kRows * D + row0 + n * 16 + lane] = st.m[n];
            part[kRows * D + kRows + row0 + n * 16 + lane] = st.l[n][0];
          }
        }
      }
    }
    first = false;
    at = base + it.first + u1;
  }
}

// Joins the parts of the item that work-group blockIdx.x began and did not end.
// blockIdx.y: 16 rows of it.
template <int D, int ROWS>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a, Shape s, const float* parts, int wgs) {
  constexpr int kM = D / 16;
  __shared__ int64_t red[6];
  __shared__ float rows[16][D + 4];
  const int64_t wg = blockIdx.x;
  // the last unit of work-group wg is of the item
  const Walk walk = find_walk(a, s, red, [&](int64_t total) { return share_of(total, wg + 1, wgs) - 1; });
  const int64_t begin = share_of(walk.total, wg, wgs), end = share_of(walk.total, wg + 1, wgs);
  if (begin >= end) return;
  const Seq q = seq_of(a, s, walk.seq);
  const Item it = item_of(q, s, end - 1 - walk.base);
  const int64_t from = walk.base + it.first, to = from + it.units;
  if (from < begin || to <= end) return;  // begun before, or ended here
  const int tile = (int)blockIdx.y;
  const float* own = parts + (wg * 2 + (from > begin ? 1 : 0)) * kPartFloats<D, ROWS>;
  const int n = threadIdx.x & 15;
  const float* stats = own + ROWS * D + tile * 16 + n;
  // the parts that follow are the first ones of their work-groups; those without
  // units are passed over
  float m = stats[0];
  int64_t w_end = wg + 1;
  while (w_end < wgs && share_of(walk.total, w_end, wgs) < to) ++w_end;
  for (int64_t w = wg + 1; w < w_end; ++w)
    if (share_of(walk.total, w + 1, wgs) > share_of(walk.total, w, wgs))
      m = fmaxf(m, parts[w * 2 * kPartFloats<D, ROWS> + ROWS * D + tile * 16 + n]);
  f32x4 o[(kM + 3) / 4];
  float l = 0.0f;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < (kM + 3) / 4; ++j) o[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int64_t w = wg; w < w_end; ++w) {
    const float* p = w == wg ? own : parts + w * 2 * kPartFloats<D, ROWS>;
    if (w != wg && share_of(walk.total, w + 1, wgs) == share_of(walk.total, w, wgs)) continue;
    const float f = exp2_fast(p[ROWS * D + tile * 16 + n] - m);
    l += p[ROWS * D + ROWS + tile * 16 + n] * f;
#pragma unroll
    for (int j = 0; j < kM / 4; ++j)
      o[j] += reinterpret_cast<const f32x4*>(p)[(tile * kM + wave + 4 * j) * 64 + lane] * f;
  }
  const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
#pragma unroll
  for (int j = 0; j < kM / 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) rows[n][(lane >> 4) * (D / 4) + e * kM + wave + 4 * j] = o[j][e] * inv;
  __syncthreads();
  for (int r = wave; r < 16; r += 4) {
    int token, head;
    if (!row_of(q, it, s, tile * 16 + r, &token, &head)) continue;
    for (int d = lane; d < D; d += 64)
      store_out(a.out, a.out_type, token * a.ldo + head * a.ldoh + d, rows[r][d]);
  }
  if (a.lse && threadIdx.x < 16) {
    int token, head;
    if (row_of(q, it, s, tile * 16 + n, &token, &head))
      a.lse[token * a.hq + head] = l == 0.0f ? -INFINITY : 0.69314718055994530942f * (m + __log2f(l));
  }
}

int log2_of(int64_t v) {
  int s = 0;
  while (((int64_t)1 << (s + 1)) <= v) ++s;
  return s;
}

// Which kernel, by the rows that a KV head's queries have at most in a sequence:
// four waves split the tokens while a wave can hold the rows (NR tiles of 16),
// beyond they split the rows.
struct Variant {
  int nr;
  bool split;
  int rows;
  int wgs;
};
Variant variant_of(int64_t group, int64_t d, int64_t max_q) {
  const int64_t rows = group * max_q;
  Variant v;
  if (rows <= 16) v = {1, true, 16, 512};
  else if (rows <= 32 || (d == 256 && rows <= 64)) v = {2, true, 32, 256};
  else if (rows <= 64) v = {4, true, 64, 256};
  else if (d == 256) v = {2, false, 128, 256};
  else v = {4, false, 256, 256};
  return v;
}

template <int D, int NR, bool SPLIT>
void launch_one(const AttnArgs& a, const Shape& s, const Variant& v, float* parts, hipStream_t st) {
  attn_kernel<D, NR, SPLIT><<<v.wgs, kThreads, 0, st>>>(a, s, parts);
  constexpr int kRows = SPLIT ? 16 * NR : 64 * NR;
  attn_join_kernel<D, kRows><<<dim3(v.wgs, kRows / 16), kThreads, 0, st>>>(a, s, parts, v.wgs);
}

template <int D>
void launch_d(const AttnArgs& a, const Shape& s, const Variant& v, float* parts, hipStream_t st) {
  if (v.split && v.nr == 1) launch_one<D, 1, true>(a, s, v, parts, st);
  else if (v.split && v.nr == 2) launch_one<D, 2, true>(a, s, v, parts, st);
  if constexpr (D == 256) {
    if (!v.split) launch_one<D, 2, false>(a, s, v, parts, st);
  } else {
    if (v.split && v.nr == 4) launch_one<D, 4, true>(a, s, v, parts, st);
    else if (!v.split) launch_one<D, 4, false>(a, s, v, parts, st);
  }
}

}  // namespace

size_t attention_workspace_bytes(int64_t hq, int64_t heads, int64_t d, int64_t max_q) {
  const Variant v = variant_of(hq / heads, d, max_q);
  return (size_t)v.wgs * 2 * v.rows * (size_t)(d + 2) * sizeof(float);
}

hipError_t launch_attention(const AttnArgs& a, void* ws, hipStream_t st) {
  const int64_t group = a.hq / a.heads;
  const Variant v = variant_of(group, a.d, a.max_q);
  Shape s;
  s.group = (int)group;
  s.part = (int)min(group, (int64_t)v.rows);
  s.parts = (int)((group + s.part - 1) / s.part);
  s.tok_shift = log2_of(v.rows / s.part);
  // a unit: 128 tokens, or the tile's tokens where they are more
  s.unit_shift = max(0, 7 - s.tok_shift);
  s.page_shift = log2_of(a.page);
  if (a.d == 64) launch_d<64>(a, s, v, static_cast<float*>(ws), st);
  else if (a.d == 128) launch_d<128>(a, s, v, static_cast<float*>(ws), st);
  else launch_d<256>(a, s, v, static_cast<float*>(ws), st);
  return hipGetLastError();
}

}  // namespace lowbit
