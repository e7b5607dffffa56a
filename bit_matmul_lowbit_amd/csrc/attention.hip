// Attention of the queries of many sequences over a paged cache held in 4 bits.
//
//   o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q.k_t - m),   t <= last(q)
//
// in one pass over the cache: the running maximum m, the sum of p and the
// unnormalised o stay in registers, FP32.
//
// Rows.  The queries of a KV head's `group` query heads read the same keys: a
// tile is a power of two of tokens by the group (or a part of it), up to 16, 32 or 64
// rows where the four waves of a work-group have the same rows and take the cache's tokens in
// turn, and up to 128 (64 of 256 values) where each has rows of its own.
//
// Products.  Both are v_mfma_f32_16x16x32_f16 with the cache as the A operand:
//   S^T = K Q^T : a lane holds, of one token, the quarter of the head that its
//     16 lanes belong to -- d / 8 neighbouring bytes; Q is put in the order of
//     the nibbles once.
//   O^T = V^T P^T : the cache keeps four tokens of a pair of values in a
//     dword, so a lane has four tokens of d / 16 values in one load, and the
//     tokens that it needs of P are those that S^T gave it: P is rounded to FP16
//     and used where it is.
// With few rows the codes go straight from memory to the lane that needs them, never
// through LDS; with many, the four waves make an operand each and hand it round in LDS.
// A code becomes FP16(a (1 + c / 16) + b) with a shift, a mask and half a packed
// FMA: it is put into the mantissa of 1.0.  Keys and values of the cache are FP16
// numbers by definition, so nothing is lost there; BF16 queries are scaled by a power
// of two a row, which is exact down to 2^-31 of the row's largest (FP16's least numbers: what is
// smaller is off by 2^-39 of the largest).  The sum of p is a product with ones, of the same
// rounded p.
//
// m is not the maximum but lies 7 below the one that set it, and is set again only where a score
// passes it by more than 15, which FP16 still holds.  So p has all of FP16's bits down to 2^-21 of
// the largest and is off by 2^-32 of that at most below (with m at the maximum: 2^-14 and 2^-25,
// and what many tokens have together behind one of most of the mass was 25 % off, or gone).  Most
// steps neither exchange lanes nor rescale o.  m lower still takes away from what a score may rise:
// 10 below costs chunks of three prompts 1 %, 12 below 4 %.
//
// Work.  All (sequence, KV head, tile) items are cut into units of 128 tokens (or as
// many as a tile has, if they are more), and the units of all items, one after another, are
// shared out evenly over the work-groups from the lengths on the device: a work-group may
// end one item and begin others.  An item that does not end where it began leaves its
// parts (m, sum, o) in the workspace, and a second launch joins them in the order of
// their work-groups.  No atomics; equal inputs give equal bits.
//
// Measured (a 1 GiB copy moves 5.2 TB/s, an 8192^3 product of the library 1.2 PFLOP/s here):
//   one token over 262144, 24 heads on 4 of 256: 65 us and 8 for the join, 335 MB, the
//     cache read at 5.2 TB/s: bound by memory
//   16 chats, 1 to 32767 tokens, the same heads: 57 and 8 us
//   one token over 4096, 16 heads on 8 of 128: 8.0 and 5.4 us: latency (the lists, q, three
//     steps of loads and products, the join's launch)
//   four tokens of those 16 chats: 86 us for the same bytes.  attn_kernel<256, 2> keeps 12 registers in
//     memory, <128, 4> 47 and <64, 4> 13
//   chunks of up to 2048 on three prompts, 32 heads on 8 of 128: 420 us, 713 TFLOP/s of the
//     two products: what the exponentials and the rounding of p take from the matrix units' issue,
//     with two waves a SIMD for the registers of o
#include "kv4.h"

namespace lowbit {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr float kEmpty = -3.4028234663852886e38f;  // m of nothing: no score lies below it
// log2 of the largest p where m is set, and of what p may reach before it is set again (FP16 holds
// less than 2^16).  Where a step of the scores is 8, m may lie 8 below instead of 7; where it is
// larger, m is the maximum.
constexpr float kSet = 7.0f, kRaise = 15.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// To the nearest: cut off, p would put the result 2.5e-4 off (relative, FP16's own rounding being
// 2.1e-4), so 2e-4 at most
__device__ __forceinline__ f16x2 to_f16x2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_convertvector((f32x2{a, b}), f16x2);
}

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

// What a kernel reads of the call's lists: nothing writes them meanwhile, so
// they come through the scalar cache
typedef const __attribute__((address_space(4))) int32_t* list_t;
__device__ __forceinline__ list_t list_of(const int32_t* p) { return (list_t)(uintptr_t)p; }

// What beginning an item costs, in units: an item counts as so many units more
// than its tokens are.  (Three prompts of 8192, 2729 and 510 tokens, chunks of up to
// 2048: 541 us without, 442 with one.)
constexpr int kBegin = 1;

// How rows and tokens are cut; made on the host.
struct Shape {
  int group;        // query heads of a KV head
  int part;         // of them in a tile
  int parts;        // tiles beside each other for all of them
  int tok_shift;    // a tile's tokens: 1 << tok_shift
  int unit_shift;   // log2(tokens of a unit / tokens of a tile)
  int page_shift;
};

// sum of kBegin + ceil(y / r) for y = 1..x, r = 1 << shift: the units of the tiles
// whose last row sees up to x tiles' worth of tokens
template <class T>
__device__ __forceinline__ T units_up_to(T x, int shift) {
  const T a = x >> shift, b = x & (((T)1 << shift) - 1);
  return ((a * (a + 1) / 2) << shift) + b * (a + 1) + kBegin * x;
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
    const list_t start = list_of(a.q_start);
    q0 = min(max((int64_t)start[i], (int64_t)0), a.m);
    q1 = min(max((int64_t)start[i + 1], q0), a.m);
  }
  q.q0 = (int)q0;
  q.nq = (int)(q1 - q0);
  q.len = min(max(list_of(a.lengths)[i], 0), (int)a.tcap << s.page_shift);
  q.off = q.len - q.nq;
  const int tt = 1 << s.tok_shift;
  q.before = (max(q.off, 0) + tt - 1) >> s.tok_shift;
  const int tiles = (q.nq + tt - 1) >> s.tok_shift;
  q.per = units_up_to((int64_t)q.before + tiles, s.unit_shift) - units_up_to((int64_t)q.before, s.unit_shift);
  q.units = q.per * a.heads * s.parts;
  return q;
}

// Even shares of all units: the first `more` work-groups have one unit more.
// Work-groups without a unit come last.
struct Shares {
  int64_t each, more;
  __device__ __forceinline__ int64_t begin(int64_t i) const { return i * each + min(i, more); }
};

__device__ __forceinline__ Shares shares_of(int64_t total, int64_t wgs) {
  Shares h;
  // few units: no 64-bit division (a hundred instructions in a row)
  h.each = total <= INT32_MAX ? (int64_t)((uint32_t)total / (uint32_t)wgs) : total / wgs;
  h.more = total - h.each * wgs;
  return h;
}

// Which work-group does what, found by every work-group for itself.
struct Walk {
  int seq;          // of the unit that was asked for
  int64_t base;     // first unit of that sequence
  Shares share;
};

// The shares, and the sequence that unit `pick(shares)` is of: the threads take
// neighbouring sequences each, and add up.
template <class F>
__device__ __forceinline__ Walk find_walk(const AttnArgs& a, const Shape& s, int64_t* red, int64_t wgs, F pick) {
  const int t = threadIdx.x, n = (int)a.b;
  if (n == 1) {
    const int64_t total = uniform64(seq_of(a, s, 0).units);
    return {0, 0, shares_of(total, wgs)};
  }
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
  const Shares share = shares_of(uniform64(total), wgs);
  const int64_t want = pick(share);
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
  return {uniform((int)red[4]), uniform64(red[5]), share};
}

// one item: a tile of a KV head of a sequence
struct Item {
  int head, part, tile;
  int64_t first;   // its units begin there, counted from the start of the sequence's
  int units;
};
template <class T>
__device__ __forceinline__ Item item_by(const Seq& q, const Shape& s, T unit) {
  Item it;
  const T per = (T)q.per, which = unit / per, rest = unit - which * per;
  it.head = (int)which / s.parts;
  it.part = (int)which - it.head * s.parts;
  // the tile that unit `rest` is of: the last one whose units begin at or before it
  const T zero = units_up_to((T)q.before, s.unit_shift);
  int lo = 0, hi = (q.nq + (1 << s.tok_shift) - 1) >> s.tok_shift;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (units_up_to((T)(q.before + mid), s.unit_shift) - zero <= rest) lo = mid;
    else hi = mid;
  }
  it.tile = lo;
  const T begin = units_up_to((T)(q.before + lo), s.unit_shift) - zero;
  it.units = (int)(units_up_to((T)(q.before + lo + 1), s.unit_shift) - zero - begin);
  it.first = (int64_t)(which * per + begin);
  return it;
}
// Scalar 32-bit arithmetic wherever the numbers allow it: 64-bit divisions and
// products cost some microseconds an item.
__device__ __forceinline__ Item item_of(const Seq& q, const Shape& s, int64_t unit) {
  const int64_t most = units_up_to((int64_t)q.before + ((q.nq + (1 << s.tok_shift) - 1) >> s.tok_shift), s.unit_shift);
  if (uniform(most <= INT32_MAX && q.units <= INT32_MAX)) {
    Seq u = q;
    u.per = uniform((int)q.per);
    return item_by<uint32_t>(u, s, (uint32_t)uniform((int)unit));
  }
  return item_by<int64_t>(q, s, unit);
}

// Codes and params of 32 tokens' keys, and of their values, as a lane needs them
template <int D>
struct Keys {
  static constexpr int kP = D / 32 >= 8 ? 2 : 1;  // groups of 32 values that a lane's part falls into
  uint32_t code[2][D / 32], param[2][kP];
};
template <int D>
struct Values {
  uint32_t code[2][D / 32], param[2][4];
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&out)[W], __amdgpu_buffer_rsrc_t part, uint32_t lane, int at) {
  if constexpr (W == 1) {
    out[0] = __builtin_amdgcn_raw_buffer_load_b32(part, lane, at, 0);
  } else if constexpr (W == 2) {
    const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(part, lane, at, 0);
    out[0] = x[0], out[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(part, lane, at + 16 * i, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[4 * i + e] = x[e];
    }
  }
}

// Where the two halves of 32 tokens lie: the part of the page that belongs to the
// head, as a buffer (of no bytes if there is no such page: loads give zeros)
struct Place {
  __amdgpu_buffer_rsrc_t part[2];
  int in[2];
  bool there[2];
};
__device__ __forceinline__ Place place_of(list_t table, int page_shift, const uint8_t* head, int64_t page_bytes,
                                          int part_bytes, int pages, int end, int t) {
  Place p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int u = t + 16 * h;
    const int id = u < end ? table[u >> page_shift] : -1;
    p.there[h] = id >= 0 && id < pages;
    p.part[h] = buffer_rsrc(head + (p.there[h] ? id : 0) * page_bytes, p.there[h] ? part_bytes : 0);
    p.in[h] = u & ((1 << page_shift) - 1);
  }
  return p;
}

// a lane's places in the codes and params of 16 tokens
template <int D>
struct Lane {
  uint32_t k, kp, v, vp;
  __device__ __forceinline__ explicit Lane(int lane) {
    const int m = lane & 15, g = lane >> 4;
    k = m * (D / 2) + g * (D / 8);
    kp = (m * (D / 32) + g * (D / 32) / 4) * 4;
    v = g * (D * 2) + m * (D / 8);
    vp = (g * (D / 32) + m * D / 512) * 16;
  }
};

template <int D>
__device__ __forceinline__ void load_keys(Keys<D>& r, const Place& p, const KvHead& lay, const Lane<D>& at) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_words(r.code[h], p.part[h], at.k, p.in[h] * (D / 2));
    load_words(r.param[h], p.part[h], at.kp, lay.k_params() + p.in[h] * (D / 8));
  }
}
template <int D>
__device__ __forceinline__ void load_values(Values<D>& r, const Place& p, const KvHead& lay, const Lane<D>& at) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_words(r.code[h], p.part[h], at.v, lay.v_codes() + p.in[h] * (D / 2));
    load_words(r.param[h], p.part[h], at.vp, lay.v_params() + p.in[h] * (D / 8));
  }
}

__device__ __forceinline__ f16x2 splat_lo(uint32_t w) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w, w, 0x01000100u));
}
__device__ __forceinline__ f16x2 splat_hi(uint32_t w) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(w, w, 0x03020302u));
}
// a and b of four tokens' values, zeros where a code would stand for infinity or NaN: for tokens
// that not all rows see or that lie past the end, which a row takes p = 0 of, and 0 times that is
// no 0.  (All codes' values lie between the first one's and the last one's.)  Three prompts in chunks
// take 420 us with it for 412 without; the other kernels lose nothing.
__device__ __forceinline__ void finite_only(uint32_t (&ab)[4]) {
  constexpr uint32_t kExponents = 0x7C007C00u;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const f16x2 a = __builtin_bit_cast(f16x2, ab[e]), b = __builtin_bit_cast(f16x2, ab[e + 2]);
    const f16x2 one = {(_Float16)1.0f, (_Float16)1.0f}, most = {(_Float16)1.9375f, (_Float16)1.9375f};
    const uint32_t first = __builtin_bit_cast(uint32_t, fma2(a, one, b)) & kExponents;
    const uint32_t last = __builtin_bit_cast(uint32_t, fma2(a, most, b)) & kExponents;
    const bool lo = (first & 0x7C00u) < 0x7C00u && (last & 0x7C00u) < 0x7C00u;
    const bool hi = first < 0x7C000000u && last < 0x7C000000u;
    const uint32_t keep = (lo ? 0x0000FFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
    ab[e] &= keep;
    ab[e + 2] &= keep;
  }
}
__device__ __forceinline__ f16x8 join(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
  return (f16x8){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The running state of NR tiles of 16 rows: a lane belongs to row lane % 16
template <int D, int NR>
struct State {
  static constexpr int kM = D / 16;
  f32x4 o[NR][kM];
  float l[NR], m[NR];  // l: of the tokens that this lane had
};

// Q of a wave's rows as the B operand.  Where it would take more than 32
// registers it stays in LDS (which leaves o in the vector registers and two waves
// a SIMD: o in accumulation registers was copied back and forth every step).
template <int D, int NR>
constexpr bool kQInLds = NR * D > 256;

// S^T of 32 tokens: two tiles of 16 of them, four to a lane.  q(n, w): the
// operand of tile n's rows, step w
template <int D, int NR, class Q>
__device__ __forceinline__ void scores(f32x4 (&s)[NR][2], const Keys<D>& r, Q q, uint32_t ones) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < NR; ++n) s[n][h] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    if (kQInLds<D, NR>) __builtin_amdgcn_sched_barrier(0);  // registers: one step's keys at a time
    f16x8 key[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t ab = r.param[h][Keys<D>::kP == 2 ? w / 4 : 0], x = r.code[h][w];
      const f16x2 a = splat_lo(ab), b = splat_hi(ab);
      key[h] = join(fma2(nibbles<0>(x, ones), a, b), fma2(nibbles<1>(x, ones), a, b),
                    fma2(nibbles<2>(x, ones), a, b), fma2(nibbles<3>(x, ones), a, b));
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const f16x8 qn = q(n, w);
#pragma unroll
      for (int h = 0; h < 2; ++h) s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key[h], qn, s[n][h], 0, 0, 0);
    }
  }
}

// p of the 32 tokens in the order of the product with V, and the state's maximum
// and sum with them
template <int D, int NR, class C>
__device__ __forceinline__ void weigh(State<D, NR>& st, f16x8 (&p)[NR], const f32x4 (&s)[NR][2], C c, uint32_t ones) {
  const f16x2 one = __builtin_bit_cast(f16x2, ones);
  // two tiles at a time, for which there is one question whether a maximum rises
  constexpr int kTogether = NR < 2 ? 1 : 2;
#pragma unroll
  for (int n0 = 0; n0 < NR; n0 += kTogether) {
    // scaled first, m taken away after: equal scores have equal weights however
    // large they are
    f32x4 x[kTogether][2];
    float most[kTogether];
    bool rises = false;
#pragma unroll
    for (int n = 0; n < kTogether; ++n) {
      const float f = c(n0 + n);
#pragma unroll
      for (int h = 0; h < 2; ++h) x[n][h] = s[n0 + n][h] * f;
      const f32x4 u = x[n][0], v = x[n][1];
      most[n] = fmaxf(fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])), fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
      rises = rises || most[n] - st.m[n0 + n] > kRaise;
    }
    if (__builtin_amdgcn_ballot_w64(rises) != 0) {
#pragma unroll
      for (int n = 0; n < kTogether; ++n) {
        const float m = fmaxf(st.m[n0 + n], max_groups(most[n]) - kSet);
        const float f = exp2_fast(st.m[n0 + n] - m);
        st.m[n0 + n] = m;
        st.l[n0 + n] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[n0 + n][i] *= f;
      }
    }
#pragma unroll
    for (int n = 0; n < kTogether; ++n) {
      f16x2 pk[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        pk[e] = to_f16x2(exp2_fast(x[n][e >> 1][2 * (e & 1)] - st.m[n0 + n]),
                         exp2_fast(x[n][e >> 1][2 * (e & 1) + 1] - st.m[n0 + n]));
      p[n0 + n] = join(pk[0], pk[1], pk[2], pk[3]);
      // the sum of the rounded p, as the product with V takes them
#pragma unroll
      for (int e = 0; e < 4; ++e) st.l[n0 + n] = __builtin_amdgcn_fdot2(pk[e], one, st.l[n0 + n], false);
    }
  }
}

// O^T += V^T P^T
template <int D, int NR>
__device__ __forceinline__ void gather(State<D, NR>& st, const Values<D>& r, const f16x8 (&p)[NR], uint32_t ones) {
  f16x2 a[2][2], b[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    a[h][0] = __builtin_bit_cast(f16x2, r.param[h][0]);
    a[h][1] = __builtin_bit_cast(f16x2, r.param[h][1]);
    b[h][0] = __builtin_bit_cast(f16x2, r.param[h][2]);
    b[h][1] = __builtin_bit_cast(f16x2, r.param[h][3]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    if (kQInLds<D, NR>) __builtin_amdgcn_sched_barrier(0);
    const uint32_t x = r.code[0][e], y = r.code[1][e];
    const f16x8 even = join(fma2(nibbles<0>(x, ones), a[0][0], b[0][0]), fma2(nibbles<2>(x, ones), a[0][1], b[0][1]),
                            fma2(nibbles<0>(y, ones), a[1][0], b[1][0]), fma2(nibbles<2>(y, ones), a[1][1], b[1][1]));
    const f16x8 odd = join(fma2(nibbles<1>(x, ones), a[0][0], b[0][0]), fma2(nibbles<3>(x, ones), a[0][1], b[0][1]),
                           fma2(nibbles<1>(y, ones), a[1][0], b[1][0]), fma2(nibbles<3>(y, ones), a[1][1], b[1][1]));
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

// What a work-group that began an item and did not end it leaves for the join:
// the number of parts (in a list of its own, 0: nothing to join), which of its own
// two is the first, and where the item's rows go.
struct alignas(16) Join {
  int slot;
  int token, tokens;  // first row of q, and how many there are
  int head, heads;    // first head, and how many
  int pad[3];
};
// The work-group whose share holds unit `to` - 1, counted from the first
__device__ __forceinline__ int64_t holder(const Shares& h, int64_t to) {
  const int64_t longer = h.more * (h.each + 1);  // units of the work-groups that have one more
  if (to <= longer) return (to - 1) / (h.each + 1);
  return h.more + (to - 1 - longer) / h.each;
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

// ln of a sum l of 2^(x - m); nothing: -inf.  (kSet is taken out of the logarithm, which has its
// rounding there.)
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -INFINITY : 0.69314718055994530942f * ((m + kSet) + __log2f(l * __builtin_exp2f(-kSet)));
}
__device__ __forceinline__ float inverse_of(float l) { return l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l; }  // NaN stays

// row `row` of an item: its row of q and its head; false if it has none
__device__ __forceinline__ bool row_of(const Seq& q, const Item& it, const Shape& s, int row, int* token, int* head) {
  const int t = row / s.part, h = row - t * s.part;
  const int tok = (it.tile << s.tok_shift) + t;
  const int in = it.part * s.part + h;
  *token = q.q0 + tok;
  *head = it.head * s.group + in;
  return t < (1 << s.tok_shift) && tok < q.nq && in < s.group;
}

// A quarter of a row of q, as the B operand of the scores, FP16, the values in
// the order of the nibbles.  Returns what the row's scores are to be multiplied
// by (with log2 e, for 2^x), never 0: a hidden score is -inf times this.
template <int D>
__device__ __forceinline__ float load_q(f16x8 (&out)[D / 32], const AttnArgs& a, bool have, int token, int head, int g) {
  uint32_t w[D / 8];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) w[j] = 0;
  if (have)
    __builtin_memcpy(w, static_cast<const uint16_t*>(a.q) + token * a.ldq + head * a.ldqh + g * (D / 4), sizeof(w));
  const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;  // a negative scale turns q around
#pragma unroll
  for (int j = 0; j < D / 8; ++j) w[j] ^= sign;
  float c = fabsf(a.scale) * 1.44269504088896340736f;
  if (a.q_type == 3) {
    // BF16: times the power of two that puts the row's largest near 2^14
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) big = max(big, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    const int e = (int)(__builtin_bit_cast(uint32_t, max_groups(__builtin_bit_cast(float, big << 16))) >> 23);
    const int up = max(min(127 + 14 - e, 126), -126);
    const float f = __builtin_bit_cast(float, (uint32_t)(127 + up) << 23);
    c *= __builtin_bit_cast(float, (uint32_t)(127 - up) << 23);
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
    out[j] = (f16x8){x.x, z.x, x.y, z.y, y.x, u.x, y.y, u.y};  // 0 4 1 5 2 6 3 7
  }
  return fmaxf(c, 1e-37f);
}

// What the rows of a wave came to: their results, where the item is whole, or a
// part for the join.
template <int D, int NR, int ROWS>
__device__ __forceinline__ void finish(const State<D, NR>& st, const AttnArgs& a, const Shape& s, const Seq& q,
                                       const Item& it, int row0, bool whole, float* part, int lane) {
  constexpr int kM = D / 16;
  const int g = lane >> 4;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    int token, head;
    if (!row_of(q, it, s, row0 + n * 16 + (lane & 15), &token, &head)) continue;
    if (whole) {
      const float l = st.l[n], f = inverse_of(l);
      const int64_t to = token * a.ldo + head * a.ldoh + g * (D / 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[kM];
#pragma unroll
        for (int j = 0; j < kM; ++j) v[j] = st.o[n][j][e] * f;
        store_row(a.out, a.out_type, to + e * kM, v);
      }
      if (a.lse && g == 0)
        a.lse[token * a.hq + head] = log_sum(st.m[n], l);
    } else {
#pragma unroll
      for (int j = 0; j < kM; ++j) reinterpret_cast<f32x4*>(part)[((row0 / 16 + n) * kM + j) * 64 + lane] = st.o[n][j];
      if (g == 0) reinterpret_cast<float2*>(part + ROWS * D)[row0 + n * 16 + lane] = make_float2(st.m[n], st.l[n]);
    }
  }
}

// A work-group's note on its last item for the join
__device__ __forceinline__ void leave(int* counts, Join* joins, const Shares& share, int64_t wg, bool first,
                                      const Shape& s, const Seq& q, const Item& it, int64_t base, bool more) {
  counts[wg] = more ? (int)(holder(share, base + it.first + it.units) - wg) + 1 : 0;
  Join j = {};
  j.slot = first ? 0 : 1;
  j.token = q.q0 + (it.tile << s.tok_shift);
  j.tokens = min(1 << s.tok_shift, q.nq - (it.tile << s.tok_shift));
  j.head = it.head * s.group + it.part * s.part;
  j.heads = min(s.part, s.group - it.part * s.part);
  joins[wg] = j;
}

// Few rows: the four waves take a unit's tokens in turn for the same rows and are
// joined through LDS.
template <int D, int NR>
__global__ __launch_bounds__(kThreads, 2) void attn_kernel(AttnArgs a, Shape s, float* parts, int* counts, Join* joins) {
  constexpr int kM = D / 16;
  constexpr int kRows = 16 * NR;
  __shared__ int64_t red[6];
  constexpr bool kLds = kQInLds<D, NR>;
  __shared__ f32x4 swap[2 * kM * 64];
  __shared__ f16x8 q_lds[kLds ? NR * (D / 32) * 64 : 1];
  __shared__ float c_lds[kLds ? kRows : 1];
  __shared__ int last_lds[kLds ? kRows : 1];
  __shared__ float stat[4 * 2 * 16 * NR];
  // where every work-group has work, neighbouring shares go to one of the eight
  // dies, whose L2 then holds few heads
  const int64_t wgs = gridDim.x;
  auto number = [&](const Shares& h) {
    return h.each > 0 ? (int64_t)(blockIdx.x & 7) * (wgs / 8) + (blockIdx.x >> 3) : (int64_t)blockIdx.x;
  };
  const Walk walk = find_walk(a, s, red, wgs, [&](const Shares& h) { return h.begin(number(h)); });
  const int64_t wg = number(walk.share);
  const int64_t end = walk.share.begin(wg + 1);
  int64_t at = walk.share.begin(wg);
  if (at >= end) {
    if (threadIdx.x == 0) counts[wg] = 0;
    return;
  }
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4;
  const Lane<D> place(lane);
  const uint32_t ones = ones_of();
  const KvHead lay(1 << s.page_shift, D);
  const int64_t page_bytes = a.heads * lay.bytes();
  const int unit_tokens_shift = s.unit_shift + s.tok_shift;
  int i = walk.seq;
  int64_t base = walk.base;
  bool first = true;
  while (at < end) {
    Seq q = seq_of(a, s, i);
    q.q0 = uniform(q.q0);
    q.nq = uniform(q.nq);
    q.off = uniform(q.off);
    q.len = uniform(q.len);
    if (at >= base + q.units) {
      base += q.units;
      ++i;
      continue;
    }
    Item it = item_of(q, s, at - base);
    // one item for the whole work-group: its numbers belong into scalar registers
    it.head = uniform(it.head);
    it.part = uniform(it.part);
    it.tile = uniform(it.tile);
    const int seq = uniform(i);
    // its units of this work-group, and those of them that have tokens
    const int v0 = uniform((int)(at - base - it.first)), v1 = uniform((int)min(end - base - it.first, (int64_t)it.units));
    const int u0 = max(v0 - kBegin, 0), u1 = max(v1 - kBegin, 0);
    // the tokens that any of its rows sees, and those that all of them see (rows
    // that are not there may count what they like)
    const int tile_end = uniform(min(q.len, q.off + ((it.tile + 1) << s.tok_shift)));
    const int open = uniform(min(q.len, q.off + (it.tile << s.tok_shift) + 1));
    const list_t table = list_of(a.table + (int64_t)seq * a.ldt);
    const uint8_t* head_base = a.pages + (int64_t)it.head * lay.bytes();
    const int t_end = uniform((int)min((int64_t)tile_end, (int64_t)u1 << unit_tokens_shift));
    constexpr int kStep = 128;
    int t = uniform((u0 << unit_tokens_shift) + wave * 32);
    auto find = [&](int from) __attribute__((always_inline)) {
      return place_of(table, s.page_shift, head_base, page_bytes, lay.bytes(), (int)a.n_pages, t_end, from);
    };
    // keys and values are on their way before q is; page numbers go a step ahead
    Place now = find(t), then = find(t + kStep);
    Keys<D> keys;
    Values<D> values;
    load_keys<D>(keys, now, lay, place);
    load_values<D>(values, now, lay, place);
    // its rows
    f16x8 qf[kLds ? 1 : NR][D / 32];
    f16x8* q_own = q_lds + lane;
    if (kLds) __syncthreads();  // the last item's rows are done with
    // a row's factor of the scores and the last token that it sees
    float c_of[kLds ? 1 : NR];
    int last_of[kLds ? 1 : NR];
    State<D, NR> st;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = n * 16 + (lane & 15);
      int token, head;
      const bool have = row_of(q, it, s, row, &token, &head);
      const int last = have ? q.off + (token - q.q0) : -1;
      f16x8 qr[D / 32];
      const float c = load_q<D>(qr, a, have, token, head, g);
      if constexpr (kLds) {
        if (g == 0) {
          c_lds[row] = c;
          last_lds[row] = last;
        }
      } else {
        c_of[n] = c;
        last_of[n] = last;
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        if constexpr (kLds) {
          if (wave == n % 4) q_own[(n * (D / 32) + j) * 64] = qr[j];
        } else {
          qf[n][j] = qr[j];
        }
      }
      st.m[n] = kEmpty;
      st.l[n] = 0.0f;
#pragma unroll
      for (int j = 0; j < kM; ++j) st.o[n][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    if (kLds) __syncthreads();
    auto q_of = [&](int n, int w) __attribute__((always_inline)) {
      if constexpr (kLds) return q_own[(n * (D / 32) + w) * 64];
      else return qf[n][w];
    };
    auto c_at = [&](int n) __attribute__((always_inline)) {
      if constexpr (kLds) return c_lds[n * 16 + (lane & 15)];
      else return c_of[n];
    };
    auto last_at = [&](int n) __attribute__((always_inline)) {
      if constexpr (kLds) return last_lds[n * 16 + (lane & 15)];
      else return last_of[n];
    };
    // (a step past the last one loads nothing: there is no page for it)
    for (int steps = uniform(max(0, (t_end - t + kStep - 1) / kStep)); steps > 0; --steps) {
      f32x4 sc[NR][2];
      f16x8 p[NR];
      scores<D, NR>(sc, keys, q_of, ones);
      __builtin_amdgcn_sched_barrier(0);
      load_keys<D>(keys, then, lay, place);
      const bool there = now.there[0] && now.there[1];
      if (t + 32 > open || !there) {
        // tokens past the row's last one or of no page: a score of -inf, whatever the bits say
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int first = t + 16 * h + 4 * g;
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const int sees = now.there[h] ? last_at(n) - first : -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][h][e] = e <= sees ? sc[n][h][e] : -INFINITY;
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      weigh<D, NR>(st, p, sc, c_at, ones);
      __builtin_amdgcn_sched_barrier(0);
      if (t + 32 > open) {  // (here, where the scores' registers are free: fewer are spilled)
        finite_only(values.param[0]);
        finite_only(values.param[1]);
      }
      gather<D, NR>(st, values, p, ones);
      __builtin_amdgcn_sched_barrier(0);
      load_values<D>(values, then, lay, place);
      t += kStep;
      now = then;
      then = find(t + kStep);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {  // over the four groups of lanes
      st.l[n] += __shfl_xor(st.l[n], 16);
      st.l[n] += __shfl_xor(st.l[n], 32);
    }
    {
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
        if (g == 0) stat[64 * NR + wave * 16 * NR + n * 16 + lane] = st.l[n];
      }
      // waves 2 and 3 hand over to 0 and 1, then 1 to 0
#pragma unroll
      for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int half = 2; half >= 1; half >>= 1) {
          if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int j = 0; j < kM; ++j) swap[((wave - half) * kM + j) * 64 + lane] = st.o[n][j];
          }
          __syncthreads();
          if (wave < half) {
#pragma unroll
            for (int j = 0; j < kM; ++j) st.o[n][j] += swap[(wave * kM + j) * 64 + lane];
          }
          __syncthreads();
        }
      }
      if (wave == 0) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float l = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) l += stat[64 * NR + w * 16 * NR + n * 16 + (lane & 15)];
          st.l[n] = l;
        }
      }
    }
    if (wave == 0) {
      finish<D, NR, kRows>(st, a, s, q, it, 0, v0 == 0 && v1 == it.units,
                           parts + (wg * 2 + (first ? 0 : 1)) * kPartFloats<D, kRows>, lane);
    }
    if (threadIdx.x == 0 && base + it.first + v1 == end)  // its last item
      leave(counts, joins, walk.share, wg, first, s, q, it, base, v0 == 0 && v1 < it.units);
    first = false;
    at = base + it.first + v1;
  }
}

// A wave's share of 32 tokens' operands: kPer of the D / 16 operands of K (16
// tokens, 32 values) and as many of V (32 tokens, 16 values)
template <int D>
struct Shared {
  static constexpr int kPer = D / 64, kOps = D / 16;  // a wave's, all
  static constexpr int kW = D == 64 ? 1 : D / 128;    // dwords of K, and of V, that they are of
  uint32_t k[kPer], kp[kPer], v[kW][2], vp[2][4];
  bool there[2];
  int at;
};
template <int D>
__device__ __forceinline__ void load_shared(Shared<D>& r, const Place& p, int t, const KvHead& lay, const Lane<D>& at,
                                            int wave) {
  constexpr int kPer = Shared<D>::kPer;
  r.at = t;
#pragma unroll
  for (int h = 0; h < 2; ++h) r.there[h] = p.there[h];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int f = wave * kPer + j, w = f >> 1;
    const auto part = D == 64 ? ((f & 1) ? p.part[1] : p.part[0]) : p.part[j & 1];
    const int in = D == 64 ? ((f & 1) ? p.in[1] : p.in[0]) : p.in[j & 1];
    r.k[j] = __builtin_amdgcn_raw_buffer_load_b32(part, at.k, in * (D / 2) + 4 * w, 0);
    r.kp[j] = __builtin_amdgcn_raw_buffer_load_b32(part, at.kp, lay.k_params() + in * (D / 8) + (w / 4) * 4, 0);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int e = 0; e < Shared<D>::kW; ++e) {
      const int w = (wave * kPer) / 2 + e;
      r.v[e][h] = __builtin_amdgcn_raw_buffer_load_b32(p.part[h], at.v, lay.v_codes() + p.in[h] * (D / 2) + 4 * w, 0);
    }
    load_words(r.vp[h], p.part[h], at.vp, lay.v_params() + p.in[h] * (D / 8));
  }
}
// ... as FP16 into LDS, where a lane of any wave finds its 16 bytes of them
template <int D>
__device__ __forceinline__ void spread_shared(f16x8* lds, Shared<D>& r, int open, int lane, int wave, uint32_t ones) {
  constexpr int kPer = Shared<D>::kPer;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t x = r.k[j];
    const f16x2 a = splat_lo(r.kp[j]), b = splat_hi(r.kp[j]);
    lds[(wave * kPer + j) * 64 + lane] = join(fma2(nibbles<0>(x, ones), a, b), fma2(nibbles<1>(x, ones), a, b),
                                              fma2(nibbles<2>(x, ones), a, b), fma2(nibbles<3>(x, ones), a, b));
  }
  f16x2 a[2][2], b[2][2];
  if (r.at + 32 > open && (r.there[0] || r.there[1])) {  // (what is of no page is zeros already)
    finite_only(r.vp[0]);
    finite_only(r.vp[1]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    a[h][0] = __builtin_bit_cast(f16x2, r.vp[h][0]);
    a[h][1] = __builtin_bit_cast(f16x2, r.vp[h][1]);
    b[h][0] = __builtin_bit_cast(f16x2, r.vp[h][2]);
    b[h][1] = __builtin_bit_cast(f16x2, r.vp[h][3]);
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int f = wave * kPer + j;
    const uint32_t x = r.v[j >> 1][0], y = r.v[j >> 1][1];
    // even operands: nibbles 0 and 2, odd ones: 1 and 3
    const int down = D == 64 ? (f & 1) * 4 : (j & 1) * 4;
    const uint32_t xs = x >> down, ys = y >> down;
    lds[(Shared<D>::kOps + f) * 64 + lane] =
        join(fma2(nibbles<0>(xs, ones), a[0][0], b[0][0]), fma2(nibbles<2>(xs, ones), a[0][1], b[0][1]),
             fma2(nibbles<0>(ys, ones), a[1][0], b[1][0]), fma2(nibbles<2>(ys, ones), a[1][1], b[1][1]));
  }
}

// Many rows: every wave has kWaveRows of its own, and the four make the operands
// of 32 tokens together, one step ahead, in two LDS buffers in turn (each wave
// making all of them for itself, 64 rows a wave, was bound by that: three prompts in chunks of
// 2048 take 967 us by that kernel, 420 by this one).
// A wave has 32 rows, or 16 of 256 values (32 of those and their q do not fit its registers).
template <int D>
constexpr int kManyTiles = D == 256 ? 1 : 2;
template <int D>
constexpr int kManyRows = 64 * kManyTiles<D>;
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attn_rows_kernel(AttnArgs a, Shape s, float* parts, int* counts,
                                                                Join* joins) {
  constexpr int kM = D / 16, kOps = Shared<D>::kOps, kTiles = kManyTiles<D>, kWaveRows = 16 * kTiles;
  __shared__ int64_t red[6];
  __shared__ f16x8 lds[2][2 * kOps * 64];
  // where every work-group has work, neighbouring shares go to one of the eight
  // dies, whose L2 then holds few heads
  const int64_t wgs = gridDim.x;
  auto number = [&](const Shares& h) {
    return h.each > 0 ? (int64_t)(blockIdx.x & 7) * (wgs / 8) + (blockIdx.x >> 3) : (int64_t)blockIdx.x;
  };
  const Walk walk = find_walk(a, s, red, wgs, [&](const Shares& h) { return h.begin(number(h)); });
  const int64_t wg = number(walk.share);
  const int64_t end = walk.share.begin(wg + 1);
  int64_t at = walk.share.begin(wg);
  if (at >= end) {
    if (threadIdx.x == 0) counts[wg] = 0;
    return;
  }
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), g = lane >> 4;
  const Lane<D> place(lane);
  const uint32_t ones = ones_of();
  const KvHead lay(1 << s.page_shift, D);
  const int64_t page_bytes = a.heads * lay.bytes();
  const int unit_tokens_shift = s.unit_shift + s.tok_shift;
  int i = walk.seq;
  int64_t base = walk.base;
  bool first = true;
  while (at < end) {
    Seq q = seq_of(a, s, i);
    q.q0 = uniform(q.q0);
    q.nq = uniform(q.nq);
    q.off = uniform(q.off);
    q.len = uniform(q.len);
    if (at >= base + q.units) {
      base += q.units;
      ++i;
      continue;
    }
    Item it = item_of(q, s, at - base);
    it.head = uniform(it.head);
    it.part = uniform(it.part);
    it.tile = uniform(it.tile);
    const int seq = uniform(i);
    // its units of this work-group, and those of them that have tokens
    const int v0 = uniform((int)(at - base - it.first)), v1 = uniform((int)min(end - base - it.first, (int64_t)it.units));
    const int u0 = max(v0 - kBegin, 0), u1 = max(v1 - kBegin, 0);
    const int tile_end = uniform(min(q.len, q.off + ((it.tile + 1) << s.tok_shift)));
    const int open = uniform(min(q.len, q.off + (it.tile << s.tok_shift) + 1));
    const list_t table = list_of(a.table + (int64_t)seq * a.ldt);
    const uint8_t* head_base = a.pages + (int64_t)it.head * lay.bytes();
    const int t_end = uniform((int)min((int64_t)tile_end, (int64_t)u1 << unit_tokens_shift));
    int t = uniform(u0 << unit_tokens_shift);
    auto find = [&](int from) __attribute__((always_inline)) {
      return place_of(table, s.page_shift, head_base, page_bytes, lay.bytes(), (int)a.n_pages, t_end, from);
    };
    Shared<D> raw;
    load_shared<D>(raw, find(t), t, lay, place, wave);
    Place then = find(t + 32);
    f16x8 q_op[kTiles][D / 32];
    float c[kTiles];
    int last[kTiles];
    State<D, kTiles> st;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      int token, head;
      const bool have = row_of(q, it, s, wave * kWaveRows + n * 16 + (lane & 15), &token, &head);
      last[n] = have ? q.off + (token - q.q0) : -1;
      c[n] = load_q<D>(q_op[n], a, have, token, head, g);
      st.m[n] = kEmpty;
      st.l[n] = 0.0f;
#pragma unroll
      for (int j = 0; j < kM; ++j) st.o[n][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    bool there0 = raw.there[0], there1 = raw.there[1];
    spread_shared<D>(lds[0], raw, open, lane, wave, ones);
    load_shared<D>(raw, then, t + 32, lay, place, wave);
    then = find(t + 64);
    __syncthreads();
    int turn = 0;
    for (int steps = uniform(max(0, (t_end - t + 31) / 32)); steps > 0; --steps) {
      const f16x8* ops = lds[turn];
      f32x4 sc[kTiles][2];
      f16x8 p[kTiles];
      // operands leave LDS kAhead at a time, before what stands between them and
      // their products: the next step's operands, and the weights
      constexpr int kAhead = kOps < 8 ? kOps : 8;
      f16x8 op[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) op[j] = ops[j * 64 + lane];
      const bool now0 = there0, now1 = there1;
      there0 = raw.there[0];
      there1 = raw.there[1];
      // the next step's operands, and the codes of the one after it
      spread_shared<D>(lds[turn ^ 1], raw, open, lane, wave, ones);
      load_shared<D>(raw, then, t + 64, lay, place, wave);
      then = find(t + 96);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) sc[n][0] = sc[n][1] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j0 = 0; j0 < kOps; j0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
            sc[n][j & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(op[j], q_op[n][(j0 + j) >> 1], sc[n][j & 1], 0, 0, 0);
          // then the operands that follow: of K, and after them the first of V
          op[j] = ops[(j0 + kAhead + j) * 64 + lane];
        }
      }
      if (t + 32 > open || !now0 || !now1) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            const int sees = (h ? now1 : now0) ? last[n] - (t + 16 * h + 4 * g) : -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][h][e] = e <= sees ? sc[n][h][e] : -INFINITY;
          }
      }
      // ahead of the other work-group's waves, whose products go on beside it (the three prompts
      // above: 4 % less time)
      __builtin_amdgcn_s_setprio(1);
      weigh<D, kTiles>(st, p, sc, [&](int n) { return c[n]; }, ones);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
#pragma unroll
      for (int j0 = 0; j0 < kM; j0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
            st.o[n][j0 + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(op[j], p[n], st.o[n][j0 + j], 0, 0, 0);
          if (j0 + kAhead < kM) op[j] = ops[(kOps + j0 + kAhead + j) * 64 + lane];
        }
      }
      __syncthreads();
      t += 32;
      turn ^= 1;
    }
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {  // over the four groups of lanes
      st.l[n] += __shfl_xor(st.l[n], 16);
      st.l[n] += __shfl_xor(st.l[n], 32);
    }
    finish<D, kTiles, kManyRows<D>>(st, a, s, q, it, wave * kWaveRows, v0 == 0 && v1 == it.units,
                                 parts + (wg * 2 + (first ? 0 : 1)) * kPartFloats<D, kManyRows<D>>, lane);
    if (threadIdx.x == 0 && base + it.first + v1 == end)  // its last item
      leave(counts, joins, walk.share, wg, first, s, q, it, base, v0 == 0 && v1 < it.units);
    first = false;
    at = base + it.first + v1;
  }
}

constexpr int kMostParts = 512;  // work-groups of the first launch

// The work-group that began the `nth` item whose parts are to be joined, and how
// many they are; {.., 0} if there are not so many.  Every thread of a
// work-group of at least 256 calls it.
struct Owner {
  int wg, parts;
};
__device__ __forceinline__ Owner find_owner(const int* counts, int wgs, int nth, int* lds) {
  // lds: [0..7] owners of a wave's work-groups, [8] and [9] the result
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int c[2] = {0, 0};
  if (t < 256) {
    c[0] = counts[t];
    if (wgs > 256) c[1] = counts[t + 256];
  }
  if (t == 0) lds[9] = 0;
  const uint64_t b0 = __builtin_amdgcn_ballot_w64(c[0] != 0), b1 = __builtin_amdgcn_ballot_w64(c[1] != 0);
  if (lane == 0 && wave < 4) {
    lds[wave] = __popcll(b0);
    lds[wave + 4] = __popcll(b1);
  }
  __syncthreads();
  if (wave < 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int before = 0;
      for (int w = 0; w < h * 4 + wave; ++w) before += lds[w];
      const uint64_t b = h ? b1 : b0;
      if (c[h] != 0 && before + __popcll(b & (((uint64_t)1 << lane) - 1)) == nth) {
        lds[8] = h * 256 + t;
        lds[9] = c[h];
      }
    }
  }
  __syncthreads();
  return {uniform(lds[8]), uniform(lds[9])};
}

// Joins the parts of item blockIdx.x of those that are to be joined, of a kernel
// whose waves split the tokens.  blockIdx.y: 16 rows of it and kJ of the head's
// tiles.  Eight waves take the parts in turn; all that is loaded first goes out
// at once.
constexpr int kJoinThreads = 512, kJoinWaves = kJoinThreads / 64, kJ = 2;
template <int D, int ROWS>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a, int part, const float* parts,
                                                                 const int* counts, const Join* joins, int wgs) {
  constexpr int kM = D / 16, kY = kM / kJ;
  __shared__ float weight[kMostParts][16];
  __shared__ f32x4 swap[kJoinWaves - 1][kJ * 64];
  __shared__ float most8[kJoinWaves][16], sum8[kJoinWaves][16];
  __shared__ int lds[10];
  const Owner own = find_owner(counts, wgs, (int)blockIdx.x, lds);
  if (own.parts == 0) return;
  const int count = own.parts;
  const int tile = (int)blockIdx.y / kY, column = ((int)blockIdx.y % kY) * kJ;
  const int t = threadIdx.x, lane = t & 63, wave = uniform(t >> 6), n = lane & 15;
  const Join* jp = joins + own.wg;
  const int slot = uniform(jp->slot), tokens = uniform(jp->tokens), heads = uniform(jp->heads);
  if (tile * 16 / part >= tokens) return;  // no row of the tile is there
  // a part's floats; those that follow the first are the first ones of their work-groups
  auto at = [&](int k) {
    return parts + ((int64_t)(own.wg + k) * 2 + (k == 0 ? slot : 0)) * kPartFloats<D, ROWS>;
  };
  const int row = tile * 16 + n, tok = row / part, h = row - tok * part;
  const bool there = tok < tokens && h < heads;  // the parts have no other rows
  constexpr int kAhead = 8, kRound = kJoinThreads / 16;
  f32x4 x[kAhead][kJ];
  auto fetch = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int k = k0 + e * kJoinWaves;
      if (k < count && there) {
#pragma unroll
        for (int c = 0; c < kJ; ++c)
          x[e][c] = reinterpret_cast<const f32x4*>(at(k))[(tile * kM + column + c) * 64 + lane];
      }
    }
  };
  fetch(wave);
  float2 ml[kMostParts / kRound];
#pragma unroll
  for (int e = 0; e < kMostParts / kRound; ++e) {
    ml[e] = make_float2(kEmpty, 0.0f);
    const int k = (t >> 4) + e * kRound;
    if (e * kRound < count && k < count) ml[e] = reinterpret_cast<const float2*>(at(k) + ROWS * D)[row];
  }
  float m = kEmpty;
#pragma unroll
  for (int e = 0; e < kMostParts / kRound; ++e) m = fmaxf(m, ml[e].x);
  m = max_groups(m);
  if (lane < 16) most8[wave][n] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) m = fmaxf(m, most8[w][n]);
  float l = 0.0f;
#pragma unroll
  for (int e = 0; e < kMostParts / kRound; ++e) {
    if (e * kRound < count) {
      const float g = exp2_fast(ml[e].x - m);
      weight[(t >> 4) + e * kRound][n] = g;
      l += g * ml[e].y;
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (lane < 16) sum8[wave][n] = l;
  __syncthreads();
  f32x4 o[kJ];
#pragma unroll
  for (int c = 0; c < kJ; ++c) o[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave; k0 < count; k0 += kJoinWaves * kAhead) {
    if (k0 != wave) fetch(k0);
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int k = k0 + e * kJoinWaves;
      if (k < count) {
        const float g = weight[k][n];
#pragma unroll
        for (int c = 0; c < kJ; ++c) o[c] += x[e][c] * g;
      }
    }
  }
  if (wave > 0)
#pragma unroll
    for (int c = 0; c < kJ; ++c) swap[wave - 1][c * 64 + lane] = o[c];
  __syncthreads();
  if (wave > 0) return;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) l += sum8[w][n];
#pragma unroll
  for (int w = 0; w < kJoinWaves - 1; ++w)
#pragma unroll
    for (int c = 0; c < kJ; ++c) o[c] += swap[w][c * 64 + lane];
  if (!there) return;
  const float inv = inverse_of(l);
  const int token = jp->token + tok, head = jp->head + h;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v[kJ];
#pragma unroll
    for (int c = 0; c < kJ; ++c) v[c] = o[c][e] * inv;
    store_row(a.out, a.out_type, token * a.ldo + head * a.ldoh + (lane >> 4) * (D / 4) + e * kM + column, v);
  }
  if (a.lse && column == 0 && lane < 16)
    a.lse[token * a.hq + head] = log_sum(m, l);
}

// The same for a kernel whose waves have rows of their own: items have many rows
// and few parts, so a wave takes 16 rows and walks their parts.
template <int D, int ROWS>
__global__ __launch_bounds__(kThreads) void attn_join_rows_kernel(AttnArgs a, int part, const float* parts,
                                                                  const int* counts, const Join* joins, int wgs) {
  constexpr int kM = D / 16;
  __shared__ int lds[10];
  const Owner own = find_owner(counts, wgs, (int)blockIdx.x, lds);
  if (own.parts == 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15;
  const int tile = (int)blockIdx.y * 4 + wave, row = tile * 16 + n;
  const Join* jp = joins + own.wg;
  const int slot = uniform(jp->slot), tokens = uniform(jp->tokens), heads = uniform(jp->heads);
  const int tok = row / part, h = row - tok * part;
  if (tok >= tokens || h >= heads) return;  // the parts have no such row
  float m = kEmpty, l = 0.0f;
  f32x4 o[kM];
#pragma unroll
  for (int c = 0; c < kM; ++c) o[c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < own.parts; ++k) {
    const float* p = parts + ((int64_t)(own.wg + k) * 2 + (k == 0 ? slot : 0)) * kPartFloats<D, ROWS>;
    const float2 ml = reinterpret_cast<const float2*>(p + ROWS * D)[row];
    f32x4 x[kM];
#pragma unroll
    for (int c = 0; c < kM; ++c) x[c] = reinterpret_cast<const f32x4*>(p)[(tile * kM + c) * 64 + lane];
    const float most = fmaxf(m, ml.x), f = exp2_fast(m - most), g = exp2_fast(ml.x - most);
    m = most;
    l = l * f + ml.y * g;
#pragma unroll
    for (int c = 0; c < kM; ++c) o[c] = o[c] * f + x[c] * g;
  }
  const float inv = inverse_of(l);
  const int token = jp->token + tok, head = jp->head + h;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v[kM];
#pragma unroll
    for (int c = 0; c < kM; ++c) v[c] = o[c][e] * inv;
    store_row(a.out, a.out_type, token * a.ldo + head * a.ldoh + (lane >> 4) * (D / 4) + e * kM, v);
  }
  if (a.lse && lane < 16)
    a.lse[token * a.hq + head] = log_sum(m, l);
}

int log2_of(int64_t v) {
  int s = 0;
  while (((int64_t)1 << (s + 1)) <= v) ++s;
  return s;
}

// Which kernel, by the rows that a KV head's queries have at most in a sequence:
// the waves split the tokens while one of them can hold the rows (nr tiles of 16),
// beyond they split the rows.  Both sides, us a call replayed from a graph:
//   up to 16 rows, for 16 or 32: one chat of 4096 13.7 and 15.9, of 262144 81 and 83,
//     16 mixed chats 57 and 67
//   17 to 32, for 32 or 64: 8 tokens of a chat of 4096 18 and 26, of 16 chats 49 and 71;
//     4 tokens of 16 mixed chats, heads of 256, for 32 or by rows 82 and 150
//   33 to 64, split by tokens or by rows: 16 tokens of a chat of 4096 29 and 38, of 32768 54
//     and 71, of four of those 90 and 109; but of 16 chats of 4096 89 and 63.  The lengths are on
//     the device; the longer ones decide.  (Heads of 256 would need 64 more registers.)
//   beyond: chunks of 2048 of three prompts 420 by rows, 967 by tokens; 128 rows of a chat of
//     4096 40 and 37
struct Variant {
  int nr;  // 0: attn_rows_kernel
  int rows;
};
// Two a unit.  Half as many take 641 us for those chunks, 768 take 470 (and 90 for the chat of
// 262144, whose parts are more).
constexpr int kWgs = 512;
Variant variant_of(int64_t group, int64_t d, int64_t max_q) {
  const int64_t rows = group * max_q;
  if (rows <= 16) return {1, 16};
  if (rows <= 32) return {2, 32};
  if (rows <= 64 && d < 256) return {4, 64};
  return {0, d == 256 ? kManyRows<256> : kManyRows<128>};
}

template <int D, int NR>
void launch_one(const AttnArgs& a, const Shape& s, void* ws, hipStream_t st) {
  constexpr int kRows = NR ? 16 * NR : kManyRows<D>;
  int* counts = static_cast<int*>(ws);
  Join* joins = reinterpret_cast<Join*>(counts + kWgs);
  float* parts = reinterpret_cast<float*>(joins + kWgs);
  // no more items than this, and of a work-group one at most
  const int64_t items = min(a.m, a.b + (a.m >> s.tok_shift)) * a.heads * s.parts;
  const unsigned most = (unsigned)min((int64_t)kWgs, items);
  if constexpr (NR > 0) {
    attn_kernel<D, NR><<<kWgs, kThreads, 0, st>>>(a, s, parts, counts, joins);
    attn_join_kernel<D, kRows><<<dim3(most, kRows / 16 * (D / 16 / kJ)), kJoinThreads, 0, st>>>(
        a, s.part, parts, counts, joins, kWgs);
  } else {
    attn_rows_kernel<D><<<kWgs, kThreads, 0, st>>>(a, s, parts, counts, joins);
    attn_join_rows_kernel<D, kRows><<<dim3(most, kRows / 64), kThreads, 0, st>>>(a, s.part, parts, counts, joins,
                                                                                kWgs);
  }
}

template <int D>
void launch_d(const AttnArgs& a, const Shape& s, const Variant& v, void* ws, hipStream_t st) {
  if (v.nr == 1) launch_one<D, 1>(a, s, ws, st);
  else if (v.nr == 2) launch_one<D, 2>(a, s, ws, st);
  else if (v.nr == 0) launch_one<D, 0>(a, s, ws, st);
  else if constexpr (D < 256) launch_one<D, 4>(a, s, ws, st);
}

}  // namespace

size_t attention_workspace_bytes(int64_t hq, int64_t heads, int64_t d, int64_t max_q) {
  const Variant v = variant_of(hq / heads, d, max_q);
  return (size_t)kWgs * (sizeof(int) + sizeof(Join) + 2 * v.rows * (size_t)(d + 2) * sizeof(float));
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
  if (a.d == 64) launch_d<64>(a, s, v, ws, st);
  else if (a.d == 128) launch_d<128>(a, s, v, ws, st);
  else launch_d<256>(a, s, v, ws, st);
  return hipGetLastError();
}

}  // namespace lowbit
