// Rotary positions, and a cache of keys and values in 4-bit codes as it is written
// and read back.
//
// [P2] 7minutos.es, "PrismML lanza Bonsai 27B ...", "La memoria es la
//      restriccion vinculante": the cache of 262144 tokens takes a quarter in 4
//      bits of what it takes in FP16.  With a and b here it is 5 bits, 5/16.
//
// Angles: a pair turns by position * frequency.  The frequency is held as a 64-bit
// fraction of a turn, so the product wraps by itself and no position is too far:
// the angle is off by 2^-62 of a half turn times the position at most.  Sine and
// cosine are FP64 (which runs at the rate of FP32 here), rounded once to FP32, one
// pair per token and frequency, kept in LDS for all heads.
//
// Quantiser: 32 neighbouring values of a head share a and b (FP16); a code c in
// 0..15 stands for FP16(a (1 + c / 16) + b), one packed FMA on the code spread
// into the mantissa of 1.0.
//
// What bounds them: memory where tokens are many, a launch and two latencies
// where they are few.  Measured (a 1 GiB copy moves 5.2 TB/s here):
//   8192 tokens of 32 heads of 128 turned: 28.5 us, 4.7 TB/s
//   4096 tokens written, 32 heads of q turned beside 8 of K and V: 27.1 us, 3.3 TB/s (the q's part
//     alone takes 14, K and V 10; a row's loads wait for the cosines and their barrier, one
//     memory latency after another in work-groups as short as these)
//   32768 tokens of 4 heads of 256 read back: 40.6 us, 4.3 TB/s
//   one token written and read back: 3.6 and 2.1 us
#include "kv4.h"
#include "pieces.h"

namespace lowbit {
namespace {

constexpr int kThreads = 256;

// i / divisor by a multiplication, for i and divisor below 2^16
struct Divide {
  uint32_t by, magic;
};
Divide divide(int by) { return {(uint32_t)by, (uint32_t)(((uint64_t(1) << 32) + by - 1) / by)}; }
__device__ __forceinline__ int quotient(uint32_t i, Divide d) {
  return d.by == 1 ? (int)i : (int)__umulhi(i, d.magic);
}

// Cosines and sines of `tokens` tokens from `first` on, into cs[token][rot / 2]
__device__ __forceinline__ void fill_turns(float2* cs, const int32_t* positions, const uint64_t* turns, int64_t first,
                                           int tokens, int half, Divide by_half, double gain) {
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int t = quotient(i, by_half), f = i - t * half;
    const int64_t phase = (int64_t)((uint64_t)(int64_t)positions[first + t] * turns[f]);
    double s, c;
    sincospi((double)phase * 0x1p-63, &s, &c);
    cs[i] = make_float2((float)(gain * c), (float)(gain * s));
  }
}

// x1 c - x2 s and x2 c + x1 s, every product and sum rounded to FP32
__device__ __forceinline__ float2 turned(float x1, float x2, float2 cs) {
#pragma clang fp contract(off)
  const float a = x1 * cs.x, b = x2 * cs.y, c = x2 * cs.x, d = x1 * cs.y;
  return make_float2(a - b, c + d);
}

// What one head of one token is cut into: pieces of eight, pieces that turn
// first.  In the half layout a piece is eight pairs (x[j], x[j + rot / 2]).
struct Pieces {
  int rot, half, d, turn, all, inter;
  Divide by_all;
};
Pieces pieces_of(int rot, int d, bool inter, bool in_place) {
  Pieces p;
  p.rot = rot;
  p.half = rot / 2;
  p.d = d;
  p.inter = inter;
  p.turn = ((inter ? rot : rot / 2) + 7) / 8;
  p.all = p.turn + (in_place ? 0 : (d - rot + 7) / 8);
  p.by_all = divide(p.all);
  return p;
}

// Elements [from, from + n) of a row, n <= 8
template <int S>
__device__ __forceinline__ void load_some(const void* p, int type, int64_t from, int n, float (&v)[8]) {
  if (n == 8) {
    widen<S>(load8<S>(p, from), type, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < n) {
      if constexpr (S == 4) v[j] = static_cast<const float*>(p)[from + j];
      else if (type == 2) v[j] = (float)static_cast<const _Float16*>(p)[from + j];
      else v[j] = (float)static_cast<const bf16_t*>(p)[from + j];
    }
  }
}
__device__ __forceinline__ void store_some(void* p, int type, int64_t from, int n, const float (&v)[8]) {
  if (n == 8) {
    store8(p, type, from, 0, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < n) {
      if (type == 1) static_cast<float*>(p)[from + j] = v[j];
      else if (type == 2) static_cast<_Float16*>(p)[from + j] = (_Float16)v[j];
      else static_cast<bf16_t*>(p)[from + j] = (bf16_t)v[j];
    }
  }
}

// Piece `p` of the head whose elements start at x[at] and go to out[to]
template <int S>
__device__ __forceinline__ void turn_piece(const Pieces& g, int p, const void* x, int x_type, int64_t at, void* out,
                                           int out_type, int64_t to, const float2* cs) {
  float v[8], w[8];
  if (p >= g.turn) {  // what does not turn
    const int c = g.rot + (p - g.turn) * 8, n = min(8, g.d - c);
    load_some<S>(x, x_type, at + c, n, v);
    store_some(out, out_type, to + c, n, v);
  } else if (g.inter) {
    const int c = p * 8, n = min(8, g.rot - c);
    load_some<S>(x, x_type, at + c, n, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 o = turned(v[2 * j], v[2 * j + 1], cs[2 * j < n ? c / 2 + j : 0]);
      v[2 * j] = o.x;
      v[2 * j + 1] = o.y;
    }
    store_some(out, out_type, to + c, n, v);
  } else {
    const int c = p * 8, n = min(8, g.half - c);
    load_some<S>(x, x_type, at + c, n, v);
    load_some<S>(x, x_type, at + g.half + c, n, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 o = turned(v[j], w[j], cs[j < n ? c + j : 0]);
      v[j] = o.x;
      w[j] = o.y;
    }
    store_some(out, out_type, to + c, n, v);
    store_some(out, out_type, to + g.half + c, n, w);
  }
}

// A work-group takes `tokens` tokens and `heads` heads of them.
struct RopeGrid {
  int tokens, heads;
  Pieces pieces;
  Divide by_half, by_token;  // rot / 2; pieces of a token's heads
};

template <int S>
__device__ __forceinline__ void rope_part(const RopeArgs& a, const RopeGrid& g, int64_t first, int head0, float2* cs) {
  const int tokens = (int)min((int64_t)g.tokens, a.m - first), heads = min(g.heads, (int)a.heads - head0);
  fill_turns(cs, a.positions, a.turns, first, tokens, g.pieces.half, g.by_half, a.gain);
  __syncthreads();
  const int per_token = g.heads * g.pieces.all;
  for (int i = threadIdx.x; i < tokens * per_token; i += kThreads) {
    const int t = quotient(i, g.by_token), r = i - t * per_token;
    const int h = quotient(r, g.pieces.by_all), p = r - h * g.pieces.all;
    if (h >= heads) continue;
    turn_piece<S>(g.pieces, p, a.x, a.x_type, (first + t) * a.ldx + (head0 + h) * a.ldxh, a.out, a.out_type,
                  (first + t) * a.ldo + (head0 + h) * a.ldoh, cs + t * g.pieces.half);
  }
}

extern __shared__ float2 shared_turns[];

template <int S>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, RopeGrid g) {
  rope_part<S>(a, g, (int64_t)blockIdx.x * g.tokens, (int)blockIdx.y * g.heads, shared_turns);
}

// Pieces that a work-group takes: one a thread while that leaves fewer than two
// work-groups a unit, eight a thread beyond, where the cosines are made for more of them (8 tokens
// of 24 heads of 256: 4.5 us, with eight a thread 14; 8192 of 32 heads of 128: 27.6 us, with
// one a thread 30.4)
constexpr int kSmall = kThreads, kLarge = 8 * kThreads;
constexpr int kMostTurns = 2048;  // pairs of a cosine and a sine in LDS

RopeGrid rope_grid(const RopeArgs& a, bool in_place) {
  RopeGrid g;
  g.pieces = pieces_of((int)a.rot, (int)a.d, a.inter, in_place);
  const int64_t per_token = a.heads * g.pieces.all;
  const int64_t target = a.m * per_token <= 512 * kSmall ? kSmall : kLarge;
  g.heads = (int)max((int64_t)1, min(a.heads, target / g.pieces.all));
  g.tokens = (int)max((int64_t)1, min((int64_t)kMostTurns / g.pieces.half, target / (g.heads * g.pieces.all)));
  g.tokens = (int)min((int64_t)g.tokens, a.m);
  g.by_half = divide(g.pieces.half);
  g.by_token = divide(g.heads * g.pieces.all);
  return g;
}

// ---------------------------------------------------------------------------
// the cache

// What is kept of a value: finite, with room for a (1 + 15/16) + b in FP16, and
// zero without a sign (which of two zeros is the smaller one is nobody's to say)
__device__ __forceinline__ float bounded(float x) {
  x = x != x ? 0.0f : x + 0.0f;
  return fminf(fmaxf(x, -16384.0f), 16384.0f);
}

template <int CTRL>
__device__ __forceinline__ float quad_perm(float v) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The codes of eight values (value j in nibble j), and a | b << 16 of the 32 that
// four neighbouring lanes hold.
__device__ __forceinline__ uint32_t quantise8(float (&v)[8], uint32_t* params) {
#pragma clang fp contract(off)
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = bounded(v[j]);
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    lo = fminf(lo, v[j]);
    hi = fmaxf(hi, v[j]);
  }
  lo = fminf(lo, quad_perm<0xB1>(lo));  // lane ^ 1
  hi = fmaxf(hi, quad_perm<0xB1>(hi));
  lo = fminf(lo, quad_perm<0x4E>(lo));  // lane ^ 2
  hi = fmaxf(hi, quad_perm<0x4E>(hi));
  float range = (hi - lo) * (16.0f / 15.0f);
  __asm__("" : "+v"(range));  // rounded to FP32 before it is to FP16
  const _Float16 a = (_Float16)range;
  float below = lo - (float)a;
  __asm__("" : "+v"(below));
  const _Float16 b = (_Float16)below;
  *params = (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
  const float first = (float)a + (float)b, step = (float)a * 0.0625f;
  const float inv = __builtin_amdgcn_rcpf(step);
  uint32_t codes = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // the nearest whole number to off / step, ties to even, exactly: an FMA tells
    // on which side of half a step the value lies.  An estimate that is off by
    // one at a whole number is put right by the same comparison.
    const float off = v[j] - first;
    float c = floorf(off * inv);
    const float left = __builtin_fmaf(-(c + 0.5f), step, off);
    const bool odd = ((int)c & 1) != 0;
    c += left > 0.0f || (left == 0.0f && odd) ? 1.0f : 0.0f;
    c = step > 0.0f ? fminf(fmaxf(c, 0.0f), 15.0f) : 0.0f;
    codes |= (uint32_t)c << (4 * j);
  }
  return codes;
}

// where token `slot` lies: its page and its place there; false if it is outside
__device__ __forceinline__ bool place_of(int slot, int shift, int64_t pages, int64_t* at, int* t) {
  *at = (int64_t)slot >> shift;
  *t = slot & ((1 << shift) - 1);
  return slot >= 0 && *at < pages;
}

struct KvGrid {
  int tokens;            // of a work-group (4 or 1 of them to an item of V)
  int shift;             // page = 1 << shift
  int q_parts, kv_parts; // of the grid's second dimension: q's, then K's, then V's
  RopeGrid q;            // q's pieces; its cosines are K's too
  int heads;             // KV heads of a work-group
  Divide by_head, by_token;  // pieces of a head, of a work-group's heads of one token
};

// Eight elements of a head from `c` on, and those that they turn with in the half layout
template <int S>
__device__ __forceinline__ void load_key(const KvStoreArgs& a, int64_t at, int c, Raw8<S>* own, Raw8<S>* other) {
  const int half = (int)a.rot / 2;
  *own = load8<S>(a.k, at + c);
  *other = load8<S>(a.k, at + (c >= a.rot || a.inter ? c : c < half ? c + half : c - half));
}
// ... turned where they have to be
template <int S>
__device__ __forceinline__ void turn_key(const KvStoreArgs& a, const Raw8<S>& own, const Raw8<S>& other, int c,
                                         const float2* cs, float (&v)[8]) {
  const int half = (int)a.rot / 2;
  widen<S>(own, a.in_type, v);
  if (c >= a.rot) return;  // rot is a multiple of 16: a piece turns or does not
  if (a.inter) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 o = turned(v[2 * j], v[2 * j + 1], cs[c / 2 + j]);
      v[2 * j] = o.x;
      v[2 * j + 1] = o.y;
    }
  } else {
    const bool low = c < half;
    float w[8];
    widen<S>(other, a.in_type, w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = low ? turned(v[j], w[j], cs[c + j]).x : turned(w[j], v[j], cs[c - half + j]).y;
  }
}

__device__ __forceinline__ void put_v_token(uint8_t* head, const KvHead& lay, int d, int t, int p, uint32_t codes,
                                            uint32_t params) {
  uint8_t* c = head + lay.v_codes() + (int64_t)((t >> 2) * (d / 2) + p * 4) * 4 + v_byte(t & 3);
#pragma unroll
  for (int e = 0; e < 4; ++e) c[4 * e] = (uint8_t)(codes >> (8 * e));
  if ((p & 3) == 0) {
    uint16_t* q = reinterpret_cast<uint16_t*>(head + lay.v_params()) + ((t >> 2) * (d / 32) + (p >> 2)) * 8 + (t & 3);
    q[0] = (uint16_t)params;
    q[4] = (uint16_t)(params >> 16);
  }
}

// byte e of each of four tokens' codes, in the order of v_byte
__device__ __forceinline__ uint32_t gather_bytes(const uint32_t (&w)[4], int e) {
  const uint32_t sel = (uint32_t)e | ((uint32_t)(e + 4) << 8) | 0x0C0C0000u;
  const uint32_t even = __builtin_amdgcn_perm(w[2], w[0], sel), odd = __builtin_amdgcn_perm(w[3], w[1], sel);
  return even | (odd << 16);
}

// FOUR: an item of V is four tokens, which is one 16-byte store where they
// are four neighbours of a page that start at a multiple of four; the others go byte by byte.  The
// host does not see the slots: for four tokens and more, of which a prompt's are the many.  Both
// sides, us, by fours and one by one (inputs from memory; 8 heads of 128, BF16, 32 of q): 4096 tokens in
// order 27.6 and 28.2, in order from another slot 29.6 and 28.7, scattered 34.9 and 33.1; 500 in order 8.0
// and 8.0.  4 heads of 256, FP32: single tokens of 61 chats 6.6 and 6.6, of 1000 20.0 and 17.6.
template <int S, bool FOUR>
__global__ __launch_bounds__(kThreads) void kv_store_kernel(KvStoreArgs a, KvGrid g) {
  const int64_t first = (int64_t)blockIdx.x * g.tokens;
  int part = (int)blockIdx.y;
  if (part < g.q_parts) {
    RopeArgs r = {a.q, a.q_out, a.positions, a.turns, a.ldq, a.ldqh, a.ldqo, a.ldqoh, a.m, a.hq, a.d, a.rot,
                  a.gain, a.inter, a.in_type, a.qo_type};
    rope_part<S>(r, g.q, first, part * g.q.heads, shared_turns);
    return;
  }
  part -= g.q_parts;
  const int tokens = (int)min((int64_t)g.tokens, a.m - first);
  const bool values = part >= g.kv_parts;
  const int head0 = (values ? part - g.kv_parts : part) * g.heads;
  const int heads = min(g.heads, (int)a.heads - head0), d = (int)a.d;
  const int per_head = d / 8, per_token = g.heads * per_head;
  const KvHead lay(1 << g.shift, d);
  const int64_t page_bytes = a.heads * lay.bytes();
  if (!values) {
    const int half = (int)a.rot / 2;
    if (a.turns) {
      fill_turns(shared_turns, a.positions, a.turns, first, tokens, half, g.q.by_half, a.gain);
      __syncthreads();
    }
    constexpr int kPieces = FOUR ? 4 : 1;
    for (int i0 = threadIdx.x; i0 < tokens * per_token; i0 += kPieces * kThreads) {
      Raw8<S> own[kPieces], other[kPieces];
      int token[kPieces], head[kPieces], piece[kPieces], slot[kPieces];
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int i = i0 + e * kThreads;
        const int t = quotient(i, g.by_token), r = i - t * per_token, h = quotient(r, g.by_head);
        token[e] = t;
        head[e] = head0 + h;
        piece[e] = r - h * per_head;
        slot[e] = -1;
        if (i < tokens * per_token && h < heads) {
          slot[e] = a.slots[first + t];
          load_key<S>(a, (first + t) * a.ldk + head[e] * a.ldkh, piece[e] * 8, &own[e], &other[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        int64_t at;
        int in;
        if (!place_of(slot[e], g.shift, a.n_pages, &at, &in)) continue;
        const int p = piece[e];
        float v[8];
        turn_key<S>(a, own[e], other[e], p * 8, shared_turns + token[e] * half, v);
        uint32_t params;
        const uint32_t codes = quantise8(v, &params);
        uint8_t* to = a.pages + at * page_bytes + (int64_t)head[e] * lay.bytes();
        reinterpret_cast<uint32_t*>(to)[in * (d / 8) + p] = codes;
        if ((p & 3) == 0) reinterpret_cast<uint32_t*>(to + lay.k_params())[in * (d / 32) + (p >> 2)] = params;
      }
    }
    return;
  }
  constexpr int kTok = FOUR ? 4 : 1;
  const int items = (tokens + kTok - 1) / kTok * per_token;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int t = quotient(i, g.by_token), r = i - t * per_token;
    const int h = quotient(r, g.by_head), p = r - h * per_head;
    if (h >= heads) continue;
    const int64_t token = first + t * kTok;
    const int have = min(kTok, tokens - t * kTok);
    uint32_t codes[4], params[4];
    int slot[4];
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      // past the end: the last token again, which is not written twice
      const int64_t row = token + min(j, have - 1);
      slot[j] = j < have ? a.slots[row] : -1;
      float v[8];
      widen<S>(load8<S>(a.v, row * a.ldv + (head0 + h) * a.ldvh + p * 8), a.in_type, v);
      codes[j] = quantise8(v, &params[j]);
    }
    int64_t at;
    int in;
    const int64_t off = (int64_t)(head0 + h) * lay.bytes();
    if constexpr (FOUR) {
      if ((slot[0] & 3) == 0 && slot[1] == slot[0] + 1 && slot[2] == slot[0] + 2 && slot[3] == slot[0] + 3) {
        if (!place_of(slot[0], g.shift, a.n_pages, &at, &in)) continue;
        uint8_t* head = a.pages + at * page_bytes + off;
        reinterpret_cast<uint4*>(head + lay.v_codes())[((in >> 2) * (d / 2) + p * 4) / 4] =
            make_uint4(gather_bytes(codes, 0), gather_bytes(codes, 1), gather_bytes(codes, 2), gather_bytes(codes, 3));
        if ((p & 3) == 0)
          reinterpret_cast<uint4*>(head + lay.v_params())[(in >> 2) * (d / 32) + (p >> 2)] =
              make_uint4(__builtin_amdgcn_perm(params[1], params[0], 0x05040100u),
                         __builtin_amdgcn_perm(params[3], params[2], 0x05040100u),
                         __builtin_amdgcn_perm(params[1], params[0], 0x07060302u),
                         __builtin_amdgcn_perm(params[3], params[2], 0x07060302u));
        continue;
      }
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (place_of(slot[j], g.shift, a.n_pages, &at, &in))
        put_v_token(a.pages + at * page_bytes + off, lay, d, in, p, codes[j], params[j]);
  }
}

// eight codes (code j in nibble j) as values in the order of the nibbles
__device__ __forceinline__ void values8(uint32_t w, uint32_t params, float (&v)[8]) {
  const f16x2 ab = __builtin_bit_cast(f16x2, params);
  const f16x2 a = {ab.x, ab.x}, b = {ab.y, ab.y};
  const uint32_t ones = ones_of();
  const f16x2 x[4] = {fma2(nibbles<0>(w, ones), a, b), fma2(nibbles<1>(w, ones), a, b),
                      fma2(nibbles<2>(w, ones), a, b), fma2(nibbles<3>(w, ones), a, b)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = (float)x[j].x;
    v[j + 4] = (float)x[j].y;
  }
}

// Pieces of K that a thread has on their way (32768 tokens, 4 heads of 256: 43.7 us, 50 with one)
constexpr int kAhead = 4;

// FOUR as above, us by fours and one by one (a graph's calls): 4096 tokens of 8 heads of 128 in order 6.5
// and 8.7, from another slot 8.1 and 8.4; 32768 of 4 of 256 28.8 and 34.7, from another slot 35.0 and
// 35.4; 64 in order 3.2 and 3.4, but single tokens of 61 chats 4.1 and 3.4.
template <bool FOUR>
__global__ __launch_bounds__(kThreads) void kv_load_kernel(KvLoadArgs a, KvGrid g) {
  const int64_t first = (int64_t)blockIdx.x * g.tokens;
  const int part = (int)blockIdx.y;
  const int tokens = (int)min((int64_t)g.tokens, a.m - first);
  const bool values = a.k == nullptr || part >= g.kv_parts;
  const int head0 = (part >= g.kv_parts ? part - g.kv_parts : part) * g.heads;
  const int heads = min(g.heads, (int)a.heads - head0), d = (int)a.d;
  const int per_head = d / 8, per_token = g.heads * per_head;
  const KvHead lay(1 << g.shift, d);
  const int64_t page_bytes = a.heads * lay.bytes();
  const int kTok = values && FOUR ? 4 : 1;
  const int items = (tokens + kTok - 1) / kTok * per_token;
  if (!values) {
    for (int i0 = threadIdx.x; i0 < items; i0 += kAhead * kThreads) {
      int64_t to[kAhead];
      int slot[kAhead], head[kAhead], piece[kAhead];
      uint32_t codes[kAhead], params[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int i = min(i0 + e * kThreads, items - 1);
        const int t = quotient(i, g.by_token), r = i - t * per_token;
        const int h = quotient(r, g.by_head);
        piece[e] = r - h * per_head;
        head[e] = i0 + e * kThreads < items && h < heads ? head0 + h : -1;
        slot[e] = a.slots[first + t];
        to[e] = (first + t) * a.ldk + (head0 + h) * a.ldkh + piece[e] * 8;
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        int64_t at;
        int in;
        codes[e] = params[e] = 0;
        if (place_of(slot[e], g.shift, a.n_pages, &at, &in) && head[e] >= 0) {
          const uint8_t* from = a.pages + at * page_bytes + (int64_t)head[e] * lay.bytes();
          codes[e] = reinterpret_cast<const uint32_t*>(from)[in * (d / 8) + piece[e]];
          params[e] = reinterpret_cast<const uint32_t*>(from + lay.k_params())[in * (d / 32) + (piece[e] >> 2)];
        }
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (head[e] < 0) continue;
        float v[8];
        values8(codes[e], params[e], v);
        store8(a.k, a.out_type, to[e], 0, v);
      }
    }
    return;
  }
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int t = quotient(i, g.by_token), r = i - t * per_token;
    const int h = quotient(r, g.by_head), p = r - h * per_head;
    if (h >= heads) continue;
    const int64_t off = (int64_t)(head0 + h) * lay.bytes();
    int64_t at;
    int in;
    float v[8];
    const int64_t token = first + t * kTok;
    const int have = min(kTok, tokens - t * kTok);
    if constexpr (FOUR) {
      const int s0 = a.slots[token];
      if (have == 4 && (s0 & 3) == 0 && a.slots[token + 1] == s0 + 1 && a.slots[token + 2] == s0 + 2 &&
          a.slots[token + 3] == s0 + 3) {
        uint4 c = make_uint4(0, 0, 0, 0), q = make_uint4(0, 0, 0, 0);
        if (place_of(s0, g.shift, a.n_pages, &at, &in)) {
          const uint8_t* head = a.pages + at * page_bytes + off;
          c = reinterpret_cast<const uint4*>(head + lay.v_codes())[((in >> 2) * (d / 2) + p * 4) / 4];
          q = reinterpret_cast<const uint4*>(head + lay.v_params())[(in >> 2) * (d / 32) + (p >> 2)];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int byte = (j & 1) * 2 + (j >> 1);
          const uint32_t lo = (uint32_t)byte * 0x0101u + 0x0400u;  // this byte of two dwords, side by side
          const uint32_t codes = __builtin_amdgcn_perm(c.y, c.x, lo | 0x0C0C0000u) |
                                 (__builtin_amdgcn_perm(c.w, c.z, lo | 0x0C0C0000u) << 16);
          const uint32_t aa = j < 2 ? q.x : q.y, bb = j < 2 ? q.z : q.w;
          values8(codes, __builtin_amdgcn_perm(bb, aa, (j & 1) ? 0x07060302u : 0x05040100u), v);
          store8(a.v, a.out_type, (token + j) * a.ldv + (head0 + h) * a.ldvh + p * 8, 0, v);
        }
        continue;
      }
    }
    for (int j = 0; j < have; ++j) {
      uint32_t codes = 0, params = 0;
      if (place_of(a.slots[token + j], g.shift, a.n_pages, &at, &in)) {
        const uint8_t* head = a.pages + at * page_bytes + off;
        const uint8_t* c = head + lay.v_codes() + (int64_t)((in >> 2) * (d / 2) + p * 4) * 4 + v_byte(in & 3);
#pragma unroll
        for (int e = 0; e < 4; ++e) codes |= (uint32_t)c[4 * e] << (8 * e);
        const uint16_t* q = reinterpret_cast<const uint16_t*>(head + lay.v_params()) +
                            ((in >> 2) * (d / 32) + (p >> 2)) * 8 + (in & 3);
        params = (uint32_t)q[0] | ((uint32_t)q[4] << 16);
      }
      values8(codes, params, v);
      store8(a.v, a.out_type, (token + j) * a.ldv + (head0 + h) * a.ldvh + p * 8, 0, v);
    }
  }
}

// Tokens and heads of a work-group for the cache's part
void kv_grid(KvGrid* g, int64_t m, int64_t heads, int64_t d, int64_t page, int64_t half) {
  g->shift = 0;
  while ((1 << g->shift) < page) ++g->shift;
  const int per_head = (int)d / 8;
  const int64_t per_token = heads * per_head;
  const int64_t target = m * per_token <= 512 * kSmall ? kSmall : 4 * kThreads;
  g->heads = (int)max((int64_t)1, min(heads, target / per_head));
  int64_t tokens = max((int64_t)1, target / (g->heads * per_head));
  if (half) tokens = min(tokens, kMostTurns / half);
  tokens = min(tokens, m);
  g->tokens = (int)(m >= 4 ? max((int64_t)4, tokens / 4 * 4) : tokens);
  g->kv_parts = (int)((heads + g->heads - 1) / g->heads);
  g->by_head = divide(per_head);
  g->by_token = divide(g->heads * per_head);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t st) {
  const RopeGrid g = rope_grid(a, a.out == a.x);
  const dim3 grid((unsigned)((a.m + g.tokens - 1) / g.tokens), (unsigned)((a.heads + g.heads - 1) / g.heads));
  const size_t lds = (size_t)g.tokens * g.pieces.half * sizeof(float2);
  if (a.x_type == 1) rope_kernel<4><<<grid, kThreads, lds, st>>>(a, g);
  else rope_kernel<2><<<grid, kThreads, lds, st>>>(a, g);
  return hipGetLastError();
}

hipError_t launch_kv_store(const KvStoreArgs& a, hipStream_t st) {
  KvGrid g = {};
  const int64_t half = a.turns ? a.rot / 2 : 0;
  kv_grid(&g, a.m, a.heads, a.d, a.page, half);
  g.q.by_half = divide(half ? (int)half : 1);
  if (a.q) {
    RopeArgs r = {};
    r.m = a.m;
    r.heads = a.hq;
    r.d = a.d;
    r.rot = a.rot;
    r.inter = a.inter;
    g.q = rope_grid(r, a.q_out == a.q);
    // The token groups of the cache's part, and as many heads as make up its pieces; four times
    // as many where there is work for all, since each work-group has the cosines to make (4096
    // tokens, 32 heads of 128: 29.7 -> 28.6 us; 61 tokens, 24 heads of 256 would take 14 for 6)
    g.q.tokens = g.tokens;
    const bool many = a.m * (a.heads * a.d / 8) > 512 * kSmall;
    const int64_t target = many ? 16 * kThreads : max((int64_t)kSmall, (int64_t)g.tokens * g.heads * a.d / 8);
    g.q.heads = (int)max((int64_t)1, min(a.hq, target / ((int64_t)g.tokens * g.q.pieces.all)));
    g.q.by_token = divide(g.q.heads * g.q.pieces.all);
    g.q_parts = (int)((a.hq + g.q.heads - 1) / g.q.heads);
  }
  const dim3 grid((unsigned)((a.m + g.tokens - 1) / g.tokens), (unsigned)(g.q_parts + 2 * g.kv_parts));
  const size_t lds = (size_t)g.tokens * half * sizeof(float2);
  const bool four = g.tokens >= 4;
  if (a.in_type == 1) {
    if (four) kv_store_kernel<4, true><<<grid, kThreads, lds, st>>>(a, g);
    else kv_store_kernel<4, false><<<grid, kThreads, lds, st>>>(a, g);
  } else {
    if (four) kv_store_kernel<2, true><<<grid, kThreads, lds, st>>>(a, g);
    else kv_store_kernel<2, false><<<grid, kThreads, lds, st>>>(a, g);
  }
  return hipGetLastError();
}

hipError_t launch_kv_load(const KvLoadArgs& a, hipStream_t st) {
  KvGrid g = {};
  kv_grid(&g, a.m, a.heads, a.d, a.page, 0);
  const dim3 grid((unsigned)((a.m + g.tokens - 1) / g.tokens), (unsigned)(g.kv_parts * ((a.k != nullptr) + (a.v != nullptr))));
  if (g.tokens >= 4) kv_load_kernel<true><<<grid, kThreads, 0, st>>>(a, g);
  else kv_load_kernel<false><<<grid, kThreads, 0, st>>>(a, g);
  return hipGetLastError();
}

}  // namespace lowbit
