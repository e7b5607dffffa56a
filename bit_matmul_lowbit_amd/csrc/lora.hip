// Low-rank adapters of many requests beside a shared low-bit projection:
//   v[i][j]  = scale[s] * sum_k A[s][j][k] x[i][k],  s = ids[i], j < rank[s]
//   y[i][o] += sum_j B[s][o][j] v[i][j]
//
// [P2] 7minutos.es, "PrismML lanza Bonsai 27B ...", "Como funciona la
//      compresion": every projection of the model is a frozen low-bit matrix;
//      what is learned on top of it lives in such adapters.
//
// Rows are grouped by adapter, so that an adapter's matrices meet all of its
// rows at once.  An item is up to 32 rows of one adapter (16 where adapters
// have few rows).  Up to 64 rows, a lane to a row, are grouped by the first
// wave of every work-group for itself (no launch, no memory); more are sorted
// by one work-group first (lora_plan_kernel).
//
// The first product runs on v_mfma_f32_16x16x32, the second on that (BF16) or on
// v_mfma_f32_16x16x4 (FP16; a lane holds one value of an operand's four columns).
//   A operand (16 x 32): lane l holds row l % 16, 8 values at 8 (l / 16)
//   B operand (32 x 16): lane l holds column l % 16, 8 values at 8 (l / 16)
//   D (16 x 16): lane l, register e holds row 4 (l / 16) + e, column l % 16
//
// A small call does both in one launch (lora_small_kernel), others in two:
// shrink: v^T = A x^T, one work-group per (16 rows of an item, up to 48 of
// its ranks, slice of k); its eight waves split the slice and are summed
// through LDS.  The slices' FP32 sums go to the workspace.  Operands taken
// straight from memory would have neighbouring lanes in 16 different rows,
// and such loads run at a quarter of the rate of contiguous ones; a wave
// loads 128 contiguous bytes of a row by eight lanes instead and passes them
// to the lanes that need them through LDS of its own.
// expand: y += v B^T, one work-group per (item, share of the outputs, 256 at a
// time); B goes through LDS in the same manner.  v is summed over the slices and
// scaled.  With BF16 it is split into three pieces whose sum holds its 24 bits,
// with FP16, which reaches less far than a row's inner values may lie apart, it
// stays FP32 and B is widened: a single 16-bit v would be the least exact
// value of the whole sum.  No atomics anywhere: every value has one writer and
// its sum one order.
//
// What bounds it.  Few rows: the bytes of A and B and the latencies before
// they can be asked for (ids, then v).  8 rows of 8 adapters, r 64, 5120 ->
// 34816: 4.0 + 13 us for 7 + 36 MB (more of B in flight changes nothing; with
// B's rows all one expand takes 9.2 us).  Many rows: y, read and written.  4096
// rows of 8 adapters, r 32, 5120 -> 17408, BF16: plan 7.2, shrink 21, expand
// 71 us for 285 MB of y (4.0 TB/s; a large copy reaches 4.8); with FP16 and many
// ranks the FP32 matrix instructions as well (4096 rows, r 128, 5120 -> 5120: 139 us
// a call).  One row, 2048 -> 6144, r 16: 6.8 us in one launch.
#include "common.h"

namespace lowbit {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kInlineRows = 64;  // rows that one wave groups by itself
constexpr int kItemRows = 32;    // most rows of an item
constexpr int kShrinkWaves = 8;
constexpr int kTilesN = 4;                 // 16-output tiles of a wave in expand
constexpr int kWaveN = 16 * kTilesN;       // 64 outputs per wave
constexpr int kBlockN = 4 * kWaveN;        // 256 outputs per work-group
constexpr int kFewRows = 4;                // rows of an FP16 item that go without matrix instructions
constexpr int kMaxSlots = 4096;
constexpr int kMaxSlices = 8;              // slices of k at most

template <int XT> struct Mma;
template <> struct Mma<2> {
  static __device__ __forceinline__ f32x4 run(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <> struct Mma<3> {
  static __device__ __forceinline__ f32x4 run(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};

// How v stands in LDS for the second product: as FP32, or as BF16 pieces, each
// [tm][pitch]; the pad after a row's ranks moves the next one to other banks.
template <int XT> struct Held;
template <> struct Held<2> {
  typedef float type;
  static constexpr int pieces = 1, pad = 4;
};
template <> struct Held<3> {
  typedef bf16_t type;
  static constexpr int pieces = 3, pad = 8;
};
template <int XT>
constexpr int inner_pitch(int r) { return (r + 31) / 32 * 32 + Held<XT>::pad; }
template <int XT>
constexpr size_t inner_bytes(int tm, int r) {
  return sizeof(typename Held<XT>::type) * Held<XT>::pieces * tm * inner_pitch<XT>(r);
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int64_t s) {
  if (!a.ranks) return (int)a.r;
  const int v = a.ranks[s];
  return v < 0 ? 0 : (v > (int)a.r ? (int)a.r : v);
}

// the row's adapter, or -1 for a row that nothing is added to
__device__ __forceinline__ int slot_of(const LoraArgs& a, int64_t i) {
  const int s = a.ids[i];
  return s >= 0 && s < a.slots && rank_of(a, s) > 0 ? s : -1;
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                        __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// What a plan holds, at the head of the workspace: the number of items, the items, and their rows, tm places to an
// item.  All three are found by the item's number alone, so that they are read
// in one memory latency.
struct Item {
  int slot, count, rank;
  float scale;
};
struct Plan {
  int* items_used;
  Item* items;
  int* rows;
  int most;  // items there is room for
};

// inclusive prefix sum over the wave's lanes, by DPP
__device__ __forceinline__ int wave_scan(int v) {
#define LOWBIT_SCAN(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false)
  LOWBIT_SCAN(0x111, 0xF);  // row_shr:1
  LOWBIT_SCAN(0x112, 0xF);  // row_shr:2
  LOWBIT_SCAN(0x114, 0xF);  // row_shr:4
  LOWBIT_SCAN(0x118, 0xF);  // row_shr:8
  LOWBIT_SCAN(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
  LOWBIT_SCAN(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef LOWBIT_SCAN
  return v;
}

// What a work-group shares of its item.
struct Found {
  Item it;
  int rows[kItemRows];
  int64_t y_at[kItemRows];  // where they begin in y (64-bit products at each use cost 1 to 2 % of a call)
};

// Item number `item` (tm rows at most), in every thread: its count is 0 if
// there is none; its rows are in found.rows (LDS).  The call holds a barrier.
// INLINE: the first wave finds it among up to 64 rows, a lane to a row: a ballot
// for each bit of the adapters' numbers gives every lane the rows of its own,
// the first row of each stands for the adapter's items, and a prefix sum
// numbers them.  (Passing the adapters one by one took up to 0.3 us for each.)
// Otherwise: from the plan.
template <bool INLINE>
__device__ __forceinline__ Item find_item(const LoraArgs& a, const Plan& plan, int item, int tm, Found& found) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    Item it = {0, 0, 0, 1.0f};
    if constexpr (INLINE) {
      const int m = (int)a.m;
      const int s = lane < m ? slot_of(a, lane) : -1;
      uint64_t same = __ballot(s >= 0);  // the rows of this lane's adapter, by the bits of its number
      for (int bit = 0; bit < 32 - __builtin_clz((int)a.slots | 1); ++bit) {
        const bool on = (s >> bit) & 1;
        const uint64_t all_on = __ballot(on);
        same &= on ? all_on : ~all_on;
      }
      const int all = __popcll(same), before = lanes_below(same);
      const int parts = s >= 0 && before == 0 ? (all + tm - 1) / tm : 0;
      const int end = wave_scan(parts);
      const uint64_t hit = __ballot(item < end && item >= end - parts);
      if (hit) {
        const int leader = __builtin_ctzll(hit);
        const int first = (item - __builtin_amdgcn_readlane(end - parts, leader)) * tm;
        const int left = __builtin_amdgcn_readlane(all, leader) - first;
        it.slot = __builtin_amdgcn_readlane(s, leader);
        it.count = left < tm ? left : tm;
        it.rank = rank_of(a, it.slot);
        const int at = before - first;
        if (s == it.slot && at >= 0 && at < it.count) {
          found.rows[at] = lane;
          found.y_at[at] = lane * a.ldy;
        }
      }
    } else if (item < plan.most) {
      const int used = *plan.items_used;
      const Item got = plan.items[item];
      const int row = plan.rows[item * tm + (lane & (tm - 1))];
      if (item < used) {
        it = got;
        if (lane < it.count) {
          found.rows[lane] = row;
          found.y_at[lane] = row * a.ldy;
        }
      }
    }
    if (lane == 0) found.it = it;
  }
  __syncthreads();
  Item it;
  it.slot = __builtin_amdgcn_readfirstlane(found.it.slot);
  it.count = __builtin_amdgcn_readfirstlane(found.it.count);
  it.rank = __builtin_amdgcn_readfirstlane(found.it.rank);
  // (asked for here, it is there when v is)
  it.scale = INLINE ? (a.scales ? a.scales[it.slot] : 1.0f) : found.it.scale;
  return it;
}

// Rows sorted by adapter, in one work-group: each row takes the next place
// among its adapter's (a counter in LDS); a prefix sum over the adapters'
// items gives each adapter's first item.  Rows of one adapter keep nearly
// their order; which place one gets changes no result, each row being a row
// of the products of its own.  A wave whose rows share one adapter, as in a
// long prompt, adds to the counter once.  The work-group's first 4096 rows
// keep their places in registers, later ones in `place`.
__global__ __launch_bounds__(1024) void lora_plan_kernel(LoraArgs a, Plan plan, int tm, int* place) {
  constexpr int kHeld = 4;
  __shared__ int cnt[kMaxSlots], first[kMaxSlots];
  __shared__ int wave_items[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int slot[kHeld], at[kHeld];
#pragma unroll
  for (int t = 0; t < kHeld; ++t) slot[t] = t * 1024 + tid < a.m ? slot_of(a, t * 1024 + tid) : -1;
  for (int s = tid; s < a.slots; s += 1024) cnt[s] = 0;
  __syncthreads();
  auto take = [&](int s) __attribute__((always_inline)) {
    const int s0 = __builtin_amdgcn_readfirstlane(s);
    if (__ballot(s == s0) == ~0ull) {
      if (s0 < 0) return 0;
      int got = 0;
      if (lane == 0) got = atomicAdd(&cnt[s0], 64);
      return __builtin_amdgcn_readfirstlane(got) + lane;
    }
    return s >= 0 ? atomicAdd(&cnt[s], 1) : 0;
  };
  const int64_t steps = (a.m + 1023) / 1024;
#pragma unroll
  for (int t = 0; t < kHeld; ++t)
    if (t < steps) at[t] = take(slot[t]);
  for (int64_t t = kHeld; t < steps; ++t) {
    const int64_t i = t * 1024 + tid;
    const int p = take(i < a.m ? slot_of(a, i) : -1);
    if (i < a.m) place[i] = p;
  }
  __syncthreads();
  int own[4], items = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    own[u] = tid * 4 + u < a.slots ? (cnt[tid * 4 + u] + tm - 1) / tm : 0;
    items += own[u];
  }
  const int items_to = wave_scan(items);
  if (lane == 63) wave_items[wave] = items_to;
  __syncthreads();
  const int waves_to = wave_scan(lane < 16 ? wave_items[lane] : 0);
  int it = items_to - items + (wave ? __builtin_amdgcn_readlane(waves_to, wave - 1) : 0);
  if (tid == 0) *plan.items_used = __builtin_amdgcn_readlane(waves_to, 15);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (tid * 4 + u < a.slots) first[tid * 4 + u] = it;
    it += own[u];
  }
  __syncthreads();
  auto put = [&](int s, int p, int i) __attribute__((always_inline)) {
    const int item = first[s] + p / tm, at = p % tm;
    plan.rows[item * tm + at] = i;
    if (at == 0) {
      const int left = cnt[s] - p;
      plan.items[item] = Item{s, left < tm ? left : tm, rank_of(a, s), a.scales ? a.scales[s] : 1.0f};
    }
  };
#pragma unroll
  for (int t = 0; t < kHeld; ++t)
    if (slot[t] >= 0) put(slot[t], at[t], t * 1024 + tid);
  for (int64_t t = kHeld; t < steps; ++t) {
    const int64_t i = t * 1024 + tid;
    const int s = i < a.m ? slot_of(a, i) : -1;
    if (s >= 0) put(s, place[i], (int)i);
  }
}

// The first product for 16 rows and RT * 16 ranks from r0 on, over part `part`
// of `parts` of k for this wave: the work-group's waves are summed, and thread
// 64 t + lane (t < RT) returns v[row lane % 16][r0 + 16 t + 4 (lane / 16) ..+3]
// of the parts of all its waves.  Rows past the `here` given ones and ranks
// past the adapter's repeat the last one (each is a row or column of the MFMA
// of its own) and are not to be used.
//
// `stage`, per wave: a step of each tile, 16 rows of 8 pieces of 16 bytes,
// piece p of row i at p ^ (i & 7) (the lanes of a read then fall into
// different banks); afterwards the waves' sums.  The call ends with reads of
// it.
template <int XT, int RT, int WAVES>
__device__ __forceinline__ f32x4 shrink16(const LoraArgs& a, int slot, int rank, int r0, const int* rows,
                                          int here, uint4 (*stage)[1 + RT][16][8], int part, int parts) {
  constexpr int T = 1 + RT;                          // 16-row tiles of a step: x, then A's
  constexpr int U = RT >= 3 ? 2 : RT == 2 ? 3 : 4;   // steps in flight
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;    // as an operand's lane
  const int lr = lane >> 3, lp = lane & 7;   // as a loading lane: rows lr and lr + 8, piece lp
  const uint16_t* xp[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = lr + 8 * h;
    xp[h] = static_cast<const uint16_t*>(a.x) + (int64_t)rows[at < here ? at : here - 1] * a.ldx;
  }
  const uint16_t* ap = static_cast<const uint16_t*>(a.a) + (int64_t)slot * a.r * a.k;
  uint32_t aoff[RT][2];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = r0 + t * 16 + lr + 8 * h;
      aoff[t][h] = (uint32_t)(j < rank ? j : rank - 1) * (uint32_t)a.k;
    }
  const int k = (int)a.k, steps = (k + 63) / 64;
  // steps part, part + parts, ...: the waves that run together read
  // neighbouring 128 bytes
  const int mine = part < steps ? (steps - part + parts - 1) / parts : 0;

  f32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  uint4 in[U][T][2];
  auto load = [&](int u, int i) __attribute__((always_inline)) {
    int at = (part + i * parts) * 64 + lp * 8;
    at = at < k ? at : k - 8;  // pieces past k are zeroed below
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      in[u][0][h] = *reinterpret_cast<const uint4*>(xp[h] + at);
#pragma unroll
      for (int t = 0; t < RT; ++t)
        in[u][1 + t][h] = *reinterpret_cast<const uint4*>(ap + (aoff[t][h] + (uint32_t)at));
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < mine) load(u, u);
  for (int i = 0; i < mine; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < mine) {
        const int s = part + (i + u) * parts;
        if (s * 64 + 64 > k && s * 64 + lp * 8 >= k) {
#pragma unroll
          for (int t = 0; t < T; ++t) in[u][t][0] = in[u][t][1] = make_uint4(0, 0, 0, 0);
        }
        // a wave's LDS accesses are carried out in their order; the empty asm
        // statements keep the compiler to it
        __asm__ volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) stage[wave][t][lr + 8 * h][lp ^ (lr & 7)] = in[u][t][h];
        __asm__ volatile("" ::: "memory");
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint4 b = stage[wave][0][c][(w * 4 + q) ^ (c & 7)];
#pragma unroll
          for (int t = 0; t < RT; ++t)
            acc[t] = Mma<XT>::run(stage[wave][1 + t][c][(w * 4 + q) ^ (c & 7)], b, acc[t]);
        }
        if (i + U + u < mine) load(u, i + U + u);
      }
    }
  }
  __syncthreads();
  f32x4(*red)[RT][64] = reinterpret_cast<f32x4(*)[RT][64]>(&stage[0][0][0][0]);
#pragma unroll
  for (int t = 0; t < RT; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  f32x4 sum = (f32x4){0.f, 0.f, 0.f, 0.f};
  if (wave < RT) {
    sum = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += red[w][wave][lane];
  }
  return sum;
}

// v[slice][row][j] for 16 rows of an item and RT * 16 ranks: blockIdx.x =
// item * subs + (16-row part of the item), y = part of the ranks, z = slice.
template <int XT, int RT, bool INLINE>
__global__ __launch_bounds__(512) void lora_shrink_kernel(LoraArgs a, Plan plan, int tm, int subs,
                                                          float* __restrict__ v) {
  __shared__ Found found;
  const int* rows = found.rows;
  __shared__ uint4 stage[kShrinkWaves][1 + RT][16][8];
  const int item = blockIdx.x / subs, sub = blockIdx.x % subs;
  const Item it = find_item<INLINE>(a, plan, item, tm, found);
  const int here = it.count - sub * 16 < 16 ? it.count - sub * 16 : 16;
  if (here <= 0) return;
  const int rank = it.rank, r0 = (int)blockIdx.y * RT * 16;
  if (r0 >= rank) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const f32x4 sum = shrink16<XT, RT, kShrinkWaves>(a, it.slot, rank, r0, rows + sub * 16, here, stage,
                                     (int)blockIdx.z * kShrinkWaves + wave, kShrinkWaves * (int)gridDim.z);
  const int c = threadIdx.x & 15, j = r0 + wave * 16 + ((threadIdx.x >> 4) & 3) * 4;
  // j .. j + 3 lie in the row (r is a multiple of 8); what is past the rank is not read
  if (wave < RT && c < here && j < rank)
    *reinterpret_cast<f32x4*>(v + ((int64_t)blockIdx.z * a.m + rows[sub * 16 + c]) * a.r + j) = sum;
}

// FP32 value -> its pieces.  The three are cut, not rounded, 8 bits each: they
// hold the value's 24, none of a finite value is infinite, and all have its
// sign.  One that nothing is left for takes half of the one before, so that an
// infinite entry of B meets no zero unless the value is one.
__device__ __forceinline__ void split(float v, float (&p)[1]) { p[0] = v; }
__device__ __forceinline__ void split(float v, bf16_t (&p)[3]) {
  const auto cut = [](float f) __attribute__((always_inline)) {
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, f) & 0xFFFF0000u);
  };
  float hi = v, mid = v, lo = v;
  if (__builtin_isfinite(v)) {
    hi = cut(v);
    mid = cut(v - hi);
    lo = v - hi - mid;
    if (mid == 0.0f) {
      hi *= 0.5f;
      mid = hi;
      lo = 0.0f;
    }
    if (lo == 0.0f) {
      mid *= 0.5f;
      lo = mid;
    }
  }
  p[0] = (bf16_t)hi;
  p[1] = (bf16_t)mid;
  p[2] = (bf16_t)lo;
}

// acc[s][t] += the products of 32 ranks: of v's rows (`v`: at this lane's first
// rank, in its row of the first of SUBS 16-row parts) and of B's in `w`.
//
// FP16: FP32 products, an eighth of the rate of two FP16 pieces, but a piece's
// smallest step (2^-38 of the row's largest value) and what its zeros make of an
// infinite entry of B do not show in y.  HALVES: a lane's ranks are four of the
// first 16 and, if `both`, four of the others, so that 16 ranks take half of the
// instructions (342 rows, r 16, 768 -> 12378: 27.9 -> 24.7 us a call; FP16 pieces
// 22.7).  4096 rows, r 128, 5120 -> 5120: 139 us, FP16 pieces 112.
template <int SUBS, bool HALVES>
__device__ __forceinline__ void multiply(const float* v, int pitch, int, int count, bool both,
                                         const uint4 (&w)[kTilesN], f32x4 (&acc)[SUBS][kTilesN]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && !both) break;
    f32x4 a[SUBS];
#pragma unroll
    for (int s = 0; s < SUBS; ++s)
      if (s * 16 < count) a[s] = *reinterpret_cast<const f32x4*>(v + s * 16 * pitch + h * (HALVES ? 16 : 4));
#pragma unroll
    for (int t = 0; t < kTilesN; ++t) {
      const f16x8 b = __builtin_bit_cast(f16x8, w[t]);
#pragma unroll
      for (int s = 0; s < SUBS; ++s) {
        if (s * 16 < count) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[s][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s][i], (float)b[h * 4 + i], acc[s][t], 0, 0, 0);
        }
      }
    }
  }
}
template <int SUBS, bool>
__device__ __forceinline__ void multiply(const bf16_t* v, int pitch, int tm, int count, bool,
                                         const uint4 (&w)[kTilesN], f32x4 (&acc)[SUBS][kTilesN]) {
#pragma unroll
  for (int s = 0; s < SUBS; ++s) {
    if (s * 16 < count) {
#pragma unroll
      for (int p = 0; p < Held<3>::pieces; ++p) {
        const uint4 a = *reinterpret_cast<const uint4*>(v + (p * tm + s * 16) * pitch);
#pragma unroll
        for (int t = 0; t < kTilesN; ++t) acc[s][t] = Mma<3>::run(a, w[t], acc[s][t]);
      }
    }
  }
}

// FP16, up to kFewRows rows, for which a matrix instruction's 16 would be mostly
// empty: each lane sums its own 8 ranks (`v`: at the first of them, of the first
// row), and few_end() joins the four lanes of an output.  8 rows of 8 adapters, r
// 64, 5120 -> 34816: 16.8 us a call, 19.9 by matrix instructions; 1 x 2048 -> 6144,
// r 16: 6.8 and 7.5.
__device__ __forceinline__ void few(const float* v, int pitch, int count, const uint4 (&w)[kTilesN],
                                    f32x4 (&acc)[kTilesN]) {
#pragma unroll
  for (int e = 0; e < kFewRows; ++e) {
    if (e < count) {
      float a[8];
      __builtin_memcpy(a, __builtin_assume_aligned(v + e * pitch, 16), 32);
#pragma unroll
      for (int t = 0; t < kTilesN; ++t) {
        const f16x8 b = __builtin_bit_cast(f16x8, w[t]);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t][e] = __builtin_fmaf((float)b[i], a[i], acc[t][e]);
      }
    }
  }
}
__device__ __forceinline__ void few_end(int count, f32x4 (&acc)[kTilesN]) {
#pragma unroll
  for (int e = 0; e < kFewRows; ++e)
    if (e < count) {
#pragma unroll
      for (int t = 0; t < kTilesN; ++t) {
        const float half = acc[t][e] + __shfl_xor(acc[t][e], 16, 64);
        acc[t][e] = half + __shfl_xor(half, 32, 64);
      }
    }
}

// four consecutive outputs of a row, as they are stored
template <int YT>
struct Out4 {
  uint32_t d[YT == 1 ? 4 : 2];
};

// + what is added, rounded once
__device__ __forceinline__ Out4<1> add4(Out4<1> z, float a0, float a1, float a2, float a3) {
  const float add[4] = {a0, a1, a2, a3};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    z.d[u] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, z.d[u]) + add[u]);
  return z;
}
__device__ __forceinline__ Out4<3> add4(Out4<3> z, float a0, float a1, float a2, float a3) {
  const float add[4] = {a0, a1, a2, a3};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float lo = __builtin_bit_cast(float, z.d[u] << 16) + add[2 * u];
    const float hi = __builtin_bit_cast(float, z.d[u] & 0xFFFF0000u) + add[2 * u + 1];
    z.d[u] = (uint32_t)__builtin_bit_cast(uint16_t, (bf16_t)lo) |
             ((uint32_t)__builtin_bit_cast(uint16_t, (bf16_t)hi) << 16);
  }
  return z;
}

// the first n < 4 of them (a row's last outputs)
__device__ __forceinline__ void load_tail(Out4<1>& z, const float* p, int n) {
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (u < n) z.d[u] = __builtin_bit_cast(uint32_t, p[u]);
}
__device__ __forceinline__ void load_tail(Out4<3>& z, const bf16_t* p, int n) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
  z.d[0] = n > 0 ? h[0] : 0u;
  if (n > 1) z.d[0] |= (uint32_t)h[1] << 16;
  z.d[1] = n > 2 ? h[2] : 0u;
}
__device__ __forceinline__ void store_tail(const Out4<1>& z, float* p, int n) {
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (u < n) p[u] = __builtin_bit_cast(float, z.d[u]);
}
__device__ __forceinline__ void store_tail(const Out4<3>& z, bf16_t* p, int n) {
  uint16_t* h = reinterpret_cast<uint16_t*>(p);
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (u < n) h[u] = (uint16_t)(z.d[u >> 1] >> ((u & 1) * 16));
}

// The second product for an item of up to SUBS * 16 rows: share `share` of
// `shares` of the outputs, WAVES * 64 at a time.  Column c of a wave's tile t
// is output 4 c + t, so that a lane's four tiles are four consecutive outputs
// and 16 lanes read and write 256 contiguous bytes of an FP32 row (128 of
// BF16).  The first outputs and the first ranks of B are on their way while v
// is made ready: first() brings about what inner(row, j), four sums of v from
// rank j on, needs.
template <int XT, int YT, bool INLINE, int SUBS, int WAVES, class First, class Inner>
__device__ __forceinline__ void expand_item(const LoraArgs& a, const Item& it, const Found& found,
                                            typename Held<XT>::type* pieces, int tm, uint4* staged, int share,
                                            int shares, First first, Inner inner) {
  // Four lanes load 64 contiguous bytes of a row of B and pass them on through
  // LDS, as in shrink: 8 rows of 8 adapters 17.8 -> 16.8 us a call, 4096 rows
  // 101.4 -> 97.8 (not in the small kernel, whose first product holds that LDS).
  constexpr bool kStaged = WAVES == 4;
  constexpr int P = Held<XT>::pieces;
  constexpr bool kHalves = XT == 2 && !INLINE;  // a lane's ranks of 32: 4 q .. + 3 and those 16 on; else 8 q .. + 7
  typedef typename Held<XT>::type V;
  typedef typename Elem<XT>::type X;
  typedef typename Elem<YT>::type Y;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int slot = it.slot, count = it.count, rank = it.rank;
  const float scale = it.scale;
  const int chunks = (rank + 31) / 32, pitch = inner_pitch<XT>(rank);
  const X* bs = static_cast<const X*>(a.b) + (int64_t)slot * a.n * a.r;
  // where row 4 q + e of a part, one of the item's, has its outputs n0 + 4 c
  // ...; made anew at each use (kept, the pointers would cost a wave of occupancy)
  auto yrow = [&](int s, int e, int64_t n0) __attribute__((always_inline)) {
    return static_cast<Y*>(a.y) + (found.y_at[s * 16 + q * 4 + e] + n0 + c * 4);
  };

  // by how much the four pieces of row `r` of B change places in LDS, so that 32
  // lanes that read 8 bytes of 16 rows find them in different banks
  auto turn = [](int r) __attribute__((always_inline)) { return (r >> 2 & 1) * 2 + (r >> 3 & 1); };
  uint4 w[2][kTilesN];
  // B's rows from n0 on: a uniform base and 32-bit offsets
  auto load_w = [&](uint4 (&d)[kTilesN], int64_t n0, int rc) __attribute__((always_inline)) {
    int j = rc * 32 + (kStaged ? lane & 3 : q) * 8;
    j = j < (int)a.r ? j : (int)a.r - 8;  // past r: any, masked below
    const int last = a.n - n0 < kWaveN ? (int)(a.n - n0) - 1 : kWaveN - 1;
    const X* base = bs + n0 * a.r;
#pragma unroll
    for (int t = 0; t < kTilesN; ++t) {
      const int o = (kStaged ? lane >> 2 : c) * kTilesN + t;
      // an output past the last is not stored
      d[t] = *reinterpret_cast<const uint4*>(base + (uint32_t)((o < last ? o : last) * (int)a.r + j));
    }
  };
  Out4<YT> z[SUBS][4] = {};
  auto load_y = [&](int64_t n0) __attribute__((always_inline)) {
    const int64_t left = a.n - n0 - c * 4;
#pragma unroll
    for (int s = 0; s < SUBS; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (s * 16 + q * 4 + e < count) {
          const Y* at = yrow(s, e, n0);
          if (left >= 4) __builtin_memcpy(&z[s][e], at, sizeof(z[s][e]));
          else load_tail(z[s][e], at, (int)left);
        }
  };
  const int64_t step = (int64_t)shares * (WAVES * kWaveN);
  int64_t n0 = ((int64_t)share * WAVES + wave) * kWaveN;
  // B in a ring of two: its (outputs, 32 ranks) pieces in the order in which
  // they are used, two of them ahead
  int64_t pn = n0;
  int prc = 0;
  auto request = [&](uint4 (&d)[kTilesN]) __attribute__((always_inline)) {
    if (pn >= a.n) return;
    load_w(d, pn, prc);
    if (++prc == chunks) {
      prc = 0;
      pn += step;
    }
  };
  request(w[0]);
  if (n0 < a.n) load_y(n0);
  request(w[1]);

  first();
  // v of the item's rows, 16 lanes to a row, 64 ranks at a time
  for (int sub = 0; sub * 16 < count; ++sub) {
    if (WAVES > 4 && wave >= 4) break;  // 256 threads are 16 rows
    const int at = sub * 16 + (tid >> 4), j0 = (tid & 15) * 4;
    const bool live = at < count;
    auto scaled = [&](int j) __attribute__((always_inline)) {
      f32x4 sum = (f32x4){0.f, 0.f, 0.f, 0.f};
      if (live && j < rank) {
        sum = inner(at, j);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = j + e < rank ? sum[e] * scale : 0.0f;
      }
      return sum;
    };
#pragma unroll 1
    for (int j = j0; j < chunks * 32; j += 64) {
      const f32x4 val = scaled(j);
      V p[4][P];
#pragma unroll
      for (int e = 0; e < 4; ++e) split(val[e], p[e]);
#pragma unroll
      for (int u = 0; u < P; ++u) {
        V o[4] = {p[0][u], p[1][u], p[2][u], p[3][u]};
        __builtin_memcpy(__builtin_assume_aligned(pieces + (u * tm + at) * pitch + j, sizeof(o)), o, sizeof(o));
      }
    }
  }
  __syncthreads();

  // (Only where an adapter's rows are dealt to its items in their order, so that
  // which form a row goes through depends on nothing but the call's arguments.)
  constexpr bool kFew = XT == 2 && INLINE;
  const bool is_few = kFew && count <= kFewRows;
  f32x4 acc[SUBS][kTilesN];
  int rc = 0;
  // one piece of B; with the last ranks of an output, y is written
  auto advance = [&](uint4 (&d)[kTilesN]) __attribute__((always_inline)) {
    if (rc == 0) {
#pragma unroll
      for (int s = 0; s < SUBS; ++s)
#pragma unroll
        for (int t = 0; t < kTilesN; ++t) acc[s][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    const int j = rc * 32 + q * (kHalves ? 4 : 8);
    const bool both = !kHalves || rank - rc * 32 > 16;
    if constexpr (kStaged) {
      uint4* own = staged + wave * (kTilesN * 64);
#pragma unroll
      for (int t = 0; t < kTilesN; ++t) own[t * 64 + (lane ^ (kHalves ? turn(lane >> 2) : 0))] = d[t];
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int t = 0; t < kTilesN; ++t) {
        if constexpr (kHalves) {
          const uint2* row = reinterpret_cast<const uint2*>(own + t * 64 + c * 4);
          const uint2 lo = row[q ^ (2 * turn(c))], hi = row[(4 + q) ^ (2 * turn(c))];
          d[t] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          d[t] = own[t * 64 + c * 4 + q];
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
    if (rc * 32 + 32 > rank) {  // entries past the rank may hold anything
      uint32_t keep[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int left = rank - j - 2 * h - (kHalves && h >= 2 ? 12 : 0);
        keep[h] = left >= 2 ? 0xFFFFFFFFu : (left == 1 ? 0xFFFFu : 0u);
      }
#pragma unroll
      for (int t = 0; t < kTilesN; ++t) {
        d[t].x &= keep[0];
        d[t].y &= keep[1];
        d[t].z &= keep[2];
        d[t].w &= keep[3];
      }
    }
    if constexpr (kFew) {
      if (is_few) few(pieces + j, pitch, count, d, acc[0]);
      else multiply<SUBS, kHalves>(pieces + c * pitch + j, pitch, tm, count, both, d, acc);
    } else {
      multiply<SUBS, kHalves>(pieces + c * pitch + j, pitch, tm, count, both, d, acc);
    }
    request(d);
    if (++rc < chunks) return;
    rc = 0;
    if constexpr (kFew) {
      if (is_few) few_end(count, acc[0]);
    }
#pragma unroll
    for (int s = 0; s < SUBS; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        z[s][e] = add4(z[s][e], acc[s][0][e], acc[s][1][e], acc[s][2][e], acc[s][3][e]);
    const int64_t left = a.n - n0 - c * 4;
#pragma unroll
    for (int s = 0; s < SUBS; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (s * 16 + q * 4 + e < count) {
          Y* at = yrow(s, e, n0);
          if (left >= 4) __builtin_memcpy(at, &z[s][e], sizeof(z[s][e]));
          else store_tail(z[s][e], at, (int)left);
        }
    n0 += step;
    if (n0 < a.n) load_y(n0);
  };
  while (n0 < a.n) {
    advance(w[0]);
    if (n0 < a.n) advance(w[1]);
  }
}

// One item, every gridDim.x-th 256 outputs.
template <int XT, int YT, bool INLINE, int SUBS>
__global__ __launch_bounds__(256, SUBS == 1 ? 4 : YT == 3 ? 3 : 2) void lora_expand_kernel(
    LoraArgs a, Plan plan, int tm, int slices, const float* __restrict__ v) {
  extern __shared__ uint4 dyn[];  // v (Held)
  __shared__ Found found;
  const int* rows = found.rows;
  __shared__ uint4 staged[4 * kTilesN * 64];
  for (int item = blockIdx.y;; item += gridDim.y) {
    const Item it = find_item<INLINE>(a, plan, item, tm, found);
    if (!it.count) return;
    auto inner = [&](int at, int j) __attribute__((always_inline)) {
      const float* vr = v + (int64_t)rows[at] * a.r + j;
      f32x4 sum = (f32x4){0.f, 0.f, 0.f, 0.f};
      // four slices at a time (all loads out before the first add)
#pragma unroll 1
      for (int u0 = 0; u0 < slices; u0 += 4) {
        f32x4 part[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          part[u] = *reinterpret_cast<const f32x4*>(vr + (int64_t)(u0 + u < slices ? u0 + u : u0) * a.m * a.r);
#pragma unroll
        for (int u = 0; u < 4; ++u) __asm__ volatile("" : "+v"(part[u]));  // not one by one, as they are added
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u0 + u < slices) sum += part[u];
      }
      return sum;
    };
    expand_item<XT, YT, INLINE, SUBS, 4>(a, it, found, reinterpret_cast<typename Held<XT>::type*>(dyn), tm, staged,
                                         (int)blockIdx.x, (int)gridDim.x, [] {}, inner);
    __syncthreads();  // the next item's rows and pieces
  }
}

// Both products in one launch, for few rows with small adapters: every
// work-group forms its item's v by itself (reading all of A, which the cache
// then holds) and goes on to its 512 outputs.
template <int XT, int YT, int RT>
__global__ __launch_bounds__(512) void lora_small_kernel(LoraArgs a) {
  constexpr int kWaves = 8, kPitch = RT * 16 + 4;
  __shared__ Found found;
  const int* rows = found.rows;
  __shared__ uint4 stage[kWaves][1 + RT][16][8];
  __shared__ __align__(16) float inner_v[16][kPitch];
  __shared__ uint4 pieces[inner_bytes<XT>(16, RT * 16) / 16];
  const Item it = find_item<true>(a, Plan{}, (int)blockIdx.y, 16, found);
  if (!it.count) return;
  auto first = [&]() __attribute__((always_inline)) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const f32x4 sum = shrink16<XT, RT, kWaves>(a, it.slot, it.rank, 0, rows, it.count, stage, wave, kWaves);
    if (wave < RT)
      *reinterpret_cast<f32x4*>(&inner_v[threadIdx.x & 15][wave * 16 + ((threadIdx.x >> 4) & 3) * 4]) = sum;
    __syncthreads();
  };
  auto inner = [&](int at, int j) __attribute__((always_inline)) {
    return *reinterpret_cast<const f32x4*>(&inner_v[at][j]);
  };
  expand_item<XT, YT, true, 1, kWaves>(a, it, found, reinterpret_cast<typename Held<XT>::type*>(pieces), 16, nullptr,
                                       (int)blockIdx.x, (int)gridDim.x, first, inner);
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// Rows of an item at most: 32 halve the reads of an adapter that many rows
// share; with few rows to an adapter the second 16 would be empty work-groups.
int item_rows(int64_t m, int64_t slots) { return m <= kInlineRows || m <= 16 * slots ? 16 : kItemRows; }

int64_t max_items(int64_t m, int64_t slots, int64_t tm) {
  // every item but an adapter's last is full
  const int64_t most = slots + m / tm;
  return most < m ? most : m;
}

int64_t plan_bytes(int64_t m, int64_t slots, int64_t tm) {
  return m <= kInlineRows ? 0 : 256 + round256(max_items(m, slots, tm) * (16 + tm * 4));
}

// 16-row units of the first product: of all items, as many as there can be
int64_t shrink_units(int64_t m, int64_t slots) {
  const int64_t items = max_items(m, slots, item_rows(m, slots)), rows = (m + 15) / 16;
  return items > rows ? items : rows;
}

// Ranks a work-group of the first product takes, in 16s.  Few rows: 16, for
// many work-groups, each reading x again (from the cache); many rows: x, the
// larger operand, is read once per 48 ranks, which are shared out evenly (with
// 64 one work-group fills a compute unit's LDS: 4096 x 5120 -> 5120, r 40: 66 us a
// call against 57, r 64 75 and 71, r 128 103 and 98; 1302 x 13568 -> 6355, ranks
// 56, 28, 53 and 0: 38 against 41).
int ranks_per_block(int64_t m, int64_t r, int64_t slots) {
  if (r <= 16 || shrink_units(m, slots) * ((r + 15) / 16) <= 256) return 1;
  const int tiles = (int)((r + 15) / 16), groups = (tiles + 2) / 3;
  return (tiles + groups - 1) / groups;
}

// k in slices as long as all work-groups run at once (two to a compute unit); a
// wave keeps at least 64 of k
int64_t slices_of(int64_t m, int64_t k, int64_t r, int64_t slots) {
  const int rt = ranks_per_block(m, r, slots);
  const int64_t groups = shrink_units(m, slots) * ((r + rt * 16 - 1) / (rt * 16));
  int64_t s = 512 / groups;
  const int64_t most = k / (64 * kShrinkWaves);
  s = s < most ? s : most;
  return s < 1 ? 1 : (s > kMaxSlices ? kMaxSlices : s);
}

// One launch instead of two pays while reading all of A costs a work-group
// less than the launch and the way of v through memory, and while the
// work-groups all run at once (one to a compute unit).  Measured as a graph,
// one launch against two: 1 x 2048 -> 6144, r 16 (A: 64 KB) 6.7 : 8.3 us; 16
// rows, r 32 (128 KB) 7.9 : 8.8; 1 x 5120 -> 5120, r 16 (160 KB) 8.7 : 9.2; 1 x
// 2048 -> 2048, r 64 (256 KB) 9.5 : 8.6; 4 x 2048 -> 34816, r 32 (272
// work-groups) 14.0 : 9.0.
bool small_ok(const LoraArgs& a) {
  return a.m <= 16 && a.r <= 64 && a.r * a.k * 2 <= (160 << 10) &&
         max_items(a.m, a.slots, 16) * ((a.n + 511) / 512) <= 256;
}

template <int XT, int YT>
hipError_t launch_small(const LoraArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.n + 511) / 512), (unsigned)max_items(a.m, a.slots, 16));
  if (a.r <= 16) hipLaunchKernelGGL((lora_small_kernel<XT, YT, 1>), grid, dim3(512), 0, st, a);
  else if (a.r <= 32) hipLaunchKernelGGL((lora_small_kernel<XT, YT, 2>), grid, dim3(512), 0, st, a);
  else hipLaunchKernelGGL((lora_small_kernel<XT, YT, 4>), grid, dim3(512), 0, st, a);
  return hipGetLastError();
}

template <int XT, int YT, bool INLINE>
hipError_t launch(const LoraArgs& a, const Plan& plan, float* v, hipStream_t st) {
  const int tm = item_rows(a.m, a.slots), rt = ranks_per_block(a.m, a.r, a.slots);
  const int64_t items = max_items(a.m, a.slots, tm);
  const int64_t rows = a.m < tm ? a.m : tm;
  const int subs = (int)((rows + 15) / 16);
  const int slices = (int)slices_of(a.m, a.k, a.r, a.slots);
  const dim3 gs((unsigned)(items * subs), (unsigned)((a.r + rt * 16 - 1) / (rt * 16)), (unsigned)slices);
  if (rt == 1)
    hipLaunchKernelGGL((lora_shrink_kernel<XT, 1, INLINE>), gs, dim3(512), 0, st, a, plan, tm, subs, v);
  else if (INLINE || rt == 3)  // (up to 64 rows take more than 16 ranks at once above 64 alone: in threes)
    hipLaunchKernelGGL((lora_shrink_kernel<XT, 3, INLINE>), gs, dim3(512), 0, st, a, plan, tm, subs, v);
  else if constexpr (!INLINE)
    hipLaunchKernelGGL((lora_shrink_kernel<XT, 2, false>), gs, dim3(512), 0, st, a, plan, tm, subs, v);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Work-groups: as many as run at once (three to a compute unit) where two
  // shares of the outputs each are enough for that, else four times as many.
  // One that takes several shares finds its rows and makes v ready (a chain of
  // four memory latencies) once for all of them.
  const int64_t tiles = (a.n + kBlockN - 1) / kBlockN, all = tiles * items;
  int64_t each = all <= 1536 ? (all + 767) / 768 : (all + 2999) / 3000;
  each = each < tiles ? each : tiles;
  const dim3 ge((unsigned)((tiles + each - 1) / each), (unsigned)(items < 32768 ? items : 32768));
  const size_t lds = inner_bytes<XT>(tm, (int)a.r);
  if (INLINE || tm == 16) {
    hipLaunchKernelGGL((lora_expand_kernel<XT, YT, INLINE, 1>), ge, dim3(256), lds, st, a, plan, tm, slices, v);
  } else if constexpr (!INLINE) {  // rows not sorted first make no items of 32
    hipLaunchKernelGGL((lora_expand_kernel<XT, YT, false, 2>), ge, dim3(256), lds, st, a, plan, tm, slices, v);
  }
  return hipGetLastError();
}

template <bool INLINE>
hipError_t launch_typed(const LoraArgs& a, const Plan& plan, float* v, hipStream_t st) {
  if (a.x_type == 2) return launch<2, 1, INLINE>(a, plan, v, st);
  return a.y_type == 1 ? launch<3, 1, INLINE>(a, plan, v, st) : launch<3, 3, INLINE>(a, plan, v, st);
}

}  // namespace

size_t lora_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t r, int64_t slots) {
  (void)n;
  return (size_t)(plan_bytes(m, slots, item_rows(m, slots)) + round256(slices_of(m, k, r, slots) * m * r * 4));
}

hipError_t launch_lora_accumulate(const LoraArgs& a, void* ws, hipStream_t st) {
  const int tm = item_rows(a.m, a.slots);
  char* base = static_cast<char*>(ws);
  float* v = reinterpret_cast<float*>(base + plan_bytes(a.m, a.slots, tm));
  Plan plan = {};
  if (small_ok(a)) {
    if (a.x_type == 2) return launch_small<2, 1>(a, st);
    return a.y_type == 1 ? launch_small<3, 1>(a, st) : launch_small<3, 3>(a, st);
  }
  if (a.m <= kInlineRows) return launch_typed<true>(a, plan, v, st);
  plan.items_used = reinterpret_cast<int*>(base);
  plan.items = reinterpret_cast<Item*>(base + 256);
  plan.most = (int)max_items(a.m, a.slots, tm);
  plan.rows = reinterpret_cast<int*>(base + 256 + (int64_t)plan.most * 16);
  hipLaunchKernelGGL(lora_plan_kernel, dim3(1), dim3(1024), 0, st, a, plan, tm,
                     reinterpret_cast<int*>(v));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_typed<false>(a, plan, v, st);
}

}  // namespace lowbit
