// bf16_tile.h — matrix products of bf16 rows, in tiles staged through LDS:
// the experts' products, their gradients and the projection with adapters.
//
// A workgroup of four waves computes 256 columns x BM rows of an output (BM =
// 64 JT), a wave 128 columns x 32 JT rows: 4 x JT accumulators of 32 x 32 by
// v_mfma_f32_32x32x16_bf16. The first operand holds the output's columns, so
// that a lane ends with consecutive elements of an output row: column r =
// lane % 32 of the product is row r of the tile, and with h = lane / 32, rows
// 8a + 4h + b of the product are at accumulator 4a + b.
//
// A stage takes 64 elements of the reduction, in two steps of 32. Its operands
// are copied from memory into LDS without passing registers, 64 KB (JT = 4) in
// two buffers, and read from there into registers a step before their
// products. That empties a buffer's columns a quarter into step 0, and its rows
// at its end: the stage two ahead is copied there under the rest of step 0 and
// under step 1. The stages of a workgroup's tiles form one sequence, so that a
// tile's first copies run under the end of the tile before it.
//
// An operand comes in one of two layouts:
//  * kRows: its rows are contiguous along the reduction (weights in the
//    forward product). LDS holds 128 bytes of each, the 16-byte piece c at
//    place c ^ swizzle; a lane reads its 8 elements at once, and 16 lanes
//    meet every bank once.
//  * kCols: the reduction steps from row to row (weights in the gradient of
//    the rows, both operands in the gradient of the weights). LDS holds the
//    64 rows as they are, the 16-byte piece c of row k at place c ^ 4 (k % 4);
//    ds_read_b64_tr_b16 gives 16 lanes 4 rows of 16 columns, column by column
//    (lane i gets elements i % 4 of the addresses of lanes i / 4 + {0, 4, 8,
//    12}), so that a lane has its 8 elements after two reads; 32 lanes read
//    4 rows of 64 bytes, which the swizzle puts on all banks.
// Which elements of the reduction a product takes does not matter as long as
// both operands agree: product (step e, u) takes piece 4e + 2h + u of the
// stage's eight, in both layouts.
//
// Measured, 16384 x 7168 x 7168: 1.34 PFLOP/s in the product and the rows'
// gradient, 1.14 in the weights' (a library product reaches 1.60, 1.39 and
// 1.21 on the same operands). A stage takes 2420 cycles, 2048 of them
// products: what a wave issues between two products goes past their 32
// cycles here and there, and power holds the clock at 1.4 to 1.9 GHz in calls
// of a millisecond and more. A tile costs 17 to 20 thousand cycles more, half
// of them stores, which the next tile's first stage covers in part; slots
// whose rows are no multiple of 256 and reductions of 2048 and 4096 elements
// therefore run at 0.95 to 1.05. Tiles are whole to a workgroup: 600 of them
// on 256 CUs take three rounds, in which a CU is busy 70 % of the time (8192
// rows of 8 experts, 4096 outputs: 0.85 to 0.95). LDS has no bank conflicts.
// Four waves hold 256 accumulators each and all of the vector registers, so
// there is one to a SIMD. Eight waves of 128 x 64 would read LDS 1.5 times as
// much for each product, within what it can deliver; they were not built. Row
// tiles walked together (kGroupM) 1, 2, 4 or 8: within 2 %. The gates'
// gradient spills 48 vector registers at 256 rows, between tiles and around
// their stores, the adapters' product about 200, in its part after the stages.
//
// What lies outside an operand is read as zeros, by the length in the buffer
// descriptor: rows and reduction rows past the end, pieces past the end of a
// kRows row. Columns past the end of a kCols row hold the next row's, and
// meet only outputs that are not stored.
#pragma once

#include <type_traits>

#include "mb_internal.h"
#include "rowio.h"
#include "slots.h"

namespace mb {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum TileMode {
  kTileProduct,   // y[p] = a[p] w[e]^T
  kTileGated,     // silu(gate) up of a[p] w[e]^T, w's rows being gate, then up
  kTileRowGrad,   // y[p] = a[p] w[e]
  kTileGateGrad,  // the same, times the activation's derivatives at pre[p]
  kTileWeightGrad, // y[e] = sum over e's rows of a[p]^T w[p]
  kTileWeightAdd,  // the same, added to y
  kTileLora,      // y[t] = a[t] w^T + v[t] b[adapter[t]]^T
  kTileSplit      // y[part][t] = a[t] w^T over a part of the reduction
};

struct TileArgs {
  const uint16_t* a;  // the rows
  const uint16_t* w;  // the columns: weights, or (weights' gradient) rows
  void* y;
  uint16_t* pre;
  const int32_t* cu;
  const int32_t* rep;
  const int32_t* status;
  int P, E, Eh, NS, R, cap;
  int n;  // columns of the output
  int k;  // length of the reduction; weights' gradient: rows of the output
  // kTileLora, kTileSplit: one slot of `cap` rows
  const float* v;          // [parts][cap][rank], whose sum over the parts counts
  const uint16_t* b;       // [L][n][rank]
  const int32_t* adapter;  // [cap]
  int rank, L, parts;
  int splits, split_stages;  // kTileSplit: parts, and stages (64 elements) of one
};

// The adapter of a row; none (INT32_MAX) where its number is not one.
__device__ __forceinline__ int adapter_of(const TileArgs& p, int row) {
  const int a = p.adapter[row];
  return (unsigned)a < (unsigned)p.L ? a : INT32_MAX;
}

// Elements [at, at + 8) of a row of v, each as three bf16 that together hold
// all of its 24 bits: v is not rounded. A part is the largest bf16 below what
// is left, not that itself, so that none of a value's parts is zero: times an
// infinity they are its sign's. (Of values below 2^-94 a part may be.) An
// infinity or a NaN is all three parts, apart from the rest, which it would
// slow down (4096 rows of 64 adapters in turn, rank 64: 990 us, 937 as it is,
// 898 with zero parts).
__device__ __forceinline__ void load_v(const TileArgs& p, int row, int at, bool on, i32x4* v3) {
  float s[8] = {};
  if (on && at < p.rank)
    for (int i = 0; i < p.parts; ++i) {
      float v[8];
      load8<false>(p.v + ((size_t)i * p.cap + row) * p.rank + at, 0, v);
#pragma unroll
      for (int x = 0; x < 8; ++x) s[x] += v[x];
    }
  uint32_t part[3][8];
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const uint32_t below = s[x] != 0.0f;
    float left = s[x];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      part[q][x] = (__float_as_uint(left) - (q < 2 ? below : 0)) & 0xffff0000u;
      left -= __uint_as_float(part[q][x]);
    }
  }
  float most = 0.0f;
#pragma unroll
  for (int x = 0; x < 8; ++x) most += fabsf(s[x]);
  if (__builtin_expect(__ballot(!(most < INFINITY)) != 0, 0))
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (!(fabsf(s[x]) < INFINITY))
        part[0][x] = part[1][x] = part[2][x] = __float_as_uint(s[x]) & 0xffff0000u;
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int x = 0; x < 4; ++x) v3[q][x] = (int)(part[q][2 * x] >> 16 | part[q][2 * x + 1]);
}

// o[0..4) += outputs [n, n + 4) of a row's adapter. A lane by itself: rows may
// have different adapters, and an output's ranks are consecutive in memory.
__device__ __forceinline__ void add_adapter(const TileArgs& p, int row, int n, float* o) {
  const int id = adapter_of(p, row);
  if (id == INT32_MAX) return;
  const uint16_t* b = p.b + ((size_t)id * p.n + n) * p.rank;
#pragma unroll 2
  for (int q = 0; q < p.rank; q += 8) {
    float v[8] = {};
    for (int i = 0; i < p.parts; ++i) {
      float w[8];
      load8<false>(p.v + ((size_t)i * p.cap + row) * p.rank + q, 0, w);
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] += w[x];
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float w[8];
      load8<true>(b + y * p.rank + q, 0, w);
#pragma unroll
      for (int x = 0; x < 8; ++x) o[y] = fmaf(v[x], w[x], o[y]);
    }
  }
}

// sigmoid(g) as a product of two factors, and 1 - sigmoid(g). kFar: from t =
// exp(-|g| / 2), since 1 / (1 + exp(-g)) falls below the normal numbers at
// -87.3, where g * sigmoid(g) is still one.
template <bool kFar>
struct Sigmoid {
  float a, b, rest;
  __device__ __forceinline__ explicit Sigmoid(float g) {
    if constexpr (kFar) {
      const float t = __expf(-0.5f * fabsf(g)), q = t * t, r = __builtin_amdgcn_rcpf(1.0f + q);
      a = g < 0 ? t : 1.0f;
      b = g < 0 ? t * r : r;
      rest = g < 0 ? r : q * r;
    } else {
      a = 1.0f;
      b = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
      rest = 1.0f - b;
    }
  }
  __device__ __forceinline__ float times(float v) const { return kFar ? v * a * b : v * b; }
};

// Whether one of the wave's gates is that far (every lane active).
template <int N>
__device__ __forceinline__ bool far_gate(const float* g) {
  float least = g[0];
#pragma unroll
  for (int i = 1; i < N; ++i) least = fminf(least, g[i]);
  return __ballot(least < -80.0f) != 0;
}

// o = silu(g) u; far, one of the factors goes to u, so that what the two make
// together does not vanish where u is large enough to bring it back.
template <int N, bool kFar>
__device__ __forceinline__ void gate_of(const float* g, const float* u, float* o) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Sigmoid<kFar> s(g[i]);
    o[i] = kFar ? (g[i] * s.a) * (s.b * u[i]) : s.times(g[i]) * u[i];
  }
}

template <int N>
__device__ __forceinline__ void gated(const float* g, const float* u, float* o) {
  if (far_gate<N>(g))
    gate_of<N, true>(g, u, o);
  else
    gate_of<N, false>(g, u, o);
}

// From d, the gradient of silu(g) u: those of g (in place) and of u.
template <int N, bool kFar>
__device__ __forceinline__ void gate_grad_of(const float* g, const float* u, float* d, float* du) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Sigmoid<kFar> s(g[i]);
    du[i] = s.times(d[i] * g[i]);
    d[i] = s.times(d[i] * u[i]) * fmaf(g[i], s.rest, 1.0f);
  }
}

template <int N>
__device__ __forceinline__ void gate_grad(const float* g, const float* u, float* d, float* du) {
  if (far_gate<N>(g))
    gate_grad_of<N, true>(g, u, d, du);
  else
    gate_grad_of<N, false>(g, u, d, du);
}

__device__ __forceinline__ f32x16 mfma_bf16(i32x4 a, i32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ i32x4 read_tr(const uint8_t* lo, const uint8_t* hi) {
  typedef __attribute__((address_space(3))) s16x4* tr_ptr;
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 a = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)lo));
  const i32x2 b = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)hi));
  return i32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// What the copies of one operand read in a stage. kRows: `left` bytes from
// `at`. kCols: of `left` reduction rows those that a wave copies, from column
// `col` on. Nothing where left is 0 or less.
template <bool kCols>
struct Operand {
  const uint16_t* at;
  int left, col;

  __device__ __forceinline__ i32x4 buffer(int pitch) const {
    return buffer_of(at, kCols ? max(uniform(min(max(left, 0), 16)) * pitch - col * 2, 0)
                               : max(left, 0));
  }
  __device__ __forceinline__ void next(int pitch) {
    at += kCols ? 32 * (int64_t)pitch : 64;
    left -= kCols ? 64 : 128;
  }
};

template <int JT>
struct alignas(16) BfTileLds {
  uint8_t w[2][kTileN * 128];
  uint8_t a[2][64 * JT * 128];
};

// The rows of every slot and its expert (-1: no rows), and the row tiles of
// the slots before it.
struct SlotTable {
  int first[kMaxPlanSlots + 1];
  int lo[kMaxPlanSlots], hi[kMaxPlanSlots];
  int16_t e[kMaxPlanSlots];
};

// The rows of every slot, and of every expert the slots with rows, for sums
// over an expert's rows.
struct ExpertLists {
  int lo[kMaxPlanSlots];
  int n[kMaxPlanSlots];
  int stages[kMaxExperts];       // of an expert's sum; one, of zeros, without rows
  int16_t next[kMaxPlanSlots];   // the expert's next slot with rows, -1: none
  int16_t first[kMaxExperts];    // its first, -1: none
};

template <int BM, class Args>
__device__ void slot_table(const Args& p, int nslots, SlotTable& t, int* part) {
  tile_table<BM>(p, nslots, t.first, part);
  for (int j = threadIdx.x; j < nslots; j += kExpertThreads) {
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    t.lo[j] = lo;
    t.hi[j] = hi;
    t.e[j] = hi > lo ? e : -1;
  }
  __syncthreads();
}

// The slot whose tiles hold row tile t: the last whose first tile is not
// behind t, found in two reads by the wave.
__device__ __forceinline__ int slot_at(const SlotTable& s, int nslots, int t, int lane) {
  constexpr int kEach = kMaxPlanSlots / 64;
  const int a = lane * kEach;
  const int group = __builtin_popcountll(__ballot(a < nslots && s.first[a] <= t)) - 1;
  const int b = group * kEach + lane;
  return group * kEach - 1 +
         __builtin_popcountll(__ballot(lane < kEach && b < nslots && s.first[b] <= t));
}

// The lists of the plan: an expert's home slot, then its replicas in
// ascending order. One wave links the replica slots, 64 at a time from the
// last to the first: a lane's next is the first behind it that holds the same
// expert, found by one ballot for every bit of its number, else the head of
// the expert's list so far. (1024 of them: 4 us of the call. A search of the
// slots behind each took 900.)
template <class Args>
__device__ void expert_lists(const Args& p, int nslots, ExpertLists& t) {
  static_assert(kMaxExperts == 1 << 10, "the bits of an expert's number");
  for (int j = threadIdx.x; j < nslots; j += kExpertThreads) {
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    t.lo[j] = lo;
    t.n[j] = hi - lo;
    t.next[j] = hi > lo ? e : -1;  // its expert, for now
  }
  for (int e = threadIdx.x; e < p.E; e += kExpertThreads) t.first[e] = -1;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x, replicas = p.P * p.R;
    auto slot = [&](int q) { return q / p.R * p.NS + p.Eh + q % p.R; };
    for (int q = (replicas - 1) & ~63; q >= 0; q -= 64) {
      const bool in = q + lane < replicas;
      const int s = in ? slot(q + lane) : 0, e = in ? t.next[s] : -1;
      uint64_t same = __ballot(e >= 0);
#pragma unroll
      for (int b = 0; b < 10; ++b) {
        const uint64_t set = __ballot(e >> b & 1);
        same &= e >> b & 1 ? set : ~set;
      }
      if (e >= 0) {
        const uint64_t behind = same & (~1ull << lane);
        t.next[s] = behind ? slot(q + __builtin_ctzll(behind)) : t.first[e];
        if (lane == __builtin_ctzll(same)) t.first[e] = s;
      }
      __builtin_amdgcn_wave_barrier();  // the next 64 read the heads after these wrote them
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kExpertThreads) {
    const int rank = e / p.Eh, home = rank * p.NS + e - rank * p.Eh;
    t.next[home] = t.first[e];
    const int first = t.n[home] ? home : t.first[e];
    int s = 0;
    for (int j = first; j >= 0; j = t.next[j]) s += (t.n[j] + 63) / 64;
    t.first[e] = first;
    t.stages[e] = max(s, 1);
  }
  __syncthreads();
}

// ---- few rows: operands straight from memory --------------------------------
//
// The columns' operand is read once for every slot, and sets the pace: 128 rows
// over 80 slots, 58 of them with rows, 7168 -> 2 x 2048 and back, in 0.62 and
// 0.30 ms, 5.5 and 5.7 TB/s of weights (a contiguous read here: 6.7). A
// workgroup computes 16 outputs of 16 rows, whatever a slot holds of them; its
// waves take 32 U elements of the reduction at a time by turns, so that a
// weight row is read in whole lines by waves that follow each other, and add up
// in LDS. v_mfma_f32_16x16x32_bf16: a lane (r = lane % 16, g = lane / 16) holds
// elements 8g.. of row r of 32, and ends with outputs 4g.. of row r.
__device__ __forceinline__ f32x4 mfma_few(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int kMode, bool kBF16, int kWaves, int U>
__global__ __launch_bounds__(64 * kWaves) void k_bf16_few(TileArgs p) {
  constexpr bool kLora = kMode == kTileLora, kGated = kMode == kTileGated;
  constexpr int NG = kGated ? 2 : 1;  // weight rows to an output
  constexpr int kStep = 32 * U;
  static_assert(kLora || 64 * kWaves == kExpertThreads, "the threads that make the tile table");
  __shared__ f32x4 sums[kWaves][NG][64];
  __shared__ int first[kLora ? 1 : kMaxPlanSlots + 1];
  __shared__ int part[kWaves];
  if (!kLora && (p.status[0] & MB_ST_FATAL)) return;
  const int nslots = p.P * p.NS;
  if constexpr (!kLora) tile_table<16>(p, nslots, first, part);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (p.n + 15) / 16;
  const int64_t total = (int64_t)(kLora ? (p.cap + 15) / 16 : first[nslots]) * ntn;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int mt = (int)(t / ntn), n0 = (int)(t - (int64_t)mt * ntn) * 16;
    int lo = 0, hi = p.cap, e = 0, m0 = mt * 16;
    if constexpr (!kLora) {
      const int j = slot_of(first, nslots, mt);
      slot_rows(p, j, lo, hi, e);
      m0 = lo + (mt - first[j]) * 16;
    }
    // rows past the slot's or the weights' end read the last one instead
    const uint16_t* w[NG];
#pragma unroll
    for (int i = 0; i < NG; ++i)
      w[i] = p.w + (((int64_t)e * NG + i) * p.n + min(n0 + r, p.n - 1)) * p.k + g * 8;
    const uint16_t* a = p.a + (int64_t)min(m0 + r, hi - 1) * p.k + g * 8;
    f32x4 acc[NG] = {};
    int k = wave * kStep;
    for (; k + kStep <= p.k; k += kWaves * kStep) {
      i32x4 wv[NG][U], av[U];
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int u = 0; u < U; ++u) wv[i][u] = load16(w[i] + k + u * 32);
#pragma unroll
      for (int u = 0; u < U; ++u) av[u] = load16(a + k + u * 32);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NG; ++i) acc[i] = mfma_few(wv[i][u], av[u], acc[i]);
    }
    for (; k < p.k; k += 32) {  // the wave whose turn the rest of the rows is
      const bool in = k + g * 8 < p.k;
      const i32x4 av = in ? load16(a + k) : i32x4{};
#pragma unroll
      for (int i = 0; i < NG; ++i)
        acc[i] = mfma_few(in ? load16(w[i] + k) : i32x4{}, av, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) sums[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave == 0) {
      f32x4 o[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        o[i] = sums[0][i][lane];
#pragma unroll
        for (int x = 1; x < kWaves; ++x) o[i] += sums[x][i][lane];
      }
      const int m = m0 + r, nn = n0 + 4 * g;
      float h[4] = {o[0][0], o[0][1], o[0][2], o[0][3]};
      if constexpr (kGated) {
        const float x[4] = {h[0], h[1], h[2], h[3]};
        const float u[4] = {o[1][0], o[1][1], o[1][2], o[1][3]};
        gated<4>(x, u, h);
      }
      if constexpr (kLora) {
        if (nn < p.n) add_adapter(p, min(m, hi - 1), nn, h);
      }
      if (m < hi && nn < p.n) {
        if constexpr (kBF16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + (size_t)m * p.n + nn) =
              uint2{bf16x2_rne(h[0], h[1]), bf16x2_rne(h[2], h[3])};
        else
          *reinterpret_cast<f32x4*>(static_cast<float*>(p.y) + (size_t)m * p.n + nn) =
              f32x4{h[0], h[1], h[2], h[3]};
        if constexpr (kGated) {
          if (p.pre)
#pragma unroll
            for (int i = 0; i < NG; ++i)
              *reinterpret_cast<uint2*>(p.pre + ((size_t)m * NG + i) * p.n + nn) =
                  uint2{bf16x2_rne(o[i][0], o[i][1]), bf16x2_rne(o[i][2], o[i][3])};
        }
      }
    }
    __syncthreads();
  }
}

// What a stage of 256 rows costs, in eighths of one of 128 (measured: 1.6 to
// 1.9 times as much, the less the fewer CUs work).
constexpr int kLongTile = 13;

// ---- tiles staged through LDS ------------------------------------------------
struct BfTile {
  int m0, hi, n0, e;
};

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// An output, or what its gradient needs, from a tile's first row on. Lanes
// behind the last row, or with a negative offset, read zeros and write
// nothing, without a branch: every wave issues the same number of stores for
// a tile, which the wait in the next tile's first stage counts on.
struct RowBuffer {
  __amdgpu_buffer_rsrc_t at;
  __device__ __forceinline__ RowBuffer(void* p, int rows, int pitch)
      : at(__builtin_amdgcn_make_buffer_rsrc(scalar(p), 0, uniform(max(rows, 0) * pitch),
                                             0x00020000)) {}
  static __device__ __forceinline__ void* scalar(void* p) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<void*>((uint64_t)(uint32_t)uniform((int)(at >> 32)) << 32 |
                                   (uint32_t)uniform((int)at));
  }
  __device__ __forceinline__ void store(int off, u32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, at, off, 0, 0);
  }
  __device__ __forceinline__ u32x4 load(int off) const {
    return __builtin_amdgcn_raw_buffer_load_b128(at, off, 0, 0);
  }
};

// Exchanges the odd rows of 16 lanes of a with the even ones of b. Where a
// lane (r = lane % 32, h = lane / 32) has two 16-byte pieces of row r of an
// output, this leaves one of rows 0 to 15 and one of rows 16 to 31, such that
// four lanes hold 64 consecutive bytes: whole requests to memory. It undoes
// itself.
__device__ __forceinline__ void swap16(u32x4& a, u32x4& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto v = __builtin_amdgcn_permlane16_swap(a[i], b[i], false, false);
    a[i] = v[0];
    b[i] = v[1];
  }
}

__device__ __forceinline__ u32x4 bf16x8_rne(const float* v) {
  return u32x4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
               bf16x2_rne(v[6], v[7])};
}

__device__ __forceinline__ void bf16_of(u32x4 u, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Waits until this wave's LDS reads are done and at most N of its memory
// operations, or the 63 that can be counted, are outstanding.
template <int N>
__device__ __forceinline__ void wait_stores() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N < 63 ? N : 63) : "memory");
}

template <int kMode, bool kBF16, int JT>
__global__ __launch_bounds__(kExpertThreads, 1) void k_bf16_tile(TileArgs p) {
  constexpr int BM = 64 * JT;
  constexpr bool kSplit = kMode == kTileSplit, kLora = kMode == kTileLora || kSplit;
  constexpr bool kGated = kMode == kTileGated;
  constexpr bool kGateGrad = kMode == kTileGateGrad, kAdd = kMode == kTileWeightAdd;
  constexpr bool kSum = kMode == kTileWeightGrad || kAdd;
  constexpr bool kColW = kMode == kTileRowGrad || kGateGrad || kSum, kColA = kSum;
  constexpr int BN = kGated ? kTileN / 2 : kTileN;  // outputs of a tile's columns
  constexpr int kElt = kBF16 ? 2 : 4;
  // stores of a wave for 32 rows of a tile (without pre)
  constexpr int kStores = kGated ? 4 : kGateGrad ? 16 : 8 * kElt / 2;
  static_assert(BM <= kMaxTileRows, "rows behind a tile's last are numbered in int32");
  __shared__ BfTileLds<JT> lds;
  __shared__ typename std::conditional<kSum, ExpertLists, SlotTable>::type table;
  __shared__ int part[kExpertThreads / 64];
  if (!kLora && (p.status[0] & MB_ST_FATAL)) return;
  const int nslots = p.P * p.NS;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int hn = wave >> 1, hm = wave & 1;
  const int ntn = (p.n + BN - 1) / BN;
  int mtiles = 0, total = 0;  // row tiles (of an expert, where it sums), tiles
  if constexpr (kSum) {
    expert_lists(p, nslots, table);
    mtiles = (p.k + BM - 1) / BM;
    total = mtiles * ntn * p.E;
  } else if constexpr (kLora) {
    mtiles = (p.cap + BM - 1) / BM;
    total = mtiles * ntn * (kSplit ? p.splits : 1);
  } else {
    slot_table<BM>(p, nslots, table, part);
    mtiles = uniform(table.first[nslots]);
    total = mtiles * ntn;
  }
  // workgroups go round the XCDs: those of one XCD take runs of consecutive
  // tiles, which share their rows and columns in its L2
  const int per = gridDim.x / kXcds;
  const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  auto tile_index = [&](int it) { return (it * kXcds + xcd) * per + local; };
  // (quotients are computed in vector registers: read back, or all that
  // follows from them, the copies' buffers too, would be held there)
  auto tile_of = [&](int t) {
    BfTile o;
    int e = 0;
    if constexpr (kSum || kSplit) {
      e = uniform(t / (mtiles * ntn));
      t -= e * mtiles * ntn;
    }
    const int group = uniform(t / (kGroupM * ntn)), rem = t - group * (kGroupM * ntn);
    const int gm = min(kGroupM, mtiles - group * kGroupM);
    const int column = uniform(rem / gm);
    const int mt = group * kGroupM + rem - column * gm;
    o.n0 = column * BN;
    if constexpr (kSum || kLora) {
      o.m0 = mt * BM;
      o.hi = kSum ? p.k : p.cap;
      o.e = e;
    } else {
      const int j = slot_at(table, nslots, mt, lane);
      o.m0 = uniform(table.lo[j]) + (mt - uniform(table.first[j])) * BM;
      o.hi = uniform(table.hi[j]);
      o.e = uniform(table.e[j]);
    }
    return o;
  };
  auto stages_of = [&](int e) {
    if constexpr (kSum)
      return uniform(table.stages[e]);
    else if constexpr (kSplit)
      return min(p.split_stages, (p.k + 63) / 64 - e * p.split_stages);
    else
      return (p.k + 63) / 64;
  };
  if (tile_index(0) >= total) return;
  const int tiles = (total - tile_index(0) + gridDim.x - 1) / gridDim.x;

  // ---- the copies ----
  // Bytes from a row to the next, of the columns' operand and of the rows'.
  const int pw = (kColW ? p.n : p.k) * 2, pa = p.k * 2;
  // What a lane copies: of 8 rows (kRows), piece (lane % 8) ^ swizzle of row
  // lane / 8; the swizzle of product row i is i / 2 % 8, and blocks of 8 rows
  // differ in it by constants. Of 2 or 4 rows (kCols), piece (lane % pieces)
  // ^ 4 (row % 4). cut: its lanes whose piece lies behind a row in its last
  // stage.
  constexpr int kPiecesA = kColA ? 8 * JT : 8;
  const int tail = pa - ((p.k + 63) / 64 - 1) * 128;  // bytes of a row in its last stage
  uint32_t cw[2], ca[2], cut_w[2], cut_a[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (kColW) {
      cw[j] = (lane >> 5) * pw + (((lane & 31) ^ ((2 * j + (lane >> 5)) << 2)) << 4);
      cut_w[j] = 0;
    } else {
      const int crow = lane >> 3;
      const int piece = (lane & 7) ^ (((crow >> 1) & 1) | (crow & 4)) ^ (j << 1);
      cw[j] = crow * pw + (piece << 4);
      cut_w[j] = piece * 16 >= tail ? 0x80000000u : 0u;
    }
    if constexpr (kColA) {
      const int row = lane / kPiecesA;
      const int k4 = JT == 4 ? 2 * j + row : row;
      ca[j] = row * pa + (((lane & (kPiecesA - 1)) ^ (k4 << 2)) << 4);
      cut_a[j] = 0;
    } else {
      const int crow = lane >> 3;
      const int piece = (lane & 7) ^ (crow >> 1) ^ (j << 2);
      ca[j] = crow * pa + (piece << 4);
      cut_a[j] = piece * 16 >= tail ? 0x80000000u : 0u;
    }
  }
  constexpr int kRowsW = kColW ? 2 : 8, kRowsA = kColA ? 64 / kPiecesA : 8;  // of a copy
  // Place of the copies in the sequence of stages: one ahead of the products,
  // two from the first quarter of a stage on.
  // A wave copies a quarter of each operand. Past the last tile the buffers
  // are empty: zeros, unused.
  Operand<kColW> ow;
  Operand<kColA> oa;
  int c_it = 0, c_left = 0, c_buf = 0, c_slot = 0, c_n0 = 0, c_m0 = 0;
  // the tile that the copies are at, and the one before it: when the products
  // come to a tile, the copies are at its second stage or at the next tile
  BfTile at0 = {}, at1 = {};
  // kSum: the rows of slot j, none where it is negative
  auto sum_slot = [&](int j) {
    if constexpr (kSum) {
      c_slot = j;
      const int at = uniform(j < 0 ? 0 : table.lo[j]) + wave * 16;
      const int rows = uniform(j < 0 ? 0 : table.n[j]) - wave * 16;
      ow = {p.w + (int64_t)at * p.n + c_n0, rows, c_n0};
      oa = {p.a + (int64_t)at * p.k + c_m0, rows, c_m0};
    }
  };
  auto aim = [&](int it) {
    const BfTile t = tile_of(tile_index(it));
    at1 = at0;
    at0 = t;
    c_left = stages_of(t.e);
    if constexpr (kSum) {
      c_n0 = t.n0;
      c_m0 = t.m0;
      sum_slot(uniform(table.first[t.e]));
    } else {
      const int m = t.m0 + wave * 16 * JT, nm = uniform(min(max(t.hi - m, 0), 16 * JT));
      oa = {p.a + (int64_t)m * p.k, nm * pa, 0};
      if constexpr (kColW) {  // reduction rows, each wave its 16 of a stage
        ow = {p.w + ((int64_t)t.e * p.k + wave * 16) * p.n + t.n0, p.k - wave * 16, t.n0};
      } else if constexpr (kGated) {
        // waves 0 and 2 copy gate rows, 1 and 3 the up rows of the same outputs
        const int n = t.n0 + (wave >> 1) * 64, nn = uniform(min(max(p.n - n, 0), 64));
        ow = {p.w + (((int64_t)t.e * 2 + (wave & 1)) * p.n + n) * p.k, nn * pw, 0};
      } else {
        const int n = t.n0 + wave * 64, nn = uniform(min(max(p.n - n, 0), 64));
        if constexpr (kSplit) {  // from the part's first element of every row
          const int k0 = t.e * p.split_stages * 64;
          oa = {p.a + (int64_t)m * p.k + k0, nm * pa - k0 * 2, 0};
          ow = {p.w + (int64_t)n * p.k + k0, nn * pw - k0 * 2, 0};
        } else {
          ow = {p.w + ((int64_t)t.e * p.n + n) * p.k, nn * pw, 0};
        }
      }
    }
  };
  auto next_stage = [&] {
    c_buf ^= 1;
    ow.next(pw);
    oa.next(pa);
    if (--c_left == 0) {
      ++c_it;
      if (c_it < tiles) {
        aim(c_it);
        return;
      }
      ow.left = oa.left = 0;
      c_left = 1 << 30;
      at1 = at0;
    } else if constexpr (kSum) {
      if (__builtin_expect(c_it < tiles && ow.left + wave * 16 <= 0, 0))
        sum_slot(uniform(table.next[c_slot]));
    }
  };
  // A pitch that the compiler does not know to be the same every time: it
  // would keep offsets that follow from it in registers of their own, and
  // spill them.
  auto fresh = [](int v) {
    asm volatile("" : "+s"(v));
    return v;
  };
  // A stage's copies. (The buffers are put together in every stage: kept from
  // stage to stage, the compiler may hold them in vector registers.) The
  // copies of one operand are issued in order, each moving its lanes' offsets
  // on: between two products there is room for seven instructions.
  struct Copies {
    i32x4 buf;
    uint32_t at[2];
    int step;
  };
  auto last_stage = [&] {  // of a row
    return c_left == 1 && (!kSplit || at0.e == p.splits - 1) ? 0xffffffffu : 0u;
  };
  auto offsets_w = [&](Copies& c) {
    const int pitch = fresh(pw);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      c.at[j] = (cw[j] + j * kRowsW * pitch) | (kColW ? 0u : cut_w[j] & last_stage());
    c.step = 2 * kRowsW * pitch;
  };
  auto offsets_a = [&](Copies& c) {
    const int pitch = fresh(pa);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      c.at[j] = (ca[j] + j * kRowsA * pitch) | (kColA ? 0u : cut_a[j] & last_stage());
    c.step = 2 * kRowsA * pitch;
  };
  auto copy_w = [&](Copies& c, int y) {
    copy16<0>(c.buf, (lds_ptr)(lds.w[c_buf] + (wave * 8 + y) * 1024), c.at[y & 1], 0);
    c.at[y & 1] += c.step;
  };
  auto copy_a = [&](Copies& c, int y) {
    copy16<0>(c.buf, (lds_ptr)(lds.a[c_buf] + (wave * 2 * JT + y) * 1024), c.at[y & 1], 0);
    c.at[y & 1] += c.step;
  };

  // ---- operands of the matrix unit, [step][accumulator][product] ----
  // A step's are read from LDS under the products of the step before. Column n
  // of a wave's 32 enters the matrix unit as row swap23(n), bits 2 and 3
  // exchanged, which leaves a lane 8 consecutive outputs in 8 consecutive
  // accumulators.
  i32x4 fw[2][4][2], fa[2][JT][2];
  constexpr int kPitchW = kTileN * 2, kPitchA = BM * 2;  // of reduction rows (kCols)
  const int piece = ((2 * h) ^ ((r >> 1) & 7)) << 4;     // kRows: of (step 0, h, 0)
  const int swapped = (r & 19) | ((r & 4) << 1) | ((r & 8) >> 1);
  int at_w[4], at_a[JT];
  {
    // kCols: lane i of 16 addresses row i / 4, 4 columns; group lane / 16 % 2
    // takes columns 16 on
    const int i = lane & 15, g = (lane >> 4) & 1;
    const int chunk = ((i & 1) << 1) | ((i >> 1) & 1);  // swap23 of columns 4 (i % 4)
#pragma unroll
    for (int t = 0; t < 4; ++t)
      at_w[t] = kColW ? (16 * h + (i >> 2)) * kPitchW +
                            (((hn * 16 + t * 4 + g * 2 + (chunk >> 1)) ^ (i >> 2 << 2)) << 4) +
                            (chunk & 1) * 8
                      : (hn * 128 + t * 32 + swapped) * 128;
#pragma unroll
    for (int t = 0; t < JT; ++t)
      at_a[t] = kColA ? (16 * h + (i >> 2)) * kPitchA +
                            ((((2 * t + hm) * 4 + g * 2 + ((i & 3) >> 1)) ^ (i >> 2 << 2)) << 4) +
                            (i & 1) * 8
                      : ((2 * t + hm) * 32 + r) * 128;
  }
  auto read_w = [&](int buf, int step, int t, int u) {
    if constexpr (kColW) {
      const uint8_t* s = lds.w[buf] + at_w[t] + (step * 32 + u * 8) * kPitchW;
      fw[step][t][u] = read_tr(s, s + 4 * kPitchW);
    } else {
      fw[step][t][u] = load16(lds.w[buf] + at_w[t] + (piece ^ (step * 64 + u * 16)));
    }
  };
  auto read_a = [&](int buf, int step, int t, int u) {
    if constexpr (kColA) {
      const uint8_t* s = lds.a[buf] + at_a[t] + (step * 32 + u * 8) * kPitchA;
      fa[step][t][u] = read_tr(s, s + 4 * kPitchA);
    } else {
      fa[step][t][u] = load16(lds.a[buf] + at_a[t] + (piece ^ (step * 64 + u * 16)));
    }
  };
  // What step 1 reads for the next stage, y of kNext: all operands of its step
  // 0, in the order in which the products need them (of each u, column 0, the
  // rows, columns 1 to 3), then the columns of its step 1's first products.
  constexpr int kNext = 2 * (4 + JT) + 4;
  auto read_next = [&](int buf, int y) {
    const int u = y / (4 + JT), i = y % (4 + JT);
    if (u > 1)
      read_w(buf, 1, i, 0);
    else if (i == 0)
      read_w(buf, 0, 0, u);
    else if (i <= JT)
      read_a(buf, 0, i - 1, u);
    else
      read_w(buf, 0, i - JT, u);
  };

  aim(0);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s) next_stage();
    Copies to_w = {settled(ow.buffer(pw))}, to_a = {settled(oa.buffer(pa))};
    offsets_w(to_w);
    offsets_a(to_a);
#pragma unroll
    for (int y = 0; y < 8; ++y) copy_w(to_w, y);
#pragma unroll
    for (int y = 0; y < 2 * JT; ++y) copy_a(to_a, y);
  }
  wait_barrier<0>();
  int buf = 0;
#pragma unroll
  for (int y = 0; y < kNext; ++y) read_next(0, y);

  // A tile of fewer rows (a slot's last) leaves out accumulators of every
  // wave, 64 rows at a time, the waves' row tiles taking turns: JN of JT are
  // left. stored: JN of the tile before, 0 before the first.
  auto run = [&](const BfTile& tile, int stored, auto jn_) {
    constexpr int JN = decltype(jn_)::value;
    f32x16 acc[4][JN];
    // Under the products of a stage: the rest of its own operands (step 0),
    // those that read_next names of the next (step 1), and the copies of the
    // stage two ahead, the columns' from the moment when all waves have read
    // the present ones (step 0), the rows' in step 1. A product takes 32 cycles,
    // a wave issues in order, and there is one wave to a SIMD: what stands
    // between two products beyond those cycles leaves the matrix unit idle, so
    // no more than a few instructions do, and the copies (16 cycles each of
    // the address unit that the four waves share) are spread evenly.
    auto stage = [&](auto first_) {
      constexpr bool kFirst = decltype(first_)::value;
      constexpr int kProducts = 8 * JN;  // of a step
      constexpr int kRead = 3 * JN;  // from here on the stage's columns are copied over
      Copies to_w, to_a;
#pragma unroll
      for (int x = 0; x < kProducts; ++x) {
        const int c = x / JN, j = x % JN, u = c >> 2, i = c & 3;
        // all columns of the stage are in this wave's registers; after the
        // barrier, in every wave's
        if (x == kRead) read_barrier();
        // where the copies of the stage two ahead read
        if (x == JN) next_stage();
        if (x == 2 * JN) to_w.buf = settled(ow.buffer(pw));
        if (x == 2 * JN + 1) offsets_w(to_w);
        if (x == 5 * JN) to_a.buf = settled(oa.buffer(pa));
        if (x == 5 * JN + 1) offsets_a(to_a);
        acc[i][j] = mfma_bf16(fw[0][i][u], fa[0][j][u], kFirst && !u ? f32x16{} : acc[i][j]);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (y * JN / 2 == x) read_w(buf, 1, y, 1);
#pragma unroll
        for (int y = 0; y < 2 * JN; ++y)
          if (3 * JN + y * 15 / 8 == x) read_a(buf, 1, y % JN, y / JN);
#pragma unroll
        for (int y = 0; y < 8; ++y)
          if (kRead + y * (kProducts - kRead) / 8 == x) copy_w(to_w, y);
        __builtin_amdgcn_sched_barrier(0);
      }
      // this wave has read all of the stage, and its copies of the next have
      // landed (the eight just issued are of the one after); after the barrier
      // that holds for all waves. In a tile's first stage the stores of the tile
      // before lie between the two, kStores at least for each 32 rows, and may
      // still be under way.
      if constexpr (kFirst) {
        if (JT > 3 && stored > 3)
          wait_stores<4 * kStores + 8>();
        else if (JT > 2 && stored > 2)
          wait_stores<3 * kStores + 8>();
        else if (stored > 1)
          wait_stores<2 * kStores + 8>();
        else if (stored > 0)
          wait_stores<kStores + 8>();
        else
          wait_stores<8>();
        asm volatile("s_barrier" ::: "memory");
      } else {
        wait_barrier<8>();
      }
#pragma unroll
      for (int x = 0; x < kProducts; ++x) {
        const int c = x / JN, j = x % JN, u = c >> 2, i = c & 3;
        acc[i][j] = mfma_bf16(fw[1][i][u], fa[1][j][u], acc[i][j]);
#pragma unroll
        for (int y = 0; y < kNext; ++y)
          if (y * kProducts / kNext == x) read_next(buf ^ 1, y);
#pragma unroll
        for (int y = 0; y < 2 * JT; ++y)
          if (y * kProducts / (2 * JT) == x) copy_a(to_a, y);
        __builtin_amdgcn_sched_barrier(0);
      }
      buf ^= 1;
    };
    const int stages = stages_of(tile.e);
    stage(std::true_type());
    for (int s = 1; s < stages; ++s) stage(std::false_type());
    // the accumulators are in the matrix unit's registers (nothing runs here:
    // it keeps the allocator from moving them in and out in the loop)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < JN; ++j) asm volatile("" : "+a"(acc[i][j]));
    if constexpr (kLora && !kSplit) {
      // the reduction goes on over the ranks of the rows' adapters, 32 rows at
      // a time. In runs they are all of one; else each adapter's part is made
      // for all and taken by its rows alone, so that what is not finite in
      // one stays out of the others.
#pragma unroll
      for (int j = 0; j < JN; ++j) {
        const int row = min(tile.m0 + (2 * j + hm) * 32 + r, tile.hi - 1), id = adapter_of(p, row);
        auto ranks = [&](int ad, f32x16& c0, f32x16& c1, f32x16& c2, f32x16& c3) {
          for (int q = 0; q < p.rank; q += 16) {
            const int at = q + h * 8;
            i32x4 b[4], v[3];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = tile.n0 + hn * 128 + i * 32 + swapped;
              b[i] = i32x4{};
              if (n < p.n && at < p.rank)
                b[i] = load16(p.b + ((size_t)ad * p.n + n) * p.rank + at);
            }
            load_v(p, row, at, id == ad, v);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
              c0 = mfma_bf16(b[0], v[x], c0);
              c1 = mfma_bf16(b[1], v[x], c1);
              c2 = mfma_bf16(b[2], v[x], c2);
              c3 = mfma_bf16(b[3], v[x], c3);
            }
          }
        };
        int ad = wave_min_i32(id);
        if (__ballot(id == ad) == ~0ull) {
          if (ad != INT32_MAX) ranks(ad, acc[0][j], acc[1][j], acc[2][j], acc[3][j]);
        } else {
          f32x16 sum[4] = {};
          while (ad != INT32_MAX) {
            f32x16 one[4] = {};
            ranks(ad, one[0], one[1], one[2], one[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int x = 0; x < 16; ++x) sum[i][x] = id == ad ? one[i][x] : sum[i][x];
            ad = wave_min_i32(id > ad ? id : INT32_MAX);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][j] += sum[i];
        }
      }
    }
    // ---- the outputs ----
    // A lane's pieces of 64 bytes of 32 rows, a and b, to the rows from
    // 32 (2 j + hm) on (see swap16): `col` is where the 64 bytes begin in the
    // row, `end` where the row's valid ones end.
    const int rows = min(tile.hi - tile.m0, BM);
    int row0 = hm * 32 + (lane & 15);  // + 64 j
    asm volatile("" : "+v"(row0));     // as `fresh`
    // h's pieces are next to each other in bf16 rows, a and b in fp32 rows
    const int byte = (lane >> 5) * (kBF16 ? 16 : 32) + ((lane >> 4) & 1) * (kBF16 ? 32 : 16);
    auto place = [&](int j, int pitch, int col, int end) {
      return col + byte < end ? (row0 + 64 * j) * pitch + col + byte : INT32_MIN;
    };
    auto put = [&](const RowBuffer& to, int at, int pitch, u32x4 a, u32x4 b) {
      swap16(a, b);
      to.store(at, a);
      to.store(at < 0 ? at : at + 16 * pitch, b);
    };
    if constexpr (kGated) {
      // accumulators 0, 1 are gates, 2, 3 the same outputs' ups
      const int pitch = fresh(p.n * 2);
      const RowBuffer y(static_cast<uint16_t*>(p.y) + (size_t)tile.m0 * p.n, rows, pitch);
      const RowBuffer pre(p.pre + (size_t)tile.m0 * 2 * p.n, p.pre ? rows : 0, 2 * pitch);
#pragma unroll
      for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u32x4 g2[2], u2[2], o2[2];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            float g[8], u[8], o[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
              g[x] = acc[i][j][8 * v + x], u[x] = acc[i + 2][j][8 * v + x];
            gated<8>(g, u, o);
            g2[v] = bf16x8_rne(g);
            u2[v] = bf16x8_rne(u);
            o2[v] = bf16x8_rne(o);
          }
          const int col = (tile.n0 + hn * 64 + i * 32) * 2;
          put(y, place(j, pitch, col, pitch), pitch, o2[0], o2[1]);
          if (p.pre) {
            const int at = place(j, 2 * pitch, col, pitch);
            put(pre, at, 2 * pitch, g2[0], g2[1]);
            put(pre, at < 0 ? at : at + pitch, 2 * pitch, u2[0], u2[1]);
          }
          __builtin_amdgcn_sched_barrier(0);  // a few accumulators at a time: no spills
        }
    } else {
      const int wide = kGateGrad ? 2 * p.n : p.n;
      const int pitch = fresh(wide * kElt), half = fresh(p.n * 2), end = kGateGrad ? half : pitch;
      const size_t m = (kSum ? (size_t)tile.e * p.k : kSplit ? (size_t)tile.e * p.cap : 0) + tile.m0;
      uint8_t* const to = static_cast<uint8_t*>(p.y) + m * pitch;
      const RowBuffer y(to, rows, pitch);
      const RowBuffer in(kGateGrad ? static_cast<void*>(p.pre + m * wide) : to,
                         kGateGrad || kAdd ? rows : 0, pitch);
      // 64 bytes at a time: 32 bf16 of an accumulator, or half as many fp32
      constexpr int kPieces = 4 * kElt / 2;
      auto where = [&](int j, int c) {
        return place(j, pitch, (tile.n0 + hn * 128) * kElt + c * 64, end);
      };
      // what a piece needs is read kPieces pieces before it
      u32x4 ahead[kPieces][kGateGrad ? 4 : 2];
      auto fetch = [&](int j, int c) {
        if constexpr (kGateGrad || kAdd) {
          const int at = where(j, c);
#pragma unroll
          for (int q = 0; q < (kGateGrad ? 4 : 2); ++q)
            ahead[c][q] = in.load(at < 0 ? at : at + (q & 1) * 16 * pitch + (q >> 1) * half);
        }
      };
#pragma unroll
      for (int c = 0; c < kPieces; ++c) fetch(0, c);
#pragma unroll
      for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const int at = where(j, c);
          if constexpr (kGateGrad) {
            swap16(ahead[c][0], ahead[c][1]);
            swap16(ahead[c][2], ahead[c][3]);
            u32x4 dg[2], du[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              float g[8], u[8], d[8], e[8];
              bf16_of(ahead[c][v], g);
              bf16_of(ahead[c][2 + v], u);
#pragma unroll
              for (int x = 0; x < 8; ++x) d[x] = acc[c][j][8 * v + x];
              gate_grad<8>(g, u, d, e);
              dg[v] = bf16x8_rne(d);
              du[v] = bf16x8_rne(e);
            }
            if (j + 1 < JN) fetch(j + 1, c);
            put(y, at, pitch, dg[0], dg[1]);
            put(y, at < 0 ? at : at + half, pitch, du[0], du[1]);
          } else {
            if constexpr (kAdd) swap16(ahead[c][0], ahead[c][1]);
            u32x4 o2[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              if constexpr (kBF16) {
                float o[8], b[8] = {};
                if constexpr (kAdd) bf16_of(ahead[c][v], b);
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] = kAdd ? acc[c][j][8 * v + x] + b[x] : acc[c][j][8 * v + x];
                o2[v] = bf16x8_rne(o);
              } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  float o = acc[c >> 1][j][(c & 1) * 8 + 4 * v + x];
                  if constexpr (kAdd) o += __uint_as_float(ahead[c][v][x]);
                  o2[v][x] = __float_as_uint(o);
                }
              }
            }
            if constexpr (kAdd)
              if (j + 1 < JN) fetch(j + 1, c);
            put(y, at, pitch, o2[0], o2[1]);
          }
          if (kGateGrad || kAdd || c == kPieces - 1) __builtin_amdgcn_sched_barrier(0);
        }
    }
  };
  int stored = 0;
  for (int it = 0; it < tiles; ++it) {
    const BfTile tile = c_it == it ? at0 : at1;
    // (outputs of sums over an expert's rows, and of one long batch, have one
    // such tile in a column)
    const int jn = kSum || kLora ? JT : min((tile.hi - tile.m0 + 63) / 64, JT);
    if (jn == JT)
      run(tile, stored, std::integral_constant<int, JT>());
    else if constexpr (!kSum && !kLora) {
      if (JT > 3 && jn == 3)
        run(tile, stored, std::integral_constant<int, (JT > 3 ? 3 : 1)>());
      else if (JT > 2 && jn == 2)
        run(tile, stored, std::integral_constant<int, (JT > 2 ? 2 : 1)>());
      else
        run(tile, stored, std::integral_constant<int, 1>());
    }
    stored = jn;
  }
  // no copy may reach LDS after the workgroup has given it back
  wait_barrier<0>();
}

}  // namespace mb
