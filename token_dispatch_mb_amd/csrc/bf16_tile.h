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
// A stage takes 64 elements of the reduction. Its operands are copied from
// memory into LDS without passing registers, 64 KB (JT = 4) in two buffers:
// the stage two ahead is copied over the present one, the columns once all of
// these are in registers, the rows half a step later. The stages of a
// workgroup's tiles form one sequence, so that a tile's first copies run
// under the end of the tile before it.
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
  kTileWeightGrad // y[e] = sum over e's rows of a[p]^T w[p]
};

struct TileArgs {
  const uint16_t* a;  // the rows
  const uint16_t* w;  // the columns: weights, or (kTileWeightGrad) rows
  void* y;
  uint16_t* pre;
  const int32_t* cu;
  const int32_t* rep;
  const int32_t* status;
  int P, E, Eh, NS, R, cap;
  int n;  // columns of the output
  int k;  // length of the reduction; kTileWeightGrad: rows of the output
  int add;  // kTileWeightGrad: add to y
};

// silu(g) and its derivative. exp(-g) passes binary32 where g is below -88,
// and both go to their limit 0 there.
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

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

// Eight consecutive elements of an output row.
template <bool kBF16>
__device__ __forceinline__ void store8_at(void* y, size_t at, const float* v) {
  if constexpr (kBF16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at) =
        uint4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
              bf16x2_rne(v[6], v[7])};
  } else {
    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(y) + at);
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// What the copies of one operand read in a stage. kRows: `left` bytes from
// `at`. kCols: of `left` reduction rows those that a wave copies, from column
// `col` on. Nothing where left is 0 or less.
template <bool kCols>
struct Operand {
  const uint16_t* at;
  int left, col;

  __device__ __forceinline__ i32x4 buffer(int pitch) const {
    return buffer_of(at, kCols ? max(min(max(left, 0), 16) * pitch - col * 2, 0) : max(left, 0));
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

// The rows of every slot and the slots of every expert, for sums over an
// expert's rows.
struct ExpertLists {
  int lo[kMaxPlanSlots];
  int n[kMaxPlanSlots];
  int next[kMaxPlanSlots];  // the next slot of the same expert, -1: none
};

struct BfTile {
  int m0, hi, n0, e;
};

template <int kMode, bool kBF16, int JT>
__global__ __launch_bounds__(kExpertThreads, 1) void k_bf16_tile(TileArgs p) {
  constexpr int BM = 64 * JT, JH = JT / 2;
  constexpr bool kColW = kMode >= kTileRowGrad, kColA = kMode == kTileWeightGrad;
  constexpr bool kSum = kMode == kTileWeightGrad;
  constexpr int BN = kMode == kTileGated ? kTileN / 2 : kTileN;  // outputs of a tile's columns
  static_assert(BM <= kMaxTileRows, "rows behind a tile's last are numbered in int32");
  __shared__ BfTileLds<JT> lds;
  __shared__ typename std::conditional<kSum, ExpertLists, int[kMaxPlanSlots + 1]>::type table;
  __shared__ int part[kExpertThreads / 64];
  if (p.status[0] & MB_ST_FATAL) return;
  const int nslots = p.P * p.NS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int hn = wave >> 1, hm = wave & 1;
  const int ntn = (p.n + BN - 1) / BN;
  int mtiles = 0, total = 0;  // row tiles (of an expert, where it sums), tiles
  if constexpr (kSum) {
    for (int j = threadIdx.x; j < nslots; j += kExpertThreads) {
      int lo, hi, e;
      slot_rows(p, j, lo, hi, e);
      table.lo[j] = lo;
      table.n[j] = hi - lo;
      table.next[j] = hi > lo ? e : -1;  // its expert, for now
    }
    __syncthreads();
    // an expert's home slot, then its replicas in ascending order
    constexpr int kEach = kMaxPlanSlots / kExpertThreads;
    int nx[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = threadIdx.x + i * kExpertThreads;
      nx[i] = -1;
      if (j >= nslots) continue;
      const int rank = j / p.NS, at = j - rank * p.NS;
      const bool home = at < p.Eh;
      const int e = home ? rank * p.Eh + at : table.next[j];
      if (e < 0) continue;
      for (int q = home ? 0 : rank * p.R + at - p.Eh + 1; q < p.P * p.R; ++q) {
        const int s = q / p.R * p.NS + p.Eh + q % p.R;
        if (table.next[s] == e) {
          nx[i] = s;
          break;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (threadIdx.x + i * kExpertThreads < nslots) table.next[threadIdx.x + i * kExpertThreads] = nx[i];
    __syncthreads();
    mtiles = (p.k + BM - 1) / BM;
    total = mtiles * ntn * p.E;
  } else {
    tile_table<BM>(p, nslots, table, part);
    mtiles = __builtin_amdgcn_readfirstlane(table[nslots]);
    total = mtiles * ntn;
  }
  // workgroups go round the XCDs: those of one XCD take runs of consecutive
  // tiles, which share their rows and columns in its L2
  const int per = gridDim.x / kXcds;
  const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  auto tile_index = [&](int it) { return (it * kXcds + xcd) * per + local; };
  auto tile_of = [&](int t) {
    BfTile o;
    int e = 0;
    if constexpr (kSum) {
      e = t / (mtiles * ntn);
      t -= e * mtiles * ntn;
    }
    const int group = t / (kGroupM * ntn), rem = t - group * (kGroupM * ntn);
    const int gm = min(kGroupM, mtiles - group * kGroupM);
    const int mt = group * kGroupM + rem % gm;
    o.n0 = rem / gm * BN;
    if constexpr (kSum) {
      o.m0 = mt * BM;
      o.hi = p.k;
      o.e = e;
    } else {
      const int j = slot_of(table, nslots, mt);
      int lo;
      slot_rows(p, j, lo, o.hi, o.e);
      o.m0 = lo + (mt - __builtin_amdgcn_readfirstlane(table[j])) * BM;
    }
    return o;
  };
  // kSum: the first slot of the list from j that holds rows
  auto with_rows = [&](int j) {
    if constexpr (kSum)
      while (j >= 0 && !__builtin_amdgcn_readfirstlane(table.n[j]))
        j = __builtin_amdgcn_readfirstlane(table.next[j]);
    return j;
  };
  auto home_of = [&](int e) {
    const int rank = e / p.Eh;
    return rank * p.NS + e - rank * p.Eh;
  };
  // stages of a tile; a sum over no rows takes one, of zeros
  auto stages_of = [&](int e) {
    if constexpr (kSum) {
      int s = 0;
      for (int j = with_rows(home_of(e)); j >= 0;
           j = with_rows(__builtin_amdgcn_readfirstlane(table.next[j])))
        s += (__builtin_amdgcn_readfirstlane(table.n[j]) + 63) / 64;
      return max(s, 1);
    } else {
      return (p.k + 63) / 64;
    }
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
  // Place of the copies in the sequence of stages: two ahead of the product.
  // A wave copies a quarter of each operand. Past the last tile the buffers
  // are empty: zeros, unused.
  Operand<kColW> ow;
  Operand<kColA> oa;
  int c_it = 0, c_left = 0, c_buf = 0, c_slot = 0, c_n0 = 0, c_m0 = 0;
  // kSum: `rows` rows from `at` on
  auto sum_at = [&](int64_t at, int rows) {
    ow = {p.w + (at + wave * 16) * p.n + c_n0, rows - wave * 16, c_n0};
    oa = {p.a + (at + wave * 16) * p.k + c_m0, rows - wave * 16, c_m0};
  };
  auto aim = [&](int it) {
    const BfTile t = tile_of(tile_index(it));
    c_left = stages_of(t.e);
    if constexpr (kSum) {
      c_n0 = t.n0;
      c_m0 = t.m0;
      c_slot = with_rows(home_of(t.e));
      if (c_slot >= 0)
        sum_at(__builtin_amdgcn_readfirstlane(table.lo[c_slot]),
               __builtin_amdgcn_readfirstlane(table.n[c_slot]));
      else
        sum_at(0, 0);
    } else {
      const int m = t.m0 + wave * 16 * JT, nm = min(max(t.hi - m, 0), 16 * JT);
      oa = {p.a + (int64_t)m * p.k, nm * pa, 0};
      if constexpr (kColW) {  // reduction rows, each wave its 16 of a stage
        ow = {p.w + ((int64_t)t.e * p.k + wave * 16) * p.n + t.n0, p.k - wave * 16, t.n0};
      } else if constexpr (kMode == kTileGated) {
        // waves 0 and 2 copy gate rows, 1 and 3 the up rows of the same outputs
        const int n = t.n0 + (wave >> 1) * 64, nn = min(max(p.n - n, 0), 64);
        ow = {p.w + (((int64_t)t.e * 2 + (wave & 1)) * p.n + n) * p.k, nn * pw, 0};
      } else {
        const int n = t.n0 + wave * 64, nn = min(max(p.n - n, 0), 64);
        ow = {p.w + ((int64_t)t.e * p.n + n) * p.k, nn * pw, 0};
      }
    }
  };
  auto next_stage = [&] {
    c_buf ^= 1;
    if (--c_left == 0) {
      if (++c_it < tiles) {
        aim(c_it);
        return;
      }
      ow.left = oa.left = 0;
      c_left = 1 << 30;
    } else {
      ow.next(pw);
      oa.next(pa);
      if constexpr (kSum) {
        if (ow.left + wave * 16 <= 0) {  // the next of the expert's slots
          c_slot = with_rows(__builtin_amdgcn_readfirstlane(table.next[c_slot]));
          sum_at(__builtin_amdgcn_readfirstlane(table.lo[c_slot]),
                 __builtin_amdgcn_readfirstlane(table.n[c_slot]));
        }
      }
    }
  };
  // A stage's copies from buffer b. (The buffer is put together just before
  // they are issued: kept from stage to stage, the compiler may hold it in
  // vector registers.) last: all ones in a tile's last stage (kRows).
  auto last_stage = [&] { return c_left == 1 ? 0xffffffffu : 0u; };
  auto copy_w = [&](i32x4 b, uint32_t last, int c) {
    copy16(b, (lds_ptr)(lds.w[c_buf] + (wave * 8 + c) * 1024),
           (cw[c & 1] + c * kRowsW * pw) | (kColW ? 0u : cut_w[c & 1] & last), 0);
  };
  auto copy_a = [&](i32x4 b, uint32_t last, int c) {
    copy16(b, (lds_ptr)(lds.a[c_buf] + (wave * 2 * JT + c) * 1024),
           (ca[c & 1] + c * kRowsA * pa) | (kColA ? 0u : cut_a[c & 1] & last), 0);
  };

  // ---- operands of the matrix unit, [accumulator][product of the step] ----
  // Each register is read from LDS for the next step as soon as its last
  // product of this one is issued: the rows in two halves, the columns along
  // the second half. Column n of a wave's 32 enters the matrix unit as row
  // swap23(n), bits 2 and 3 exchanged, which leaves a lane 8 consecutive
  // outputs in 8 consecutive accumulators.
  i32x4 fw[4][2], fa[JT][2];
  constexpr int kPitchW = kTileN * 2, kPitchA = BM * 2;  // of reduction rows (kCols)
  const int piece = ((2 * h) ^ ((r >> 1) & 7)) << 4;     // kRows: of (step 0, h, 0)
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
                      : (hn * 128 + t * 32 + ((r & 19) | ((r & 4) << 1) | ((r & 8) >> 1))) * 128;
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
      fw[t][u] = read_tr(s, s + 4 * kPitchW);
    } else {
      fw[t][u] = load16(lds.w[buf] + at_w[t] + (piece ^ (step * 64 + u * 16)));
    }
  };
  auto read_a = [&](int buf, int step, int t, int u) {
    if constexpr (kColA) {
      const uint8_t* s = lds.a[buf] + at_a[t] + (step * 32 + u * 8) * kPitchA;
      fa[t][u] = read_tr(s, s + 4 * kPitchA);
    } else {
      fa[t][u] = load16(lds.a[buf] + at_a[t] + (piece ^ (step * 64 + u * 16)));
    }
  };

  aim(0);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const i32x4 bw = ow.buffer(pw), ba = oa.buffer(pa);
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_w(bw, last_stage(), c);
#pragma unroll
    for (int c = 0; c < 2 * JT; ++c) copy_a(ba, last_stage(), c);
    next_stage();
  }
  wait_barrier<0>();
  int buf = 0;
#pragma unroll
  for (int t = 0; t < 4; ++t) read_w(0, 0, t, 0), read_w(0, 0, t, 1);
#pragma unroll
  for (int t = 0; t < JH; ++t) read_a(0, 0, t, 0), read_a(0, 0, t, 1);

  // A tile of no more than half its rows (a slot's last) leaves the second
  // half of every wave's accumulators out, the waves' row tiles taking turns.
  auto run = [&](const BfTile& tile, auto half_) {
    constexpr bool kHalf = decltype(half_)::value;
    constexpr int JN = kHalf ? JH : JT;
    f32x16 acc[4][JN] = {};
    const int stages = stages_of(tile.e);
    for (int s = 0; s < stages; ++s) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const i32x4 bw = ow.buffer(pw), ba = oa.buffer(pa);
        const uint32_t last = last_stage();
        // first half: the rows of the second are read under it
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int u = c >> 2, i = c & 3;
#pragma unroll
          for (int j = 0; j < JH; ++j) acc[i][j] = mfma_bf16(fw[i][u], fa[j][u], acc[i][j]);
          if (!kHalf && c < JT) read_a(buf, e, JH + (c >> 1), c & 1);
          if (e) copy_w(bw, last, c);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (e) {
          // this wave has read all of the stage, and its copies of the next
          // have landed (the eight just issued are of the one after); after
          // the barrier that holds for all waves
          wait_barrier<8>();
          buf ^= 1;
        }
        // second half: the next step's operands are read under it, and the
        // stage two ahead copied into the buffer just read
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int u = c >> 2, i = c & 3;
#pragma unroll
          for (int j = JH; j < JN; ++j) acc[i][j] = mfma_bf16(fw[i][u], fa[j][u], acc[i][j]);
          read_w(buf, 1 - e, i, u);
          if (c < JT) read_a(buf, 1 - e, c >> 1, c & 1);
          if (e) {
#pragma unroll
            for (int d = c * JT / 4; d < (c + 1) * JT / 4; ++d) copy_a(ba, last, d);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (!e) read_barrier();  // all columns of the stage are in registers
      }
      next_stage();
    }
    // ---- the outputs ----
#pragma unroll
    for (int j = 0; j < JN; ++j) {
      const int m = tile.m0 + (2 * j + hm) * 32 + r;
      const bool row = m < tile.hi;
      if constexpr (kMode == kTileGated) {
        // accumulators 0, 1 are gates, 2, 3 the same outputs' ups
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int v = 0; v < 16; v += 8) {
            const int nn = tile.n0 + hn * 64 + i * 32 + v * 2 + h * 8;
            float g[8], u[8], o[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              g[x] = acc[i][j][v + x];
              u[x] = acc[i + 2][j][v + x];
              o[x] = g[x] * sigmoid(g[x]) * u[x];
            }
            if (row && nn < p.n) {
              store8_at<true>(p.y, (size_t)m * p.n + nn, o);
              if (p.pre) {
                store8_at<true>(p.pre, (size_t)m * 2 * p.n + nn, g);
                store8_at<true>(p.pre, (size_t)m * 2 * p.n + p.n + nn, u);
              }
            }
            __builtin_amdgcn_sched_barrier(0);  // a few accumulators at a time: no spills
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int v = 0; v < 16; v += 8) {
            const int nn = tile.n0 + hn * 128 + i * 32 + v * 2 + h * 8;
            if (kMode == kTileGateGrad || kSum) __builtin_amdgcn_sched_barrier(0);
            if (!row || nn >= p.n) continue;
            float o[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) o[x] = acc[i][j][v + x];
            if constexpr (kMode == kTileGateGrad) {
              float g[8], u[8], du[8];
              load8<true>(p.pre + (size_t)m * 2 * p.n + nn, 0, g);
              load8<true>(p.pre + (size_t)m * 2 * p.n + p.n + nn, 0, u);
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float s = sigmoid(g[x]);
                du[x] = o[x] * g[x] * s;
                o[x] = o[x] * u[x] * s * (1.0f + g[x] * (1.0f - s));
              }
              store8_at<true>(p.y, (size_t)m * 2 * p.n + nn, o);
              store8_at<true>(p.y, (size_t)m * 2 * p.n + p.n + nn, du);
            } else if constexpr (kSum) {
              const size_t at = ((size_t)tile.e * p.k + m) * p.n + nn;
              if (p.add) {
                float b[8];
                load8<kBF16>(static_cast<char*>(p.y) + at * (kBF16 ? 2 : 4), 0, b);
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] += b[x];
              }
              store8_at<kBF16>(p.y, at, o);
            } else {
              store8_at<kBF16>(p.y, (size_t)m * p.n + nn, o);
            }
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // one row of accumulators at a time: no spills
    }
  };
  for (int it = 0; it < tiles; ++it) {
    const BfTile tile = tile_of(tile_index(it));
    if (kSum || tile.hi - tile.m0 > BM / 2)
      run(tile, std::false_type());
    else
      run(tile, std::true_type());
  }
  // no copy may reach LDS after the workgroup has given it back
  wait_barrier<0>();
}

}  // namespace mb
