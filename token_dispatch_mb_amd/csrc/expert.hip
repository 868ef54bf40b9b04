// expert.hip — the experts' products over the dispatch layout, from
// microscaled 4-bit rows and weights (mb_expert_mx4).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands as e2m1 with an e8m0
// scale per 32 elements of k: a lane (r = lane % 16, g = lane / 16) holds the
// 32 elements g of row r of its operand's 128 (16 bytes, the packed order of
// the rows in memory) and their scale byte. The weights are the first
// operand, so that a lane ends with four consecutive outputs of one row:
// column r of the product is row r of the tile, rows 4g..4g+3 its outputs.
#include <type_traits>

#include "mb_internal.h"
#include "rowio.h"
#include "slots.h"

namespace mb {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct ExpertArgs {
  const uint8_t* a;
  const uint8_t* a_scale;
  const uint8_t* w;
  const uint8_t* w_scale;
  void* y;
  const int32_t* cu;
  const int32_t* rep;
  const int32_t* status;
  int P, E, Eh, NS, R, cap, n, k;
};

__device__ __forceinline__ f32x4 mfma_mx4(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const i32x8 b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, sa, 0, sb);
}

// u: which byte of the lanes' scales (the builtin takes it as a constant).
__device__ __forceinline__ f32x16 mfma_mx4(i32x4 a, i32x4 b, f32x16 c, int sa, int sb, int u) {
  const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  const i32x8 b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return u ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, 1, sa, 1, sb)
           : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, 0, sa, 0, sb);
}

// The scales of four steps; rows of scales are whole words.
__device__ __forceinline__ i32x4 scales16(const uint8_t* p) {
  i32x4 v;
  __builtin_memcpy(&v, __builtin_assume_aligned(p, 4), 16);
  return v;
}

template <bool kBF16>
__device__ __forceinline__ void store4(void* y, size_t at, f32x4 v) {
  if constexpr (kBF16) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) =
        uint2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(y) + at) = v;
  }
}

// Outputs [at, at + 8) of a row, as many as are left (a multiple of 4).
template <bool kBF16>
__device__ __forceinline__ void store8_of(void* y, size_t at, int left, f32x4 v, f32x4 u) {
  if constexpr (kBF16) {
    if (left >= 8)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at) =
          uint4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(u[0], u[1]),
                bf16x2_rne(u[2], u[3])};
  } else {
    if (left >= 4) store4<false>(y, at, v);
    if (left >= 8) store4<false>(y, at + 4, u);
  }
}

// ---- tiles staged through LDS -----------------------------------------------
//
// A workgroup of four waves computes 256 outputs x BM rows (BM = 64 JT), a
// wave 128 outputs x 32 JT rows: 4 x JT accumulators of 32 x 32 by
// v_mfma_scale_f32_32x32x64_f8f6f4 (lane r = lane % 32 of an operand's rows,
// h = lane / 32 of its two blocks of 32 elements; outputs 8a + 4h + b of row
// r at accumulator 4a + b).
//
// A step takes 128 elements of k. Rows are copied from memory into LDS,
// without passing registers, in pairs of steps: 128 bytes of every row, one
// cache line. (With single steps, 64 bytes of a row and 4 of its scales at a
// time, the L2's requests set the pace.) The scales are copied in groups of
// four steps, 16 bytes of every row. Two pairs and two groups are in LDS; the
// pair two ahead is copied over the present one, its weights once all of
// these are in registers, its rows half a step later, its scales under the
// next pair's first half step. (All copies in one half step held up the
// products: the address unit takes 16 cycles for each of 64, and 64 for each
// of the scales' eight, which fetch from 64 lines.) The pairs of a workgroup's tiles form one sequence, so that a
// tile's first copies run under the end of the tile before it.
//
// LDS layout of a pair: rows of 128 bytes, the 16-byte piece c of a row at
// place c ^ swizzle; the copy writes 64 consecutive pieces (8 rows), so the
// swizzle is in the piece each lane fetches. A read of one piece of 32 rows
// then meets every bank once in 16 lanes. Block (step, h, u) of a pair, u the
// product of the step, is piece 4 step + 2 h + u: a lane's two scales of a
// step are then neighbours. Weight row n enters the matrix unit as row
// swap23(n % 32), bits 2 and 3 exchanged, which leaves a lane 8 consecutive
// outputs in 8 consecutive accumulators: 16-byte bf16 stores.
//
// Measured on MI355X: 1048576 rows, 7168 x 2048, 288 slots: 7.7-8.0 ms, 3.9
// PFLOP/s. What it spends, from variants with a part left out: the products
// and the stores 5.4 ms (the stores 0.8), the copies 2, reads of LDS 0.5.
// With random operands the card's power sets the clock (1.7 GHz; the products
// alone, in a loop, reach 6.3 PFLOP/s, and 10 on zeros), so the parts add up
// though they overlap. Accumulators of 16 x 16 x 128 took 8.4 ms here.
constexpr int kFewGroups = 2048;

struct Tile {
  int m0, hi, n0, e;
};

template <int JT>
struct alignas(16) TileLds {
  uint8_t w[2][kTileN * 128];
  uint8_t a[2][64 * JT * 128];
  uint8_t ws[2][kTileN * 16];
  uint8_t as[2][kTileN * 16];  // 64 JT rows, and what the other waves copy
  uint8_t none[kTileN * 16];   // zeros: where copies of nothing go, the scales behind a row
  int first[kMaxPlanSlots + 1];
  int part[kExpertThreads / 64];
};

template <bool kBF16, int JT>
__global__ __launch_bounds__(kExpertThreads, 1) void k_expert_tile(ExpertArgs p) {
  constexpr int BM = 64 * JT, JH = JT / 2;
  static_assert(BM <= kMaxTileRows, "rows behind a tile's last are numbered in int32");
  __shared__ TileLds<JT> lds;
  if (p.status[0] & MB_ST_FATAL) return;
  const int nslots = p.P * p.NS;
  reinterpret_cast<uint4*>(lds.none)[threadIdx.x] = uint4{};
  tile_table<BM>(p, nslots, lds.first, lds.part);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int hn = wave >> 1, hm = wave & 1;
  const int ntn = (p.n + kTileN - 1) / kTileN;
  const int mtiles = __builtin_amdgcn_readfirstlane(lds.first[nslots]);
  const int total = mtiles * ntn;
  const int kb = p.k / 2, ks = p.k / 32, steps = p.k / 128;
  const int pairs = (steps + 1) / 2;
  // workgroups go round the XCDs: those of one XCD take runs of consecutive
  // tiles, which share their rows and weights in its L2
  const int per = gridDim.x / kXcds;
  const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  auto tile_index = [&](int it) { return (it * kXcds + xcd) * per + local; };
  auto tile_of = [&](int t) {
    Tile o;
    const int group = t / (kGroupM * ntn), rem = t - group * (kGroupM * ntn);
    const int gm = min(kGroupM, mtiles - group * kGroupM);
    const int mt = group * kGroupM + rem % gm;
    const int j = slot_of(lds.first, nslots, mt);
    int lo;
    slot_rows(p, j, lo, o.hi, o.e);
    o.m0 = lo + (mt - __builtin_amdgcn_readfirstlane(lds.first[j])) * BM;
    o.n0 = rem / gm * kTileN;
    return o;
  };
  if (tile_index(0) >= total) return;
  const int tiles = (total - tile_index(0) + gridDim.x - 1) / gridDim.x;

  // What a lane copies: of 8 rows, piece (lane % 8) ^ swizzle of row crow.
  // The swizzle of matrix-unit row i is i / 2 % 8; blocks of 8 rows differ in
  // it by constants. cut: its lanes whose piece lies in the second step.
  const int crow = lane >> 3;
  uint32_t ca[2], cw[2], cut_a[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    ca[j] = crow * kb + (((lane & 7) ^ (crow >> 1) ^ (j << 2)) << 4);
    cw[j] = crow * kb + (((lane & 7) ^ (((crow >> 1) & 1) | (crow & 4)) ^ (j << 1)) << 4);
    cut_a[j] = ((lane ^ (j << 2)) & 4) ? 0x80000000u : 0u;
  }
  const uint32_t cut_w = ((lane ^ crow) & 4) ? 0x80000000u : 0u;
  // scales: a lane a row; none (zeros) past the tile's rows when JT = 2
  const uint32_t csw = (wave * 64 + lane) * ks;
  const uint32_t csa = wave * 64 < BM ? csw : 0x80000000u;

  // the copies' place in the sequence of pairs: two ahead of the product.
  // Past the last tile its last pair is copied again, unused.
  i32x4 rw, ra, rws, ras;
  Tile next;
  int c_buf = 0, c_group = 1;
  auto aim = [&](int it) {
    next = tile_of(tile_index(it));
    const size_t wrow = (size_t)next.e * p.n + next.n0;
    const int nw = min(kTileN, p.n - next.n0), na = min(BM, next.hi - next.m0);
    rw = buffer_of(p.w + wrow * kb, (uint32_t)nw * kb);
    rws = buffer_of(p.w_scale + wrow * ks, (uint32_t)nw * ks);
    ra = buffer_of(p.a + (size_t)next.m0 * kb, (uint32_t)na * kb);
    ras = buffer_of(p.a_scale + (size_t)next.m0 * ks, (uint32_t)na * ks);
  };
  // Copy c of a pair's rows: 8 of weights, then 2 JT, from a buffer that is
  // settled for all of them. With an odd number of steps the second half of
  // the last pair lies behind the row: its lanes read out of range, zeros.
  auto copy_w = [&](i32x4 rows, int pair, int c) {
    const uint32_t last = 2 * pair + 1 == steps ? 0x80000000u : 0u;
    copy16<0>(rows, (lds_ptr)(lds.w[c_buf] + (wave * 8 + c) * 1024),
           (cw[c & 1] + (wave * 8 + c) * 8 * kb) | (cut_w & last), pair * 128);
  };
  auto copy_a = [&](i32x4 rows, int pair, int c) {
    const uint32_t last = 2 * pair + 1 == steps ? 0x80000000u : 0u;
    copy16<0>(rows, (lds_ptr)(lds.a[c_buf] + (wave * 2 * JT + c) * 1024),
           (ca[c & 1] + (wave * 2 * JT + c) * 8 * kb) | (cut_a[c & 1] & last), pair * 128);
  };
  // The scales of a pair and the next; nothing in the second pair of a group.
  // They follow half a pair after the rows, by when the rows' descriptors may
  // be those of the next tile.
  i32x4 late_ws, late_as;
  int late_pair = 0;
  auto copy_scales = [&](int c) {
    const bool group = !(late_pair & 1);
    const uint32_t none = group ? 0u : 0x80000000u;
    if (c == 0) {
      c_group ^= group ? 1 : 0;
      copy16(late_ws, (lds_ptr)((group ? lds.ws[c_group] : lds.none) + wave * 1024), csw | none,
             (late_pair >> 1) * 16);
    } else {
      copy16(late_as, (lds_ptr)((group ? lds.as[c_group] : lds.none) + wave * 1024), csa | none,
             (late_pair >> 1) * 16);
    }
  };

  // Operands of the matrix unit, [accumulator][product of the step]. Each
  // register is read from LDS for the next step as soon as its last product
  // of this one is issued: the rows in two halves, the weights along the
  // second half.
  i32x4 fw[4][2], fa[JT][2];
  int sw[4], sa[JT];
  const int rn = (r & 19) | ((r & 4) << 1) | ((r & 8) >> 1);  // swap23
  const int ow = (hn * 128 + rn) * 128, oa = (hm * 32 + r) * 128;
  const int piece = ((2 * h) ^ ((r >> 1) & 7)) << 4;  // of (step 0, h, 0)
  auto read_w = [&](int buf, int step, int t, int u) {
    fw[t][u] = load16(lds.w[buf] + ow + (piece ^ (step * 64 + u * 16)) + t * 32 * 128);
  };
  auto read_a = [&](int buf, int step, int t, int u) {
    fa[t][u] = load16(lds.a[buf] + oa + (piece ^ (step * 64 + u * 16)) + t * 64 * 128);
  };
  // the two scales of a step (0..3 of its group), all rows at s
  auto scales = [&](const uint8_t* s, int row, int step) {
    return (int)*reinterpret_cast<const uint16_t*>(s + row * 16 + step * 4 + 2 * h);
  };

  aim(0);
#pragma unroll
  for (int pair = 0; pair < 2; ++pair) {
    const i32x4 w = settled(rw), a = settled(ra);
#pragma unroll
    for (int c = 0; c < 8; ++c) copy_w(w, pair, c);
#pragma unroll
    for (int c = 0; c < 2 * JT; ++c) copy_a(a, pair, c);
    c_buf ^= 1;
  }
  late_ws = rws, late_as = ras;
  copy_scales(0);
  copy_scales(1);
  late_pair = 1;
  wait_barrier<0>();
  int buf = 0, grp = 0, ahead = 2;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    read_w(0, 0, t, 0), read_w(0, 0, t, 1);
    sw[t] = scales(lds.ws[0], hn * 128 + t * 32 + rn, 0);
  }
#pragma unroll
  for (int t = 0; t < JH; ++t) {
    read_a(0, 0, t, 0), read_a(0, 0, t, 1);
    sa[t] = scales(lds.as[0], (2 * t + hm) * 32 + r, 0);
  }
  // A tile of no more than half its rows (a slot's last) leaves the second
  // half of every wave's accumulators out, the waves' row tiles taking turns:
  // their products are skipped (65536 rows over 320 slots, 2048 x 7168: 4 %).
  auto run = [&](int it, auto half_) {
    constexpr bool kHalf = decltype(half_)::value;
    constexpr int JN = kHalf ? JH : JT;
    f32x16 acc[4][JN] = {};
    Tile tile = next;
    for (int s = 0; s < pairs; ++s) {
      if (ahead == pairs) {  // at the end of the last pair but two
        tile = next;
        ahead = pairs - 1;
        if (it + 1 < tiles) {
          aim(it + 1);
          ahead = 0;
        }
      }
      const bool behind = 2 * s + 1 == steps;  // the second step is behind the row
      const int gs = 2 * s & 2;                // the pair's first step in its group
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* as = e && behind ? lds.none : lds.as[grp];
        i32x4 w, a;
        if (e) w = settled(rw);
        // first half: the rows of the second are read under it
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int u = c >> 2, i = c & 3;
#pragma unroll
          for (int j = 0; j < JH; ++j)
            acc[i][j] = mfma_mx4(fw[i][u], fa[j][u], acc[i][j], sw[i], sa[j], u);
          if (!kHalf && c < JT) read_a(buf, e, JH + (c >> 1), c & 1);
          if (!kHalf && c < JH) sa[JH + c] = scales(as, (2 * (JH + c) + hm) * 32 + r, gs + e);
          if (e) copy_w(w, ahead, c);
          if (!e && c < 2) copy_scales(c);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (e) {
          // this wave has read all of the pair, and its copies of the next
          // have landed (the eight just issued are of the one after); after
          // the barrier that holds for all waves
          wait_barrier<8>();
          buf ^= 1;
          grp ^= s + 1 == pairs || gs ? 1 : 0;
        }
        const int ns = e ? (s + 1 == pairs ? 0 : (gs + 2) & 2) : gs + 1;  // the next step in its group
        const uint8_t* nas = !e && behind ? lds.none : lds.as[grp];
        const uint8_t* nws = !e && behind ? lds.none : lds.ws[grp];
        if (e) a = settled(ra);
        // second half: the next step's operands are read under it, and the
        // pair two ahead copied into the buffer just read
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int u = c >> 2, i = c & 3;
#pragma unroll
          for (int j = JH; j < JN; ++j)
            acc[i][j] = mfma_mx4(fw[i][u], fa[j][u], acc[i][j], sw[i], sa[j], u);
          read_w(buf, 1 - e, i, u);
          if (u) sw[i] = scales(nws, hn * 128 + i * 32 + rn, ns);
          if (c < JT) read_a(buf, 1 - e, c >> 1, c & 1);
          if (c < JH) sa[c] = scales(nas, (2 * c + hm) * 32 + r, ns);
          if (e) {
#pragma unroll
            for (int d = c * JT / 4; d < (c + 1) * JT / 4; ++d) copy_a(a, ahead, d);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (!e) read_barrier();  // all weights of the pair are in registers
      }
      late_ws = rws, late_as = ras;
      late_pair = ahead++;
      c_buf ^= 1;
    }
#pragma unroll
    for (int j = 0; j < JN; ++j) {
      const int m = tile.m0 + (2 * j + hm) * 32 + r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int v = 0; v < 16; v += 8) {
          const int nn = tile.n0 + hn * 128 + i * 32 + v * 2 + h * 8;
          const f32x16& c = acc[i][j];
          if (m < tile.hi)
            store8_of<kBF16>(p.y, (size_t)m * p.n + nn, p.n - nn,
                             f32x4{c[v], c[v + 1], c[v + 2], c[v + 3]},
                             f32x4{c[v + 4], c[v + 5], c[v + 6], c[v + 7]});
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // one row of accumulators at a time: no spills
    }
  };
  for (int it = 0; it < tiles; ++it) {
    if (next.hi - next.m0 > BM / 2)  // of tile `it`: the copies are two pairs ahead at most
      run(it, std::false_type());
    else
      run(it, std::true_type());
  }
  // no copy may reach LDS after the workgroup has given it back
  wait_barrier<0>();
}

// ---- few rows to an expert: operands straight from memory --------------------
//
// The weights are read once each, and set the pace. A wave computes 16
// outputs of 16 RT rows; a workgroup's four waves take 64 consecutive outputs
// and share the rows through the caches. Four steps' weights (64 bytes of a
// row a step) and the 16 bytes of their scales are fetched together.
// Measured on MI355X: 512 rows over 320 slots, 7168 x 2048: 0.30 ms, the 1.6
// GB of the weights in use at 5.4 TB/s; 1024 to 4096 workgroups take the same
// time, 16384 1 % more.
template <bool kBF16, int RT>
__global__ __launch_bounds__(kExpertThreads) void k_expert_few(ExpertArgs p) {
  __shared__ int first[kMaxPlanSlots + 1];
  __shared__ int part[kExpertThreads / 64];
  if (p.status[0] & MB_ST_FATAL) return;
  const int nslots = p.P * p.NS;
  tile_table<16 * RT>(p, nslots, first, part);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (p.n + 63) / 64;
  const int64_t total = (int64_t)first[nslots] * ntn;
  const int kb = p.k / 2, ks = p.k / 32, steps = p.k / 128;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int mt = (int)(t / ntn), nt = (int)(t - (int64_t)mt * ntn);
    const int j = slot_of(first, nslots, mt);
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    const int m0 = lo + (mt - first[j]) * 16 * RT;
    const int n0 = nt * 64 + wave * 16;
    if (n0 >= p.n) continue;
    // rows past the slot's or the weights' end read the last one instead
    const size_t wr = (size_t)e * p.n + min(n0 + r, p.n - 1);
    const uint8_t* w = p.w + wr * kb + g * 16;
    const uint8_t* ws = p.w_scale + wr * ks;
    const uint8_t *a[RT], *as[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const size_t ar = min(m0 + i * 16 + r, hi - 1);
      a[i] = p.a + ar * kb + g * 16;
      as[i] = p.a_scale + ar * ks;
    }
    f32x4 acc[RT] = {};
    int s = 0;
    for (; s + 4 <= steps; s += 4) {
      i32x4 wv[4], av[RT][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) wv[u] = load16(w + (s + u) * 64);
      const i32x4 wd = scales16(ws + s * 4);
      i32x4 ad[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
#pragma unroll
        for (int u = 0; u < 4; ++u) av[i][u] = load16(a[i] + (s + u) * 64);
        ad[i] = scales16(as[i] + s * 4);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[i] = mfma_mx4(wv[u], av[i][u], acc[i], (uint32_t)wd[u] >> (8 * g),
                            (uint32_t)ad[i][u] >> (8 * g));
    }
    for (; s < steps; ++s) {
      const i32x4 wv = load16(w + s * 64);
#pragma unroll
      for (int i = 0; i < RT; ++i)
        acc[i] = mfma_mx4(wv, load16(a[i] + s * 64), acc[i], ws[s * 4 + g], as[i][s * 4 + g]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int m = m0 + i * 16 + r, nn = n0 + 4 * g;
      if (m < hi && nn < p.n) store4<kBF16>(p.y, (size_t)m * p.n + nn, acc[i]);
    }
  }
}

// Which kernel, from the rows expected in a slot. Measured on MI355X, us, for
// k_expert_few<1>, k_expert_few<4>, 128-row and 256-row tiles (weights n x k):
//   320 slots, 2048 x 7168:   2 rows 332, 526, 335, 370; 8 rows 538, 716, 411,
//     452; 32 rows 1258, 1260, 449, 485; 128 rows 4405, 3210, 666, 653; 256 rows
//     8616, 6035, 1014, 921; 512 rows 17023, 11678, 1762, 1465
//   16 slots, 4096 x 4096:    2 rows 27, 42, 26, 27; 8 rows 35, 53, 26, 27; 128
//     rows 297, 206, 49, 37; 256 rows 571, 394, 67, 69; 512 rows 1126, 743, 107, 101
//   9 slots, 2048 x 2048:     8 rows 11, 11, 14, 16; 32 rows 16, 17, 16, 17; 256
//     rows 79, 56, 19, 25; 512 rows 149, 102, 28, 27
//   144 slots, 2048 x 256:    16 rows 23, 26; 32 rows 33, 32; 256 rows 179, 130
// So the tiles need enough of them to occupy the CUs, and k of two pairs of
// steps; 128 rows to a tile waste less of it, 256 copy less. Near a whole number
// of tiles per CU the rule can miss the better one (16 slots at 128 rows: 49, not 37).
template <bool kBF16>
void launch_expert_t(const ExpertArgs& p, int64_t rows, hipStream_t st) {
  const int64_t slots = (int64_t)p.P * p.NS, columns = (p.n + kTileN - 1) / kTileN;
  const bool tiles = p.k >= 384 && rows >= slots * (slots * columns < kCus / 2 ? 32 : 2);
  const dim3 block(kExpertThreads);
  if (tiles && rows >= slots * 160 && (rows / 256 + slots) * columns > 2 * kCus)
    hipLaunchKernelGGL((k_expert_tile<kBF16, 4>), dim3(kCus), block, 0, st, p);
  else if (tiles)
    hipLaunchKernelGGL((k_expert_tile<kBF16, 2>), dim3(kCus), block, 0, st, p);
  else if (p.k < 384 && rows >= slots * 24)
    hipLaunchKernelGGL((k_expert_few<kBF16, 4>), dim3(kFewGroups), block, 0, st, p);
  else
    hipLaunchKernelGGL((k_expert_few<kBF16, 1>), dim3(kFewGroups), block, 0, st, p);
}

}  // namespace

hipError_t launch_expert_mx4(const mb_dims& d, const Geometry& g, const mb_plan_bufs& o,
                             int32_t n_out, int32_t k_in, const uint8_t* a,
                             const uint8_t* a_scale, const uint8_t* w, const uint8_t* w_scale,
                             void* y, hipStream_t st) {
  if (d.n_tokens == 0) return hipSuccess;
  const ExpertArgs p = {a,         a_scale, w,           w_scale, y,
                        o.cu_seqlens, o.rep_expert, o.status, d.n_ranks, d.n_experts,
                        g.Eh,      g.NS,    d.slots_per_rank, d.cap, n_out, k_in};
  const int64_t rows = (int64_t)d.n_tokens * d.top_k;
  if (d.dtype_out == MB_BF16)
    launch_expert_t<true>(p, rows, st);
  else
    launch_expert_t<false>(p, rows, st);
  return hipGetLastError();
}

}  // namespace mb
