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
#include "wave.h"

namespace mb {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kExpertThreads = 256;
constexpr int kMaxPlanSlots = kMaxExperts + kMaxRanks * kMaxSlots;

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

typedef const __attribute__((address_space(4))) int32_t* plan_ptr;

// Rows [lo, hi) of slot j (r = j / NS), absolute in the buffer, and its
// expert; empty when it holds none. Only a broken plan needs the clamps.
__device__ __forceinline__ void slot_rows(const ExpertArgs& p, int j, int& lo, int& hi, int& e) {
  const int r = j / p.NS, i = j - r * p.NS;
  // the plan does not change under the kernel: constant memory
  auto cu = (plan_ptr)(p.cu + (size_t)r * (p.NS + 1) + i);
  lo = min(max(cu[0], 0), p.cap);
  hi = min(max(cu[1], lo), p.cap);
  e = i < p.Eh ? r * p.Eh + i : ((plan_ptr)p.rep)[(size_t)r * p.R + i - p.Eh];
  if ((unsigned)e >= (unsigned)p.E) hi = lo;
  lo += r * p.cap;
  hi += r * p.cap;
}

// first[j] = row tiles of the slots before j, first[nslots] = all of them.
template <int BM>
__device__ void tile_table(const ExpertArgs& p, int nslots, int* first, int* part) {
  const int per = (nslots + kExpertThreads - 1) / kExpertThreads;
  const int j0 = threadIdx.x * per;
  int sum = 0;
  for (int j = j0; j < min(j0 + per, nslots); ++j) {
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    sum += (hi - lo + BM - 1) / BM;
  }
  const int incl = wave_inclusive_sum(sum);
  if ((threadIdx.x & 63) == 63) part[threadIdx.x >> 6] = incl;
  __syncthreads();
  int base = incl - sum;
  for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) base += part[i];
  for (int j = j0; j < min(j0 + per, nslots); ++j) {
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    first[j] = base;
    base += (hi - lo + BM - 1) / BM;
  }
  if (threadIdx.x == kExpertThreads - 1) first[nslots] = base;
  __syncthreads();
}

// The slot whose tiles hold row tile t.
__device__ __forceinline__ int slot_of(const int* first, int nslots, int t) {
  int lo = 0, hi = nslots;  // first[lo] <= t < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
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

// Waits until this wave's LDS reads are done and at most N of its memory
// operations (copies to LDS, stores) are outstanding, oldest first, then for
// the other waves.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// ---- tiles staged through LDS -----------------------------------------------
//
// A workgroup of four waves computes 256 outputs x BM rows (BM = 32 MT), a
// wave 128 outputs x 16 MT rows: 8 x MT accumulators of 16 x 16. A step takes
// 128 elements of k. Rows are copied from memory into LDS, without passing
// registers, in pairs of steps: 128 bytes of every row, one cache line. (With
// single steps, 64 bytes of a row and 4 of its scales at a time, the L2's
// requests set the pace: 10.5 ms for 1048576 rows of 7168 by 2048, twice the
// requests for rows and eight times those for scales.) The scales are copied
// in groups of four steps, 16 bytes of every row. Two pairs and two groups
// are in LDS; the pair two ahead is copied as soon as the last operand of the
// present one is in registers. The pairs of a workgroup's tiles form one
// sequence, so that a tile's first copies run under the end of the tile
// before it.
//
// LDS layout of a pair: rows of 128 bytes, the 16-byte piece c of a row at
// place c ^ swizzle; the copy writes 64 consecutive pieces (8 rows), so the
// swizzle is in the piece each lane fetches. A read of one piece of 16 rows
// then meets every bank once. Weight rows enter the matrix unit in the order
// n(t, i) = (t / 2) 32 + (i / 4) 8 + (t % 2) 4 + i % 4 (accumulator t, row i),
// which leaves a lane 8 consecutive outputs in two accumulators: 16-byte
// bf16 stores, 64 consecutive bytes per row.
constexpr int kTileN = 256;
constexpr int kCus = 256, kXcds = 8;
constexpr int kGroupM = 4;  // row tiles whose columns are walked together

typedef __attribute__((address_space(3))) void* lds_ptr;

// Buffer descriptor of `bytes` bytes at p (wave-uniform). A read at voff +
// soff gives 0 where voff >= bytes - soff: soff must be below bytes, so what
// may pass the end is always in voff.
__device__ __forceinline__ i32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane((int)at),
               __builtin_amdgcn_readfirstlane((int)(at >> 32) & 0xffff),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Copies 64 lanes' 16 or 4 bytes at buf[voff + soff] to consecutive places of
// LDS from `to` (wave-uniform). No register is written. In assembly because
// the compiler, for its builtin, waits for every copy in flight before the
// next read of any LDS; the waits that order copies and reads are
// wait_barrier's.
__device__ __forceinline__ void copy16(i32x4 buf, lds_ptr to, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               ::"s"((uint32_t)(uintptr_t)to), "v"(voff), "s"(buf), "s"(soff)
               : "memory");
}
__device__ __forceinline__ i32x4 piece_at(const uint8_t* p) {
  return *static_cast<const i32x4*>(__builtin_assume_aligned(p, 16));
}

struct Tile {
  int m0, hi, n0, e;
};

template <int MT>
struct alignas(16) TileLds {
  uint8_t w[2][kTileN * 128];
  uint8_t a[2][32 * MT * 128];
  uint8_t ws[2][kTileN * 16];
  uint8_t as[2][kTileN * 16];  // 32 MT rows, copied by four waves: twice over when MT = 4
  uint8_t none[4 * 1024];      // where copies of nothing go
  int first[kMaxPlanSlots + 1];
  int part[kExpertThreads / 64];
};

template <bool kBF16, int MT>
__global__ __launch_bounds__(kExpertThreads, 1) void k_expert_tile(ExpertArgs p) {
  constexpr int BM = 32 * MT, MH = MT / 2;
  __shared__ TileLds<MT> lds;
  if (p.status[0] & MB_ST_FATAL) return;
  const int nslots = p.P * p.NS;
  tile_table<BM>(p, nslots, lds.first, lds.part);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
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

  // What a lane copies: of 8 rows, piece (lane % 8) ^ swizzle of row lane / 8.
  // The swizzle of row i of 16 in the matrix unit is i / 2; blocks of 8 rows
  // differ in it by constants.
  const int crow = lane >> 3;
  uint32_t ca[2], cw[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) ca[j] = crow * kb + (((lane & 7) ^ (crow >> 1) ^ (j << 2)) << 4);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    cw[j] = crow * kb + (((lane & 7) ^ ((crow >> 1) & 1) ^ (j << 1)) << 4);
  // scales: lane = row, in the order of the accumulators' rows
  const int q = wave * 64 + lane, qi = q & 15, qt = (q >> 4) & 7;
  const uint32_t csw = ((q >> 7) * 128 + (qt >> 1) * 32 + (qi >> 2) * 8 + (qt & 1) * 4 + (qi & 3)) * ks;
  const uint32_t csa = (q % BM) * ks;

  // the copies' place in the sequence of pairs: two ahead of the product.
  // Past the last tile its last pair is copied again, unused.
  i32x4 rw, ra, rws, ras;
  Tile next;
  int c_buf = 0, c_group = 0;
  auto aim = [&](int it) {
    next = tile_of(tile_index(it));
    const size_t wrow = (size_t)next.e * p.n + next.n0;
    const int nw = min(kTileN, p.n - next.n0), na = min(BM, next.hi - next.m0);
    rw = buffer_of(p.w + wrow * kb, (uint32_t)nw * kb);
    rws = buffer_of(p.w_scale + wrow * ks, (uint32_t)nw * ks);
    ra = buffer_of(p.a + (size_t)next.m0 * kb, (uint32_t)na * kb);
    ras = buffer_of(p.a_scale + (size_t)next.m0 * ks, (uint32_t)na * ks);
  };
  auto copy = [&](int pair) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      copy16(rw, (lds_ptr)(lds.w[c_buf] + (wave * 8 + j) * 1024),
             cw[j & 3] + (wave * 8 + j) * 8 * kb, pair * 128);
#pragma unroll
    for (int j = 0; j < MT; ++j)
      copy16(ra, (lds_ptr)(lds.a[c_buf] + (wave * MT + j) * 1024),
             ca[j & 1] + (wave * MT + j) * 8 * kb, pair * 128);
    // the scales of this pair and the next; nothing in the second of a group
    const bool group = !(pair & 1);
    c_group ^= group ? 1 : 0;
    const uint32_t none = group ? 0u : 0x80000000u;
    copy16(rws, (lds_ptr)((group ? lds.ws[c_group] : lds.none) + wave * 1024), csw | none,
           (pair >> 1) * 16);
    copy16(ras, (lds_ptr)((group ? lds.as[c_group] : lds.none) + wave * 1024), csa | none,
           (pair >> 1) * 16);
    c_buf ^= 1;
  };

  // Operands of the matrix unit. Each register is read from LDS for the next
  // step as soon as its last product of this one is issued: the rows in two
  // halves, the weights along the second half.
  i32x4 fw[8], fa[MT];
  int sw[8], sa[MT];
  const int ow = (hn * 128 + (r >> 2) * 8 + (r & 3)) * 128, oa = (hm * 16 * MT + r) * 128;
  const int piece = (g ^ (r >> 1)) << 4;  // of the first step of a pair; the second's is piece ^ 64
  auto read_w = [&](int buf, int half, int t) {
    fw[t] = piece_at(lds.w[buf] + ow + (piece ^ half * 64) + ((t >> 1) * 32 + (t & 1) * 4) * 128);
  };
  auto read_a = [&](int buf, int half, int t) {
    fa[t] = piece_at(lds.a[buf] + oa + (piece ^ half * 64) + t * 16 * 128);
  };
  auto scale = [&](const uint8_t* s, int row, int step) {
    return (int)s[(row + r) * 16 + (step & 3) * 4 + g];
  };

  aim(0);
  c_group = 1;
  copy(0);
  copy(1);
  wait_barrier<0>();
  int buf = 0, grp = 0, ahead = 2;
#pragma unroll
  for (int t = 0; t < 8; ++t) read_w(0, 0, t), sw[t] = scale(lds.ws[0], hn * 128 + t * 16, 0);
#pragma unroll
  for (int t = 0; t < MH; ++t) read_a(0, 0, t), sa[t] = scale(lds.as[0], (hm * MT + t) * 16, 0);
  for (int it = 0; it < tiles; ++it) {
    f32x4 acc[8][MT] = {};
    Tile tile = next;
    for (int s = 0; s < steps; ++s) {
      if (ahead == pairs) {  // at the end of the last pair but two
        tile = next;
        ahead = pairs - 1;
        if (it + 1 < tiles) {
          aim(it + 1);
          ahead = 0;
        }
      }
      // the second half of this step's rows is read under the products of the
      // first half
#pragma unroll
      for (int t = MH; t < MT; ++t)
        read_a(buf, s & 1, t), sa[t] = scale(lds.as[grp], (hm * MT + t) * 16, s);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < MH; ++j) acc[i][j] = mfma_mx4(fw[i], fa[j], acc[i][j], sw[i], sa[j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      const int step = s + 1 < steps ? s + 1 : 0;  // the next
      if (!(step & 1)) {
        // this wave has read all of the pair, and its copies of the next have
        // landed; after the barrier that holds for all waves
        wait_barrier<0>();
        copy(ahead++);
        buf ^= 1;
        grp ^= step & 2 ? 0 : 1;
      }
      // the next step's operands, under the products of the second half
#pragma unroll
      for (int t = 0; t < MH; ++t)
        read_a(buf, step & 1, t), sa[t] = scale(lds.as[grp], (hm * MT + t) * 16, step);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = MH; j < MT; ++j) acc[i][j] = mfma_mx4(fw[i], fa[j], acc[i][j], sw[i], sa[j]);
        read_w(buf, step & 1, i), sw[i] = scale(lds.ws[grp], hn * 128 + i * 16, step);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int m = tile.m0 + (hm * MT + j) * 16 + r;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const int nn = tile.n0 + hn * 128 + (i >> 1) * 32 + g * 8;
        if (m < tile.hi)
          store8_of<kBF16>(p.y, (size_t)m * p.n + nn, p.n - nn, acc[i][j], acc[i + 1][j]);
      }
      __builtin_amdgcn_sched_barrier(0);  // one row of accumulators at a time: no spills
    }
  }
  // no copy may reach LDS after the workgroup has given it back
  wait_barrier<0>();
}

// 64 x 64 tiles, operands straight from memory: wave w holds 16 outputs of
// all 64 rows. Workgroups stride over the tiles.
template <bool kBF16>
__global__ __launch_bounds__(kExpertThreads) void k_expert_mx4(ExpertArgs p) {
  __shared__ int first[kMaxPlanSlots + 1];
  __shared__ int part[kExpertThreads / 64];
  if (p.status[0] & MB_ST_FATAL) return;
  const int nslots = p.P * p.NS;
  tile_table<64>(p, nslots, first, part);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (p.n + 63) / 64;
  const int total = first[nslots];
  const size_t kb = p.k / 2, ks = p.k / 32;
  for (int64_t t = blockIdx.x; t < (int64_t)total * ntn; t += gridDim.x) {
    const int mt = (int)(t / ntn), nt = (int)(t - (int64_t)mt * ntn);
    const int j = slot_of(first, nslots, mt);
    int lo, hi, e;
    slot_rows(p, j, lo, hi, e);
    const int m0 = lo + (mt - first[j]) * 64;
    const int n0 = nt * 64 + wave * 16;
    if (n0 >= p.n) continue;
    // rows past the slot's or the weights' end read the last one instead
    const size_t wr = (size_t)e * p.n + min(n0 + r, p.n - 1);
    size_t ar[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ar[i] = min(m0 + i * 16 + r, hi - 1);
    f32x4 acc[4] = {};
    for (int kk = 0; kk < p.k / 128; ++kk) {
      const i32x4 wv = *reinterpret_cast<const i32x4*>(p.w + wr * kb + kk * 64 + g * 16);
      const int ws = p.w_scale[wr * ks + kk * 4 + g];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const i32x4 av = *reinterpret_cast<const i32x4*>(p.a + ar[i] * kb + kk * 64 + g * 16);
        const int as = p.a_scale[ar[i] * ks + kk * 4 + g];
        acc[i] = mfma_mx4(wv, av, acc[i], ws, as);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + i * 16 + r, nn = n0 + 4 * g;
      if (m < hi && nn < p.n) store4<kBF16>(p.y, (size_t)m * p.n + nn, acc[i]);
    }
  }
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
  if (k_in >= 384 && rows >= (int64_t)d.n_ranks * g.NS * 128) {
    if (d.dtype_out == MB_BF16)
      hipLaunchKernelGGL((k_expert_tile<true, 8>), dim3(kCus), dim3(kExpertThreads), 0, st, p);
    else
      hipLaunchKernelGGL((k_expert_tile<false, 8>), dim3(kCus), dim3(kExpertThreads), 0, st, p);
    return hipGetLastError();
  }
  if (k_in >= 384 && rows >= (int64_t)d.n_ranks * g.NS * 32) {
    if (d.dtype_out == MB_BF16)
      hipLaunchKernelGGL((k_expert_tile<true, 4>), dim3(kCus), dim3(kExpertThreads), 0, st, p);
    else
      hipLaunchKernelGGL((k_expert_tile<false, 4>), dim3(kCus), dim3(kExpertThreads), 0, st, p);
    return hipGetLastError();
  }
  const int grid = 1024;
  if (d.dtype_out == MB_BF16)
    hipLaunchKernelGGL(k_expert_mx4<true>, dim3(grid), dim3(kExpertThreads), 0, st, p);
  else
    hipLaunchKernelGGL(k_expert_mx4<false>, dim3(grid), dim3(kExpertThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace mb
