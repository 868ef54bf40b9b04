// expert.hip — the experts' products over the dispatch layout, from
// microscaled 4-bit rows and weights (mb_expert_mx4).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands as e2m1 with an e8m0
// scale per 32 elements of k: a lane (r = lane % 16, g = lane / 16) holds the
// 32 elements g of row r of its operand's 128 (16 bytes, the packed order of
// the rows in memory) and their scale byte. The weights are the first
// operand, so that a lane ends with four consecutive outputs of one row:
// column r of the product is row r of the tile, rows 4g..4g+3 its outputs.
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

// Rows [lo, hi) of slot j (r = j / NS), absolute in the buffer, and its
// expert; empty when it holds none. Only a broken plan needs the clamps.
__device__ __forceinline__ void slot_rows(const ExpertArgs& p, int j, int& lo, int& hi, int& e) {
  const int r = j / p.NS, i = j - r * p.NS;
  const int32_t* cu = p.cu + (size_t)r * (p.NS + 1) + i;
  lo = min(max(cu[0], 0), p.cap);
  hi = min(max(cu[1], lo), p.cap);
  e = i < p.Eh ? r * p.Eh + i : p.rep[(size_t)r * p.R + i - p.Eh];
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
  return lo;
}

template <bool kBF16>
__device__ __forceinline__ void store4(void* y, size_t at, f32x4 v) {
  if constexpr (kBF16) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) =
        uint2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(y) + at) = v;
  }
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
  const int grid = 1024;
  if (d.dtype_out == MB_BF16)
    hipLaunchKernelGGL(k_expert_mx4<true>, dim3(grid), dim3(kExpertThreads), 0, st, p);
  else
    hipLaunchKernelGGL(k_expert_mx4<false>, dim3(grid), dim3(kExpertThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace mb
