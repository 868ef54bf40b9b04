// combine_grad.hip — the gradients of the combine (mb_combine_grad):
//   dy_exp[pos[t][k]] = w[t][k] dy[t],  dw[t][k] = <dy[t], y_exp[pos[t][k]]>.
#include "mb_internal.h"
#include "rowio.h"
#include "wave.h"

namespace mb {
namespace {

constexpr int kGradThreads = 256;
constexpr unsigned kGradGroups = 1u << 20;  // of one launch at most; they go round the tokens

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The 16 bytes of a lane: 8 bf16 or 4 fp32 elements.
template <bool kBF16>
struct Chunk {
  static constexpr int kElems = kBF16 ? 8 : 4;
  float v[kElems];
  __device__ __forceinline__ explicit Chunk(u32x4 u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBF16) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(u[i]);
      }
    }
  }
  __device__ __forceinline__ u32x4 times(float w) const {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBF16)
        o[i] = bf16x2_rne(w * v[2 * i], w * v[2 * i + 1]);
      else
        o[i] = __float_as_uint(w * v[i]);
    }
    return o;
  }
};

// `wpt` waves (1, 2 or 4) take a token's row, 16 bytes a lane at a time: dy's
// are read once, and for every k those of its expert row, which meet dy in
// the weight's sum, and the weighted ones are written. A wave's sums are
// added over its lanes, then over the token's waves in LDS.
//
// Bound by HBM: 32768 tokens of 8 experts, 7168 bf16: 1.60 ms, 5.0 TB/s of
// scattered rows read and written in turn; 4096 x 2, 4096 fp32: 50 us, 6.7
// TB/s (partly from the last-level cache). A wave for every pair instead took
// 1.59 ms. More waves than `chunks` feed would idle: a token has one wave to
// 1024 bytes, at most four. K of 1, 2, 4 and 8 are unrolled, which holds the
// sums in registers; others go through a loop of the largest.
template <int KT, bool kBF16>
__global__ __launch_bounds__(kGradThreads) void k_combine_grad(
    const u32x4* __restrict__ dy, const u32x4* __restrict__ ye, const float* __restrict__ w,
    const int32_t* __restrict__ pos, const int32_t* __restrict__ status, u32x4* __restrict__ dye,
    float* __restrict__ dw, int N, int K_, int chunks, int wpt, int rows) {
  constexpr int KM = KT ? KT : kMaxTopK;
  const int K = KT ? KT : K_;
  __shared__ float sums[kGradThreads / 64][KM];
  if (status[0] & MB_ST_FATAL) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tpb = kGradThreads / 64 / wpt, part = wave % wpt;
  for (int64_t first = (int64_t)blockIdx.x * tpb; first < N; first += (int64_t)gridDim.x * tpb) {
    const int64_t t = first + wave / wpt;
    const bool on = t < N;
    float acc[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k) acc[k] = 0.0f;
    if (on) {
      const int32_t* pt = pos + t * K;
      const float* wt = w + t * K;
      for (int c = part * 64 + lane; c < chunks; c += wpt * 64) {
        const Chunk<kBF16> d(dy[t * chunks + c]);
#pragma unroll
        for (int k = 0; k < KM; ++k) {
          if (k >= K) break;
          const int p = pt[k];
          if ((unsigned)p >= (unsigned)rows) continue;  // only a broken plan
          const size_t at = (size_t)p * chunks + c;
          if (dw) {
            const Chunk<kBF16> y(ye[at]);
#pragma unroll
            for (int i = 0; i < Chunk<kBF16>::kElems; ++i) acc[k] = fmaf(d.v[i], y.v[i], acc[k]);
          }
          if (dye) __builtin_nontemporal_store(d.times(wt[k]), dye + at);
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int k = 0; k < KM; ++k) {
      if (k >= K) break;
      const float s = wave_sum_f32(acc[k]);
      if (lane == 0) sums[wave][k] = s;
    }
    __syncthreads();
    if (on && part == 0 && lane < K) {
      float s = 0.0f;
      for (int i = 0; i < wpt; ++i) s += sums[wave + i][lane];
      dw[t * K + lane] = s;
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_combine_grad(const mb_dims& d, const mb_plan_bufs& o, const void* dy,
                               const void* ye, const float* w, void* dye, float* dw,
                               hipStream_t st) {
  if (d.n_tokens == 0) return hipSuccess;
  const int chunks = (int)(d.hidden * elt_bytes(d.dtype_out) / 16), rows = d.n_ranks * d.cap;
  const int wpt = chunks <= 64 ? 1 : chunks <= 128 ? 2 : 4;
  const int tpb = kGradThreads / 64 / wpt;
  const dim3 grid(min((unsigned)(((int64_t)d.n_tokens + tpb - 1) / tpb), kGradGroups));
  const dim3 block(kGradThreads);
  const auto *dyv = static_cast<const u32x4*>(dy), *yev = static_cast<const u32x4*>(ye);
  auto* dyev = static_cast<u32x4*>(dye);
#define MB_G(KT)                                                                              \
  do {                                                                                        \
    if (d.dtype_out == MB_BF16)                                                               \
      hipLaunchKernelGGL((k_combine_grad<KT, true>), grid, block, 0, st, dyv, yev, w, o.pos,    \
                         o.status, dyev, dw, d.n_tokens, d.top_k, chunks, wpt, rows);          \
    else                                                                                      \
      hipLaunchKernelGGL((k_combine_grad<KT, false>), grid, block, 0, st, dyv, yev, w, o.pos,   \
                         o.status, dyev, dw, d.n_tokens, d.top_k, chunks, wpt, rows);          \
  } while (0)
  switch (d.top_k) {
    case 1: MB_G(1); break;
    case 2: MB_G(2); break;
    case 4: MB_G(4); break;
    case 8: MB_G(8); break;
    default: MB_G(0); break;
  }
#undef MB_G
  return hipGetLastError();
}

}  // namespace mb
