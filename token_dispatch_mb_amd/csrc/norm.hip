// norm.hip — root-mean-square norm with the residual's addition, rows out in
// fp8 with a scale per 128 elements (mb_rmsnorm_fp8).
#include <math.h>

#include "mb_internal.h"
#include "rowio.h"
#include "wave.h"

namespace mb {
namespace {

constexpr int kNormThreads = 512;
static_assert(MB_MAX_NORM_HIDDEN <= 4 * 8 * kNormThreads, "at most four chunks to a lane");
constexpr float kE4m3Max = 448.0f;

// Mean squares (with epsilon) below kTinyMean, of which squares below the
// normal numbers are a part that counts, are taken again from rows times
// kLift: sums of at most 2^14 such squares stay below 2^114, and the smallest
// number's square is 2^-98.
constexpr float kTinyMean = 0x1p-100f, kLift = 0x1p100f;

// Sum over the workgroup, the same in every lane.
__device__ __forceinline__ float group_sum(float v, float* part) {
  v = wave_sum_f32(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 64; ++i) v += part[i];
  return v;
}

// One workgroup per row, a lane per 8 consecutive elements, the row in
// registers between its two passes (sum of squares; scales and codes), so
// that memory is read and written once and bounds it. Squares are summed in
// binary32; the normed value is rounded once, to e4m3 (and once more, from
// the same binary32 value, to dtype in y). Measured on MI355X: 131072 x 7168
// bf16 with the residual 1.11-1.14 ms, 5.8-6.0 TB/s of 6.6 GB; 4099 x 4224 fp32 28
// us, 5.5 TB/s; one row 3.0 us. 256 or 1024 lanes to a row were 2 and 4 % slower
// on the first, 8 and 1 % on the second. Short rows leave most lanes idle and
// are bound by their workgroups, not by memory: 60000 bf16 rows of 128, 512,
// 1024, 2048 take 69, 70, 93, 114 us (0.3, 1.3, 2.0, 3.3 TB/s).
template <bool kBF16, int CPT>
__global__ __launch_bounds__(kNormThreads) void k_rmsnorm_fp8(
    const void* x, const void* res, const void* weight, void* res_out, void* y, uint32_t* q,
    float* q_scale, int chunks, float eps) {
  __shared__ float part[kNormThreads / 64];
  const size_t row = (size_t)blockIdx.x * chunks;
  float h[CPT][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = i * kNormThreads + threadIdx.x;
    if (c < chunks) {
      load8<kBF16>(x, row + c, h[i]);
      if (res) {
        float r[8];
        load8<kBF16>(res, row + c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        if (res_out) store8<kBF16>(res_out, row + c, h[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
  }
  ss = group_sum(ss, part);
  float ms = ss / (float)(chunks * 8) + eps;
  if (ms < kTinyMean) {  // the same for every lane
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      if (i * kNormThreads + (int)threadIdx.x < chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i][j] *= kLift;
          ss = fmaf(h[i][j], h[i][j], ss);
        }
      }
    }
    __syncthreads();  // every lane has read the first sums
    ss = group_sum(ss, part);
    ms = ss / (float)(chunks * 8) + eps * kLift * kLift;
  }
  float inv = ms > 0.0f ? 1.0f / sqrtf(ms) : 0.0f;
  const bool bad = !(ss < INFINITY);  // a NaN or an infinity in the row, or a sum past binary32
  if (bad) inv = NAN;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = i * kNormThreads + threadIdx.x;
    if (c < chunks) {
      float g[8], v[8];
      uint32_t bits = 0;
      load8<kBF16>(weight, c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = h[i][j] * inv * g[j];
        bits = max(bits, __float_as_uint(v[j]) & 0x7fffffffu);
      }
      if (y) store8<kBF16>(y, row + c, v);  // all NaN when bad: inv is
      // 16 lanes of 8 elements share a block
      const float amax = __uint_as_float(row_max_u32(bits));
      const bool tiny = amax < 0x1p-110f;
      const float scale = tiny ? 1.0f : amax / kE4m3Max;
      // y / scale as division rounds it: the product with the rounded
      // reciprocal, less its remainder's (signs so that -0 stays -0)
      const bool flat = tiny || amax == INFINITY;  // finite values give zeros
      const float d = flat ? 0.0f : scale, f = flat ? 0.0f : 1.0f / scale;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = v[j] * f;
        v[j] = fmaf(fmaf(t, d, -v[j]), -f, t);
      }
      const uint2 o = {fp8x4(v[0], v[1], v[2], v[3]), fp8x4(v[4], v[5], v[6], v[7])};
      reinterpret_cast<uint2*>(q)[row + c] = bad ? uint2{0x7f7f7f7fu, 0x7f7f7f7fu} : o;
      if ((threadIdx.x & 15) == 0) q_scale[(row + c) >> 4] = bad ? NAN : scale;
    }
  }
}

template <bool kBF16>
void launch_norm_t(int n_rows, int hidden, float eps, const void* x, const void* res,
                   const void* weight, void* res_out, void* y, uint8_t* q, float* q_scale,
                   hipStream_t st) {
  const int chunks = hidden / 8;
  const int cpt = (chunks + kNormThreads - 1) / kNormThreads;
  auto at = [&](const void* p, int row) {  // row `row` of p, null where there is none
    return p ? static_cast<const char*>(p) + (size_t)row * hidden * (kBF16 ? 2 : 4) : nullptr;
  };
  // a launch holds fewer than 2^32 threads
  constexpr int kMost = kMaxWaves / (kNormThreads / 64);
  for (int row = 0; row < n_rows; row += kMost) {
    const dim3 grid(min(n_rows - row, kMost));
    uint32_t* q4 = reinterpret_cast<uint32_t*>(q + (size_t)row * hidden);
#define MB_N(C)                                                                              \
  hipLaunchKernelGGL((k_rmsnorm_fp8<kBF16, C>), grid, dim3(kNormThreads), 0, st, at(x, row), \
                     at(res, row), weight, const_cast<char*>(at(res_out, row)),              \
                     const_cast<char*>(at(y, row)), q4, q_scale + (size_t)row * (hidden / 128), \
                     chunks, eps)
    if (cpt <= 1)
      MB_N(1);
    else if (cpt <= 2)
      MB_N(2);
    else
      MB_N(4);
#undef MB_N
  }
}

}  // namespace

hipError_t launch_rmsnorm_fp8(int32_t n_rows, int32_t hidden, bool bf16, float eps, const void* x,
                              const void* res, const void* weight, void* res_out, void* y,
                              uint8_t* q, float* q_scale, hipStream_t st) {
  if (n_rows == 0) return hipSuccess;
  if (bf16)
    launch_norm_t<true>(n_rows, hidden, eps, x, res, weight, res_out, y, q, q_scale, st);
  else
    launch_norm_t<false>(n_rows, hidden, eps, x, res, weight, res_out, y, q, q_scale, st);
  return hipGetLastError();
}

}  // namespace mb
