// mx4.hip — rows to microscaled 4-bit floats and back (mb_quantize_mx4,
// mb_dequantize_mx4; OCP Microscaling Formats v1.0).
#include <math.h>

#include "mb_internal.h"
#include "rowio.h"
#include "wave.h"

namespace mb {
namespace {

constexpr int kMxThreads = 256;

// A lane per 8 elements, four lanes per block of 32.
//
// Scale byte of a block from its largest magnitude: 127 + floor(log2(amax))
// - 2, at least 0; the exponent of a finite value is at most 127, so it never
// reaches 254.
__device__ __forceinline__ int scale_byte(float amax) {
  if (amax == 0.0f) return 0;
  // frexp's exponent is floor(log2) + 1, denormals included
  return max(__builtin_amdgcn_frexp_expf(amax) + 124, 0);
}

__device__ __forceinline__ uint32_t quantize8(const float* v, int s) {
  uint32_t o = 0;
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = ldexpf(v[i], 127 - s);  // below 8 in magnitude
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[0], u[1], 1.0f, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[2], u[3], 1.0f, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[4], u[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[6], u[7], 1.0f, 3);
}

// One wave per 64 chunks of a row, a row's parts on consecutive waves.
template <bool kBF16, bool kSwiglu>
__global__ __launch_bounds__(kMxThreads) void k_quantize_mx4(const void* x,
                                                             const int32_t* row_src, uint32_t* q,
                                                             uint8_t* q_scale, int n_rows,
                                                             int chunks, int wpr) {
  const int lane = threadIdx.x & 63;
  const int gw = __builtin_amdgcn_readfirstlane(blockIdx.x * (kMxThreads / 64) + (threadIdx.x >> 6));
  const int row = gw / wpr, c = (gw - row * wpr) * 64 + lane;
  if (row >= n_rows) return;
  if (row_src && row_src[row] < 0) return;
  if (c >= chunks) return;  // whole blocks: chunks is a multiple of 4
  const size_t at = (size_t)row * chunks + c;
  float v[8];
  if constexpr (kSwiglu) {
    float up[8];
    load8<kBF16>(x, (size_t)row * 2 * chunks + c, v);
    load8<kBF16>(x, ((size_t)row * 2 + 1) * chunks + c, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.0f + __expf(-v[i])) * up[i];
  } else {
    load8<kBF16>(x, at, v);
  }
  float amax = 0.0f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    amax = fmaxf(amax, fabsf(v[i]));  // skips NaN
    nan |= v[i] != v[i];
  }
  if (nan) amax = INFINITY;
  amax = quad_max_f32(amax);
  const bool bad = amax == INFINITY;
  const int s = bad ? 255 : scale_byte(amax);
  q[at] = bad ? 0u : quantize8(v, s);
  if ((lane & 3) == 0) q_scale[at >> 2] = (uint8_t)s;
}

template <bool kBF16>
__global__ __launch_bounds__(kMxThreads) void k_dequantize_mx4(const uint32_t* q,
                                                               const uint8_t* q_scale, void* x,
                                                               int n_rows, int chunks, int wpr) {
  const int lane = threadIdx.x & 63;
  const int gw = __builtin_amdgcn_readfirstlane(blockIdx.x * (kMxThreads / 64) + (threadIdx.x >> 6));
  const int row = gw / wpr, c = (gw - row * wpr) * 64 + lane;
  if (row >= n_rows || c >= chunks) return;
  const size_t at = (size_t)row * chunks + c;
  const uint32_t u = q[at];
  const int s = q_scale[at >> 2];
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // e2m1: twice the magnitude is 0, 1, 2, 3, 4, 6, 8, 12
    const uint32_t m = (u >> (4 * i)) & 7u;
    const uint32_t twice = m < 4 ? m : (2u | (m & 1u)) << ((m >> 1) - 1);
    const float f = ldexpf((float)twice, s - 128);
    v[i] = s == 255 ? NAN : (u >> (4 * i)) & 8u ? -f : f;
  }
  store8<kBF16>(x, at, v);
}

}  // namespace

hipError_t launch_quantize_mx4(int32_t n_rows, int32_t hidden, bool bf16, bool swiglu,
                               const void* x, const int32_t* row_src, uint8_t* q,
                               uint8_t* q_scale, hipStream_t st) {
  if (n_rows == 0) return hipSuccess;
  const int chunks = hidden / 8, wpr = (chunks + 63) / 64;
  const int64_t waves = (int64_t)n_rows * wpr;
  const dim3 grid((unsigned)((waves + kMxThreads / 64 - 1) / (kMxThreads / 64)));
  uint32_t* q4 = reinterpret_cast<uint32_t*>(q);
#define MB_Q(B, S)                                                                            \
  hipLaunchKernelGGL((k_quantize_mx4<B, S>), grid, dim3(kMxThreads), 0, st, x, row_src, q4, \
                     q_scale, n_rows, chunks, wpr)
  if (bf16) {
    if (swiglu) MB_Q(true, true);
    else MB_Q(true, false);
  } else {
    if (swiglu) MB_Q(false, true);
    else MB_Q(false, false);
  }
#undef MB_Q
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(int32_t n_rows, int32_t hidden, bool bf16, const uint8_t* q,
                                 const uint8_t* q_scale, void* x, hipStream_t st) {
  if (n_rows == 0) return hipSuccess;
  const int chunks = hidden / 8, wpr = (chunks + 63) / 64;
  const int64_t waves = (int64_t)n_rows * wpr;
  const dim3 grid((unsigned)((waves + kMxThreads / 64 - 1) / (kMxThreads / 64)));
  const uint32_t* q4 = reinterpret_cast<const uint32_t*>(q);
  if (bf16)
    hipLaunchKernelGGL(k_dequantize_mx4<true>, grid, dim3(kMxThreads), 0, st, q4, q_scale, x,
                       n_rows, chunks, wpr);
  else
    hipLaunchKernelGGL(k_dequantize_mx4<false>, grid, dim3(kMxThreads), 0, st, q4, q_scale, x,
                       n_rows, chunks, wpr);
  return hipGetLastError();
}

}  // namespace mb
