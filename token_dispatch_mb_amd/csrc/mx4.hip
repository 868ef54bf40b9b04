// mx4.hip — rows to microscaled 4-bit floats and back (mb_quantize_mx4,
// mb_dequantize_mx4; OCP Microscaling Formats v1.0).
#include <math.h>

#include "mb_internal.h"
#include "rowio.h"
#include "wave.h"

namespace mb {
namespace {

constexpr int kMxThreads = 256;

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Both directions are bound by memory: a lane per 8 elements (16 bytes of
// bf16, 4 of codes), four lanes per block of 32. Measured on MI355X for 8192 x
// 7168 bf16 rows: 22-25 us to quantise, 21 us back, 47 in all (6.4 TB/s: the
// codes stay in the last-level cache). With two or four chunks of a lane in
// flight both together took 2 and 8 % longer (51, 54 against 50 us, all three
// with plain stores).

// Scale byte of a block from the bits of its largest magnitude: 127 +
// floor(log2(amax)) - 2, at least 0, which is the bits' exponent less 2 for a
// normal amax (a denormal one gives 0 either way); 255 for infinities and
// NaN, whose bits are the largest.
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  const int e = (int)(amax >> 23);
  return e == 255 ? 255 : max(e - 2, 0);
}

// v[0..8) under scale byte s, as packed codes.
__device__ __forceinline__ uint32_t quantize8(const float* v, int s) {
  uint32_t o = 0;
  float u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __builtin_amdgcn_ldexpf(v[i], 127 - s);  // below 8 in magnitude
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[0], u[1], 1.0f, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[2], u[3], 1.0f, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[4], u[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, u[6], u[7], 1.0f, 3);
}

// Chunk `at` of the output, of a block whose four lanes are neighbours.
__device__ __forceinline__ void quantize_chunk(const float* v, size_t at, uint32_t* q,
                                               uint8_t* q_scale) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  amax = quad_max_u32(amax);
  const int s = scale_byte(amax);
  q[at] = s == 255 ? 0u : quantize8(v, s);
  if ((at & 3) == 0) q_scale[at >> 2] = (uint8_t)s;
}

// g / (1 + exp(-g)) * up for gates from kNearGate on: the exponential's
// argument is off by |g| 2^-24 of rounding, so the whole by less than 2^-19.
constexpr float kNearGate = -16.0f;

__device__ __forceinline__ float swiglu_near(float g, float up) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * up;
}

// The same for any gate, by h = exp(-|g| / 2): g / (1 + h h) * up, and two
// factors h more for a negative g, one on each side, so that nothing on the
// way overflows or falls below the normal numbers before the result does (the
// reciprocal of 1 + exp(-g) does from -87.3). What the exponential's argument
// loses by its rounding and its constant's comes back as a factor: below 2^-20.
// 65536 rows of 2 x 2048 bf16 by this alone take 116 us, by the near form 106.
__device__ __forceinline__ float swiglu_any(float g, float up) {
  constexpr float kHalfLog2e = 0x1.715476p-1f, kLn2 = 0x1.62e43p-1f;
  constexpr float kRest = 0x1.cab1b6p-28f;  // log2(e) / 2 less its constant, times ln 2
  const float m = -fabsf(g), t = m * kHalfLog2e;
  const float rest = fmaf(m, kRest, fmaf(m, kHalfLog2e, -t) * kLn2);
  float h = __builtin_amdgcn_exp2f(t);
  h = fmaf(h, rest, h);
  const float r = __builtin_amdgcn_rcpf(fmaf(h, h, 1.0f)), f = g < 0.0f ? h : 1.0f;
  return g * f * r * (f * up);
}

// All rows of x, one after the other.
template <bool kBF16>
__global__ __launch_bounds__(kMxThreads) void k_quantize_mx4(const void* x, uint32_t* q,
                                                             uint8_t* q_scale, size_t chunks) {
  const size_t at = (size_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (at >= chunks) return;  // whole blocks: chunks is a multiple of 4
  float v[8];
  load8<kBF16>(x, at, v);
  quantize_chunk(v, at, q, q_scale);
}

// Row by row, for rows with an activation or that may be skipped: one wave
// per 64 chunks of a row, a row's parts on consecutive waves. The activation
// is not rounded before it is quantised. 65536 rows of 2 x 2048 bf16: 106 us,
// 5.7 TB/s.
template <bool kBF16, bool kSwiglu>
__global__ __launch_bounds__(kMxThreads) void k_quantize_mx4_rows(const void* x,
                                                                  const int32_t* row_src,
                                                                  uint32_t* q, uint8_t* q_scale,
                                                                  int n_rows, int chunks, int wpr) {
  const int lane = threadIdx.x & 63;
  const int gw = __builtin_amdgcn_readfirstlane(blockIdx.x * (kMxThreads / 64) + (threadIdx.x >> 6));
  const int row = gw / wpr, c = (gw - row * wpr) * 64 + lane;
  if (row >= n_rows || c >= chunks) return;  // whole blocks: chunks is a multiple of 4
  float v[8];
  if constexpr (kSwiglu) {
    float up[8];
    load8<kBF16>(x, (size_t)row * 2 * chunks + c, v);
    load8<kBF16>(x, ((size_t)row * 2 + 1) * chunks + c, up);
    if (row_src && row_src[row] < 0) return;
    float low = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) low = fminf(low, v[i]);
    if (ballot64(low < kNearGate) == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = swiglu_near(v[i], up[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = swiglu_any(v[i], up[i]);
    }
  } else {
    load8<kBF16>(x, (size_t)row * chunks + c, v);
    if (row_src && row_src[row] < 0) return;
  }
  quantize_chunk(v, (size_t)row * chunks + c, q, q_scale);
}

template <bool kBF16>
__global__ __launch_bounds__(kMxThreads) void k_dequantize_mx4(const uint32_t* q,
                                                               const uint8_t* q_scale, void* x,
                                                               size_t chunks) {
  const size_t at = (size_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (at >= chunks) return;
  const uint32_t u = q[at];
  const int s = q_scale[at >> 2];
  const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 0),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 2),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 3)};
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = s == 255 ? NAN : __builtin_amdgcn_ldexpf(p[j >> 1][j & 1], s - 127);
  store8<kBF16>(x, at, v);
}

}  // namespace

hipError_t launch_quantize_mx4(int32_t n_rows, int32_t hidden, bool bf16, bool swiglu,
                               const void* x, const int32_t* row_src, uint8_t* q,
                               uint8_t* q_scale, hipStream_t st) {
  if (n_rows == 0) return hipSuccess;
  const int chunks = hidden / 8;
  uint32_t* q4 = reinterpret_cast<uint32_t*>(q);
  if (!swiglu && !row_src) {
    const size_t all = (size_t)n_rows * chunks;
    const dim3 grid((unsigned)((all + kMxThreads - 1) / kMxThreads));
    if (bf16)
      hipLaunchKernelGGL(k_quantize_mx4<true>, grid, dim3(kMxThreads), 0, st, x, q4, q_scale, all);
    else
      hipLaunchKernelGGL(k_quantize_mx4<false>, grid, dim3(kMxThreads), 0, st, x, q4, q_scale, all);
    return hipGetLastError();
  }
  const int wpr = (chunks + 63) / 64;
  const int64_t waves = (int64_t)n_rows * wpr;
  const dim3 grid((unsigned)((waves + kMxThreads / 64 - 1) / (kMxThreads / 64)));
#define MB_Q(B, S)                                                                         \
  hipLaunchKernelGGL((k_quantize_mx4_rows<B, S>), grid, dim3(kMxThreads), 0, st, x, row_src, q4, \
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
  const size_t all = (size_t)n_rows * (hidden / 8);
  const dim3 grid((unsigned)((all + kMxThreads - 1) / kMxThreads));
  const uint32_t* q4 = reinterpret_cast<const uint32_t*>(q);
  if (bf16)
    hipLaunchKernelGGL(k_dequantize_mx4<true>, grid, dim3(kMxThreads), 0, st, q4, q_scale, x, all);
  else
    hipLaunchKernelGGL(k_dequantize_mx4<false>, grid, dim3(kMxThreads), 0, st, q4, q_scale, x, all);
  return hipGetLastError();
}

}  // namespace mb
