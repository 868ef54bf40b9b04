// rowio.h — 8-element lane chunks of fp32 / bf16 rows and conversions shared
// by the norm and the 4-bit row kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mb {

// Two fp32 values to packed bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  const bf16x2 o = __builtin_convertvector(v, bf16x2);
  uint32_t u;
  __builtin_memcpy(&u, &o, 4);
  return u;
}

// v[0..8) = elements [8c, 8c + 8) of p.
template <bool kBF16>
__device__ __forceinline__ void load8(const void* p, size_t c, float* v) {
  if constexpr (kBF16) {
    const uint4 u = static_cast<const uint4*>(p)[c];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = static_cast<const float4*>(p)[2 * c], b = static_cast<const float4*>(p)[2 * c + 1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// Nontemporal: rows leave for memory (8192 x 7168 bf16 rows read back from
// 4 bits: 46-47 us with the quantisation before it, 50-51 with plain stores; the
// norm of 131072 such rows 2 % faster).
template <bool kBF16>
__device__ __forceinline__ void store8(void* p, size_t c, const float* v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  if constexpr (kBF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2_rne(v[2 * i], v[2 * i + 1]);
    __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, static_cast<u32x4*>(p) + c);
  } else {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, static_cast<f32x4*>(p) + 2 * c);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, static_cast<f32x4*>(p) + 2 * c + 1);
  }
}

// Four values as e4m3fn bytes, round to nearest even. A quotient may pass 448
// by its own rounding and its divisor's, never by half a step (16): no overflow.
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  const int o = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, o, true);
}

}  // namespace mb
