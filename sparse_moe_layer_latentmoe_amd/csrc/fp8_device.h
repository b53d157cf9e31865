// Device-side pieces of the 8-bit floating-point (e4m3) kernels.
#pragma once
#include "lmoe_device.h"

namespace lmoe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kE4M3Max = 448.f;

__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// D(16x16, fp32) = A(16x128, e4m3) * B(128x16, e4m3) from a zero accumulator.
// Lane l supplies row l%16 of A and column l%16 of B, 32 k each (which ones
// does not matter as long as both agree); result layout as mfma_bf16's.
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                          0, 0, 0);
}

// The same product with each operand converted to bf16 (exactly): the sum is
// then an fp32 sum, at half the rate.  The 8-bit instruction adds the products
// of each eight neighbouring k after cutting them to multiples of 2^(E - 13), E
// the largest sum of two codes' exponents among the eight (subnormal codes and
// zeros: -6), and the sixteen sums in about 24 bits: off by less than
// 7 2^(E - 13) for each eight (measured, up to 0.56 of that).  Of the sum of the
// products' magnitudes that is 2^-15.9 on normally distributed blocks of 128,
// 2^-11.4 on exp(2 n) with normal n and 2^-10 on exp(6 n), against 2^-25.4 here.
struct Bf16Frag {
  bf16x8 v[4];
};
__device__ __forceinline__ Bf16Frag fp8_to_bf16(i32x8 a) {
  Bf16Frag r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)a[i], 1.f, false);
    const auto hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)a[i], 1.f, true);
    r.v[i >> 1][4 * (i & 1)] = lo[0];
    r.v[i >> 1][4 * (i & 1) + 1] = lo[1];
    r.v[i >> 1][4 * (i & 1) + 2] = hi[0];
    r.v[i >> 1][4 * (i & 1) + 3] = hi[1];
  }
  return r;
}
__device__ __forceinline__ f32x4 mfma_fp8(const Bf16Frag& a, const Bf16Frag& b) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma_bf16(a.v[i], b.v[i], c);
  return c;
}

// Four values within [-448, 448] (up to rounding) as e4m3 codes, lowest byte
// first, rounded to nearest, ties to even.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return (uint32_t)v;
}

// A raw buffer over `bytes` from `base` (at most 2 GiB of them).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0,
                                           (int)(bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0),
                                           0x00020000);
}

}  // namespace lmoe
