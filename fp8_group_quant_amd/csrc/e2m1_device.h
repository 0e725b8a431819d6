// e2m1_device.h — code that the kernels which write or read 4-bit rows share: the scale rule, encoding and
// decoding 8 elements of a lane, and division by a size that the host knows.
//
// e2m1 codes: sign, 2 exponent and 1 mantissa bits (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), the even
// element in the low half of a byte.
#pragma once

#include "serving_device.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kEl = 8;  // elements of a lane, a quarter of a scale block
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Division of u < 2^30 by a constant d: (mulhi(u, mul) + u) >> shift with shift = ceil(log2 d)
// and mul = floor(2^32 (2^shift - d) / d) + 1 (Granlund and Montgomery, "Division by invariant
// integers using multiplication", PLDI'94).
struct Divider {
  uint32_t mul, shift;
};
Divider divider(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) s++;
  return Divider{static_cast<uint32_t>((((uint64_t(1) << s) - d) << 32) / d + 1), s};
}
__device__ __forceinline__ uint32_t divide(uint32_t u, Divider d) { return (__umulhi(u, d.mul) + u) >> d.shift; }

// Biased exponent of the smallest power of two >= amax / 6 for a normal amax = m * 2^e with m
// in [1, 2): 6 * 2^(e - 2) = 1.5 * 2^e reaches amax when m <= 1.5, else one exponent more.
__device__ __forceinline__ uint32_t e2m1_scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  return (bits >> 23) - 2u + ((bits & 0x7FFFFFu) > 0x400000u ? 1u : 0u);
}

// The 8 elements of a lane, as stored.
template <int DT>
struct Raw8 {
  u32x4 w[DT == FP8Q_DTYPE_F32 ? 2 : 1];
};

// Largest magnitude of the 8. bf16 and fp16 magnitudes order like their bits.
template <int DT>
__device__ __forceinline__ float amax8(const Raw8<DT>& r) {
  if constexpr (DT == FP8Q_DTYPE_F32) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) a = fmaxf(a, fabsf(__uint_as_float(r.w[i >> 2][i & 3])));
    return a;
  } else {
    u16x2 a = __builtin_bit_cast(u16x2, r.w[0][0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; i++)
      a = __builtin_elementwise_max(a, __builtin_bit_cast(u16x2, r.w[0][i] & 0x7FFF7FFFu));
    const uint32_t top = max(static_cast<uint32_t>(a[0]), static_cast<uint32_t>(a[1]));
    return DT == FP8Q_DTYPE_BF16 ? bf16_lo(top) : f16_lo(top);
  }
}

// A word as a pair of 16-bit floats. (A function: a bit cast of a vector's element itself takes
// the vector's first one.)
template <typename T>
__device__ __forceinline__ T pair(uint32_t w) { return __builtin_bit_cast(T, w); }

// The 8 codes at this scale.
template <int DT>
__device__ __forceinline__ uint32_t encode8(const Raw8<DT>& r, float scale) {
  uint32_t c = 0;
  if constexpr (DT == FP8Q_DTYPE_BF16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair<bf16x2>(r.w[0][0]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair<bf16x2>(r.w[0][1]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair<bf16x2>(r.w[0][2]), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair<bf16x2>(r.w[0][3]), scale, 3);
  } else if constexpr (DT == FP8Q_DTYPE_F16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, pair<f16x2>(r.w[0][0]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, pair<f16x2>(r.w[0][1]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, pair<f16x2>(r.w[0][2]), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, pair<f16x2>(r.w[0][3]), scale, 3);
  } else {
    auto f = [&](int i) { return __uint_as_float(r.w[i >> 2][i & 3]); };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(0), f(1), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(2), f(3), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(4), f(5), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(6), f(7), scale, 3);
  }
  return c;
}

// Whether 6, the largest code, at this scale byte passes the type's largest finite value. (255 is no
// scale: its values are NaN, and stay so.)
template <int DT>
__device__ __forceinline__ bool may_overflow(uint32_t byte) {
  constexpr uint32_t kFirst = DT == FP8Q_DTYPE_F16 ? 127 + 14 : 127 + 126;
  return byte - kFirst < 255u - kFirst;
}

// The values of 8 codes, those past the type's largest finite value as that value. Else exact in bf16
// and fp32; fp16 is rounded from the exact value.
template <int DT>
__device__ __forceinline__ Raw8<DT> decode8(uint32_t c, uint32_t byte) {
  const float scale = __uint_as_float(byte << 23);
  Raw8<DT> r;
  if constexpr (DT == FP8Q_DTYPE_BF16) {
    r.w[0][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
    r.w[0][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
    r.w[0][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
    r.w[0][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
    if (may_overflow<DT>(byte)) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const u16x2 mag = __builtin_elementwise_min(pair<u16x2>(r.w[0][i] & 0x7FFF7FFFu), u16x2{0x7F7F, 0x7F7F});
        r.w[0][i] = (r.w[0][i] & 0x80008000u) | __builtin_bit_cast(uint32_t, mag);
      }
    }
  } else {
    f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1),
                  __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3)};
    if (may_overflow<DT>(byte)) {
      constexpr float kMost = DT == FP8Q_DTYPE_F16 ? 65504.0f : __FLT_MAX__;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[i].x = fminf(fmaxf(v[i].x, -kMost), kMost);
        v[i].y = fminf(fmaxf(v[i].y, -kMost), kMost);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (DT == FP8Q_DTYPE_F16) {
        r.w[0][i] = pack16<DT>(v[i].x, v[i].y);
      } else {
        r.w[i >> 1][2 * (i & 1)] = __float_as_uint(v[i].x);
        r.w[i >> 1][2 * (i & 1) + 1] = __float_as_uint(v[i].y);
      }
    }
  }
  return r;
}

}  // namespace
}  // namespace fp8q
