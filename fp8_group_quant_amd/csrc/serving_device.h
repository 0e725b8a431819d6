// serving_device.h — device code that the serving operators share: rounding to the model's type
// and storing.
#pragma once

#include "quant_device.h"

namespace fp8q {
namespace {

// Two fp32 values as bf16 or fp16 (nearest even), the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (DT == FP8Q_DTYPE_BF16)
    return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(a))) |
           static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(b))) << 16;
  else
    return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(a))) |
           static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(b))) << 16;
}

// 16 fp32 values rounded to the model's type (nearest even) and stored.
template <int DT>
__device__ __forceinline__ void store16(void* base, int64_t idx, const float (&v)[16]) {
  if constexpr (DT == FP8Q_DTYPE_F32) {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(base) + idx);
#pragma unroll
    for (int h = 0; h < 4; h++) p[h] = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
  } else {
    u32x4 w[2];
#pragma unroll
    for (int j = 0; j < 8; j++) w[j >> 2][j & 3] = pack16<DT>(v[2 * j], v[2 * j + 1]);
    u32x4* p = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + idx);
    p[0] = w[0];
    p[1] = w[1];
  }
}

}  // namespace
}  // namespace fp8q
