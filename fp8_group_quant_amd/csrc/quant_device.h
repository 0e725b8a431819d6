// quant_device.h — device code that the kernels with group-quantized output or input share:
// wave reductions, 16-element loads and their widening to fp32, the scale rules and the
// e4m3 / int8 encode.
//
// Compile without contraction (-ffp-contract=off) and with correctly rounded fp32 division: the
// arithmetic sequence of the scale rules is part of the ABI's contract (bit-exact results).
#pragma once

#include "fp8q_internal.h"
#include "quant_math.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kPerLane = 16;    // consecutive elements owned by one lane per chunk (32 B of bf16)
constexpr int kChunk = 64 * kPerLane;  // elements per wave-wide chunk
constexpr float kFmax = 448.0f;
constexpr float kImax = 127.0f;  // int8 output: largest code used
constexpr float kEps = 0x1.b7cdfep-34f;  // 1e-10f, the amax floor

// ------------------------------------------------------------------ wave helpers
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL,
                                                    0xF, 0xF, false));
}

// Max over the LANES (2, 4 or 8) adjacent lanes holding one group; every lane of the
// group receives the result. All 64 lanes must be active.
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));                              // quad_perm [1,0,3,2]
  if constexpr (LANES >= 4) v = fmaxf(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
  if constexpr (LANES >= 8) v = fmaxf(v, dpp<0x141>(v));   // row_half_mirror
  return v;
}

// Index of the calling wave in its block as a wave-uniform (scalar) value: the per-item row
// and address arithmetic derived from it then runs on the scalar unit, not the vector ALU.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// ------------------------------------------------------------------ element loads
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Raw storage of the 16 consecutive input elements of one lane (32 or 64 bytes).
template <int DT>
struct Raw16;
template <>
struct Raw16<FP8Q_DTYPE_BF16> { u32x4 w[2]; };
template <>
struct Raw16<FP8Q_DTYPE_F16> { u32x4 w[2]; };
template <>
struct Raw16<FP8Q_DTYPE_F32> { f32x4 w[4]; };

// 16-byte loads of adjacent addresses with the default cache policy (measured ~6% faster
// than non-temporal loads on MI355X, although the input is read once).
template <int DT>
__device__ __forceinline__ void load_raw(const void* base, int64_t idx, Raw16<DT>& r) {
  if constexpr (DT == FP8Q_DTYPE_F32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + idx);
#pragma unroll
    for (int h = 0; h < 4; h++) r.w[h] = p[h];
  } else {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + idx);
    r.w[0] = p[0];
    r.w[1] = p[1];
  }
}

template <int DT>
__device__ __forceinline__ void zero_raw(Raw16<DT>& r) {
  if constexpr (DT == FP8Q_DTYPE_F32) {
#pragma unroll
    for (int h = 0; h < 4; h++) r.w[h] = f32x4{0.f, 0.f, 0.f, 0.f};
  } else {
    r.w[0] = u32x4{0u, 0u, 0u, 0u};
    r.w[1] = r.w[0];
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float f16_lo(uint32_t w) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w & 0xFFFFu)));
}
__device__ __forceinline__ float f16_hi(uint32_t w) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
}

template <int DT>
__device__ __forceinline__ void widen(const Raw16<DT>& r, float (&v)[16]) {
  if constexpr (DT == FP8Q_DTYPE_F32) {
#pragma unroll
    for (int h = 0; h < 4; h++) {
      v[4 * h] = r.w[h].x; v[4 * h + 1] = r.w[h].y; v[4 * h + 2] = r.w[h].z; v[4 * h + 3] = r.w[h].w;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const uint32_t w = r.w[h][q];
        if constexpr (DT == FP8Q_DTYPE_BF16) {
          v[8 * h + 2 * q] = bf16_lo(w);
          v[8 * h + 2 * q + 1] = bf16_hi(w);
        } else {
          v[8 * h + 2 * q] = f16_lo(w);
          v[8 * h + 2 * q + 1] = f16_hi(w);
        }
      }
    }
  }
}

// Max over all 64 lanes, returned wave-uniform: 8-lane DPP butterfly, row_mirror for 16
// lanes, then the four 16-lane rows through readlane.
__device__ __forceinline__ float wave_max(float v) {
  v = group_max<8>(v);
  v = fmaxf(v, dpp<0x140>(v));  // row_mirror: lane i with lane 15 - i of its row
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return fmaxf(fmaxf(r0, r1), fmaxf(r2, r3));
}

// ------------------------------------------------------------------ scale rules
template <int FMT, bool I8>
__device__ __forceinline__ float group_multiplier(float amax, uint32_t& scale_bits) {
  static_assert(!I8 || FMT == FP8Q_SCALE_F32, "int8 output takes fp32 scales");
  // amax >= 1e-10 (the floor), so both divisions are in their short forms' checked domains:
  // r = amax / C, then 1 / r with r in [2e-13, 3e36] or infinite
  const float r = I8 ? div_by_const<127>(amax) : div_by_const<448>(amax);
  if constexpr (FMT == FP8Q_SCALE_UE8M0) {
    const uint32_t bits = __float_as_uint(r);
    const uint32_t ex = ((bits >> 23) & 0xFFu) + ((bits & 0x7FFFFFu) != 0u ? 1u : 0u);
    scale_bits = ex;
    return __uint_as_float((254u - ex) << 23);  // 2^(127-(ex-127)), exact
  } else {
    scale_bits = __float_as_uint(r);
    return div_short(1.0f, r);
  }
}

__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

__device__ __forceinline__ float clamp448(float v) { return fminf(fmaxf(v, -kFmax), kFmax); }

// int8: four codes (int8_code_bits: clamp to +-127, round with ties to even, code in the low
// byte), packed little-endian; v_perm_b32 gathers the low bytes (selector 0x0c: zero).
__device__ __forceinline__ uint32_t cvt4_i8(float a, float b, float c, float d) {
  const uint32_t lo = __builtin_amdgcn_perm(int8_code_bits(b), int8_code_bits(a), 0x0c0c0400u);  // a, b
  const uint32_t hi = __builtin_amdgcn_perm(int8_code_bits(d), int8_code_bits(c), 0x0c0c0400u);  // c, d
  return lo | (hi << 16);
}

// 16 values times the multiplier, as 16 output codes (e4m3 after the clamp to +-448, or
// int8)
template <bool I8>
__device__ __forceinline__ u32x4 encode16(const float (&v)[16], float inv) {
  u32x4 w;
#pragma unroll
  for (int q = 0; q < 4; q++) {
    if constexpr (I8)
      w[q] = cvt4_i8(v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv);
    else
      w[q] = cvt4(clamp448(v[4 * q] * inv), clamp448(v[4 * q + 1] * inv), clamp448(v[4 * q + 2] * inv),
                  clamp448(v[4 * q + 3] * inv));
  }
  return w;
}

}  // namespace
}  // namespace fp8q
