// norm.hip — root-mean-square norm of each row, with the residual's addition before it and
// group quantization to e4m3 after it, in one pass over the data.
//
//   h = x + residual (fp32); y = (h * r) * weight with r = 1 / sqrt(mean(h^2) + eps);
//   q, s = the group quantization of y (fp8q.h, fp8q_group_quant).
//
// A row stays in registers between the sum of squares and the encode, so every input is read
// once and every output written once: 7 bytes per bf16 element with a residual (x, residual
// and its sum 2 each, the code 1). That traffic is what bounds it: 4096 x 7168 with a residual,
// 206 MB, takes 41.4 us = 5.0 TB/s, the rate of a plain copy. The arithmetic, about 13 fp32
// operations per element, shows in short rows without a residual (30011 x 576, fp16, 53 MB: 14.3
// us = 3.7 TB/s). The row's sum of squares is fp32: four sums per lane by fma, then a tree. The
// factors are carried with their rounding errors, so that y has one rounding to fp32: of the codes
// that a plain fp32 evaluation rounds to a neighbour's side of a tie, half are then right.
#include <algorithm>

#include "quant_device.h"
#include "serving.h"
#include "serving_device.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

// Reductions over the LANES (16 or 64) lanes that share a row, or a wave's part of one: the steps
// of group_max within 16 lanes, then the wave's four rows of lanes through readlane.
template <int LANES, typename F>
__device__ __forceinline__ float row_reduce(float v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  if constexpr (LANES == 16) return v;
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return f(f(r0, r1), f(r2, r3));
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }

// 16 values times their groups' multiplier as e4m3 codes. Nothing is clamped: the scale is amax / 448
// or more up to its rounding and the multiplier's, so a product stays below 448 * (1 + 2^-21),
// which rounds to 448 (from 464 on it would not).
__device__ __forceinline__ u32x4 encode16_below448(const float (&v)[16], float inv) {
  u32x4 w;
#pragma unroll
  for (int q = 0; q < 4; q++)
    w[q] = cvt4(v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv);
  return w;
}

// LANES lanes of each of WPR waves share a row (64, or 16 of one wave), each lane holding CH times
// 16 elements: lane and wave i take the elements [16 i, 16 i + 16) of every 16 * LANES * WPR.
// Waves per SIMD that the registers are kept to: one register more than four waves have would cost a
// quarter of the loads in flight (30011 x 576, fp16: 16.7 us).
constexpr int norm_waves(int CH) { return CH == 3 ? 4 : 1; }

template <int DT, int LANES, int WPR, int CH>
__global__ __launch_bounds__(WPR < 4 ? 256 : 64 * WPR, norm_waves(CH)) void rms_norm_quant_kernel(NormParams p) {
  static_assert(LANES == 64 || WPR == 1, "a row of 16 lanes is one wave's");
  // 64 values of h leave no registers for the other inputs of all passes: x and the residual come in for
  // two passes at a time, and the weight after the sum. (All at once, 36 to 116 registers went to
  // scratch: 1024 x 65536 with a residual took 149 us in bf16 and 344 in fp32, now 107 and 195.)
  constexpr bool kLong = CH == 4;
  constexpr int kAhead = 2;
  constexpr int kWaves = WPR < 4 ? 4 : WPR;
  constexpr int kRows = kWaves / WPR * (64 / LANES);  // of a block
  constexpr int kPass = LANES * WPR * kPerLane;       // elements of a row that its lanes hold at a time
  __shared__ float part[2][2][kWaves / WPR][WPR];  // by iteration parity: sums of squares, maxima
  const int lane = threadIdx.x & 63;
  const int wave = wave_index();
  const int wr = wave / WPR, wi = wave % WPR;
  const int at = (LANES == 64 ? wi * 64 + lane : lane & 15) * kPerLane;
  int par = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows; row0 < p.M;
       row0 += static_cast<int64_t>(gridDim.x) * kRows, par ^= 1) {
    const int64_t m = row0 + (LANES == 64 ? wr : wave * 4 + (lane >> 4));
    const bool live = m < p.M;
    Raw16<DT> xr[CH], rr[CH], gr[CH];
    auto load = [&](int i, bool with_weight) {
      zero_raw<DT>(xr[i]);
      zero_raw<DT>(rr[i]);
      if (with_weight) zero_raw<DT>(gr[i]);
      const int32_t k = at + kPass * i;
      if (live && k < p.K) {
        load_raw<DT>(p.x, m * p.x_sm + k, xr[i]);
        if (p.res) load_raw<DT>(p.res, m * p.r_sm + k, rr[i]);
        if (with_weight) load_raw<DT>(p.w, k, gr[i]);
      }
    };
    if constexpr (!kLong) {
#pragma unroll
      for (int i = 0; i < CH; i++) load(i, true);
    }
    float h[CH][16];
    float sq[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < CH; i++) {
      if constexpr (kLong) {
        if (i % kAhead == 0) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int a = 0; a < kAhead; a++) load(i + a, false);
        }
      }
      widen<DT>(xr[i], h[i]);
      if (p.res) {
        float r[16];
        widen<DT>(rr[i], r);
#pragma unroll
        for (int j = 0; j < 16; j++) h[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 16; j++) sq[j & 3] = fmaf(h[i][j], h[i][j], sq[j & 3]);
      const int32_t k = at + kPass * i;
      if (p.res_out && live && k < p.K) store16<DT>(p.res_out, m * p.ro_sm + k, h[i]);
    }
    float ss = row_reduce<LANES>((sq[0] + sq[1]) + (sq[2] + sq[3]), add);
    if constexpr (WPR > 1) {
      if (lane == 0) part[par][0][wr][wi] = ss;
      __syncthreads();
      float s[WPR];
#pragma unroll
      for (int i = 0; i < WPR; i++) s[i] = part[par][0][wr][i];
#pragma unroll
      for (int n = WPR / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; i++) s[i] += s[i + n];
      ss = s[0];
    }
    // r + r_lo = 1 / sqrt(v) but for r_lo's own rounding (Newton's step, its residual by fma)
    const float v = ss / p.k + p.eps, r = 1.0f / sqrtf(v), vr = v * r;
    const float left = fmaf(-vr, r, 1.0f) - fmaf(v, r, -vr) * r;
    const float r_lo = fabsf(left) < 1.0f ? 0.5f * r * left : 0.0f;  // v of 0 or infinity: no residual
    float amax[CH], row_max = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      float g[16];
      if constexpr (kLong) {
        __builtin_amdgcn_sched_barrier(0);
        zero_raw<DT>(gr[i]);
        if (live && at + kPass * i < p.K) load_raw<DT>(p.w, at + kPass * i, gr[i]);
      }
      widen<DT>(gr[i], g);
      amax[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; j++) {
        const float hr = h[i][j] * r, hr_lo = fmaf(h[i][j], r_lo, fmaf(h[i][j], r, -hr));
        h[i][j] = fmaf(hr, g[j], hr_lo * g[j]);
        amax[i] = fmaxf(amax[i], fabsf(h[i][j]));
      }
      if (p.group != 0) {
        amax[i] = group_max<2>(amax[i]);
        if (p.group >= 64) amax[i] = fmaxf(amax[i], dpp<0x4E>(amax[i]));
        if (p.group >= 128) amax[i] = fmaxf(amax[i], dpp<0x141>(amax[i]));
      } else {
        row_max = fmaxf(row_max, amax[i]);
      }
    }
    if (p.group == 0) {  // one group per row
      row_max = row_reduce<LANES>(row_max, larger);
      if constexpr (WPR > 1) {
        if (lane == 0) part[par][1][wr][wi] = row_max;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPR; i++) row_max = fmaxf(row_max, part[par][1][wr][i]);
      }
#pragma unroll
      for (int i = 0; i < CH; i++) amax[i] = row_max;
    }
#pragma unroll
    for (int i = 0; i < CH; i++) {
      int32_t k = at + kPass * i;
      if constexpr (kLong) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+v"(k));  // the passes' scale addresses are not worth registers across the rows
      }
      uint32_t sbits;
      float inv;
      if (p.ue8m0) inv = group_multiplier<FP8Q_SCALE_UE8M0, false>(fmaxf(amax[i], kEps), sbits);
      else inv = group_multiplier<FP8Q_SCALE_F32, false>(fmaxf(amax[i], kEps), sbits);
      if (live && k < p.K) {
        *reinterpret_cast<u32x4*>(p.q + m * p.q_sm + k) = encode16_below448(h[i], inv);
        // the group's first lane stores its scale
        if (p.group != 0 ? (k & (p.group - 1)) == 0 : k == 0) {
          const int32_t g = k >> p.group_shift;
          const int64_t to = p.packed ? 4 * (m * p.s_sm + (g >> 2) * p.s_sg) + (g & 3) : m * p.s_sm + g * p.s_sg;
          if (p.ue8m0) static_cast<uint8_t*>(p.s)[to] = static_cast<uint8_t>(sbits);
          else static_cast<uint32_t*>(p.s)[to] = sbits;
        }
      }
    }
  }
}

template <int DT, int LANES, int WPR, int CH>
void launch_one(const NormParams& p, hipStream_t stream) {
  constexpr int rows = (WPR < 4 ? 4 / WPR : 1) * (64 / LANES);
  const int64_t grid = std::min<int64_t>((p.M + rows - 1) / rows, 65535);
  hipLaunchKernelGGL((rms_norm_quant_kernel<DT, LANES, WPR, CH>), dim3(static_cast<unsigned>(grid)),
                     dim3(WPR < 4 ? 256 : 64 * WPR), 0, stream, p);
}

// Lanes per row by its length: short rows share a wave, four to one (each lane's fixed work, about
// 60 instructions for sums and scales, then serves up to 48 elements: 60000 x 256 takes 22.0 us,
// 38 us with a wave per row); longer ones have 16 elements per lane and as many waves as that
// takes, which is the most loads in flight (4096 x 7168: 8 waves 41.8 us, 4 waves of 32 elements
// 42.7; one row of 7168: 3.3 and 3.7 us), up to a block's 16, and then two or four passes of them (2048 x
// 24576 in bf16: 83 us with two, 162 with four, which held them all). Between 512 and 768 elements the registers decide: three
// passes fit where there is no residual and 16-bit rows (30000 x 768: 16.9 us, 19.7 with a wave per
// row; fp32 28.6 and 25.2; with a residual 35.7 and 33.1).
template <int DT>
void launch_dt(const NormParams& p, hipStream_t s) {
  if constexpr (DT != FP8Q_DTYPE_F32) {
    if (p.K > 512 && p.K <= 768 && !p.res) return launch_one<DT, 16, 1, 3>(p, s);
  }
  if (p.K <= 256) launch_one<DT, 16, 1, 1>(p, s);
  else if (p.K <= 512) launch_one<DT, 16, 1, 2>(p, s);
  else if (p.K <= 1024) launch_one<DT, 64, 1, 1>(p, s);
  else if (p.K <= 2048) launch_one<DT, 64, 2, 1>(p, s);
  else if (p.K <= 4096) launch_one<DT, 64, 4, 1>(p, s);
  else if (p.K <= 8192) launch_one<DT, 64, 8, 1>(p, s);
  else if (p.K <= 16384) launch_one<DT, 64, 16, 1>(p, s);
  else if (p.K <= 32768) launch_one<DT, 64, 16, 2>(p, s);
  else launch_one<DT, 64, 16, 4>(p, s);
}

}  // namespace

int launch_rms_norm_quant(int dtype, const NormParams& p, hipStream_t stream) {
  switch (dtype) {
    case FP8Q_DTYPE_BF16: launch_dt<FP8Q_DTYPE_BF16>(p, stream); break;
    case FP8Q_DTYPE_F16: launch_dt<FP8Q_DTYPE_F16>(p, stream); break;
    default: launch_dt<FP8Q_DTYPE_F32>(p, stream); break;
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("rms norm launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace fp8q
