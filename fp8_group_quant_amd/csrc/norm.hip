// norm.hip — root-mean-square norm of each row, with the residual's addition before it and
// group quantization to e4m3 after it, in one pass over the data.
//
//   h = x + residual (fp32); y = (h * r) * weight with r = 1 / sqrt(mean(h^2) + eps);
//   q, s = the group quantization of y (fp8q.h, fp8q_group_quant).
//
// A row stays in registers between the sum of squares and the encode, so every input is read
// once and every output written once: 7 bytes per bf16 element with a residual (x, residual
// and its sum 2 each, the code 1). That traffic is what bounds it: 4096 x 7168 with a residual,
// 206 MB, takes 41.6 us = 4.9 TB/s, the rate of a plain copy. The arithmetic, about 13 fp32
// operations per element, shows in short rows without a residual (30011 x 576, fp16, 53 MB: 14.7
// us = 3.6 TB/s; there two of the five operations per element between h and y are for the root's and
// the products' rounding errors).
//
// h is rounded to fp32. The sum of its squares is fp32 in each lane (four sums by fma) and over the first
// lanes, and 64-bit in its last additions; the mean is 64-bit, and the factors are carried with their
// rounding errors, so that y is the exact value's own rounding but for what the sum's 32-bit parts
// leave (0.2 units). Against 64 bits 11 of 1.8e8 codes are off with UE8M0 scales (4096 x 7168; a plain fp32
// evaluation 80); with fp32 scales, whose reciprocal and its product round again, 1317 and 1508.
#include <algorithm>

#include "quant_device.h"
#include "serving.h"
#include "serving_device.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

// Reductions over the LANES (16 or 64) lanes that share a row, or a wave's part of one: the steps of
// group_max within 16 lanes, then the wave's four rows of lanes through readlane.
template <int LANE>
__device__ __forceinline__ float lane_of(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), LANE));
}
template <int LANES>
__device__ __forceinline__ float row_max_of(float v) {
  v = group_max<8>(v);
  v = fmaxf(v, dpp<0x140>(v));
  if constexpr (LANES == 16) return v;
  return fmaxf(fmaxf(lane_of<0>(v), lane_of<16>(v)), fmaxf(lane_of<32>(v), lane_of<48>(v)));
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const int2 w = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{__builtin_amdgcn_update_dpp(w.x, w.x, CTRL, 0xF, 0xF, false),
                                         __builtin_amdgcn_update_dpp(w.y, w.y, CTRL, 0xF, 0xF, false)});
}
// The last additions of a sum decide its error (that of those before averages out over the parts), so
// they are done in 64 bits: of 16 lanes the sums of four, of a wave the sums of 16.
template <int LANES>
__device__ __forceinline__ double row_sum_of(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  if constexpr (LANES == 16) {
    double s = v;
    s += dpp64<0x141>(s);
    return s + dpp64<0x140>(s);
  } else {
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    return (static_cast<double>(lane_of<0>(v)) + lane_of<16>(v)) + (static_cast<double>(lane_of<32>(v)) + lane_of<48>(v));
  }
}

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
  // two passes at a time (fp32: one), and the weight after the sum. (All at once, 36 to 116 registers
  // went to memory: 1024 x 65536 with a residual took 149 us in bf16 and 344 in fp32, now 106 and 193.)
  constexpr bool kLong = CH == 4;
  constexpr int kAhead = DT == FP8Q_DTYPE_F32 ? 1 : 2;
  constexpr int kWaves = WPR < 4 ? 4 : WPR;
  constexpr int kRows = kWaves / WPR * (64 / LANES);  // of a block
  constexpr int kPass = LANES * WPR * kPerLane;       // elements of a row that its lanes hold at a time
  __shared__ double sums[2][kWaves / WPR][WPR];  // of squares, by iteration parity
  __shared__ float maxima[2][kWaves / WPR][WPR];
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
    double ss = row_sum_of<LANES>((sq[0] + sq[1]) + (sq[2] + sq[3]));
    if constexpr (WPR > 1) {
      if (lane == 0) sums[par][wr][wi] = ss;
      __syncthreads();
      ss = sums[par][wr][lane & (WPR - 1)];  // every lane one wave's, then over WPR neighbours
      ss += dpp64<0xB1>(ss);
      if constexpr (WPR >= 4) ss += dpp64<0x4E>(ss);
      if constexpr (WPR >= 8) ss += dpp64<0x141>(ss);
      if constexpr (WPR >= 16) ss += dpp64<0x140>(ss);
    }
    // r + r_lo = 1 / sqrt(v) but for r_lo's own rounding: Newton's step from the instruction's estimate
    const double v = fma(ss, p.inv_k, static_cast<double>(p.eps));
    const float r = static_cast<float>(__builtin_amdgcn_rsq(v));
    const float left = static_cast<float>(fma(-v * r, static_cast<double>(r), 1.0));
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
      row_max = row_max_of<LANES>(row_max);
      if constexpr (WPR > 1) {
        if (lane == 0) maxima[par][wr][wi] = row_max;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPR; i++) row_max = fmaxf(row_max, maxima[par][wr][i]);
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
// 24576 in bf16: 82 us with two, 162 with four). Between 512 and 768 elements the registers decide:
// three passes fit, but for two to four registers, 16-bit rows without a residual (30000 x 768: bf16 15.6 us,
// 17.4 with a wave per row, fp16 16.0 and 18.0; fp32 28.6 and 25.2; with a residual 35.7 and 33.1).
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
