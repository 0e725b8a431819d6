// norm.hip — root-mean-square norm of each row, with the residual's addition before it and
// group quantization to e4m3 after it, in one pass over the data.
//
//   h = x + residual (fp32); y = (h * r) * weight with r = 1 / sqrt(mean(h^2) + eps);
//   q, s = the group quantization of y (fp8q.h, fp8q_group_quant).
//
// A row stays in registers between the sum of squares and the encode, so every input is read
// once and every output written once: 7 bytes per bf16 element with a residual (x, residual
// and its sum 2 each, the code 1). That traffic is what bounds it; the arithmetic is about 10
// fp32 operations per element. The row's sum of squares is fp32, each lane adding 16 elements
// per chunk by fma before the lanes' sums meet.
#include <algorithm>

#include "quant_device.h"
#include "serving.h"
#include "serving_device.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

// Sum over all 64 lanes, returned wave-uniform (the steps of wave_max).
__device__ __forceinline__ float wave_sum(float v) {
  v = v + dpp<0xB1>(v);
  v = v + dpp<0x4E>(v);
  v = v + dpp<0x141>(v);
  v = v + dpp<0x140>(v);
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return (r0 + r1) + (r2 + r3);
}

// WPR waves share a row, each holding CH chunks of 1024 elements (wave w: chunks w, w + WPR,
// ...). Fewer than 4 waves to a row: a block of 4 waves takes several rows.
template <int DT, int WPR, int CH>
__global__ __launch_bounds__(WPR < 4 ? 256 : 64 * WPR) void rms_norm_quant_kernel(NormParams p) {
  constexpr int kRows = WPR < 4 ? 4 / WPR : 1;
  __shared__ float part[2][2][kRows][WPR];  // by iteration parity: sums of squares, maxima
  const int lane = threadIdx.x & 63;
  const int wave = wave_index();
  const int wr = wave / WPR, wi = wave % WPR;
  int par = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows; row0 < p.M;
       row0 += static_cast<int64_t>(gridDim.x) * kRows, par ^= 1) {
    const int64_t m = row0 + wr;
    const bool live = m < p.M;  // wave-uniform
    Raw16<DT> xr[CH], rr[CH], gr[CH];
#pragma unroll
    for (int i = 0; i < CH; i++) {
      zero_raw<DT>(xr[i]);
      zero_raw<DT>(rr[i]);
      zero_raw<DT>(gr[i]);
      const int64_t k = static_cast<int64_t>(wi + WPR * i) * kChunk + lane * kPerLane;
      if (live && k < p.K) {
        load_raw<DT>(p.x, m * p.x_sm + k, xr[i]);
        if (p.res) load_raw<DT>(p.res, m * p.r_sm + k, rr[i]);
        load_raw<DT>(p.w, k, gr[i]);
      }
    }
    float h[CH][16];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      widen<DT>(xr[i], h[i]);
      if (p.res) {
        float r[16];
        widen<DT>(rr[i], r);
#pragma unroll
        for (int j = 0; j < 16; j++) h[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 16; j++) ss = fmaf(h[i][j], h[i][j], ss);
      const int64_t k = static_cast<int64_t>(wi + WPR * i) * kChunk + lane * kPerLane;
      if (p.res_out && live && k < p.K) store16<DT>(p.res_out, m * p.ro_sm + k, h[i]);
    }
    ss = wave_sum(ss);
    if constexpr (WPR > 1) {
      if (lane == 0) part[par][0][wr][wi] = ss;
      __syncthreads();
      ss = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; i++) ss += part[par][0][wr][i];
    }
    const float r = 1.0f / sqrtf(ss * p.inv_k + p.eps);
    float amax[CH], row_max = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      float g[16];
      widen<DT>(gr[i], g);
      amax[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; j++) {
        h[i][j] = (h[i][j] * r) * g[j];
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
      row_max = wave_max(row_max);
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
      const int64_t k = static_cast<int64_t>(wi + WPR * i) * kChunk + lane * kPerLane;
      uint32_t sbits;
      float inv;
      if (p.ue8m0) inv = group_multiplier<FP8Q_SCALE_UE8M0, false>(fmaxf(amax[i], kEps), sbits);
      else inv = group_multiplier<FP8Q_SCALE_F32, false>(fmaxf(amax[i], kEps), sbits);
      if (live && k < p.K) {
        *reinterpret_cast<u32x4*>(p.q + m * p.q_sm + k) = encode16<false>(h[i], inv);
        const bool first = p.group != 0 ? (k & (p.group - 1)) == 0 : k == 0;
        if (first) {
          const int64_t g = p.group != 0 ? k / p.group : 0;
          const int64_t at = p.packed ? 4 * (m * p.s_sm + (g >> 2) * p.s_sg) + (g & 3) : m * p.s_sm + g * p.s_sg;
          if (p.ue8m0) static_cast<uint8_t*>(p.s)[at] = static_cast<uint8_t>(sbits);
          else static_cast<uint32_t*>(p.s)[at] = sbits;
        }
      }
    }
  }
}

template <int DT, int WPR, int CH>
void launch_one(const NormParams& p, hipStream_t stream) {
  constexpr int rows = WPR < 4 ? 4 / WPR : 1;
  const int64_t grid = std::min<int64_t>((p.M + rows - 1) / rows, 65535);
  hipLaunchKernelGGL((rms_norm_quant_kernel<DT, WPR, CH>), dim3(static_cast<unsigned>(grid)),
                     dim3(WPR < 4 ? 256 : 64 * WPR), 0, stream, p);
}

// Waves per row by the row's length.
template <int DT>
void launch_dt(const NormParams& p, hipStream_t s) {
  const int64_t chunks = (p.K + kChunk - 1) / kChunk;
  if (chunks <= 1) launch_one<DT, 1, 1>(p, s);
  else if (chunks <= 2) launch_one<DT, 2, 1>(p, s);
  else if (chunks <= 4) launch_one<DT, 4, 1>(p, s);
  else if (chunks <= 8) launch_one<DT, 4, 2>(p, s);
  else if (chunks <= 16) launch_one<DT, 8, 2>(p, s);
  else launch_one<DT, 16, 4>(p, s);
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
