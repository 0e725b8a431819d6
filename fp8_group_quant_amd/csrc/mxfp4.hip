// mxfp4.hip — rows as e2m1 codes with one UE8M0 byte per 32 elements (the operands of the 4-bit product),
// with silu(gate) * up before it on request, and such codes back as rows.
//
//   amax = max(max |x_i|, 1e-10) over 32 elements; 2^(byte - 127) = smallest power of two >= amax / 6;
//   code_i = e2m1_nearest_even( x_i / 2^(byte - 127) )
// The division is exact and no element saturates, so the rounding to e2m1 is the only one (silu * up is fp32).
//
// Both directions are bound by HBM traffic: 2 bytes per element on the model's side (bf16), 0.53 on the
// codes'. A lane owns 8 consecutive elements: 16 bytes per access next to the neighbour's, and a block's four
// lanes are a quad. The quantizer's lanes take one row each (2, 4 and 8 rows to a lane: 0 to 2, 1 to 12 and 2 to 20 %
// slower); the way back, whose loads are small, takes four where that still fills the device (1 row to a lane: 2 to 5 %
// slower on large tensors).
//
// us, bf16 in one launch, and bytes moved per second: 4096 x 7168 quantized 17.5 (4.2 TB/s) and back 13.9 (5.3); fp16
// gate | up 6007 x 2 x 2080 15 (3.8) and back 6.4 (4.9, mostly within the caches).
#include <algorithm>

#include "e2m1_device.h"
#include "mxfp4.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kThreads = 256;

// Inputs above the L2s' 32 MB are loaded past them, so that they do not push out the codes: 4096 x 7168 in bf16 1.0
// us less, 6007 x 2 x 2080 in fp16 1.8; 2048 x 4096, which the L2s may hold, would take 0.9 more.
constexpr int64_t kStreamed = int64_t(32) << 20;

struct Grid {
  uint32_t units, per;  // lanes with work; those of one group of rows
  Divider by_per;
};

template <int DT, bool STREAMED>
__device__ __forceinline__ Raw8<DT> load8(const uint8_t* p) {
  Raw8<DT> r;
#pragma unroll
  for (int j = 0; j < (DT == FP8Q_DTYPE_F32 ? 2 : 1); j++) {
    const u32x4* w = reinterpret_cast<const u32x4*>(p) + j;
    r.w[j] = STREAMED ? __builtin_nontemporal_load(w) : *w;
  }
  return r;
}

template <int DT>
__device__ __forceinline__ float element(const Raw8<DT>& r, int i) {
  if constexpr (DT == FP8Q_DTYPE_F32) return __uint_as_float(r.w[i >> 2][i & 3]);
  else if constexpr (DT == FP8Q_DTYPE_BF16) return i & 1 ? bf16_hi(r.w[0][i >> 1]) : bf16_lo(r.w[0][i >> 1]);
  else return i & 1 ? f16_hi(r.w[0][i >> 1]) : f16_lo(r.w[0][i >> 1]);
}

// silu(gate) * up in fp32, by the fixed exponential and the short division of the FP8 quantizer.
template <int DT>
__device__ __forceinline__ Raw8<FP8Q_DTYPE_F32> silu_mul8(const Raw8<DT>& gate, const Raw8<DT>& up) {
  Raw8<FP8Q_DTYPE_F32> y;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float g = element<DT>(gate, i);
    y.w[i >> 2][i & 3] = __float_as_uint(div_short(g, 1.0f + exp_fixed(-g)) * element<DT>(up, i));
  }
  return y;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, 0xF, 0xF, false));
}

template <int DT, bool SILU, bool STREAMED>
__global__ __launch_bounds__(kThreads) void mxfp4_quant_kernel(Mxfp4RowsParams p, Grid g) {
  constexpr int kEsz = DT == FP8Q_DTYPE_F32 ? 4 : 2;
  constexpr int kIn = SILU ? FP8Q_DTYPE_F32 : DT;  // what is encoded
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= g.units) return;  // (whole quads, and with packed scales whole rows of 16 lanes)
  const uint32_t row32 = divide(u, g.by_per);
  const int64_t row = row32, k = static_cast<int64_t>(u - row32 * g.per) * kEl;
  const uint8_t* x = static_cast<const uint8_t*>(p.x) + (row * p.x_sm + k) * kEsz;
  Raw8<kIn> v;
  if constexpr (SILU) v = silu_mul8<DT>(load8<DT, STREAMED>(x), load8<DT, STREAMED>(x + p.K * kEsz));
  else v = load8<DT, STREAMED>(x);
  // a scale block's four lanes are a quad
  float amax = amax8<kIn>(v);
  amax = fmaxf(amax, dpp<0xB1>(amax));
  amax = fmaxf(amax, dpp<0x4E>(amax));
  const uint32_t byte = e2m1_scale_byte(fmaxf(amax, kEps));
  *reinterpret_cast<uint32_t*>(p.q + row * p.q_sm + k / 2) = encode8<kIn>(v, __uint_as_float(byte << 23));
  if (p.packed) {  // the bytes of 16 lanes' four blocks
    uint32_t word = byte << (k & 96) / 4;
    word |= dpp_u32<0x124>(word);  // row_ror:4
    word |= dpp_u32<0x128>(word);  // row_ror:8
    if ((k & 127) == 0) reinterpret_cast<uint32_t*>(p.s)[row * p.s_sm + k / 128 * p.s_sg] = word;
  } else if ((k & 31) == 0) {
    p.s[row * p.s_sm + k / kMxBlock * p.s_sg] = static_cast<uint8_t>(byte);
  }
}

template <int DT, int ROWS>
__global__ __launch_bounds__(kThreads) void mxfp4_dequant_kernel(Mxfp4RowsParams p, Grid g) {
  constexpr int kEsz = DT == FP8Q_DTYPE_F32 ? 4 : 2;
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= g.units) return;
  const uint32_t group = divide(u, g.by_per);
  const int64_t row = static_cast<int64_t>(group) * ROWS, k = static_cast<int64_t>(u - group * g.per) * kEl;
  const int64_t blk = k / kMxBlock;
  uint32_t c[ROWS], byte[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    const int64_t r = min(row + i, p.M - 1);
    c[i] = *reinterpret_cast<const uint32_t*>(p.q + r * p.q_sm + k / 2);
    byte[i] = p.s[p.packed ? 4 * (r * p.s_sm + blk / 4 * p.s_sg) + blk % 4 : r * p.s_sm + blk * p.s_sg];
  }
  uint8_t* x = static_cast<uint8_t*>(p.x) + (row * p.x_sm + k) * kEsz;
#pragma unroll
  for (int i = 0; i < ROWS; i++) {
    const Raw8<DT> r = decode8<DT>(c[i], byte[i]);
    if (row + i >= p.M) return;
#pragma unroll
    for (int j = 0; j < kEsz / 2; j++) reinterpret_cast<u32x4*>(x + i * p.x_sm * kEsz)[j] = r.w[j];
  }
}

// Calls `one` with row ranges whose lanes count at most 2^30.
template <typename F>
void by_ranges(const Mxfp4RowsParams& p, int rows, int esz, F one) {
  const int64_t per = p.K / kEl;
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / per) * rows;
  for (int64_t m = 0; m < p.M; m += most) {
    Mxfp4RowsParams r = p;
    r.M = std::min(most, p.M - m);
    r.x = static_cast<uint8_t*>(p.x) + m * p.x_sm * esz;
    r.q = p.q + m * p.q_sm;
    r.s = p.s + m * p.s_sm * (p.packed ? 4 : 1);
    const Grid g{static_cast<uint32_t>((r.M + rows - 1) / rows * per), static_cast<uint32_t>(per),
                 divider(static_cast<uint32_t>(per))};
    one(r, dim3((g.units + kThreads - 1) / kThreads), g);
  }
}

template <int DT, bool SILU, bool STREAMED>
void quant(const Mxfp4RowsParams& p, hipStream_t stream) {
  by_ranges(p, 1, DT == FP8Q_DTYPE_F32 ? 4 : 2, [&](const Mxfp4RowsParams& r, dim3 grid, const Grid& g) {
    hipLaunchKernelGGL((mxfp4_quant_kernel<DT, SILU, STREAMED>), grid, dim3(kThreads), 0, stream, r, g);
  });
}
template <int DT, int ROWS>
void dequant(const Mxfp4RowsParams& p, hipStream_t stream) {
  by_ranges(p, ROWS, DT == FP8Q_DTYPE_F32 ? 4 : 2, [&](const Mxfp4RowsParams& r, dim3 grid, const Grid& g) {
    hipLaunchKernelGGL((mxfp4_dequant_kernel<DT, ROWS>), grid, dim3(kThreads), 0, stream, r, g);
  });
}

template <int DT>
void quant_any(bool silu, const Mxfp4RowsParams& p, hipStream_t stream) {
  const bool streamed = p.M > kStreamed / (p.K * (silu ? 2 : 1) * (DT == FP8Q_DTYPE_F32 ? 4 : 2));
  if (silu) streamed ? quant<DT, true, true>(p, stream) : quant<DT, true, false>(p, stream);
  else streamed ? quant<DT, false, true>(p, stream) : quant<DT, false, false>(p, stream);
}
// Four rows to a lane where that still gives every CU two blocks.
template <int DT>
void dequant_any(const Mxfp4RowsParams& p, hipStream_t stream) {
  const bool tall = p.M >= 4 && p.M / 4 * (p.K / kEl) >= int64_t(2) * kThreads * current_device_shape().cus;
  tall ? dequant<DT, 4>(p, stream) : dequant<DT, 1>(p, stream);
}

int finish(const char* what) {
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string(what) + " launch: " + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace

int launch_mxfp4_quant(int dtype, bool silu, const Mxfp4RowsParams& p, hipStream_t stream) {
  switch (dtype) {
    case FP8Q_DTYPE_BF16: quant_any<FP8Q_DTYPE_BF16>(silu, p, stream); break;
    case FP8Q_DTYPE_F16: quant_any<FP8Q_DTYPE_F16>(silu, p, stream); break;
    default: quant_any<FP8Q_DTYPE_F32>(silu, p, stream); break;
  }
  return finish("mxfp4 quantization");
}

int launch_mxfp4_dequant(int dtype, const Mxfp4RowsParams& p, hipStream_t stream) {
  switch (dtype) {
    case FP8Q_DTYPE_BF16: dequant_any<FP8Q_DTYPE_BF16>(p, stream); break;
    case FP8Q_DTYPE_F16: dequant_any<FP8Q_DTYPE_F16>(p, stream); break;
    default: dequant_any<FP8Q_DTYPE_F32>(p, stream); break;
  }
  return finish("mxfp4 dequantization");
}

}  // namespace fp8q
