// kv4.hip — writing rows into a paged cache of 4-bit codes, and reading them back.
//
// A row of D elements (one token's key or value of one head) is held as D / 2 bytes of e2m1
// codes (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; element 2i in the low half of byte i) and one
// UE8M0 byte per 32 elements: the group rule of the FP8 quantizer with 6 in the place of 448.
// The scale is a power of two and at least amax / 6, so the division by it is exact and no
// element saturates: the rounding to e2m1 (nearest, ties to even) is the only one.
//
// Both directions are bound by HBM traffic: 2 bytes per element on the model's side (bf16),
// 0.53 on the cache's. A lane owns 16 consecutive elements (half a scale block).
#include <algorithm>

#include "quant_device.h"
#include "serving.h"
#include "serving_device.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kThreads = 256;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Biased exponent of the smallest power of two >= amax / 6 for a normal amax = m * 2^e with m
// in [1, 2): 6 * 2^(e - 2) = 1.5 * 2^e reaches amax when m <= 1.5, else one exponent more.
__device__ __forceinline__ uint32_t e2m1_scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  return (bits >> 23) - 2u + ((bits & 0x7FFFFFu) > 0x400000u ? 1u : 0u);
}

// Byte offset of row (slot, head) in a cached tensor; slot is in [0, pages << page_shift).
__device__ __forceinline__ int64_t row_at(const Kv4Cache& c, int32_t slot, int32_t head, int64_t sp, int64_t st,
                                          int64_t sh) {
  const int32_t page = slot >> c.page_shift, tok = slot & ((1 << c.page_shift) - 1);
  return page * sp + tok * st + head * sh;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void kv4_write_kernel(Kv4RowsParams p, uint32_t units, uint32_t per_token) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;  // 16 elements of one row
  const int which = blockIdx.y;                            // keys, values
  if (u >= units) return;
  const uint32_t t = u / per_token, rest = u - t * per_token;
  const int32_t el = static_cast<int32_t>(rest) * kPerLane;
  const int32_t head = el / p.D, d = el - head * p.D;
  const int32_t slot = p.slots[t];
  // slots outside the cache (a padding token's -1) are skipped; both lanes of a block agree
  if (slot < 0 || slot >= (p.c.pages << p.c.page_shift)) return;
  Raw16<DT> raw;
  load_raw<DT>(p.x[which], t * p.x_st[which] + head * p.x_sh[which] + d, raw);
  float v[16];
  widen<DT>(raw, v);
  float amax = kEps;
#pragma unroll
  for (int j = 0; j < 16; j++) amax = fmaxf(amax, fabsf(v[j]));
  amax = fmaxf(amax, dpp<0xB1>(amax));  // the block's other half
  const uint32_t byte = e2m1_scale_byte(amax);
  const float scale = __uint_as_float(byte << 23);
  u32x2 w = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 2; j++) {
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], v[8 * j], v[8 * j + 1], scale, 0);
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], v[8 * j + 2], v[8 * j + 3], scale, 1);
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], v[8 * j + 4], v[8 * j + 5], scale, 2);
    w[j] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[j], v[8 * j + 6], v[8 * j + 7], scale, 3);
  }
  uint8_t* codes = (which ? p.c.v : p.c.k) + row_at(p.c, slot, head, p.c.c_sp, p.c.c_st, p.c.c_sh);
  *reinterpret_cast<u32x2*>(codes + d / 2) = w;
  if ((d & 16) == 0) {
    uint8_t* scales = (which ? p.c.vs : p.c.ks) + row_at(p.c, slot, head, p.c.s_sp, p.c.s_st, p.c.s_sh);
    scales[d / kKv4Block] = static_cast<uint8_t>(byte);
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4RowsParams p, uint32_t units, uint32_t per_token) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  const int which = blockIdx.y;
  if (u >= units) return;
  const uint32_t t = u / per_token, rest = u - t * per_token;
  const int32_t el = static_cast<int32_t>(rest) * kPerLane;
  const int32_t head = el / p.D, d = el - head * p.D;
  const int32_t slot = p.slots[t];
  float v[16];
  if (slot < 0 || slot >= (p.c.pages << p.c.page_shift)) {  // no such row: zeros
#pragma unroll
    for (int j = 0; j < 16; j++) v[j] = 0.0f;
  } else {
    const uint8_t* codes = (which ? p.c.v : p.c.k) + row_at(p.c, slot, head, p.c.c_sp, p.c.c_st, p.c.c_sh);
    const uint8_t* scales = (which ? p.c.vs : p.c.ks) + row_at(p.c, slot, head, p.c.s_sp, p.c.s_st, p.c.s_sh);
    const u32x2 w = *reinterpret_cast<const u32x2*>(codes + d / 2);
    const float scale = __uint_as_float(static_cast<uint32_t>(scales[d / kKv4Block]) << 23);
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], scale, 0);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], scale, 1);
      const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], scale, 2);
      const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], scale, 3);
      v[8 * j] = a.x; v[8 * j + 1] = a.y; v[8 * j + 2] = b.x; v[8 * j + 3] = b.y;
      v[8 * j + 4] = c.x; v[8 * j + 5] = c.y; v[8 * j + 6] = e.x; v[8 * j + 7] = e.y;
    }
  }
  store16<DT>(p.x[which], t * p.x_st[which] + head * p.x_sh[which] + d, v);
}

// Calls `one` with token ranges whose 16-element units count at most 2^30 (one launch for any
// call of up to 2^34 elements per tensor).
template <typename F>
void by_ranges(const Kv4RowsParams& p, int esz, F one) {
  const int64_t per_token = static_cast<int64_t>(p.H) * p.D / kPerLane;
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / per_token);
  for (int64_t t = 0; t < p.T; t += most) {
    Kv4RowsParams r = p;
    r.T = std::min(most, p.T - t);
    r.slots = p.slots + t;
    for (int i = 0; i < 2; i++) r.x[i] = static_cast<uint8_t*>(p.x[i]) + t * p.x_st[i] * esz;
    const int64_t units = r.T * per_token;
    one(r, dim3(static_cast<unsigned>((units + kThreads - 1) / kThreads), 2), static_cast<uint32_t>(units),
        static_cast<uint32_t>(per_token));
  }
}

template <int DT>
void launch_rows(bool write, const Kv4RowsParams& p, hipStream_t stream) {
  by_ranges(p, DT == FP8Q_DTYPE_F32 ? 4 : 2, [&](const Kv4RowsParams& r, dim3 grid, uint32_t units, uint32_t per_token) {
    if (write)
      hipLaunchKernelGGL((kv4_write_kernel<DT>), grid, dim3(kThreads), 0, stream, r, units, per_token);
    else
      hipLaunchKernelGGL((kv4_read_kernel<DT>), grid, dim3(kThreads), 0, stream, r, units, per_token);
  });
}

int launch_any(bool write, int dtype, const Kv4RowsParams& p, hipStream_t stream) {
  switch (dtype) {
    case FP8Q_DTYPE_BF16: launch_rows<FP8Q_DTYPE_BF16>(write, p, stream); break;
    case FP8Q_DTYPE_F16: launch_rows<FP8Q_DTYPE_F16>(write, p, stream); break;
    default: launch_rows<FP8Q_DTYPE_F32>(write, p, stream); break;
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess)
    return fail(FP8Q_ELAUNCH, std::string(write ? "kv4 write" : "kv4 read") + " launch: " + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace

int launch_kv4_write(int dtype, const Kv4RowsParams& p, hipStream_t stream) { return launch_any(true, dtype, p, stream); }
int launch_kv4_read(int dtype, const Kv4RowsParams& p, hipStream_t stream) { return launch_any(false, dtype, p, stream); }

}  // namespace fp8q
