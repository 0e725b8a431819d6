// kv4.hip — writing rows into a paged cache of 4-bit codes, and reading them back.
//
// A row of D elements (one token's key or value of one head) is held as D / 2 bytes of e2m1
// codes (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; element 2i in the low half of byte i) and one
// UE8M0 byte per 32 elements: the group rule of the FP8 quantizer with 6 in the place of 448.
// The scale is a power of two and at least amax / 6, so the division by it is exact and no
// element saturates: the rounding to e2m1 (nearest, ties to even) is the only one.
//
// Both directions are bound by HBM traffic: 2 bytes per element on the model's side (bf16),
// 0.53 on the cache's. A lane owns 8 consecutive elements (a quarter of a scale block) of 4
// tokens in a row: 16 bytes per lane and access on the model's side, next to the neighbour's,
// and the index arithmetic is done once for the four. Blocks of the write take keys and values in
// turn: they are often views of one projection's output, whose rows are then read whole (65536
// tokens of 8 x 128, 340 MB: 70 us, 82 us with all keys before all values; fp32 124 either way). The
// read's outputs are two tensors, written one after the other (131072 tokens, 680 MB: 131 us, in turn too).
#include <algorithm>

#include "quant_device.h"
#include "serving.h"
#include "serving_device.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

constexpr int kThreads = 256;
constexpr int kEl = 8;   // elements of a lane
constexpr int kTok = 4;  // tokens of a lane
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

struct Grid {
  uint32_t units, per;  // lanes with work per tensor; those of one group of tokens
  Divider by_per;
};

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

// Where a lane's elements lie: the first of its tokens, head and element of the row.
struct Place {
  int32_t t, head, d;
};
__device__ __forceinline__ Place place_of(const Kv4RowsParams& p, const Grid& g, uint32_t u) {
  const uint32_t group = divide(u, g.by_per), el = (u - group * g.per) * kEl;
  return Place{static_cast<int32_t>(group) * kTok, static_cast<int32_t>(el >> p.d_shift),
               static_cast<int32_t>(el & ((1u << p.d_shift) - 1u))};
}

// Slots of the lane's tokens, -1 for one that is not there or lies outside the cache.
__device__ __forceinline__ void slots_of(const Kv4RowsParams& p, int32_t t, int32_t (&slot)[kTok]) {
#pragma unroll
  for (int i = 0; i < kTok; i++) {
    slot[i] = t + i < p.T ? p.slots[t + i] : -1;
    if (slot[i] >= (p.c.pages << p.c.page_shift)) slot[i] = -1;
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void kv4_write_kernel(Kv4RowsParams p, Grid g) {
  constexpr int kEsz = DT == FP8Q_DTYPE_F32 ? 4 : 2;
  const uint32_t u = (blockIdx.x >> 1) * kThreads + threadIdx.x;
  const int which = blockIdx.x & 1;  // keys, values
  if (u >= g.units) return;
  const Place at = place_of(p, g, u);
  const uint8_t* x = static_cast<const uint8_t*>(p.x[which]) + (at.t * p.x_st[which] + at.head * p.x_sh[which] + at.d) * kEsz;
  int32_t slot[kTok];
  slots_of(p, at.t, slot);
  Raw8<DT> raw[kTok];
#pragma unroll
  for (int i = 0; i < kTok; i++) {
#pragma unroll
    for (int j = 0; j < kEsz / 2; j++) {
      raw[i].w[j] = u32x4{0u, 0u, 0u, 0u};
      if (slot[i] >= 0) raw[i].w[j] = reinterpret_cast<const u32x4*>(x + i * p.x_st[which] * kEsz)[j];
    }
  }
  uint8_t* codes = (which ? p.c.v : p.c.k) + at.head * p.c.c_sh + at.d / 2;
  uint8_t* scales = (which ? p.c.vs : p.c.ks) + at.head * p.c.s_sh + at.d / kKv4Block;
  const int32_t mask = (1 << p.c.page_shift) - 1;
#pragma unroll
  for (int i = 0; i < kTok; i++) {
    // a scale block's four lanes are neighbours in a quad and have the same token
    float amax = amax8<DT>(raw[i]);
    amax = fmaxf(amax, dpp<0xB1>(amax));
    amax = fmaxf(amax, dpp<0x4E>(amax));
    const uint32_t byte = e2m1_scale_byte(fmaxf(amax, kEps));
    const uint32_t c = encode8<DT>(raw[i], __uint_as_float(byte << 23));
    if (slot[i] >= 0) {
      const int64_t page = slot[i] >> p.c.page_shift, tok = slot[i] & mask;
      *reinterpret_cast<uint32_t*>(codes + page * p.c.c_sp + tok * p.c.c_st) = c;
      if ((at.d & (kKv4Block - 1)) == 0) scales[page * p.c.s_sp + tok * p.c.s_st] = static_cast<uint8_t>(byte);
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4RowsParams p, Grid g) {
  constexpr int kEsz = DT == FP8Q_DTYPE_F32 ? 4 : 2;
  const uint32_t half = gridDim.x >> 1;
  const int which = blockIdx.x >= half;  // all keys, then all values
  const uint32_t u = (which ? blockIdx.x - half : blockIdx.x) * kThreads + threadIdx.x;
  if (u >= g.units) return;
  const Place at = place_of(p, g, u);
  int32_t slot[kTok];
  slots_of(p, at.t, slot);
  const uint8_t* codes = (which ? p.c.v : p.c.k) + at.head * p.c.c_sh + at.d / 2;
  const uint8_t* scales = (which ? p.c.vs : p.c.ks) + at.head * p.c.s_sh + at.d / kKv4Block;
  const int32_t mask = (1 << p.c.page_shift) - 1;
  uint32_t c[kTok], byte[kTok];
#pragma unroll
  for (int i = 0; i < kTok; i++) {
    c[i] = 0;  // a slot outside the cache: zeros
    byte[i] = 127;
    if (slot[i] >= 0) {
      const int64_t page = slot[i] >> p.c.page_shift, tok = slot[i] & mask;
      c[i] = *reinterpret_cast<const uint32_t*>(codes + page * p.c.c_sp + tok * p.c.c_st);
      byte[i] = scales[page * p.c.s_sp + tok * p.c.s_st];
    }
  }
  uint8_t* x = static_cast<uint8_t*>(p.x[which]) + (at.t * p.x_st[which] + at.head * p.x_sh[which] + at.d) * kEsz;
  // Tokens decoded together before their stores, by the type: the check for infinities between the stores
  // costs more than its instructions. us for 1, 2 and 4: 131072 tokens of 8 x 128 in bf16 134, 131 and
  // 136 (128 without the check), 65536 in fp16 67, 68 and 72 (67), in fp32 142, - and 117 (125).
  constexpr int kAhead = DT == FP8Q_DTYPE_F32 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < kTok; i += kAhead) {
    Raw8<DT> r[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; a++) r[a] = decode8<DT>(c[i + a], byte[i + a]);
#pragma unroll
    for (int a = 0; a < kAhead; a++) {
      if (at.t + i + a >= p.T) return;
#pragma unroll
      for (int j = 0; j < kEsz / 2; j++) reinterpret_cast<u32x4*>(x + (i + a) * p.x_st[which] * kEsz)[j] = r[a].w[j];
    }
  }
}

// Calls `one` with token ranges whose lanes count at most 2^30 (one launch for any call of up
// to 2^35 elements per tensor).
template <typename F>
void by_ranges(const Kv4RowsParams& p, int esz, F one) {
  const int64_t per = static_cast<int64_t>(p.H) * p.D / kEl;
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / per) * kTok;
  for (int64_t t = 0; t < p.T; t += most) {
    Kv4RowsParams r = p;
    r.T = std::min(most, p.T - t);
    r.slots = p.slots + t;
    for (int i = 0; i < 2; i++) r.x[i] = static_cast<uint8_t*>(p.x[i]) + t * p.x_st[i] * esz;
    const Grid g{static_cast<uint32_t>((r.T + kTok - 1) / kTok * per), static_cast<uint32_t>(per),
                 divider(static_cast<uint32_t>(per))};
    one(r, dim3((g.units + kThreads - 1) / kThreads * 2), g);
  }
}

template <int DT>
void launch_rows(bool write, const Kv4RowsParams& p, hipStream_t stream) {
  by_ranges(p, DT == FP8Q_DTYPE_F32 ? 4 : 2, [&](const Kv4RowsParams& r, dim3 grid, const Grid& g) {
    if (write)
      hipLaunchKernelGGL((kv4_write_kernel<DT>), grid, dim3(kThreads), 0, stream, r, g);
    else
      hipLaunchKernelGGL((kv4_read_kernel<DT>), grid, dim3(kThreads), 0, stream, r, g);
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
