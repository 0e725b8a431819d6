// gemm_mxfp4.hip — Y = A B^T of two matrices of e2m1 codes with one UE8M0 scale per 32 elements of a row
// (MXFP4), rounded to bf16 once:
//   Y[m][n] = bf16( sum_k 2^(ea(m, k/32) - 127) A[m][k] * 2^(eb(n, k/32) - 127) B[n][k] )
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with 4-bit operands: lane l holds row l % 16, the 32 elements (16 bytes)
// of K block l / 16, and that block's scale byte. The operands are swapped (its "A" are rows of B), so a lane
// of the result has four consecutive n of one m.
#include <algorithm>

#include "mxfp4.h"

namespace fp8q {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // operand format

__device__ __forceinline__ v8i operand(u32x4 w) {
  return v8i{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3]), 0, 0, 0, 0};
}

__device__ __forceinline__ v4f mma(v8i b, uint32_t eb, v8i a, uint32_t ea, v4f c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, kFp4, kFp4, 0, static_cast<int>(eb), 0, static_cast<int>(ea));
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// One wave per 16 x 16 outputs, operands straight from memory.
__global__ __launch_bounds__(64) void gemm_mxfp4_simple_kernel(Mxfp4GemmParams p) {
  const int lane = threadIdx.x, r = lane & 15, h = lane >> 4;
  const int64_t m = static_cast<int64_t>(blockIdx.y) * 16 + r, n = static_cast<int64_t>(blockIdx.x) * 16 + r;
  const int64_t mr = min(m, p.M - 1), nr = min(n, p.N - 1);
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t kb = 0; kb < p.K / 128; kb++) {
    const v8i a = operand(*reinterpret_cast<const u32x4*>(p.a + mr * p.lda + kb * 64 + 16 * h));
    const v8i b = operand(*reinterpret_cast<const u32x4*>(p.b + nr * p.ldb + kb * 64 + 16 * h));
    const uint32_t ea = p.sa[4 * (mr * p.sa_sm + kb * p.sa_sk) + h], eb = p.sb[4 * (nr * p.sb_sn + kb * p.sb_sk) + h];
    acc = mma(b, eb, a, ea, acc);
  }
  if (m >= p.M) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + 4 * h + i;
    if (col < p.N) p.y[m * p.ldy + col] = bf16_bits(acc[i]);
  }
}

}  // namespace

int64_t mxfp4_gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

int launch_mxfp4_gemm(const Mxfp4GemmParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(gemm_mxfp4_simple_kernel, dim3(static_cast<unsigned>((p.N + 15) / 16), static_cast<unsigned>((p.M + 15) / 16)),
                     dim3(64), 0, stream, p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("mxfp4 product launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace fp8q
