// mxfp4.h — launchers and parameters of the 4-bit microscaled quantizer and product. Not part of the public
// ABI (include/fp8q.h).
#pragma once

#include "fp8q_internal.h"

namespace fp8q {

constexpr int kMxBlock = 32;  // elements that share one scale byte

struct Mxfp4RowsParams {
  void* x;              // [M][K], or [M][2 K] gate | up
  uint8_t* q;           // [M][K / 2]
  uint8_t* s;           // scale bytes, or words of four
  int64_t M, K;
  int64_t x_sm;         // elements
  int64_t q_sm;         // bytes
  int64_t s_sm, s_sg;   // bytes, or words
  int32_t packed;       // words of four groups
};

int launch_mxfp4_quant(int dtype, bool silu, const Mxfp4RowsParams& p, hipStream_t stream);
int launch_mxfp4_dequant(int dtype, const Mxfp4RowsParams& p, hipStream_t stream);

// A [M][K / 2] and B [N][K / 2] codes; the scales of 128 elements of a row (four bytes) are the 32-bit word
// at s + 4 * (row * s_sm + k / 128 * s_sk) bytes.
struct Mxfp4GemmParams {
  const uint8_t* a;
  const uint8_t* sa;
  const uint8_t* b;
  const uint8_t* sb;
  uint16_t* y;
  int64_t M, N, K;
  int64_t lda, ldb;  // bytes
  int64_t ldy;       // elements
  int64_t sa_sm, sa_sk, sb_sn, sb_sk;  // words
  float* ws;
  int64_t ws_bytes;
  int xcds;
  int splits;        // ranges of K
};

int64_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
int launch_mxfp4_gemm(const Mxfp4GemmParams& p, hipStream_t stream);
int launch_mxfp4_zero(const Mxfp4GemmParams& p, hipStream_t stream);  // K == 0

}  // namespace fp8q
