// api_mxfp4.hip — C ABI of the 4-bit microscaled quantizer and product: argument validation (host only, before
// any device call), the device check, then the launch. Semantics: include/fp8q.h.
#include "mxfp4.h"

namespace fp8q {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int rows_entry(const char* name, bool quant, bool silu, void* x, int dtype, int64_t M, int64_t K, int64_t x_sm, uint8_t* q,
               int64_t q_sm, void* s, int scale_fmt, int64_t s_sm, int64_t s_sg, void* stream) {
  set_error("");
  const std::string pre = std::string(name) + ": ";
  const int esz = dtype == FP8Q_DTYPE_F32 ? 4 : dtype == FP8Q_DTYPE_BF16 || dtype == FP8Q_DTYPE_F16 ? 2 : 0;
  if (esz == 0) return fail(FP8Q_EUNSUPPORTED, pre + "dtype must be BF16, F16 or F32");
  const bool packed = scale_fmt == FP8Q_SCALE_UE8M0_PACKED;
  if (!packed && scale_fmt != FP8Q_SCALE_UE8M0)
    return fail(FP8Q_EUNSUPPORTED, pre + "scale_fmt must be UE8M0 or UE8M0_PACKED");
  if (M < 0 || K < 0) return fail(FP8Q_EINVAL, pre + "negative size");
  if (K % 32 != 0) return fail(FP8Q_EINVAL, pre + "K must be a multiple of 32");
  if (packed && K % 128 != 0) return fail(FP8Q_EINVAL, pre + "packed UE8M0 scales need a multiple of 4 groups per row");
  if (K > (int64_t(1) << 30)) return fail(FP8Q_EUNSUPPORTED, pre + "rows are limited to 2^30 elements");
  if (x_sm < 0 || q_sm < 0 || s_sm < 0 || s_sg < 0) return fail(FP8Q_EINVAL, pre + "negative stride");
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x || !q || !s) return fail(FP8Q_EINVAL, pre + "null tensor pointer");
  if (quant && M > 1 && q_sm < K / 2) return fail(FP8Q_EINVAL, pre + "q rows overlap (q_sm < K / 2)");
  if (!quant && M > 1 && x_sm < K) return fail(FP8Q_EINVAL, pre + "x rows overlap (x_sm < K)");
  const int64_t ng = packed ? K / 128 : K / 32;
  const bool row_major = s_sg == 1 && (M <= 1 || s_sm >= ng);
  const bool col_major = s_sm == 1 && (ng <= 1 || s_sg >= M);
  if (!row_major && !col_major)
    return fail(FP8Q_EINVAL, pre + "scale strides are neither row-major (s_sg == 1) nor column-major (s_sm == 1)");
  if (!aligned(x, 16) || x_sm * esz % 16 != 0) return fail(FP8Q_EALIGN, pre + "x and its row stride must be 16-byte aligned");
  if (!aligned(q, 16) || q_sm % 16 != 0) return fail(FP8Q_EALIGN, pre + "q and its row stride must be 16-byte aligned");
  if (packed && !aligned(s, 4)) return fail(FP8Q_EALIGN, pre + "packed UE8M0 words must be 4-byte aligned");
  const int dev = check_current_device();
  if (dev != FP8Q_OK) return dev;
  Mxfp4RowsParams p{};
  p.x = x;
  p.q = q;
  p.s = static_cast<uint8_t*>(s);
  p.M = M;
  p.K = K;
  p.x_sm = x_sm;
  p.q_sm = q_sm;
  p.s_sm = s_sm;
  p.s_sg = s_sg;
  p.packed = packed;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return quant ? launch_mxfp4_quant(dtype, silu, p, st) : launch_mxfp4_dequant(dtype, p, st);
}

constexpr int64_t kMostStride = int64_t(1) << 24;  // bytes
bool gemm_sizes(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kMost = int64_t(1) << 26;
  return M <= kMost && N <= kMost && M * N <= (int64_t(1) << 40) && K < (int64_t(1) << 25);
}

// One operand's scales as words of four: packed words with any strides, or row-major bytes in whole words.
int scale_words(const std::string& pre, const char* which, const void* s, int fmt, int64_t rows, int64_t K, int64_t sm,
                int64_t sk, int64_t& word_sm, int64_t& word_sk) {
  if (fmt == FP8Q_SCALE_UE8M0_PACKED) {
    word_sm = sm;
    word_sk = sk;
  } else {
    if (K > 32 && sk != 1) return fail(FP8Q_EUNSUPPORTED, pre + which + " scale bytes must be row-major (or packed words)");
    if (rows > 1 && sm % 4 != 0) return fail(FP8Q_EALIGN, pre + which + " rows of scale bytes must be 4-byte aligned");
    word_sm = sm / 4;
    word_sk = 1;
  }
  if (!aligned(s, 4)) return fail(FP8Q_EALIGN, pre + which + " scales must be 4-byte aligned");
  if (rows > 1 && word_sm >= kMostStride / 4)
    return fail(FP8Q_EUNSUPPORTED, pre + which + " rows of scales must be less than 2^24 bytes apart");
  return FP8Q_OK;
}

int gemm_entry(const uint8_t* a, int64_t lda, const void* sa, int sa_fmt, int64_t sa_sm, int64_t sa_sk, const uint8_t* b,
               int64_t ldb, const void* sb, int sb_fmt, int64_t sb_sn, int64_t sb_sk, uint16_t* y, int64_t ldy, int64_t M,
               int64_t N, int64_t K, void* workspace, int64_t workspace_bytes, void* stream) {
  set_error("");
  static const std::string pre = "fp8q_gemm_mxfp4: ";
  auto e8 = [](int f) { return f == FP8Q_SCALE_UE8M0 || f == FP8Q_SCALE_UE8M0_PACKED; };
  if (!e8(sa_fmt) || !e8(sb_fmt)) return fail(FP8Q_EUNSUPPORTED, pre + "scales must be UE8M0 or UE8M0_PACKED");
  if (M < 0 || N < 0 || K < 0) return fail(FP8Q_EINVAL, pre + "negative size");
  if (K % 128 != 0) return fail(FP8Q_EINVAL, pre + "K must be a multiple of 128");
  if (!gemm_sizes(M, N, K)) return fail(FP8Q_EUNSUPPORTED, pre + "M and N up to 2^26, M * N up to 2^40, K below 2^25");
  if (lda < 0 || ldb < 0 || ldy < 0 || sa_sm < 0 || sa_sk < 0 || sb_sn < 0 || sb_sk < 0)
    return fail(FP8Q_EINVAL, pre + "negative stride");
  if (workspace_bytes < 0) return fail(FP8Q_EINVAL, pre + "negative workspace size");
  if (!aligned(workspace, 16)) return fail(FP8Q_EALIGN, pre + "workspace must be 16-byte aligned");
  if (M == 0 || N == 0 || (K == 0 && !y)) return FP8Q_OK;
  if (!y || (K > 0 && (!a || !b || !sa || !sb))) return fail(FP8Q_EINVAL, pre + "null tensor pointer");
  if ((M > 1 && lda < K / 2) || (N > 1 && ldb < K / 2)) return fail(FP8Q_EINVAL, pre + "lda and ldb must be >= K / 2");
  if (M > 1 && ldy < N) return fail(FP8Q_EINVAL, pre + "ldy must be >= N (rows of y overlap)");
  if (!aligned(y, 2)) return fail(FP8Q_EALIGN, pre + "y must be 2-byte aligned");
  Mxfp4GemmParams p{};
  p.y = y;
  p.M = M;
  p.N = N;
  p.K = K;
  p.ldy = ldy;
  if (K == 0) {  // sums of nothing
    const int rc = check_current_device();
    return rc != FP8Q_OK ? rc : launch_mxfp4_zero(p, static_cast<hipStream_t>(stream));
  }
  // (a tile's rows lie within 32 bits of its first one)
  if ((M > 1 && lda >= kMostStride) || (N > 1 && ldb >= kMostStride))
    return fail(FP8Q_EUNSUPPORTED, pre + "lda and ldb must be below 2^24");
  if (!aligned(a, 16) || !aligned(b, 16) || (M > 1 && lda % 16 != 0) || (N > 1 && ldb % 16 != 0))
    return fail(FP8Q_EALIGN, pre + "a, b and their row strides must be 16-byte aligned");
  int rc = scale_words(pre, "a's", sa, sa_fmt, M, K, sa_sm, sa_sk, p.sa_sm, p.sa_sk);
  if (rc != FP8Q_OK) return rc;
  rc = scale_words(pre, "b's", sb, sb_fmt, N, K, sb_sn, sb_sk, p.sb_sn, p.sb_sk);
  if (rc != FP8Q_OK) return rc;
  rc = check_current_device();
  if (rc != FP8Q_OK) return rc;
  p.a = a;
  p.sa = static_cast<const uint8_t*>(sa);
  p.b = b;
  p.sb = static_cast<const uint8_t*>(sb);
  p.lda = M > 1 ? lda : K / 2;
  p.ldb = N > 1 ? ldb : K / 2;
  p.ws = static_cast<float*>(workspace);
  p.ws_bytes = workspace ? workspace_bytes : 0;
  return launch_mxfp4_gemm(p, static_cast<hipStream_t>(stream));
}

}  // namespace
}  // namespace fp8q

extern "C" {

int fp8q_mxfp4_quant(const void* x, int in_dtype, int64_t M, int64_t K, int64_t x_sm, uint8_t* q, int64_t q_sm, void* s,
                     int scale_fmt, int64_t s_sm, int64_t s_sg, void* stream) {
  return fp8q::rows_entry("fp8q_mxfp4_quant", true, false, const_cast<void*>(x), in_dtype, M, K, x_sm, q, q_sm, s,
                          scale_fmt, s_sm, s_sg, stream);
}

int fp8q_silu_mul_mxfp4_quant(const void* x, int in_dtype, int64_t M, int64_t K, int64_t x_sm, uint8_t* q, int64_t q_sm,
                              void* s, int scale_fmt, int64_t s_sm, int64_t s_sg, void* stream) {
  return fp8q::rows_entry("fp8q_silu_mul_mxfp4_quant", true, true, const_cast<void*>(x), in_dtype, M, K, x_sm, q, q_sm, s,
                          scale_fmt, s_sm, s_sg, stream);
}

int fp8q_mxfp4_dequant(const uint8_t* q, int64_t q_sm, const void* s, int scale_fmt, int64_t s_sm, int64_t s_sg, void* x,
                       int out_dtype, int64_t M, int64_t K, int64_t x_sm, void* stream) {
  return fp8q::rows_entry("fp8q_mxfp4_dequant", false, false, x, out_dtype, M, K, x_sm, const_cast<uint8_t*>(q), q_sm,
                          const_cast<void*>(s), scale_fmt, s_sm, s_sg, stream);
}

int64_t fp8q_gemm_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K) {
  using namespace fp8q;
  set_error("");
  if (M <= 0 || N <= 0 || K <= 0 || !gemm_sizes(M, N, K) || K % 128 != 0 || check_current_device() != FP8Q_OK) return 0;
  return mxfp4_gemm_workspace_bytes(M, N, K);
}

int fp8q_gemm_mxfp4(const uint8_t* a, int64_t lda, const void* sa, int sa_fmt, int64_t sa_sm, int64_t sa_sk, const uint8_t* b,
                    int64_t ldb, const void* sb, int sb_fmt, int64_t sb_sn, int64_t sb_sk, uint16_t* y, int64_t ldy,
                    int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes, void* stream) {
  return fp8q::gemm_entry(a, lda, sa, sa_fmt, sa_sm, sa_sk, b, ldb, sb, sb_fmt, sb_sn, sb_sk, y, ldy, M, N, K, workspace,
                          workspace_bytes, stream);
}

}  // extern "C"
