// api_serving.hip — C ABI of the quantizing norm, the 4-bit cache, its page plan and attention: argument validation
// (host only, before any device call), the device check, then the launch. Semantics:
// include/fp8q.h.
#include <algorithm>
#include <cmath>
#include <limits>

#include "serving.h"

namespace fp8q {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int element_size(int dtype) {
  return dtype == FP8Q_DTYPE_F32 ? 4 : (dtype == FP8Q_DTYPE_BF16 || dtype == FP8Q_DTYPE_F16) ? 2 : 0;
}

// Whether rows of `row` units at the given (count, stride) steps are pairwise disjoint: sorted
// by stride, every step must clear all that lies below it.
bool disjoint(int64_t row, std::pair<int64_t, int64_t> a, std::pair<int64_t, int64_t> b,
              std::pair<int64_t, int64_t> c = {1, 0}) {
  std::pair<int64_t, int64_t> d[3] = {a, b, c};
  std::sort(d, d + 3, [](const auto& x, const auto& y) { return x.second < y.second; });
  __int128 extent = row;
  for (const auto& [n, stride] : d) {
    if (n <= 1) continue;
    if (stride < extent) return false;
    extent += static_cast<__int128>(n - 1) * stride;
  }
  return true;
}

int norm_entry(const void* x, int in_dtype, int64_t M, int64_t K, int64_t x_sm, const void* residual, int64_t r_sm,
               void* residual_out, int64_t ro_sm, const void* weight, float eps, uint8_t* q, int64_t q_sm, void* s,
               int scale_fmt, int64_t s_sm, int64_t s_sg, int group_size, void* stream) {
  set_error("");
  const std::string pre = "fp8q_rms_norm_group_quant: ";
  const int esz = element_size(in_dtype);
  if (esz == 0) return fail(FP8Q_EUNSUPPORTED, pre + "in_dtype must be BF16, F16 or F32");
  if (scale_fmt != FP8Q_SCALE_F32 && scale_fmt != FP8Q_SCALE_UE8M0 && scale_fmt != FP8Q_SCALE_UE8M0_PACKED)
    return fail(FP8Q_EUNSUPPORTED, pre + "scale_fmt must be F32, UE8M0 or UE8M0_PACKED");
  if (M < 0 || K < 0) return fail(FP8Q_EINVAL, pre + "negative size");
  const bool grouped = group_size == 32 || group_size == 64 || group_size == 128;
  if (!grouped && (group_size <= 0 || group_size != K))
    return fail(FP8Q_EUNSUPPORTED, pre + "group_size must be 32, 64, 128 or K (per-token)");
  if (K % group_size != 0) return fail(FP8Q_EINVAL, pre + "K must be a multiple of group_size");
  if (K % 16 != 0) return fail(FP8Q_EINVAL, pre + "per-token quantization needs K % 16 == 0");
  if (K > kNormMaxK) return fail(FP8Q_EUNSUPPORTED, pre + "rows are limited to 65536 elements");
  const bool packed = scale_fmt == FP8Q_SCALE_UE8M0_PACKED;
  if (packed && (K / group_size) % 4 != 0)
    return fail(FP8Q_EINVAL, pre + "packed UE8M0 scales need a multiple of 4 groups per row");
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(FP8Q_EINVAL, pre + "eps must be finite and >= 0");
  if (x_sm < 0 || r_sm < 0 || ro_sm < 0 || q_sm < 0 || s_sm < 0 || s_sg < 0)
    return fail(FP8Q_EINVAL, pre + "negative stride");
  if (residual_out && !residual) return fail(FP8Q_EINVAL, pre + "residual_out without a residual");
  if (M == 0 || K == 0) return FP8Q_OK;
  if (!x || !weight || !q || !s) return fail(FP8Q_EINVAL, pre + "null tensor pointer");
  if (M > 1 && q_sm < K) return fail(FP8Q_EINVAL, pre + "q rows overlap (q_sm < K)");
  if (residual_out && M > 1 && ro_sm < K) return fail(FP8Q_EINVAL, pre + "residual_out rows overlap (ro_sm < K)");
  const int64_t ng = packed ? K / group_size / 4 : K / group_size;
  const bool row_major = s_sg == 1 && (M <= 1 || s_sm >= ng);
  const bool col_major = s_sm == 1 && (ng <= 1 || s_sg >= M);
  if (!row_major && !col_major)
    return fail(FP8Q_EINVAL, pre + "scale strides are neither row-major (s_sg == 1) nor column-major (s_sm == 1)");
  if (!aligned(x, 16) || x_sm * esz % 16 != 0 || !aligned(weight, 16))
    return fail(FP8Q_EALIGN, pre + "x, its row stride and the weight must be 16-byte aligned");
  if (residual && (!aligned(residual, 16) || r_sm * esz % 16 != 0))
    return fail(FP8Q_EALIGN, pre + "residual and its row stride must be 16-byte aligned");
  if (residual_out && (!aligned(residual_out, 16) || ro_sm * esz % 16 != 0))
    return fail(FP8Q_EALIGN, pre + "residual_out and its row stride must be 16-byte aligned");
  if (!aligned(q, 16) || q_sm % 16 != 0) return fail(FP8Q_EALIGN, pre + "q and its row stride must be 16-byte aligned");
  if (scale_fmt != FP8Q_SCALE_UE8M0 && !aligned(s, 4))
    return fail(FP8Q_EALIGN, pre + "fp32 scales and packed UE8M0 words must be 4-byte aligned");
  const int dev = check_current_device();
  if (dev != FP8Q_OK) return dev;
  NormParams p{};
  p.x = x;
  p.res = residual;
  p.res_out = residual_out;
  p.w = weight;
  p.q = q;
  p.s = s;
  p.M = M;
  p.K = K;
  p.x_sm = x_sm;
  p.r_sm = r_sm;
  p.ro_sm = ro_sm;
  p.q_sm = q_sm;
  p.s_sm = s_sm;
  p.s_sg = s_sg;
  p.eps = eps;
  p.inv_k = 1.0 / static_cast<double>(K);
  p.group = grouped ? group_size : 0;
  p.group_shift = group_size == 32 ? 5 : group_size == 64 ? 6 : group_size == 128 ? 7 : 30;
  p.ue8m0 = scale_fmt != FP8Q_SCALE_F32;
  p.packed = packed;
  return launch_rms_norm_quant(in_dtype, p, static_cast<hipStream_t>(stream));
}

// ------------------------------------------------------------------ 4-bit cache
int log2_exact(int64_t v) {
  for (int i = 0; i < 31; i++)
    if (v == (int64_t(1) << i)) return i;
  return -1;
}

// Sizes, strides and alignment of the cached tensors; `written`: rows must not overlap.
int check_cache(const std::string& pre, const uint8_t* kc, const uint8_t* ks, const uint8_t* vc, const uint8_t* vs,
                int64_t pages, int64_t page_size, int64_t H, int64_t D, int64_t c_sp, int64_t c_st, int64_t c_sh,
                int64_t s_sp, int64_t s_st, int64_t s_sh, bool written) {
  if (D != 64 && D != 128 && D != 256) return fail(FP8Q_EUNSUPPORTED, pre + "head dimension must be 64, 128 or 256");
  if (H < 0 || pages < 0) return fail(FP8Q_EINVAL, pre + "negative size");
  if (log2_exact(page_size) < 0) return fail(FP8Q_EUNSUPPORTED, pre + "page_size must be a power of two below 2^31");
  if (H > (int64_t(1) << 20)) return fail(FP8Q_EUNSUPPORTED, pre + "at most 2^20 heads");
  if (pages >= (int64_t(1) << 31) || pages * page_size >= (int64_t(1) << 31))
    return fail(FP8Q_EUNSUPPORTED, pre + "the cache must have fewer than 2^31 slots");
  if (c_sp < 0 || c_st < 0 || c_sh < 0 || s_sp < 0 || s_st < 0 || s_sh < 0)
    return fail(FP8Q_EINVAL, pre + "negative stride");
  if (pages == 0) return FP8Q_OK;  // no slot is ever touched
  if (!kc || !ks || !vc || !vs) return fail(FP8Q_EINVAL, pre + "null cache pointer");
  if (!aligned(kc, 16) || !aligned(vc, 16) || c_sp % 16 != 0 || c_st % 16 != 0 || c_sh % 16 != 0)
    return fail(FP8Q_EALIGN, pre + "cached codes and their strides must be 16-byte aligned");
  const int64_t sn = D / kKv4Block;
  if (!aligned(ks, sn) || !aligned(vs, sn) || s_sp % sn != 0 || s_st % sn != 0 || s_sh % sn != 0)
    return fail(FP8Q_EALIGN, pre + "cached scales and their strides must be aligned to a row's D / 32 bytes");
  if (written && (!disjoint(D / 2, {pages, c_sp}, {page_size, c_st}, {H, c_sh}) ||
                  !disjoint(sn, {pages, s_sp}, {page_size, s_st}, {H, s_sh})))
    return fail(FP8Q_EINVAL, pre + "cached rows overlap");
  return FP8Q_OK;
}

Kv4Cache cache_of(const uint8_t* kc, const uint8_t* ks, const uint8_t* vc, const uint8_t* vs, int64_t pages,
                  int64_t page_size, int64_t c_sp, int64_t c_st, int64_t c_sh, int64_t s_sp, int64_t s_st,
                  int64_t s_sh) {
  Kv4Cache c{};
  c.k = const_cast<uint8_t*>(kc);
  c.ks = const_cast<uint8_t*>(ks);
  c.v = const_cast<uint8_t*>(vc);
  c.vs = const_cast<uint8_t*>(vs);
  c.pages = pages;
  c.page_shift = log2_exact(page_size);
  c.c_sp = c_sp;
  c.c_st = c_st;
  c.c_sh = c_sh;
  c.s_sp = s_sp;
  c.s_st = s_st;
  c.s_sh = s_sh;
  return c;
}

int rows_entry(bool write, const void* k, int64_t k_st, int64_t k_sh, const void* v, int64_t v_st, int64_t v_sh,
               int dtype, int64_t T, int64_t H, int64_t D, const int32_t* slots, const uint8_t* kc, const uint8_t* ks,
               const uint8_t* vc, const uint8_t* vs, int64_t pages, int64_t page_size, int64_t c_sp, int64_t c_st,
               int64_t c_sh, int64_t s_sp, int64_t s_st, int64_t s_sh, void* stream) {
  set_error("");
  const std::string pre = write ? "fp8q_kv4_write: " : "fp8q_kv4_read: ";
  const int esz = element_size(dtype);
  if (esz == 0) return fail(FP8Q_EUNSUPPORTED, pre + "dtype must be BF16, F16 or F32");
  if (T < 0) return fail(FP8Q_EINVAL, pre + "negative size");
  if (T >= (int64_t(1) << 31)) return fail(FP8Q_EUNSUPPORTED, pre + "fewer than 2^31 tokens");
  if (k_st < 0 || k_sh < 0 || v_st < 0 || v_sh < 0) return fail(FP8Q_EINVAL, pre + "negative stride");
  const int rc = check_cache(pre, kc, ks, vc, vs, pages, page_size, H, D, c_sp, c_st, c_sh, s_sp, s_st, s_sh, write);
  if (rc != FP8Q_OK) return rc;
  if (T == 0 || H == 0) return FP8Q_OK;
  if (!k || !v || !slots) return fail(FP8Q_EINVAL, pre + "null tensor pointer");
  if (!write && (!disjoint(D, {T, k_st}, {H, k_sh}) || !disjoint(D, {T, v_st}, {H, v_sh})))
    return fail(FP8Q_EINVAL, pre + "output rows overlap");
  if (!aligned(k, 16) || !aligned(v, 16) || k_st * esz % 16 != 0 || k_sh * esz % 16 != 0 || v_st * esz % 16 != 0 ||
      v_sh * esz % 16 != 0)
    return fail(FP8Q_EALIGN, pre + "k, v and their strides must be 16-byte aligned");
  if (!aligned(slots, 4)) return fail(FP8Q_EALIGN, pre + "slots must be 4-byte aligned");
  const int dev = check_current_device();
  if (dev != FP8Q_OK) return dev;
  Kv4RowsParams p{};
  p.c = cache_of(kc, ks, vc, vs, pages, page_size, c_sp, c_st, c_sh, s_sp, s_st, s_sh);
  p.x[0] = const_cast<void*>(k);
  p.x[1] = const_cast<void*>(v);
  p.x_st[0] = k_st;
  p.x_st[1] = v_st;
  p.x_sh[0] = k_sh;
  p.x_sh[1] = v_sh;
  p.slots = slots;
  p.T = T;
  p.H = static_cast<int32_t>(H);
  p.D = static_cast<int32_t>(D);
  p.d_shift = log2_exact(D);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return write ? launch_kv4_write(dtype, p, st) : launch_kv4_read(dtype, p, st);
}

// ------------------------------------------------------------------ attention
// Sizes alone; FP8Q_OK also for empty problems.
int check_attention_sizes(const std::string& pre, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                          int64_t max_tokens) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0 || max_tokens < 0) return fail(FP8Q_EINVAL, pre + "negative size");
  if (D != 64 && D != 128 && D != 256) return fail(FP8Q_EUNSUPPORTED, pre + "head dimension must be 64, 128 or 256");
  if (B == 0 || T == 0 || Hq == 0) return FP8Q_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return fail(FP8Q_EINVAL, pre + "query heads must be a multiple of cached heads");
  if (B > kMaxSequences) return fail(FP8Q_EUNSUPPORTED, pre + "at most 4096 sequences");
  if (Hq > (int64_t(1) << 20) || T >= (int64_t(1) << 31) || T * Hq >= (int64_t(1) << 31))
    return fail(FP8Q_EUNSUPPORTED, pre + "fewer than 2^31 query rows, at most 2^20 heads");
  if (max_tokens > (int64_t(1) << 30)) return fail(FP8Q_EUNSUPPORTED, pre + "at most 2^30 tokens in a sequence's pages");
  return FP8Q_OK;
}

// What tells the three attention calls apart.
struct AttnMask {
  Mask kind;
  int causal;                // kAll
  int64_t window, sinks;     // kWindow
  const int32_t* tree;       // kTree
  int64_t tree_st, tree_words;
};

int check_window(const std::string& pre, int64_t window, int64_t sinks) {
  if (window < 1) return fail(FP8Q_EINVAL, pre + "window must be at least 1");
  if (sinks < 0) return fail(FP8Q_EINVAL, pre + "sinks must be >= 0");
  return FP8Q_OK;
}

// A window, and sinks, past every possible length are as that length.
int64_t at_most_tokens(int64_t v) { return std::min(v, int64_t(1) << 30); }

int attention_entry(const std::string& pre, const AttnMask& mask, const void* q, int dtype, int64_t q_st, int64_t q_sh, const uint8_t* kc, const uint8_t* ks,
                    const uint8_t* vc, const uint8_t* vs, int64_t pages, int64_t page_size, int64_t c_sp, int64_t c_st,
                    int64_t c_sh, int64_t s_sp, int64_t s_st, int64_t s_sh, const int32_t* table, int64_t table_sb,
                    int64_t max_pages, const int32_t* kv_lens, const int32_t* q_indptr, void* out, int64_t o_st,
                    int64_t o_sh, float* lse, int64_t l_st, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                    float sm_scale, void* workspace, int64_t workspace_bytes, void* stream) {
  set_error("");
  if (dtype != FP8Q_DTYPE_BF16 && dtype != FP8Q_DTYPE_F16)
    return fail(FP8Q_EUNSUPPORTED, pre + "dtype must be BF16 or F16");
  int rc = check_cache(pre, kc, ks, vc, vs, pages, page_size, Hkv, D, c_sp, c_st, c_sh, s_sp, s_st, s_sh, false);
  if (rc != FP8Q_OK) return rc;
  if (max_pages < 0 || max_pages > (int64_t(1) << 30)) return fail(FP8Q_EINVAL, pre + "max_pages outside [0, 2^30]");
  rc = check_attention_sizes(pre, B, T, Hq, Hkv, D, max_pages * page_size);
  if (rc != FP8Q_OK) return rc;
  if (q_st < 0 || q_sh < 0 || o_st < 0 || o_sh < 0 || l_st < 0 || table_sb < 0)
    return fail(FP8Q_EINVAL, pre + "negative stride");
  if (!std::isfinite(sm_scale)) return fail(FP8Q_EINVAL, pre + "sm_scale must be finite");
  if (mask.kind == kWindow && (rc = check_window(pre, mask.window, mask.sinks)) != FP8Q_OK) return rc;
  if (mask.kind == kTree && (mask.tree_words < 0 || mask.tree_st < 0))
    return fail(FP8Q_EINVAL, pre + "negative size or stride of the tree mask");
  if (workspace_bytes < 0) return fail(FP8Q_EINVAL, pre + "workspace_bytes must be >= 0");
  if (B == 0 || T == 0 || Hq == 0) return FP8Q_OK;
  if (!q || !out || !kv_lens || (!table && max_pages > 0)) return fail(FP8Q_EINVAL, pre + "null tensor pointer");
  if (!q_indptr && T != B) return fail(FP8Q_EINVAL, pre + "without q_indptr every sequence has one query (T == B)");
  if (mask.kind == kTree && mask.tree_words > 0 && !mask.tree) return fail(FP8Q_EINVAL, pre + "null tree mask");
  if (mask.kind == kTree && mask.tree_words > (int64_t(1) << 26))
    return fail(FP8Q_EUNSUPPORTED, pre + "at most 2^26 words of the tree mask for a query");
  if (!disjoint(D, {T, o_st}, {Hq, o_sh})) return fail(FP8Q_EINVAL, pre + "output rows overlap");
  if (lse && T > 1 && l_st < Hq) return fail(FP8Q_EINVAL, pre + "lse rows overlap (l_st < Hq)");
  if (!aligned(q, 16) || q_st % 8 != 0 || q_sh % 8 != 0)
    return fail(FP8Q_EALIGN, pre + "q and its strides must be 16-byte aligned");
  if (!aligned(out, 16) || o_st % 8 != 0 || o_sh % 8 != 0)
    return fail(FP8Q_EALIGN, pre + "out and its strides must be 16-byte aligned");
  if (!aligned(table, 4) || !aligned(kv_lens, 4) || !aligned(q_indptr, 4) || !aligned(lse, 4) ||
      !aligned(mask.tree, 4))
    return fail(FP8Q_EALIGN, pre + "page table, lengths, q_indptr, tree mask and lse must be 4-byte aligned");
  if (!aligned(workspace, 16)) return fail(FP8Q_EALIGN, pre + "workspace must be 16-byte aligned");
  const int dev = check_current_device();
  if (dev != FP8Q_OK) return dev;
  Kv4AttnParams p{};
  p.c = cache_of(kc, ks, vc, vs, pages, page_size, c_sp, c_st, c_sh, s_sp, s_st, s_sh);
  p.q = q;
  p.q_st = q_st;
  p.q_sh = q_sh;
  p.out = out;
  p.o_st = o_st;
  p.o_sh = o_sh;
  p.lse = lse;
  p.l_st = l_st;
  p.table = table;
  p.table_sb = table_sb;
  p.max_tokens = pages == 0 ? 0 : max_pages * page_size;  // an empty cache holds no sequence's tokens
  p.kv_lens = kv_lens;
  p.q_indptr = q_indptr;
  p.B = B;
  p.T = T;
  p.Hq = static_cast<int32_t>(Hq);
  p.Hkv = static_cast<int32_t>(Hkv);
  p.group = static_cast<int32_t>(Hq / Hkv);
  // A scale of zero becomes the smallest number instead, so that a masked score times it is still
  // -infinity; a score below 2^127 times that is below 2^-22. (fp32 denormals are on in the kernels.)
  p.scale_log2 = std::min(std::max(std::fabs(sm_scale) * 5.770780163555854f, std::numeric_limits<float>::denorm_min()),
                          std::numeric_limits<float>::max());
  p.q_sign = sm_scale < 0.0f ? 0x80008000u : 0u;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (mask.kind == kWindow) {
    p.window = static_cast<int32_t>(at_most_tokens(mask.window));
    p.sinks = static_cast<int32_t>(at_most_tokens(mask.sinks));
    p.sink_end = static_cast<int32_t>(sink_stretch(p.sinks));
    return launch_kv4_window_attention(dtype, D, p, workspace, workspace_bytes, st);
  }
  if (mask.kind == kTree) {
    p.tree = mask.tree;
    p.tree_st = mask.tree_st;
    p.tree_words = static_cast<int32_t>(mask.tree_words);
    return launch_kv4_tree_attention(dtype, D, p, workspace, workspace_bytes, st);
  }
  p.causal = mask.causal != 0;
  return launch_kv4_attention(dtype, D, p, workspace, workspace_bytes, st);
}

int64_t attention_workspace(const char* pre, int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                            int64_t max_tokens, const AttnMask& mask) {
  set_error("");
  if (check_attention_sizes(pre, B, T, Hq, Hkv, D, max_tokens) != FP8Q_OK ||
      (dtype != FP8Q_DTYPE_BF16 && dtype != FP8Q_DTYPE_F16) || B == 0 || T == 0 || Hq == 0 ||
      (mask.kind == kWindow && check_window(pre, mask.window, mask.sinks) != FP8Q_OK) ||
      check_current_device() != FP8Q_OK)
    return 0;
  if (mask.kind == kWindow)
    max_tokens = window_tokens(max_tokens, at_most_tokens(mask.window), at_most_tokens(mask.sinks));
  return kv4_attention_workspace(dtype, B, T, Hq, Hkv, D, max_tokens, mask.kind);
}

// ------------------------------------------------------------------ page plan
struct Bytes {
  const void* at;
  int64_t n;
};
bool overlap(const Bytes& a, const Bytes& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.n > 0 && b.n > 0 && a.at && b.at && x < y + b.n && y < x + a.n;
}

int plan_entry(const int32_t* kv_lens, const int32_t* q_lens, int64_t B, const int32_t* free_pages, int64_t F, int32_t* table,
               int64_t table_sb, int64_t max_pages, int64_t pages, int64_t page_size, int32_t* new_lens, int32_t* q_indptr,
               int32_t* slots, int32_t* positions, int64_t T, int32_t* pages_taken, void* stream) {
  set_error("");
  static const std::string pre = "fp8q_kv4_plan: ";
  if (B < 0 || F < 0 || T < 0 || pages < 0 || max_pages < 0) return fail(FP8Q_EINVAL, pre + "negative size");
  if (table_sb < 0) return fail(FP8Q_EINVAL, pre + "negative stride");
  if (B > kMaxSequences) return fail(FP8Q_EUNSUPPORTED, pre + "at most 4096 sequences");
  if (log2_exact(page_size) < 0) return fail(FP8Q_EUNSUPPORTED, pre + "page_size must be a power of two below 2^31");
  if (pages >= (int64_t(1) << 31) || pages * page_size >= (int64_t(1) << 31))
    return fail(FP8Q_EUNSUPPORTED, pre + "the cache must have fewer than 2^31 slots");
  if (T >= (int64_t(1) << 30)) return fail(FP8Q_EUNSUPPORTED, pre + "fewer than 2^30 new tokens");
  if (max_pages > (int64_t(1) << 30) || max_pages * page_size > (int64_t(1) << 30))
    return fail(FP8Q_EUNSUPPORTED, pre + "at most 2^30 tokens in a sequence's pages");
  if (F >= (int64_t(1) << 31)) return fail(FP8Q_EUNSUPPORTED, pre + "fewer than 2^31 free pages");
  if (table_sb > (int64_t(1) << 40)) return fail(FP8Q_EUNSUPPORTED, pre + "a block table stride of at most 2^40");
  if (!q_indptr || !pages_taken || (B > 0 && (!kv_lens || !q_lens || !new_lens)) || (F > 0 && !free_pages) ||
      (T > 0 && !slots) || (B > 0 && max_pages > 0 && !table))
    return fail(FP8Q_EINVAL, pre + "null tensor pointer");
  if (B > 1 && table_sb < max_pages) return fail(FP8Q_EINVAL, pre + "rows of the block table overlap");
  if (!aligned(kv_lens, 4) || !aligned(q_lens, 4) || !aligned(free_pages, 4) || !aligned(table, 4) || !aligned(new_lens, 4) ||
      !aligned(q_indptr, 4) || !aligned(slots, 4) || !aligned(positions, 4) || !aligned(pages_taken, 4))
    return fail(FP8Q_EALIGN, pre + "every tensor must be 4-byte aligned");
  // Blocks read the inputs while others write: no output may share memory with anything else.
  const Bytes all[9] = {{new_lens, 4 * B}, {q_indptr, 4 * (B + 1)}, {slots, 4 * T}, {positions, 4 * T}, {pages_taken, 4},
                        {table, B > 0 ? 4 * ((B - 1) * table_sb + max_pages) : 0},
                        {kv_lens, 4 * B}, {q_lens, 4 * B}, {free_pages, 4 * F}};
  for (int i = 0; i < 6; i++)
    for (int j = i + 1; j < 9; j++)
      if (overlap(all[i], all[j])) return fail(FP8Q_EINVAL, pre + "an output overlaps another tensor");
  const int dev = check_current_device();
  if (dev != FP8Q_OK) return dev;
  Kv4PlanParams p{};
  p.kv_lens = kv_lens;
  p.q_lens = q_lens;
  p.free_pages = free_pages;
  p.table = table;
  p.table_sb = table_sb;
  p.max_tokens = max_pages * page_size;
  p.B = B;
  p.T = T;
  p.F = F;
  p.pages = pages;
  p.page_shift = log2_exact(page_size);
  p.new_lens = new_lens;
  p.q_indptr = q_indptr;
  p.slots = slots;
  p.positions = positions;
  p.pages_taken = pages_taken;
  return launch_kv4_plan(p, static_cast<hipStream_t>(stream));
}

}  // namespace
}  // namespace fp8q

extern "C" {

int fp8q_rms_norm_group_quant(const void* x, int in_dtype, int64_t M, int64_t K, int64_t x_sm, const void* residual,
                              int64_t r_sm, void* residual_out, int64_t ro_sm, const void* weight, float eps,
                              uint8_t* q, int64_t q_sm, void* s, int scale_fmt, int64_t s_sm, int64_t s_sg,
                              int group_size, void* stream) {
  return fp8q::norm_entry(x, in_dtype, M, K, x_sm, residual, r_sm, residual_out, ro_sm, weight, eps, q, q_sm, s,
                          scale_fmt, s_sm, s_sg, group_size, stream);
}

int fp8q_kv4_write(const void* k, int64_t k_st, int64_t k_sh, const void* v, int64_t v_st, int64_t v_sh, int in_dtype,
                   int64_t T, int64_t H, int64_t D, const int32_t* slots, uint8_t* kc, uint8_t* ks, uint8_t* vc,
                   uint8_t* vs, int64_t pages, int64_t page_size, int64_t c_sp, int64_t c_st, int64_t c_sh,
                   int64_t s_sp, int64_t s_st, int64_t s_sh, void* stream) {
  return fp8q::rows_entry(true, k, k_st, k_sh, v, v_st, v_sh, in_dtype, T, H, D, slots, kc, ks, vc, vs, pages,
                          page_size, c_sp, c_st, c_sh, s_sp, s_st, s_sh, stream);
}

int fp8q_kv4_read(void* k, int64_t k_st, int64_t k_sh, void* v, int64_t v_st, int64_t v_sh, int out_dtype, int64_t T,
                  int64_t H, int64_t D, const int32_t* slots, const uint8_t* kc, const uint8_t* ks, const uint8_t* vc,
                  const uint8_t* vs, int64_t pages, int64_t page_size, int64_t c_sp, int64_t c_st, int64_t c_sh,
                  int64_t s_sp, int64_t s_st, int64_t s_sh, void* stream) {
  return fp8q::rows_entry(false, k, k_st, k_sh, v, v_st, v_sh, out_dtype, T, H, D, slots, kc, ks, vc, vs, pages,
                          page_size, c_sp, c_st, c_sh, s_sp, s_st, s_sh, stream);
}

int64_t fp8q_kv4_attention_workspace_size(int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                          int64_t max_tokens) {
  return fp8q::attention_workspace("fp8q_kv4_attention_workspace_size: ", dtype, B, T, Hq, Hkv, D, max_tokens,
                                   {fp8q::kAll, 1, 0, 0, nullptr, 0, 0});
}

int fp8q_kv4_attention(
    const void* q, int dtype, int64_t q_st, int64_t q_sh, const uint8_t* kc, const uint8_t* ks,
    const uint8_t* vc, const uint8_t* vs, int64_t pages, int64_t page_size, int64_t c_sp, int64_t c_st, int64_t c_sh,
    int64_t s_sp, int64_t s_st, int64_t s_sh, const int32_t* table, int64_t table_sb, int64_t max_pages,
    const int32_t* kv_lens, const int32_t* q_indptr, void* out, int64_t o_st, int64_t o_sh, float* lse, int64_t l_st,
    int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, float sm_scale, int causal, void* workspace,
    int64_t workspace_bytes, void* stream) {
  return fp8q::attention_entry("fp8q_kv4_attention: ", {fp8q::kAll, causal, 0, 0, nullptr, 0, 0}, q, dtype, q_st, q_sh, kc, ks, vc, vs,
                               pages, page_size, c_sp, c_st, c_sh, s_sp, s_st, s_sh, table, table_sb, max_pages, kv_lens,
                               q_indptr, out, o_st, o_sh, lse, l_st, B, T, Hq, Hkv, D, sm_scale, workspace,
                               workspace_bytes, stream);
}

int64_t fp8q_kv4_window_attention_workspace_size(int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                                 int64_t max_tokens, int64_t window, int64_t sinks) {
  return fp8q::attention_workspace("fp8q_kv4_window_attention_workspace_size: ", dtype, B, T, Hq, Hkv, D, max_tokens,
                                   {fp8q::kWindow, 1, window, sinks, nullptr, 0, 0});
}

int fp8q_kv4_window_attention(
    const void* q, int dtype, int64_t q_st, int64_t q_sh, const uint8_t* kc, const uint8_t* ks,
    const uint8_t* vc, const uint8_t* vs, int64_t pages, int64_t page_size, int64_t c_sp, int64_t c_st, int64_t c_sh,
    int64_t s_sp, int64_t s_st, int64_t s_sh, const int32_t* table, int64_t table_sb, int64_t max_pages,
    const int32_t* kv_lens, const int32_t* q_indptr, void* out, int64_t o_st, int64_t o_sh, float* lse, int64_t l_st,
    int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, float sm_scale, int64_t window, int64_t sinks,
    void* workspace, int64_t workspace_bytes, void* stream) {
  return fp8q::attention_entry("fp8q_kv4_window_attention: ", {fp8q::kWindow, 1, window, sinks, nullptr, 0, 0}, q, dtype, q_st, q_sh, kc, ks, vc, vs,
                               pages, page_size, c_sp, c_st, c_sh, s_sp, s_st, s_sh, table, table_sb, max_pages, kv_lens,
                               q_indptr, out, o_st, o_sh, lse, l_st, B, T, Hq, Hkv, D, sm_scale, workspace,
                               workspace_bytes, stream);
}

int64_t fp8q_kv4_tree_attention_workspace_size(int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                               int64_t max_tokens) {
  return fp8q::attention_workspace("fp8q_kv4_tree_attention_workspace_size: ", dtype, B, T, Hq, Hkv, D, max_tokens,
                                   {fp8q::kTree, 0, 0, 0, nullptr, 0, 0});
}

int fp8q_kv4_tree_attention(
    const void* q, int dtype, int64_t q_st, int64_t q_sh, const uint8_t* kc, const uint8_t* ks,
    const uint8_t* vc, const uint8_t* vs, int64_t pages, int64_t page_size, int64_t c_sp, int64_t c_st, int64_t c_sh,
    int64_t s_sp, int64_t s_st, int64_t s_sh, const int32_t* table, int64_t table_sb, int64_t max_pages,
    const int32_t* kv_lens, const int32_t* q_indptr, void* out, int64_t o_st, int64_t o_sh, float* lse, int64_t l_st,
    int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, float sm_scale, const int32_t* tree_mask,
    int64_t tree_st, int64_t tree_words, void* workspace, int64_t workspace_bytes, void* stream) {
  return fp8q::attention_entry("fp8q_kv4_tree_attention: ", {fp8q::kTree, 0, 0, 0, tree_mask, tree_st, tree_words}, q, dtype, q_st, q_sh, kc, ks, vc, vs,
                               pages, page_size, c_sp, c_st, c_sh, s_sp, s_st, s_sh, table, table_sb, max_pages, kv_lens,
                               q_indptr, out, o_st, o_sh, lse, l_st, B, T, Hq, Hkv, D, sm_scale, workspace,
                               workspace_bytes, stream);
}

int fp8q_kv4_plan(const int32_t* kv_lens, const int32_t* q_lens, int64_t B, const int32_t* free_pages, int64_t F,
                  int32_t* table, int64_t table_sb, int64_t max_pages, int64_t pages, int64_t page_size, int32_t* new_lens,
                  int32_t* q_indptr, int32_t* slots, int32_t* positions, int64_t T, int32_t* pages_taken, void* stream) {
  return fp8q::plan_entry(kv_lens, q_lens, B, free_pages, F, table, table_sb, max_pages, pages, page_size, new_lens,
                          q_indptr, slots, positions, T, pages_taken, stream);
}

}  // extern "C"
