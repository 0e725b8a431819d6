// serving.h — launchers and parameters of the serving operators around the GEMMs: the
// quantizing norm and the 4-bit key/value cache. Not part of the public ABI (include/fp8q.h).
#pragma once

#include "fp8q_internal.h"

namespace fp8q {

// ------------------------------------------------------------------ norm
struct NormParams {
  const void* x;
  const void* res;  // nullptr: none
  void* res_out;    // nullptr: not stored
  const void* w;
  uint8_t* q;
  void* s;
  int64_t M, K;
  int64_t x_sm, r_sm, ro_sm;   // elements
  int64_t q_sm;                // bytes
  int64_t s_sm, s_sg;          // scale elements (packed UE8M0: words of 4 groups)
  float eps;
  double inv_k;                // 1 / K
  int32_t group;               // 32, 64, 128, or 0 (one group per row)
  int32_t group_shift;         // log2 of it (one group per row: any shift past the row)
  int32_t ue8m0, packed;
};

constexpr int64_t kNormMaxK = 65536;  // longest row that a block keeps in registers

int launch_rms_norm_quant(int dtype, const NormParams& p, hipStream_t stream);

// ------------------------------------------------------------------ 4-bit cache
constexpr int kKv4Block = 32;  // elements of a cached row that share one scale byte

// Row (page, token, head) of the codes is at c_sp * page + c_st * token + c_sh * head bytes,
// its D / 32 scale bytes at the same with s_*.
struct Kv4Cache {
  uint8_t* k;
  uint8_t* ks;
  uint8_t* v;
  uint8_t* vs;
  int64_t pages;
  int32_t page_shift;  // log2 of the page size
  int64_t c_sp, c_st, c_sh, s_sp, s_st, s_sh;
};

struct Kv4RowsParams {
  Kv4Cache c;
  void* x[2];           // keys, values [T][H][D]
  int64_t x_st[2], x_sh[2];
  const int32_t* slots;
  int64_t T;
  int32_t H, D, d_shift;  // D = 1 << d_shift
};

int launch_kv4_write(int dtype, const Kv4RowsParams& p, hipStream_t stream);
int launch_kv4_read(int dtype, const Kv4RowsParams& p, hipStream_t stream);

struct Kv4AttnParams {
  Kv4Cache c;
  const void* q;             // [T][Hq][D]
  int64_t q_st, q_sh;
  void* out;                 // [T][Hq][D]
  int64_t o_st, o_sh;
  float* lse;                // [T][Hq], or nullptr
  int64_t l_st;
  const int32_t* table;      // [B][max_pages]
  int64_t table_sb;
  int64_t max_tokens;        // max_pages << page_shift
  const int32_t* kv_lens;    // [B]
  const int32_t* q_indptr;   // [B + 1], or nullptr: sequence b is row b
  int64_t B, T;
  int32_t Hq, Hkv, group;    // group = Hq / Hkv
  float scale_log2;          // magnitude of the softmax scale times 4 log2(e)
  uint32_t q_sign;           // 0x80008000 where the scale is negative
  int32_t causal;
  int32_t span_shift;        // log2 of the tokens of a span
  int64_t max_units;         // query tiles x cached heads, at most
  int32_t blocks;            // split only, as the next two: blocks that share the line of spans
  int32_t* plan;             // [2][B + 1] spans and query tiles before each sequence
  float* parts;              // partial outputs, maxima and sums by piece
};

// Bytes of workspace with which attention of this shape splits the cache axis on the current
// device (0: it never does).
int64_t kv4_attention_workspace(int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_tokens);
int launch_kv4_attention(int dtype, int64_t D, Kv4AttnParams p, void* ws, int64_t ws_bytes, hipStream_t stream);

}  // namespace fp8q
