// kv4_attention.hip — attention over the paged 4-bit cache.
//
//   out[t][h] = sum_j p_j v_j, p = softmax_j(scale * q[t][h] . k_j) over the cached tokens j that
//   query t sees (all of its sequence's, or with `causal` those up to its own place).
//
// One pass over the cache with a running maximum and sum per query row (fp32, base 2). Query
// heads that share a cached head are rows of one tile, so the cache is read once for all.
//
// Tiles. A unit is 16 query rows (tokens x heads of the group) of one cached head against the
// sequence's cached tokens, cut into spans of 128 tokens. The waves of a block take 32 tokens of
// a span each, with a running softmax of their own; their results meet in LDS at the end. With a
// workspace, the spans of all units in a row are cut into equal runs, one per block, wherever
// the cuts fall: every block has the same work however ragged the lengths are. A unit that is
// cut leaves a piece per block, which a second kernel joins.
//
// Layouts (v_mfma_f32_16x16x32_bf16; lane l, r = l % 16, h = l / 16):
//   S^T = K Q^T: lane (r, h) loads dims [D/4 h, D/4 (h + 1)) of token r, one or two scale blocks
//     of which all elements share one scale, and converts them in registers. The contraction
//     index is free, so step j takes dims D/4 h + 8j .. + 7 from lane group h of both operands.
//     e2m1 times a power of two is exact in bf16: no error is added.
//   S^T leaves lane (r, h) with tokens 4h .. 4h + 3 of query row r: as the operand of O^T = V^T P^T
//     that is a permutation of the contraction index, which V^T's reads follow, so P never
//     leaves its registers.
//   V^T: V is converted to bf16 token by token, put into LDS and read transposed
//     (ds_read_b64_tr_b16: lane (r, h) gets dim r of tokens 4h .. 4h + 3).
//
// fp16 queries are the sum of two bf16 parts (8 + 3 bits of their 11), multiplied one after the
// other; the probabilities likewise for fp16 outputs. For bf16 outputs the probabilities are
// rounded to bf16 once: the error, 2^-8 of each term at most, is of the size of the output's
// own rounding.
#include <algorithm>

#include "serving.h"
#include "serving_device.h"

#pragma clang fp contract(off)

namespace fp8q {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 16;   // query rows of an item
constexpr int kTile = 32;   // tokens of a wave's step
constexpr int kSpan = kTile * kWaves;  // tokens of a block's step: chunks are whole spans
constexpr int kPadV = 16;   // elements between the V rows in LDS
constexpr int kMinRun = 2;  // spans of a block's run at least
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// Maximum and sum over the four lanes with the same l % 16.
__device__ __forceinline__ float quad_max(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ int32_t clamp32(int32_t v, int64_t hi) {
  return v < 0 ? 0 : v > hi ? static_cast<int32_t>(hi) : v;
}

struct Seq {
  int32_t q0, q_len, kv_len;
};

__device__ __forceinline__ Seq sequence(const Kv4AttnParams& p, int32_t b) {
  Seq s;
  s.q0 = b;
  s.q_len = 1;
  if (p.q_indptr) {
    s.q0 = clamp32(p.q_indptr[b], p.T);
    s.q_len = max(clamp32(p.q_indptr[b + 1], p.T) - s.q0, 0);
  }
  s.kv_len = clamp32(p.kv_lens[b], p.max_tokens);
  return s;
}

__device__ __forceinline__ int32_t tiles_of(const Kv4AttnParams& p, const Seq& s) {
  return static_cast<int32_t>((static_cast<int64_t>(s.q_len) * p.group + kRows - 1) / kRows);
}
// A sequence without cached tokens has one empty span, so that its rows are written.
__device__ __forceinline__ int32_t spans_of(const Seq& s) { return max((s.kv_len + kSpan - 1) / kSpan, 1); }

// ------------------------------------------------------------------ units and runs
// Prefixes over the sequences: first[b] the query tiles, line[b] the (tile, span) pairs before
// sequence b. Unit (b, tile, head) is number (first[b] + tile) * Hkv + head and has the places
// [line[b] * Hkv + (tile * Hkv + head) * spans, + spans) of the line of all spans.
struct Plan {
  int64_t* line;   // [B + 1]
  int32_t* first;  // [B + 1]
};

// Inclusive sum over the block's threads; `lds` holds one value per wave.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* lds, T& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T up = __shfl_up(v, off, 64);
    if (lane >= off) v += up;
  }
  if (lane == 63) lds[wave] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; w++) {
    if (w < wave) v += lds[w];
    total += lds[w];
  }
  return v;
}

// Fills the plan in LDS; every block computes the same from the lengths. A q_indptr that does
// not ascend can name more rows than there are: then the plan is empty and nothing is run.
__device__ __forceinline__ void make_plan(const Kv4AttnParams& p, const Plan& plan) {
  __shared__ long long tot_line[kWaves], tot_first[kWaves];
  const int tid = threadIdx.x;
  const int32_t B = static_cast<int32_t>(p.B);
  const int32_t per = (B + kThreads - 1) / kThreads;
  const int32_t beg = min(tid * per, B), end = min(beg + per, B);
  long long my_line = 0, my_first = 0;
  for (int32_t b = beg; b < end; b++) {
    const Seq s = sequence(p, b);
    const long long tiles = tiles_of(p, s);
    my_first += tiles;
    my_line += tiles * spans_of(s);
  }
  long long all_line, all_first;
  long long at_first = block_scan(my_first, tot_first, all_first) - my_first;
  long long at_line = block_scan(my_line, tot_line, all_line) - my_line;
  const bool fits = all_first * p.Hkv <= p.max_units;
  for (int32_t b = beg; b < end; b++) {
    const Seq s = sequence(p, b);
    plan.first[b] = fits ? static_cast<int32_t>(at_first) : 0;
    plan.line[b] = fits ? at_line : 0;
    const long long tiles = tiles_of(p, s);
    at_first += tiles;
    at_line += tiles * spans_of(s);
  }
  if (tid == kThreads - 1) {
    plan.first[B] = fits ? static_cast<int32_t>(all_first) : 0;
    plan.line[B] = fits ? all_line : 0;
  }
  __syncthreads();
}

// The last b with pref[b] <= v (pref ascending, pref[0] <= v).
template <typename T>
__device__ __forceinline__ int32_t find_seq(const T* pref, int32_t B, T v) {
  int32_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (pref[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// Spans of one block's run when `blocks` blocks share a line of `total` spans.
__device__ __forceinline__ int64_t run_length(int64_t total, int32_t blocks) {
  return max((total + blocks - 1) / blocks, static_cast<int64_t>(kMinRun));
}

// ------------------------------------------------------------------ cached rows
// A lane's part of one token's row: D / 4 elements.
template <int D>
struct Codes {
  uint32_t w[D / 32];
  uint32_t scale;  // byte i: the scale of elements 32i .. (one for D <= 128, two for D = 256)
};

template <int D>
__device__ __forceinline__ void load_codes(const uint8_t* codes, const uint8_t* scales, int h, Codes<D>& c) {
  if constexpr (D == 64) {
    const u32x2 a = *reinterpret_cast<const u32x2*>(codes + 8 * h);
    c.w[0] = a[0];
    c.w[1] = a[1];
    c.scale = scales[h >> 1];
  } else if constexpr (D == 128) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(codes + 16 * h);
#pragma unroll
    for (int i = 0; i < 4; i++) c.w[i] = a[i];
    c.scale = scales[h];
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(codes + 32 * h);
    const u32x4 b = *reinterpret_cast<const u32x4*>(codes + 32 * h + 16);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      c.w[i] = a[i];
      c.w[4 + i] = b[i];
    }
    c.scale = *reinterpret_cast<const uint16_t*>(scales + 2 * h);
  }
}

template <int D>
__device__ __forceinline__ void zero_codes(Codes<D>& c) {
#pragma unroll
  for (int i = 0; i < D / 32; i++) c.w[i] = 0u;
  c.scale = 0x7F7Fu;
}

// Word i of a lane's part as 8 bf16 values (exact).
template <int D>
__device__ __forceinline__ bf16x8 widen_codes(const Codes<D>& c, int i) {
  const uint32_t byte = D == 256 && i >= 4 ? c.scale >> 8 : c.scale & 0xFFu;
  const float s = __uint_as_float(byte << 23);
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.w[i], s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.w[i], s, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.w[i], s, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.w[i], s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// The 32 tokens of one step of a wave: tokens 0-15 in part 0, 16-31 in part 1.
template <int D>
struct Step {
  Codes<D> k[2], v[2];
  uint32_t there;  // bit i: token i is inside the range and its page is in the cache
};

// Page numbers of a step's two halves: of the whole half where a page holds 16 tokens or more
// (PAGE16, wave-uniform), else of the lane's token.
struct Pages {
  int32_t n[2];
};

template <bool PAGE16>
__device__ __forceinline__ Pages load_pages(const Kv4AttnParams& p, const int32_t* table, int32_t t, int32_t t_end) {
  Pages g;
#pragma unroll
  for (int s = 0; s < 2; s++) {
    // past the end: the last token's page, which is there to be read
    const int32_t tok = min(t + 16 * s + (PAGE16 ? 0 : static_cast<int>(threadIdx.x & 15)), t_end - 1);
    g.n[s] = table[tok >> p.c.page_shift];
  }
  return g;
}

// Loads a step's codes and scales. Every address is inside the cache: a page that is not there
// is replaced by page 0, and tokens past the end lie in the last token's page or in a valid
// one; what is loaded for them is not used (`there`).
template <int D, bool PAGE16>
__device__ __forceinline__ void load_step(const Kv4AttnParams& p, const Pages& g, int64_t head_c, int64_t head_s,
                                          int32_t t, int32_t t_end, Step<D>& st) {
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int32_t mask = (1 << p.c.page_shift) - 1;
  uint32_t there = 0;
#pragma unroll
  for (int s = 0; s < 2; s++) {
    const int32_t left = t_end - (t + 16 * s);  // tokens of this half inside the range
    int64_t c = head_c, b = head_s;
    if constexpr (PAGE16) {
      const bool ok = g.n[s] >= 0 && g.n[s] < p.c.pages;
      const int64_t page = ok ? g.n[s] : 0;
      const int64_t in = (t + 16 * s) & mask;
      c += page * p.c.c_sp + in * p.c.c_st;
      b += page * p.c.s_sp + in * p.c.s_st;
      const uint32_t bits = !ok || left <= 0 ? 0u : left >= 16 ? 0xFFFFu : (1u << left) - 1u;
      there |= bits << (16 * s);
      load_codes<D>(p.c.k + c + r * static_cast<uint32_t>(p.c.c_st), p.c.ks + b + r * static_cast<uint32_t>(p.c.s_st), h, st.k[s]);
      load_codes<D>(p.c.v + c + r * static_cast<uint32_t>(p.c.c_st), p.c.vs + b + r * static_cast<uint32_t>(p.c.s_st), h, st.v[s]);
    } else {
      const bool ok = g.n[s] >= 0 && g.n[s] < p.c.pages;
      const int64_t page = ok ? g.n[s] : 0;
      const int64_t in = min(t + 16 * s + r, t_end - 1) & mask;
      c += page * p.c.c_sp + in * p.c.c_st;
      b += page * p.c.s_sp + in * p.c.s_st;
      there |= static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(ok && r < left) & 0xFFFFu) << (16 * s);
      load_codes<D>(p.c.k + c, p.c.ks + b, h, st.k[s]);
      load_codes<D>(p.c.v + c, p.c.vs + b, h, st.v[s]);
    }
  }
  st.there = there;
}

// ------------------------------------------------------------------ the kernel
template <int DT>
__device__ __forceinline__ float to_f32(uint32_t half) {
  if constexpr (DT == FP8Q_DTYPE_BF16) return bf16_lo(half);
  else return f16_lo(half);
}

// bf16: one part. fp16: high and low parts whose sum is the value.
template <int DT, int PARTS>
__device__ __forceinline__ void split8(const u32x4 raw, bf16x8 (&out)[PARTS]) {
  if constexpr (DT == FP8Q_DTYPE_BF16) {
    out[0] = __builtin_bit_cast(bf16x8, raw);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float v = i & 1 ? f16_hi(raw[i >> 1]) : f16_lo(raw[i >> 1]);
      out[0][i] = static_cast<__bf16>(v);
      out[1][i] = static_cast<__bf16>(v - static_cast<float>(out[0][i]));
    }
  }
}

// Waves per SIMD that the registers are kept to (O^T and Q take D / 4 + D / 8 of them per lane).
constexpr int waves_per_simd(int D, int DT) { return D == 256 ? 2 : DT == FP8Q_DTYPE_F16 && D == 128 ? 3 : 4; }

template <int D, int DT, bool SPLIT, bool PAGE16>
__global__ __launch_bounds__(kThreads, waves_per_simd(D, DT)) void kv4_attention_kernel(Kv4AttnParams p) {
  constexpr int PARTS = DT == FP8Q_DTYPE_F16 ? 2 : 1;
  constexpr int kSteps = D / 32;   // contraction steps of S^T
  constexpr int kDims = D / 16;    // dim tiles of O^T
  constexpr int kRowV = D + kPadV;  // LDS row of V (bf16 elements)
  constexpr int kRowO = D + 4;      // LDS row of the joined output (floats)
  static_assert(kRows * kRowO * 4 <= kTile * kRowV * 2, "the joined output reuses V's LDS");
  __shared__ __align__(16) uint16_t lds_v[kWaves][kTile * kRowV];
  __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];
  extern __shared__ __align__(16) uint8_t lds_plan[];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int r = lane & 15, h = lane >> 4;
  const int32_t B = static_cast<int32_t>(p.B);
  const Plan plan{reinterpret_cast<int64_t*>(lds_plan), reinterpret_cast<int32_t*>(lds_plan + (B + 1) * 8)};

  // one unit per sequence and cached head, in order, unless something is split or has several tiles
  const bool direct = !SPLIT && p.q_indptr == nullptr && p.group <= kRows;
  if (!direct) make_plan(p, plan);

  // this block's places on the line: of spans when splitting, else of units
  int64_t at, stop;
  if constexpr (SPLIT) {
    const int64_t total = plan.line[B] * p.Hkv, run = run_length(total, p.blocks);
    at = min(blockIdx.x * run, total);
    stop = min(at + run, total);
    if (blockIdx.x == 0) {
      for (int32_t b = tid; b <= B; b += kThreads) {
        p.plan_line[b] = plan.line[b];
        p.plan_first[b] = plan.first[b];
      }
    }
  } else {
    at = blockIdx.x;
    stop = (direct ? p.B : static_cast<int64_t>(plan.first[B])) * p.Hkv;
  }

  while (at < stop) {
    // the unit at this place, and its spans [s0, s1) of this run
    int32_t b, tile = 0, head, s0 = 0, s1;
    Seq seq;
    int64_t next, piece = 0;
    bool whole = true;
    if constexpr (SPLIT) {
      b = __builtin_amdgcn_readfirstlane(find_seq(plan.line, B, at / p.Hkv));
      seq = sequence(p, b);
      const int32_t spans = spans_of(seq);
      const int64_t in = at - plan.line[b] * p.Hkv;
      const int32_t unit = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(in / spans));
      tile = unit / p.Hkv;
      head = unit - tile * p.Hkv;
      s0 = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(in - static_cast<int64_t>(unit) * spans));
      s1 = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(min(static_cast<int64_t>(spans), s0 + (stop - at))));
      next = at + (s1 - s0);
      whole = s0 == 0 && s1 == spans;
      piece = blockIdx.x + static_cast<int64_t>(plan.first[b]) * p.Hkv + unit;
    } else {
      const int32_t u = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(at / p.Hkv));
      head = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(at - static_cast<int64_t>(u) * p.Hkv));
      b = direct ? u : __builtin_amdgcn_readfirstlane(find_seq(plan.first, B, u));
      seq = sequence(p, b);
      if (!direct) tile = u - __builtin_amdgcn_readfirstlane(plan.first[b]);
      s1 = spans_of(seq);
      next = at + gridDim.x;
    }
    at = next;

    // this lane's query row; rows [first, last] of the tile exist
    const int64_t first = static_cast<int64_t>(tile) * kRows;
    const int64_t rows = static_cast<int64_t>(seq.q_len) * p.group;
    const int64_t last = min(first + kRows, rows) - 1;
    const bool row_there = first + r <= last;
    const int64_t idx = row_there ? first + r : last;
    const int32_t qi = static_cast<int32_t>(idx / p.group);
    const int32_t qh = head * p.group + static_cast<int32_t>(idx - static_cast<int64_t>(qi) * p.group);
    const int32_t before = seq.kv_len - seq.q_len + 1;  // tokens that query 0 sees
    const int32_t limit = p.causal ? min(before + qi, seq.kv_len) : seq.kv_len;
    const int32_t low = p.causal ? before + static_cast<int32_t>(first / p.group) : seq.kv_len;  // of the first row
    const int32_t high = p.causal ? before + static_cast<int32_t>(last / p.group) : seq.kv_len;  // of the last
    const int32_t t_end = min(min(s1 * kSpan, seq.kv_len), high);

    const int32_t* table = p.table + b * p.table_sb;
    const int64_t head_c = head * p.c.c_sh, head_s = head * p.c.s_sh;
    int32_t t = s0 * kSpan + kTile * wave;
    Step<D> st;
    Pages pages;
    if (t < t_end) {
      pages = load_pages<PAGE16>(p, table, t, t_end);
      load_step<D, PAGE16>(p, pages, head_c, head_s, t, t_end, st);
      pages = load_pages<PAGE16>(p, table, t + kSpan, t_end);
    }

    bf16x8 q[PARTS][kSteps];
    {
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + (seq.q0 + qi) * p.q_st + qh * p.q_sh + D / 4 * h;
#pragma unroll
      for (int j = 0; j < kSteps; j++) {
        u32x4 raw = {0u, 0u, 0u, 0u};
        if (row_there) raw = *reinterpret_cast<const u32x4*>(src + 8 * j);
        bf16x8 part[PARTS];
        split8<DT, PARTS>(raw, part);
#pragma unroll
        for (int a = 0; a < PARTS; a++) q[a][j] = part[a];
      }
    }

    uint16_t* vt = lds_v[wave];
    f32x4 o[kDims];
#pragma unroll
    for (int d = 0; d < kDims; d++) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = kNegInf, l = 0.0f;  // l: this lane's share of the row's sum

    for (; t < t_end; t += kSpan) {
      f32x4 s[2];
#pragma unroll
      for (int c = 0; c < 2; c++) {
        s[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kSteps; j++) {
          const bf16x8 k = widen_codes<D>(st.k[c], j);
#pragma unroll
          for (int a = 0; a < PARTS; a++) s[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[a][j], s[c], 0, 0, 0);
        }
      }
      const uint32_t there = st.there;
      const bool part = there != 0xFFFFFFFFu || t + kTile > low;  // wave-uniform
#pragma unroll
      for (int c = 0; c < 2; c++) {
        if (there != 0xFFFFFFFFu && ((there >> (16 * c + r)) & 1u) == 0u) zero_codes<D>(st.v[c]);
#pragma unroll
        for (int j = 0; j < kSteps; j++)
          *reinterpret_cast<bf16x8*>(vt + (16 * c + r) * kRowV + D / 4 * h + 8 * j) = widen_codes<D>(st.v[c], j);
      }
      // the next step's codes come in while this one's softmax and second product run
      if (t + kSpan < t_end) {
        load_step<D, PAGE16>(p, pages, head_c, head_s, t + kSpan, t_end, st);
        pages = load_pages<PAGE16>(p, table, t + 2 * kSpan, t_end);
      }

      float x[2][4], mx = kNegInf;
#pragma unroll
      for (int c = 0; c < 2; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) x[c][i] = s[c][i] * p.scale_log2;
      if (part) {
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int n = 16 * c + 4 * h + i;
            if (((there >> n) & 1u) == 0u || t + n >= limit) x[c][i] = kNegInf;
          }
      }
#pragma unroll
      for (int c = 0; c < 2; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) mx = fmaxf(mx, x[c][i]);
      mx = fmaxf(quad_max(mx), m);
      const float ms = mx == kNegInf ? 0.0f : mx;  // nothing seen yet: every p is 0
      if (__builtin_amdgcn_ballot_w64(mx > m) != 0) {
        const float alpha = exp2_fast(m - ms);
        m = mx;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < kDims; d++)
#pragma unroll
          for (int i = 0; i < 4; i++) o[d][i] *= alpha;
      }
      bf16x8 pr[PARTS];
#pragma unroll
      for (int c = 0; c < 2; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float e = exp2_fast(x[c][i] - ms);
          l += e;
          pr[0][4 * c + i] = static_cast<__bf16>(e);
          if constexpr (PARTS == 2) pr[1][4 * c + i] = static_cast<__bf16>(e - static_cast<float>(pr[0][4 * c + i]));
        }

      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int d = 0; d < kDims; d++) {
        const uint16_t* src = vt + (4 * h + (r >> 2)) * kRowV + 16 * d + 4 * (r & 3);
        const s16x4 a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src));
        const s16x4 a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 16 * kRowV));
        const auto av = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int a = 0; a < PARTS; a++)
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av), pr[a], o[d], 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }

    // join the waves
    l = quad_sum(l);
    if (h == 0) {
      lds_m[wave][r] = m;
      lds_l[wave][r] = l;
    }
    __syncthreads();
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; w++) top = fmaxf(top, lds_m[w][r]);
    {
      const float f = exp2_fast(m - (top == kNegInf ? 0.0f : top));
      float* dst = reinterpret_cast<float*>(vt) + r * kRowO + 4 * h;
#pragma unroll
      for (int d = 0; d < kDims; d++) *reinterpret_cast<f32x4*>(dst + 16 * d) = o[d] * f;
    }
    __syncthreads();
    for (int e = tid; e < kRows * (D / 8); e += kThreads) {
      const int row = e / (D / 8), col = e % (D / 8) * 8;
      if (first + row > last) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = 0.0f;
      float mm = kNegInf, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; w++) {
        const float* src = reinterpret_cast<const float*>(lds_v[w]) + row * kRowO + col;
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] += src[i];
        mm = fmaxf(mm, lds_m[w][row]);
      }
#pragma unroll
      for (int w = 0; w < kWaves; w++) ll += lds_l[w][row] * exp2_fast(lds_m[w][row] - (mm == kNegInf ? 0.0f : mm));
      if (SPLIT && !whole) {
        float* part = p.parts + piece * (kRows * (D + 2));
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          *reinterpret_cast<f32x4*>(part + row * D + col + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
        if (col == 0) {
          part[kRows * D + 2 * row] = mm;
          part[kRows * D + 2 * row + 1] = ll;
        }
      } else {
        const int64_t ri = first + row;
        const int32_t i = static_cast<int32_t>(ri / p.group);
        const int64_t row_t = seq.q0 + i, hh = head * p.group + static_cast<int32_t>(ri - static_cast<int64_t>(i) * p.group);
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] = pack16<DT>(v[2 * j] * inv, v[2 * j + 1] * inv);
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + row_t * p.o_st + hh * p.o_sh + col) = w;
        if (p.lse && col == 0)
          p.lse[row_t * p.l_st + hh] = ll > 0.0f ? (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f : kNegInf;
      }
    }
    __syncthreads();
  }
}

// Joins the pieces of one query row: a block per (token, query head). The waves take the pieces
// in turn, every lane D / 64 elements.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void kv4_join_kernel(Kv4AttnParams p) {
  constexpr int kPer = D / 64;
  __shared__ float lds_o[kWaves][D], lds_l[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int32_t t = static_cast<int32_t>(blockIdx.x / p.Hq), qh = static_cast<int32_t>(blockIdx.x % p.Hq);
  int32_t b = t;
  if (p.q_indptr) {
    // the sequence that holds row t: the last one whose clamped start is not after it
    int32_t lo = 0, hi = static_cast<int32_t>(p.B);
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (clamp32(p.q_indptr[mid], p.T) <= t) lo = mid; else hi = mid;
    }
    b = lo;
  }
  const Seq seq = sequence(p, b);
  if (t < seq.q0 || t >= seq.q0 + seq.q_len) return;
  const int32_t head = qh / p.group, spans = spans_of(seq);
  const int64_t idx = static_cast<int64_t>(t - seq.q0) * p.group + (qh - head * p.group);
  const int64_t unit = idx / kRows * p.Hkv + head;
  const int row = static_cast<int>(idx % kRows);
  // the runs that hold a part of this unit
  const int64_t total = p.plan_line[p.B] * p.Hkv;
  if (total == 0) return;
  const int64_t run = run_length(total, p.blocks), from = p.plan_line[b] * p.Hkv + unit * spans;
  const int64_t run0 = from / run, run1 = (from + spans - 1) / run;
  if (run0 == run1) return;
  const int32_t chunks = static_cast<int32_t>(run1 - run0) + 1;
  constexpr int64_t step = kRows * (D + 2);
  const float* base = p.parts + (run0 + static_cast<int64_t>(p.plan_first[b]) * p.Hkv + unit) * step;

  float top = kNegInf;
  for (int32_t c = lane; c < chunks; c += 64) top = fmaxf(top, base[c * step + kRows * D + 2 * row]);
  top = wave_max(top);
  const float ts = top == kNegInf ? 0.0f : top;
  float acc[kPer], l = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; i++) acc[i] = 0.0f;
#pragma unroll 4
  for (int32_t c = wave; c < chunks; c += kWaves) {
    const float* part = base + c * step;
    const float f = exp2_fast(part[kRows * D + 2 * row] - ts);
    l += part[kRows * D + 2 * row + 1] * f;
#pragma unroll
    for (int i = 0; i < kPer; i++) acc[i] += part[row * D + kPer * lane + i] * f;
  }
#pragma unroll
  for (int i = 0; i < kPer; i++) lds_o[wave][kPer * lane + i] = acc[i];
  if (lane == 0) lds_l[wave] = l;
  __syncthreads();
  float ll = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; w++) ll += lds_l[w];
  const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
  for (int d = 2 * tid; d < D; d += 2 * kThreads) {
    float a = 0.0f, c = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      a += lds_o[w][d];
      c += lds_o[w][d + 1];
    }
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + t * p.o_st + qh * p.o_sh + d) = pack16<DT>(a * inv, c * inv);
  }
  if (p.lse && tid == 0)
    p.lse[t * p.l_st + qh] = ll > 0.0f ? (ts + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f : kNegInf;
}

// ------------------------------------------------------------------ launch
struct Shape {
  int64_t units;   // at most
  int64_t blocks;  // that a split call's work is cut for
  int64_t line_bytes, plan_bytes, bytes;
};

Shape shape_of(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  Shape s;
  s.units = Hkv * ((T * (Hq / Hkv) + kRows - 1) / kRows + B);
  s.blocks = static_cast<int64_t>(current_device_shape().cus) * 4;
  s.line_bytes = (B + 1) * 8;
  s.plan_bytes = (s.line_bytes + (B + 1) * 4 + 255) / 256 * 256;
  s.bytes = s.plan_bytes + (s.units + s.blocks) * (kRows * (D + 2)) * 4;
  return s;
}

template <int D, int DT, bool PAGE16>
void launch_d(const Kv4AttnParams& p, bool split, unsigned grid, hipStream_t stream) {
  const size_t lds = (p.B + 1) * 12;
  if (split) {
    hipLaunchKernelGGL((kv4_attention_kernel<D, DT, true, PAGE16>), dim3(grid), dim3(kThreads), lds, stream, p);
    hipLaunchKernelGGL((kv4_join_kernel<D, DT>), dim3(static_cast<unsigned>(p.T * p.Hq)), dim3(kThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL((kv4_attention_kernel<D, DT, false, PAGE16>), dim3(grid), dim3(kThreads), lds, stream, p);
  }
}

template <int D>
void launch_dt(int dtype, bool page16, const Kv4AttnParams& p, bool split, unsigned grid, hipStream_t stream) {
  if (dtype == FP8Q_DTYPE_BF16) {
    if (page16) launch_d<D, FP8Q_DTYPE_BF16, true>(p, split, grid, stream);
    else launch_d<D, FP8Q_DTYPE_BF16, false>(p, split, grid, stream);
  } else {
    if (page16) launch_d<D, FP8Q_DTYPE_F16, true>(p, split, grid, stream);
    else launch_d<D, FP8Q_DTYPE_F16, false>(p, split, grid, stream);
  }
}

}  // namespace

int64_t kv4_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_tokens) {
  const Shape s = shape_of(B, T, Hq, Hkv, D);
  if (max_tokens <= kSpan * kMinRun || s.units >= 16 * s.blocks) return 0;
  return s.bytes;
}

int launch_kv4_attention(int dtype, int64_t D, Kv4AttnParams p, void* ws, int64_t ws_bytes, hipStream_t stream) {
  const Shape s = shape_of(p.B, p.T, p.Hq, p.Hkv, D);
  const int64_t need = kv4_attention_workspace(p.B, p.T, p.Hq, p.Hkv, D, p.max_tokens);
  const bool split = need > 0 && ws && ws_bytes >= need;
  p.max_units = s.units;
  if (split) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    p.blocks = static_cast<int32_t>(s.blocks);
    p.plan_line = reinterpret_cast<int64_t*>(base);
    p.plan_first = reinterpret_cast<int32_t*>(base + s.line_bytes);
    p.parts = reinterpret_cast<float*>(base + s.plan_bytes);
  }
  // a page of 16 tokens or more holds every 16 tokens that a wave loads together; a lane's
  // offset in them has 32 bits
  const bool page16 = p.c.page_shift >= 4 && p.c.c_st < (int64_t(1) << 27) && p.c.s_st < (int64_t(1) << 27);
  // unsplit: blocks walk the units in turn
  const unsigned grid = static_cast<unsigned>(split ? s.blocks : std::min<int64_t>(s.units, s.blocks * 4));
  if (D == 64) launch_dt<64>(dtype, page16, p, split, grid, stream);
  else if (D == 128) launch_dt<128>(dtype, page16, p, split, grid, stream);
  else launch_dt<256>(dtype, page16, p, split, grid, stream);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("kv4 attention launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace fp8q
