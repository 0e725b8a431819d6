// kv4_attention.hip — attention over the paged 4-bit cache.
//
//   out[t][h] = sum_j p_j v_j, p = softmax_j(scale * q[t][h] . k_j) over the cached tokens j that
//   query t sees (all of its sequence's, or with `causal` those up to its own place).
//
// One pass over the cache with a running maximum and sum per query row (fp32, base 2). Query
// heads that share a cached head are rows of one tile, so the cache is read once for all.
//
// Tiles. A unit is 16, 64 or 128 query rows (tokens x heads of the group) of one cached head
// against the sequence's cached tokens. With 16 rows the waves of a block share the tokens, 64 (or
// 32) of a step each, with a running softmax of their own; their results meet in LDS at the end.
// With more they share the rows (below). Short units are one block's. Long ones are cut: the units
// lie in a row, in spans of 128 tokens, and the row is cut into equal runs, one per block, wherever
// the cuts fall, so that every block has the same work however ragged the lengths are. A unit that
// is cut leaves a piece per block in the workspace, which a second kernel joins.
//
// Bounds. Few rows: the cache's bytes. 64 sequences of 3300 to 8192 tokens, 64 heads on 8 cached
// ones of 128: 408 MB in 86 us = 4.7 TB/s, and 6 us for the join. The loads decide it: with 32
// tokens to a step the whole took 102 us and its loads without any arithmetic 92 (a plain read of
// 4 KB pieces in random order: 69). One sequence of 262144 tokens: 285 MB in 56 us = 5.1 TB/s.
// Many rows: the matrix pipe together with the vector pipe, which converts K for every wave and
// exponentiates. 2 x 1434 and 2048 queries of 32 heads over 8192 tokens, 386 GFLOP: 431 us = 0.90
// PFLOP/s, 0.65 of a large bf16 library product's rate.
//
// Layouts (v_mfma_f32_16x16x32_bf16; lane l, r = l % 16, h = l / 16):
//   S^T = K Q^T: lane (r, h) loads dims [D/4 h, D/4 (h + 1)) of token r, one or two scale blocks
//     of which all elements share one scale, and converts them in registers. The contraction
//     index is free, so step j takes dims D/4 h + 8j .. + 7 from lane group h of both operands.
//     e2m1 times a power of two is exact in bf16 (a quarter of it, below): no error is added.
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
#include <type_traits>

#include "kv4_attention_shape.h"
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

constexpr int kWideWaves = 4;  // of a block of the wide kernel
constexpr int kJoinWaves = 4;
constexpr int kPadV = 16;   // elements between the V rows in LDS
constexpr float kLn2 = 0.6931471805599453f;
// Outputs are rescaled only when a row's maximum has grown by more than 2^8 since it last was:
// probabilities then reach 2^8, which costs fp32 sums and bf16 factors no precision.
constexpr float kHeadroom = 8.0f;
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

// The index arrays are only read: a load at a wave-uniform place is scalar.
typedef const __attribute__((address_space(4))) int32_t* ConstInts;
__device__ __forceinline__ int32_t read_int(const int32_t* a, int64_t i) { return ((ConstInts)a)[i]; }

struct Seq {
  int32_t q0, q_len, kv_len;
};

__device__ __forceinline__ Seq sequence(const Kv4AttnParams& p, int32_t b) {
  Seq s;
  s.q0 = b;
  s.q_len = 1;
  if (p.q_indptr) {
    s.q0 = clamp32(read_int(p.q_indptr, b), p.T);
    s.q_len = max(clamp32(read_int(p.q_indptr, b + 1), p.T) - s.q0, 0);
  }
  s.kv_len = clamp32(read_int(p.kv_lens, b), p.max_tokens);
  return s;
}

template <int ROWS>
__device__ __forceinline__ int32_t tiles_of(const Kv4AttnParams& p, const Seq& s) {
  return static_cast<int32_t>((static_cast<uint32_t>(s.q_len) * p.group + ROWS - 1) / ROWS);  // T * Hq < 2^31
}
// A sequence without cached tokens has one empty span, so that its rows are written.
__device__ __forceinline__ int32_t spans_of(const Kv4AttnParams& p, const Seq& s) {
  return max((s.kv_len + (1 << p.span_shift) - 1) >> p.span_shift, 1);
}

// ------------------------------------------------------------------ units and runs
// Prefixes over the sequences: first[b] the query tiles, line[b] the (tile, span) pairs before
// sequence b. Unit (b, tile, head) is number (first[b] + tile) * Hkv + head and has the places
// [line[b] * Hkv + (tile * Hkv + head) * spans, + spans) of the line of all spans. For a
// split call, which alone uses the line, the host chooses a span with which it has fewer than 2^31
// places.
struct Plan {
  int32_t* line;   // [B + 1]
  int32_t* first;  // [B + 1]
};

// Inclusive sum over the block's threads; `lds` holds one value per wave.
template <int WAVES>
__device__ __forceinline__ long long block_scan(long long v, long long* lds, long long& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const long long up = __shfl_up(v, off, 64);
    if (lane >= off) v += up;
  }
  if (lane == 63) lds[wave] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) {
    if (w < wave) v += lds[w];
    total += lds[w];
  }
  return v;
}

// Fills the plan in LDS; every block computes the same from the lengths. A q_indptr that does
// not ascend can name more rows than there are: then the plan is empty and nothing is run.
template <int ROWS, int WAVES>
__device__ __forceinline__ void make_plan(const Kv4AttnParams& p, const Plan& plan) {
  constexpr int kThreads = 64 * WAVES;
  __shared__ long long tot_line[WAVES], tot_first[WAVES];
  const int tid = threadIdx.x;
  const int32_t B = static_cast<int32_t>(p.B);
  const int32_t per = (B + kThreads - 1) / kThreads;
  const int32_t beg = min(tid * per, B), end = min(beg + per, B);
  long long my_line = 0, my_first = 0;
  for (int32_t b = beg; b < end; b++) {
    const Seq s = sequence(p, b);
    const long long tiles = tiles_of<ROWS>(p, s);
    my_first += tiles;
    my_line += tiles * spans_of(p, s);
  }
  long long all_line, all_first;
  long long at_first = block_scan<WAVES>(my_first, tot_first, all_first) - my_first;
  long long at_line = block_scan<WAVES>(my_line, tot_line, all_line) - my_line;
  const bool fits = all_first * p.Hkv <= p.max_units;
  for (int32_t b = beg; b < end; b++) {
    const Seq s = sequence(p, b);
    plan.first[b] = fits ? static_cast<int32_t>(at_first) : 0;
    plan.line[b] = fits ? static_cast<int32_t>(at_line) : 0;
    const long long tiles = tiles_of<ROWS>(p, s);
    at_first += tiles;
    at_line += tiles * spans_of(p, s);
  }
  if (tid == kThreads - 1) {
    plan.first[B] = fits ? static_cast<int32_t>(all_first) : 0;
    plan.line[B] = fits ? static_cast<int32_t>(all_line) : 0;
  }
  __syncthreads();
}

// The last b with pref[b] <= v (pref ascending, pref[0] <= v).
__device__ __forceinline__ int32_t find_seq(const int32_t* pref, int32_t B, int32_t v) {
  int32_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (pref[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// Spans of one block's run when `blocks` blocks share a line of `total` spans.
__device__ __forceinline__ int32_t run_length(int32_t total, int32_t blocks) {
  return max(total / blocks + (total % blocks != 0), kMinRun);
}

__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// One unit's tokens [t0, t1) of a block's run.
struct Work {
  Seq seq;
  int32_t b, tile, head, t0, t1;
  bool whole;     // all of the unit's tokens
  int32_t piece;  // else: where its partial results go
};

// A block's places [at, stop) on the line: of spans when splitting, else of units in steps of the
// grid. `direct`: one unit per sequence and cached head, in order, so that no plan is needed.
template <int ROWS, int WAVES, bool SPLIT>
struct Walk {
  const Kv4AttnParams& p;
  const Plan plan;
  const bool direct;
  int32_t at, stop;

  __device__ __forceinline__ Walk(const Kv4AttnParams& params, int32_t* lds)
      : p(params), plan{lds, lds + params.B + 1},
        direct(!SPLIT && params.q_indptr == nullptr && params.group <= ROWS) {
    const int32_t B = static_cast<int32_t>(p.B);
    if (!direct) make_plan<ROWS, WAVES>(p, plan);
    if constexpr (SPLIT) {
      const int32_t total = uniform(plan.line[B]) * p.Hkv, run = run_length(total, p.blocks);
      at = static_cast<int32_t>(min(static_cast<int64_t>(blockIdx.x) * run, static_cast<int64_t>(total)));
      stop = at + min(run, total - at);
      if (blockIdx.x == 0) {  // for the join
        for (int32_t b = threadIdx.x; b <= B; b += 64 * WAVES) {
          p.plan[b] = plan.line[b];
          p.plan[B + 1 + b] = plan.first[b];
        }
      }
    } else {
      at = blockIdx.x;
      stop = (direct ? B : uniform(plan.first[B])) * p.Hkv;
    }
  }

  __device__ __forceinline__ bool next(Work& w) {
    if (at >= stop) return false;
    const int32_t B = static_cast<int32_t>(p.B);
    int32_t s0 = 0, s1;
    if constexpr (SPLIT) {
      w.b = uniform(find_seq(plan.line, B, at / p.Hkv));
      w.seq = sequence(p, w.b);
      const int32_t spans = spans_of(p, w.seq), in = at - uniform(plan.line[w.b]) * p.Hkv, unit = in / spans;
      w.tile = unit / p.Hkv;
      w.head = unit - w.tile * p.Hkv;
      s0 = in - unit * spans;
      s1 = min(spans, s0 + (stop - at));
      at += s1 - s0;
      w.whole = s0 == 0 && s1 == spans;
      w.piece = blockIdx.x + uniform(plan.first[w.b]) * p.Hkv + unit;
    } else {
      const int32_t u = at / p.Hkv;
      w.head = at - u * p.Hkv;
      w.b = direct ? u : uniform(find_seq(plan.first, B, u));
      w.seq = sequence(p, w.b);
      w.tile = direct ? 0 : u - uniform(plan.first[w.b]);
      s1 = spans_of(p, w.seq);
      w.whole = true;
      w.piece = 0;
      at += min(static_cast<int32_t>(gridDim.x), stop - at);
    }
    w.t0 = s0 << p.span_shift;
    w.t1 = s1 == spans_of(p, w.seq) ? w.seq.kv_len : s1 << p.span_shift;
    return true;
  }
};

// The tile's query rows first .. last (at least one), and how much of the cache they see.
struct Rows {
  int32_t first, last;  // of the sequence's q_len * group rows; row i is query i / group
  int32_t before;       // tokens that query 0 sees with `causal`

  __device__ __forceinline__ Rows(const Kv4AttnParams& p, const Work& w, int rows) {
    first = w.tile * rows;
    last = min(first + rows, w.seq.q_len * p.group) - 1;
    before = w.seq.kv_len - w.seq.q_len + 1;
  }
  // Tokens that row i sees.
  __device__ __forceinline__ int32_t seen(const Kv4AttnParams& p, const Seq& s, int32_t i) const {
    return p.causal ? before + static_cast<int32_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.group)) : s.kv_len;
  }
};

// ------------------------------------------------------------------ cached rows
// A lane's part of one token's row: D / 4 elements, in the vectors that they are loaded as (taken
// apart, they are copied as soon as they arrive, and waited for there).
template <int D>
struct Codes {
  static constexpr int kWords = D == 64 ? 2 : 4;
  typedef uint32_t Vec __attribute__((ext_vector_type(kWords)));
  Vec v[D / 32 / kWords];
};

template <int D>
__device__ __forceinline__ void load_codes(const uint8_t* codes, uint32_t lane_offset, int h, Codes<D>& c) {
  codes += lane_offset + D / 8 * h;
#pragma unroll
  for (int j = 0; j < D / 32 / Codes<D>::kWords; j++) c.v[j] = reinterpret_cast<const typename Codes<D>::Vec*>(codes)[j];
}

template <int D>
__device__ __forceinline__ void zero_codes(Codes<D>& c) {
#pragma unroll
  for (int j = 0; j < D / 32 / Codes<D>::kWords; j++) c.v[j] = typename Codes<D>::Vec(0u);
}

// All scale bytes of one token's row, in one load per lane.
template <int D>
struct Scales {
  uint32_t w[D == 256 ? 2 : 1];
};

template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* scales, Scales<D>& s) {
  if constexpr (D == 64) {
    s.w[0] = *reinterpret_cast<const uint16_t*>(scales);
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; i++) s.w[i] = reinterpret_cast<const uint32_t*>(scales)[i];
  }
}

// The scales of a lane's part: of its one block, or for D = 256 its two.
template <int D>
struct Mult {
  float f[D == 256 ? 2 : 1];
};

// Byte b of w as the exponent of a power of two: a rotation puts it at bits 23-30.
__device__ __forceinline__ float pow2_of_byte(uint32_t w, uint32_t b) {
  return __uint_as_float(__builtin_amdgcn_alignbit(w, w, (8 * b + 9) & 31) & 0x7F800000u);
}

template <int D>
__device__ __forceinline__ Mult<D> mult_of(const Scales<D>& s, int h) {
  Mult<D> m;
  if constexpr (D == 256) {
    const uint32_t lo = s.w[0], hi = s.w[1], w = h & 2 ? hi : lo;
    m.f[0] = pow2_of_byte(w, 2 * (h & 1));
    m.f[1] = pow2_of_byte(w, 2 * (h & 1) + 1);
  } else {
    m.f[0] = pow2_of_byte(s.w[0], D == 64 ? h >> 1 : h);
  }
  return m;
}

// Scales of N = 2 or 4 times 16 tokens were loaded by lanes (r, h) for token r of half h % N: each
// half's for this lane's r, from the other rows of 16 lanes.
template <int D, int N>
__device__ __forceinline__ void spread_scales(const Scales<D>& s, int h, Mult<D> (&m)[N]) {
  Scales<D> half[4];
#pragma unroll
  for (int i = 0; i < (D == 256 ? 2 : 1); i++) {
    const auto x = __builtin_amdgcn_permlane16_swap(s.w[i], s.w[i], false, false);  // rows 0 0 2 2, 1 1 3 3
    half[0].w[i] = x[0];
    half[1].w[i] = x[1];
    if constexpr (N == 4) {
      const auto a = __builtin_amdgcn_permlane32_swap(x[0], x[0], false, false);
      const auto b = __builtin_amdgcn_permlane32_swap(x[1], x[1], false, false);
      half[0].w[i] = a[0];
      half[2].w[i] = a[1];
      half[1].w[i] = b[0];
      half[3].w[i] = b[1];
    }
  }
#pragma unroll
  for (int c = 0; c < N; c++) m[c] = mult_of<D>(half[c], h);
}

// Keys and values are converted as a quarter of themselves, which bf16 holds whatever the scale is: up to
// 6 * 2^127 cached (codes round up, so finite rows of the model's type are held as up to 2^128), of which
// a quarter is finite. Scores are then multiplied by four times the scale, outputs by four times
// the sum's reciprocal: all exact. (Scale bytes 0 and 1, which the write never stores, count as 2.)
__device__ __forceinline__ float quarter(float pow2) {
  return __uint_as_float(__builtin_elementwise_sub_sat(__float_as_uint(pow2), 2u << 23));
}
template <int D>
__device__ __forceinline__ void quarter_keys(Mult<D>& m) {
#pragma unroll
  for (int i = 0; i < (D == 256 ? 2 : 1); i++) m.f[i] = quarter(m.f[i]);
}
// Values also where a scale byte is 255, which is no number: a value that a row does not see, whatever
// its bytes are, adds 0 times a finite number, which is 0.
template <int D>
__device__ __forceinline__ void quarter_values(Mult<D>& m) {
#pragma unroll
  for (int i = 0; i < (D == 256 ? 2 : 1); i++) m.f[i] = quarter(__uint_as_float(min(__float_as_uint(m.f[i]), 254u << 23)));
}

template <int D>
__device__ __forceinline__ void one_mult(Mult<D>& m) {
#pragma unroll
  for (int i = 0; i < (D == 256 ? 2 : 1); i++) m.f[i] = 1.0f;
}

// Word i of a lane's part as 8 bf16 values (exact).
template <int D>
__device__ __forceinline__ bf16x8 widen_codes(const Codes<D>& c, const Mult<D>& m, int i) {
  const float s = m.f[D == 256 ? i / 4 : 0];
  const uint32_t w = c.v[i / Codes<D>::kWords][i % Codes<D>::kWords];
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// One step of a wave: N times 16 tokens.
template <int D, int N>
struct Step {
  Codes<D> k[N], v[N];
  Scales<D> ks, vs;  // of token r of half h % N
  std::conditional_t<N == 4, uint64_t, uint32_t> there;  // bit i: token i is inside the range, its page in the cache
};

template <int N>
constexpr std::conditional_t<N == 4, uint64_t, uint32_t> kAllThere = N == 4 ? ~0ull : (1ull << (16 * N % 64)) - 1;

// How a wave looks up the pages of the tokens that it loads together: for every token; for every
// 16 where a page holds that many; or once where a page holds all of them (the pages of the last
// two are wave-uniform: scalar loads and arithmetic).
constexpr int kByToken = 0, kBy16 = 1, kByStep = 2;

// Page numbers of N times 16 tokens.
template <int PAGE, int N>
struct Pages {
  int32_t n[PAGE == kByStep ? 1 : N];
};

template <int PAGE, int N>
__device__ __forceinline__ Pages<PAGE, N> load_pages(const Kv4AttnParams& p, const int32_t* table, int32_t t, int32_t t_end) {
  Pages<PAGE, N> g;
#pragma unroll
  for (int i = 0; i < (PAGE == kByStep ? 1 : N); i++) {
    // past the end: the last token's entry, which is there to be read
    const int32_t at = min(t + 16 * i + (PAGE == kByToken ? static_cast<int>(threadIdx.x & 15) : 0), t_end - 1) >> p.c.page_shift;
    g.n[i] = PAGE == kByToken ? table[at] : read_int(table, at);
  }
  return g;
}

// Makes the wave wait for pages that it has asked for.
template <int PAGE, int N>
__device__ __forceinline__ void settle(Pages<PAGE, N>& g) {
  if constexpr (PAGE != kByToken) {
#pragma unroll
    for (int i = 0; i < (PAGE == kByStep ? 1 : N); i++) g.n[i] = uniform(g.n[i]);
  }
}

// Where the rows of N times 16 tokens from t on lie, without their head, and which of them are there
// (bit i: token t + i is before t_end and its page is in the cache). Every address is inside the
// cache: a page that is not there is replaced by page 0, and tokens past the end lie in the last
// token's page or in a valid one; what is loaded for them is not used.
template <int N>
struct Spots {
  int64_t c[N], s[N];             // of the lane's token; of the first token where pages are uniform,
  uint32_t c_lane[N], s_lane[N];  // and the lane's offset from it
  uint64_t there;
};

template <int PAGE, int N>
__device__ __forceinline__ Spots<N> locate(const Kv4AttnParams& p, const Pages<PAGE, N>& g, int32_t t, int32_t t_end) {
  const int r = threadIdx.x & 15;
  const int32_t mask = (1 << p.c.page_shift) - 1;
  const uint32_t pages = static_cast<uint32_t>(p.c.pages);
  Spots<N> a;
  if constexpr (PAGE == kByToken) {
    a.there = 0;
#pragma unroll
    for (int i = 0; i < N; i++) {
      const bool ok = static_cast<uint32_t>(g.n[i]) < pages;
      const int64_t page = ok ? g.n[i] : 0, in = min(t + 16 * i + r, t_end - 1) & mask;
      a.there |= (__builtin_amdgcn_ballot_w64(ok && t + 16 * i + r < t_end) & 0xFFFFull) << (16 * i);
      a.c[i] = page * p.c.c_sp + in * p.c.c_st;
      a.s[i] = page * p.c.s_sp + in * p.c.s_st;
      a.c_lane[i] = a.s_lane[i] = 0;
    }
  } else {  // page strides and page extents fit 32 bits
    const uint32_t c_sp = static_cast<uint32_t>(p.c.c_sp), c_st = static_cast<uint32_t>(p.c.c_st);
    const uint32_t s_sp = static_cast<uint32_t>(p.c.s_sp), s_st = static_cast<uint32_t>(p.c.s_st);
    const int32_t left = t_end - t;
    a.there = left >= 16 * N ? kAllThere<N> : left <= 0 ? 0 : (1ull << left) - 1;
#pragma unroll
    for (int i = 0; i < N; i++) {
      if (PAGE == kBy16 || i == 0) {
        const uint32_t n = static_cast<uint32_t>(g.n[i]), page = n < pages ? n : 0, in = (t + 16 * i) & mask;
        a.there &= n < pages ? ~0ull : PAGE == kByStep ? 0ull : ~(0xFFFFull << (16 * i));
        a.c[i] = static_cast<uint64_t>(page) * c_sp + in * c_st;
        a.s[i] = static_cast<uint64_t>(page) * s_sp + in * s_st;
        a.c_lane[i] = r * c_st;
        a.s_lane[i] = r * s_st;
      } else {
        a.c[i] = a.c[0];
        a.s[i] = a.s[0];
        a.c_lane[i] = (r + 16 * i) * c_st;
        a.s_lane[i] = (r + 16 * i) * s_st;
      }
    }
  }
  return a;
}

// The scales of M = 2 or 4 times 16 tokens from the i-th on: lane (r, h) loads token r of half h % M.
// (The choice is made between values: between an array's elements it would put the array into memory.)
template <int D, int PAGE, int M, int N>
__device__ __forceinline__ void load_scales_of(const uint8_t* scales, const Spots<N>& a, int i, int h, Scales<D>& s) {
  if constexpr (PAGE == kByStep) {
    const uint32_t v = a.s_lane[i], w = a.s_lane[i + 1];
    uint32_t lane = h & 1 ? w : v;
    if constexpr (M == 4) {
      const uint32_t x = a.s_lane[i + 2], y = a.s_lane[i + 3], z = h & 1 ? y : x;
      lane = h & 2 ? z : lane;
    }
    load_scales<D>(scales + a.s[0] + lane, s);
  } else {
    const int64_t v = a.s[i] + a.s_lane[i], w = a.s[i + 1] + a.s_lane[i + 1];
    int64_t at = h & 1 ? w : v;
    if constexpr (M == 4) {
      const int64_t x = a.s[i + 2] + a.s_lane[i + 2], y = a.s[i + 3] + a.s_lane[i + 3], z = h & 1 ? y : x;
      at = h & 2 ? z : at;
    }
    load_scales<D>(scales + at, s);
  }
}

// Loads a step's codes and scales; k and v (with their scales) start at the unit's head.
template <int D, int PAGE, int N>
__device__ __forceinline__ void load_step(const Kv4AttnParams& p, const Kv4Cache& at, const Pages<PAGE, N>& g, int32_t t,
                                          int32_t t_end, Step<D, N>& st) {
  const int h = (threadIdx.x & 63) >> 4;
  const Spots<N> a = locate<PAGE, N>(p, g, t, t_end);
  st.there = a.there;
#pragma unroll
  for (int c = 0; c < N; c++) load_codes<D>(at.k + a.c[c], a.c_lane[c], h, st.k[c]);
  load_scales_of<D, PAGE, N>(at.ks, a, 0, h, st.ks);
#pragma unroll
  for (int c = 0; c < N; c++) load_codes<D>(at.v + a.c[c], a.c_lane[c], h, st.v[c]);
  load_scales_of<D, PAGE, N>(at.vs, a, 0, h, st.vs);
}

// The cache from cached head `head` on.
__device__ __forceinline__ Kv4Cache at_head(const Kv4Cache& c, int32_t head) {
  Kv4Cache a = c;
  a.k += head * c.c_sh;
  a.v += head * c.c_sh;
  a.ks += head * c.s_sh;
  a.vs += head * c.s_sh;
  return a;
}

// ------------------------------------------------------------------ the kernel
// bf16: one part. fp16: high and low parts whose sum is the value. `sign`: 0, or 0x80008000 to
// negate (the scale's sign: scores are then multiplied by its magnitude, after their maximum).
template <int DT, int PARTS>
__device__ __forceinline__ void split8(u32x4 raw, uint32_t sign, bf16x8 (&out)[PARTS]) {
#pragma unroll
  for (int i = 0; i < 4; i++) raw[i] ^= sign;
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

// Two outputs rounded to their type, an average past its largest finite value as that value: the cache
// holds up to 98304 of fp16's 65504 and 2^128 of bf16's (codes round up). (NaN stays.)
template <int DT>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
  constexpr float kMost = DT == FP8Q_DTYPE_F16 ? 65504.0f : 0x1.FEp127f;
  a = fabsf(a) > kMost ? copysignf(kMost, a) : a;
  b = fabsf(b) > kMost ? copysignf(kMost, b) : b;
  return pack16<DT>(a, b);
}

// V^T's operand for dims 16 d .. + 15 and the 32 tokens whose rows start at `src` (of lane (r, h): row
// 4h + r / 4, element 4 (r % 4)).
template <int ROW>
__device__ __forceinline__ bf16x8 read_v(const uint16_t* src, int d) {
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 16 * d));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 16 * d + 16 * ROW));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int D, int DT, int WAVES, int N, bool SPLIT, int PAGE>
__global__ __launch_bounds__(64 * WAVES, waves_per_simd(D, DT, N)) void kv4_attention_kernel(Kv4AttnParams p) {
  constexpr int PARTS = DT == FP8Q_DTYPE_F16 ? 2 : 1;
  constexpr int kTile = 16 * N;         // tokens of a wave's step
  constexpr int kStep = kTile * WAVES;  // and of the block's
  constexpr int kSteps = D / 32;   // contraction steps of S^T
  constexpr int kDims = D / 16;    // dim tiles of O^T
  constexpr int kRowV = D + kPadV;  // LDS row of V (bf16 elements)
  constexpr int kRowO = D + 4;      // LDS row of the joined output (floats)
  static_assert(kRows * kRowO * 4 <= kTile * kRowV * 2, "the joined output reuses V's LDS");
  __shared__ __align__(16) uint16_t lds_v[WAVES][kTile * kRowV];
  __shared__ float lds_m[WAVES][kRows], lds_l[WAVES][kRows];
  extern __shared__ int32_t lds_plan[];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int r = lane & 15, h = lane >> 4;
  Walk<kRows, WAVES, SPLIT> walk(p, lds_plan);
  Work w;
  while (walk.next(w)) {
    const Seq seq = w.seq;
    const int32_t head = w.head;
    const Rows tr(p, w, kRows);
    const int32_t first = tr.first, last = tr.last;
    const bool row_there = first + r <= last;
    const int32_t idx = row_there ? first + r : last, qi = idx / p.group, qh = head * p.group + idx - qi * p.group;
    const int32_t limit = tr.seen(p, seq, idx), low = tr.seen(p, seq, first);
    const int32_t t_end = min(w.t1, tr.seen(p, seq, last));

    const int32_t* table = p.table + w.b * p.table_sb;
    const Kv4Cache cache = at_head(p.c, head);
    int32_t t = w.t0 + kTile * wave;
    Step<D, N> st;
    Pages<PAGE, N> pages;
    if (t < t_end) {
      pages = load_pages<PAGE, N>(p, table, t, t_end);
      load_step<D, PAGE, N>(p, cache, pages, t, t_end, st);
      pages = load_pages<PAGE, N>(p, table, t + kStep, t_end);
    }

    bf16x8 q[PARTS][kSteps];
    {
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + (seq.q0 + qi) * p.q_st + qh * p.q_sh + D / 4 * h;
#pragma unroll
      for (int j = 0; j < kSteps; j++) {
        u32x4 raw = {0u, 0u, 0u, 0u};
        if (row_there) raw = *reinterpret_cast<const u32x4*>(src + 8 * j);
        bf16x8 part[PARTS];
        split8<DT, PARTS>(raw, p.q_sign, part);
#pragma unroll
        for (int a = 0; a < PARTS; a++) q[a][j] = part[a];
      }
    }

    uint16_t* vt = lds_v[wave];
    f32x4 o[kDims];
#pragma unroll
    for (int d = 0; d < kDims; d++) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = kNegInf, l = 0.0f;  // l: this lane's share of the row's sum

    for (; t < t_end; t += kStep) {
      f32x4 s[N];
      Mult<D> mk[N], mv[N];
      spread_scales<D, N>(st.ks, h, mk);
#pragma unroll
      for (int c = 0; c < N; c++) {
        s[c] = f32x4{0.f, 0.f, 0.f, 0.f};
        quarter_keys<D>(mk[c]);
#pragma unroll
        for (int j = 0; j < kSteps; j++) {
          const bf16x8 k = widen_codes<D>(st.k[c], mk[c], j);
#pragma unroll
          for (int a = 0; a < PARTS; a++) s[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[a][j], s[c], 0, 0, 0);
        }
      }
      const auto there = st.there;
      const bool part = there != kAllThere<N> || t + kTile > low;  // wave-uniform
      spread_scales<D, N>(st.vs, h, mv);
#pragma unroll
      for (int c = 0; c < N; c++) {
        quarter_values<D>(mv[c]);
        if (there != kAllThere<N> && ((there >> (16 * c + r)) & 1u) == 0u) {
          zero_codes<D>(st.v[c]);
          one_mult<D>(mv[c]);
        }
#pragma unroll
        for (int j = 0; j < kSteps; j++)
          *reinterpret_cast<bf16x8*>(vt + (16 * c + r) * kRowV + D / 4 * h + 8 * j) = widen_codes<D>(st.v[c], mv[c], j);
      }
      // the next step's codes come in while this one's softmax and second product run (past the
      // end: rows of the last page, not used)
      load_step<D, PAGE, N>(p, cache, pages, t + kStep, t_end, st);
      pages = load_pages<PAGE, N>(p, table, t + 2 * kStep, t_end);

      if (part) {
#pragma unroll
        for (int c = 0; c < N; c++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int n = 16 * c + 4 * h + i;
            if (((there >> n) & 1u) == 0u || t + n >= limit) s[c][i] = kNegInf;
          }
      }
      float mx = kNegInf;
#pragma unroll
      for (int c = 0; c < N; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) mx = fmaxf(mx, s[c][i]);
      mx = quad_max(mx) * p.scale_log2;
      if (__builtin_amdgcn_ballot_w64(mx > m + kHeadroom) != 0) {
        const float top = fmaxf(mx, m), alpha = exp2_fast(m - (top == kNegInf ? 0.0f : top));
        m = top;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < kDims; d++)
#pragma unroll
          for (int i = 0; i < 4; i++) o[d][i] *= alpha;
      }
      const float ms = m == kNegInf ? 0.0f : m;  // nothing seen yet: every p is 0
      bf16x8 pr[N / 2][PARTS];
#pragma unroll
      for (int c = 0; c < N; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float e = exp2_fast(fmaf(s[c][i], p.scale_log2, -ms));
          l += e;
          const __bf16 hi = static_cast<__bf16>(e);
          pr[c / 2][0][4 * (c % 2) + i] = hi;
          if constexpr (PARTS == 2) pr[c / 2][1][4 * (c % 2) + i] = static_cast<__bf16>(e - static_cast<float>(hi));
        }

      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      // every operand is read one product ahead
      const uint16_t* v_at = vt + (4 * h + (r >> 2)) * kRowV + 4 * (r & 3);
      bf16x8 vf[2];
      vf[0] = read_v<kRowV>(v_at, 0);
#pragma unroll
      for (int g = 0; g < N / 2 * kDims; g++) {
        const int c = g / kDims, d = g % kDims;
        if (g + 1 < N / 2 * kDims) vf[(g + 1) & 1] = read_v<kRowV>(v_at + 32 * ((g + 1) / kDims) * kRowV, (g + 1) % kDims);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int a = 0; a < PARTS; a++) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[g & 1], pr[c][a], o[d], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
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
    for (int n = 0; n < WAVES; n++) top = fmaxf(top, lds_m[n][r]);
    {
      const float f = exp2_fast(m - (top == kNegInf ? 0.0f : top));
      float* dst = reinterpret_cast<float*>(vt) + r * kRowO + 4 * h;
#pragma unroll
      for (int d = 0; d < kDims; d++) *reinterpret_cast<f32x4*>(dst + 16 * d) = o[d] * f;
    }
    __syncthreads();
    for (int e = tid; e < kRows * (D / 8); e += 64 * WAVES) {
      const int row = e / (D / 8), col = e % (D / 8) * 8;
      if (first + row > last) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = 0.0f;
      float mm = kNegInf, ll = 0.0f;
#pragma unroll
      for (int n = 0; n < WAVES; n++) {
        const float* src = reinterpret_cast<const float*>(lds_v[n]) + row * kRowO + col;
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] += src[i];
        mm = fmaxf(mm, lds_m[n][row]);
      }
#pragma unroll
      for (int n = 0; n < WAVES; n++) ll += lds_l[n][row] * exp2_fast(lds_m[n][row] - (mm == kNegInf ? 0.0f : mm));
      if (SPLIT && !w.whole) {
        float* part = p.parts + static_cast<int64_t>(w.piece) * (kRows * (D + 2));
#pragma unroll
        for (int i = 0; i < 8; i += 4)
          *reinterpret_cast<f32x4*>(part + row * D + col + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
        if (col == 0) {
          part[kRows * D + 2 * row] = mm;
          part[kRows * D + 2 * row + 1] = ll;
        }
      } else {
        const int32_t i = (first + row) / p.group;
        const int64_t row_t = seq.q0 + i, hh = head * p.group + first + row - i * p.group;
        const float inv = ll == 0.0f ? 0.0f : 4.0f / ll;
        u32x4 bits;
#pragma unroll
        for (int j = 0; j < 4; j++) bits[j] = pack_out<DT>(v[2 * j] * inv, v[2 * j + 1] * inv);
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + row_t * p.o_st + hh * p.o_sh + col) = bits;
        if (p.lse && col == 0)
          p.lse[row_t * p.l_st + hh] = ll == 0.0f ? kNegInf : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ many query rows
// The same products for tiles of 64 QT rows (QT 1 or 2): every wave has 16 QT rows of its own and all the
// tokens, 64 at a time. K's codes are converted in registers by every wave (they serve QT
// products each); V is converted once per block into LDS, a quarter of the tokens per wave, one
// step ahead of its use (two buffers, one barrier per step). Each of V's operands is read one product
// ahead of its use (529 us for 2 x 2048 queries over 8192 tokens when the compiler placed the reads,
// 484 so), and a step's 64 tokens take one page lookup where a page holds them (435).
// Waves per SIMD that the registers are kept to (fp16, D = 128, 64 rows: 452 us at 3, 468 at 2, for 2 x
// 1024 queries of 32 heads over 8192 tokens; bf16, D = 64, 128 rows: 353 and 388 for 2 x 2048). Up to 17
// registers then go through memory: in fp16 at D = 128 and 256 with one page lookup per step or per token, in bf16
// with one per token.
constexpr int wide_waves_per_simd(int D, int DT, int QT, bool split) {
  const int parts = DT == FP8Q_DTYPE_F16 ? 2 : 1;
  if (D * QT * parts <= 64) return 4;
  return (D * QT * parts <= 128 && !(D == 64 && split)) || (D == 128 && QT == 1) ? 3 : 2;
}

template <int D, int DT, int QT, bool SPLIT, int PAGE>
__global__ __launch_bounds__(64 * kWideWaves, wide_waves_per_simd(D, DT, QT, SPLIT)) void kv4_attention_wide_kernel(Kv4AttnParams p) {
  constexpr int PARTS = DT == FP8Q_DTYPE_F16 ? 2 : 1;
  constexpr int kSteps = D / 32, kDims = D / 16, kRowV = D + kPadV;
  constexpr int kHalves = kStepW / 16;
  constexpr int ROWS = 16 * QT * kWideWaves;
  static_assert(kHalves == kWideWaves, "every wave converts 16 tokens of V");
  __shared__ __align__(16) uint16_t lds_v[2][kStepW * kRowV];
  extern __shared__ int32_t lds_plan[];
  const int lane = threadIdx.x & 63, wave = wave_index();
  const int r = lane & 15, h = lane >> 4;
  Walk<ROWS, kWideWaves, SPLIT> walk(p, lds_plan);
  Work w;
  while (walk.next(w)) {
    const Seq seq = w.seq;
    const int32_t head = w.head;
    const Rows tr(p, w, ROWS);
    const int32_t wfirst = tr.first + 16 * QT * wave;  // this wave's rows
    const int32_t low = tr.seen(p, seq, min(wfirst, tr.last));
    const int32_t t0 = w.t0, t_end = min(w.t1, tr.seen(p, seq, tr.last));

    const int32_t* table = p.table + w.b * p.table_sb;
    const Kv4Cache cache = at_head(p.c, head);
    Codes<D> k[kHalves], v;
    Scales<D> ks[kHalves / 2], vs;
    uint64_t k_there = 0;
    uint32_t v_there = 0;
    Pages<PAGE, kHalves> k_page{};
    Pages<PAGE, 1> v_page{};
    auto load_k = [&](int32_t t) {
      const Spots<kHalves> a = locate<PAGE, kHalves>(p, k_page, t, t_end);
      k_there = a.there;
#pragma unroll
      for (int c = 0; c < kHalves; c += 2) {
        load_codes<D>(cache.k + a.c[c], a.c_lane[c], h, k[c]);
        load_codes<D>(cache.k + a.c[c + 1], a.c_lane[c + 1], h, k[c + 1]);
        load_scales_of<D, PAGE, 2>(cache.ks, a, c, h, ks[c / 2]);
      }
    };
    auto load_v = [&](int32_t t) {
      const Spots<1> a = locate<PAGE, 1>(p, v_page, t + 16 * wave, t_end);
      v_there = static_cast<uint32_t>(a.there);
      load_codes<D>(cache.v + a.c[0], a.c_lane[0], h, v);
      load_scales<D>(cache.vs + a.s[0] + a.s_lane[0], vs);
    };
    auto pages_v = [&](int32_t t) { return load_pages<PAGE, 1>(p, table, t + 16 * wave, t_end); };
    auto put_v = [&](int buf) {
      Mult<D> mv = mult_of<D>(vs, h);
      quarter_values<D>(mv);
      if (((v_there >> r) & 1u) == 0u) {
        zero_codes<D>(v);
        one_mult<D>(mv);
      }
#pragma unroll
      for (int j = 0; j < kSteps; j++)
        *reinterpret_cast<bf16x8*>(&lds_v[buf][(16 * wave + r) * kRowV + D / 4 * h + 8 * j]) = widen_codes<D>(v, mv, j);
    };
    if (t0 < t_end) {
      k_page = load_pages<PAGE, kHalves>(p, table, t0, t_end);
      v_page = pages_v(t0);
      load_k(t0);
      load_v(t0);
      k_page = load_pages<PAGE, kHalves>(p, table, t0 + kStepW, t_end);
      v_page = pages_v(t0 + kStepW);
    }

    bf16x8 q[QT][PARTS][kSteps];
    int32_t limit[QT];
#pragma unroll
    for (int n = 0; n < QT; n++) {
      const int32_t row = wfirst + 16 * n + r;
      const bool there = row <= tr.last;
      const int32_t idx = there ? row : tr.last, qi = idx / p.group, qh = head * p.group + idx - qi * p.group;
      limit[n] = tr.seen(p, seq, idx);
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + (seq.q0 + qi) * p.q_st + qh * p.q_sh + D / 4 * h;
#pragma unroll
      for (int j = 0; j < kSteps; j++) {
        u32x4 raw = {0u, 0u, 0u, 0u};
        if (there) raw = *reinterpret_cast<const u32x4*>(src + 8 * j);
        bf16x8 part[PARTS];
        split8<DT, PARTS>(raw, p.q_sign, part);
#pragma unroll
        for (int a = 0; a < PARTS; a++) q[n][a][j] = part[a];
      }
    }

    f32x4 o[QT][kDims];
    float m[QT], l[QT];
#pragma unroll
    for (int n = 0; n < QT; n++) {
      m[n] = kNegInf;
      l[n] = 0.0f;
#pragma unroll
      for (int d = 0; d < kDims; d++) o[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int v_at = (4 * h + (r >> 2)) * kRowV + 4 * (r & 3);
    if (t0 < t_end) {
      put_v(0);
      load_v(t0 + kStepW);
      v_page = pages_v(t0 + 2 * kStepW);
    }
    __syncthreads();
    int buf = 0;
    for (int32_t t = t0; t < t_end; t += kStepW, buf ^= 1) {
      f32x4 s[QT][kHalves];
      const uint64_t there = k_there;
      // the pages after next, waited for (below) before any LDS read is under way: scalar loads
      // return in no order, so that with one outstanding every LDS read would wait for all
      Pages<PAGE, kHalves> next_k;
      if constexpr (PAGE == kByStep) next_k.n[0] = v_page.n[0];  // V is a step ahead
      else next_k = load_pages<PAGE, kHalves>(p, table, t + 2 * kStepW, t_end);
      Pages<PAGE, 1> next_v = pages_v(t + 3 * kStepW);
#pragma unroll
      for (int c = 0; c < kHalves; c++) {
        Mult<D> mk[2];
        spread_scales<D, 2>(ks[c / 2], h, mk);
        quarter_keys<D>(mk[c % 2]);
#pragma unroll
        for (int n = 0; n < QT; n++) s[n][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kSteps; j++) {
          const bf16x8 kk = widen_codes<D>(k[c], mk[c % 2], j);
#pragma unroll
          for (int n = 0; n < QT; n++)
#pragma unroll
            for (int a = 0; a < PARTS; a++)
              s[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[n][a][j], s[n][c], 0, 0, 0);
        }
      }
      // loads past the end bring rows of the last page, which are not used
      load_k(t + kStepW);
      put_v(buf ^ 1);
      load_v(t + 2 * kStepW);
      settle<PAGE, kHalves>(next_k);
      settle<PAGE, 1>(next_v);
      k_page = next_k;
      v_page = next_v;
      const uint16_t* v_src = &lds_v[buf][v_at];
      bf16x8 vf[2];
      vf[0] = read_v<kRowV>(v_src, 0);
      {
        const bool part = there != ~0ull || t + kStepW > low;  // wave-uniform
        bf16x8 pr[QT][PARTS][kHalves / 2];
#pragma unroll
        for (int n = 0; n < QT; n++) {
          if (part) {
#pragma unroll
            for (int c = 0; c < kHalves; c++)
#pragma unroll
              for (int i = 0; i < 4; i++) {
                const int at = 16 * c + 4 * h + i;
                if (((there >> at) & 1u) == 0u || t + at >= limit[n]) s[n][c][i] = kNegInf;
              }
          }
          float mx = kNegInf;
#pragma unroll
          for (int c = 0; c < kHalves; c++)
#pragma unroll
            for (int i = 0; i < 4; i++) mx = fmaxf(mx, s[n][c][i]);
          mx = quad_max(mx) * p.scale_log2;
          if (__builtin_amdgcn_ballot_w64(mx > m[n] + kHeadroom) != 0) {
            const float top = fmaxf(mx, m[n]), alpha = exp2_fast(m[n] - (top == kNegInf ? 0.0f : top));
            m[n] = top;
            l[n] *= alpha;
#pragma unroll
            for (int d = 0; d < kDims; d++)
#pragma unroll
              for (int i = 0; i < 4; i++) o[n][d][i] *= alpha;
          }
          const float ms = m[n] == kNegInf ? 0.0f : m[n];
#pragma unroll
          for (int c = 0; c < kHalves; c++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const float e = exp2_fast(fmaf(s[n][c][i], p.scale_log2, -ms));
              l[n] += e;
              const __bf16 hi = static_cast<__bf16>(e);
              pr[n][0][c / 2][4 * (c % 2) + i] = hi;
              if constexpr (PARTS == 2) pr[n][1][c / 2][4 * (c % 2) + i] = static_cast<__bf16>(e - static_cast<float>(hi));
            }
        }
        // every operand is read one product ahead
#pragma unroll
        for (int g = 0; g < kHalves / 2 * kDims; g++) {
          const int c = g / kDims, d = g % kDims;
          if (g + 1 < kHalves / 2 * kDims)
            vf[(g + 1) & 1] = read_v<kRowV>(v_src + 32 * ((g + 1) / kDims) * kRowV, (g + 1) % kDims);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int n = 0; n < QT; n++)
#pragma unroll
            for (int a = 0; a < PARTS; a++)
              o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[g & 1], pr[n][a][c], o[n][d], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __syncthreads();
    }

#pragma unroll
    for (int n = 0; n < QT; n++) {
      const float sum = quad_sum(l[n]);
      const int32_t row = wfirst + 16 * n + r;
      if (row > tr.last) continue;
      if (SPLIT && !w.whole) {
        float* part = p.parts + static_cast<int64_t>(w.piece) * (ROWS * (D + 2));
        const int at = row - tr.first;
#pragma unroll
        for (int d = 0; d < kDims; d++) *reinterpret_cast<f32x4*>(part + at * D + 16 * d + 4 * h) = o[n][d];
        if (h == 0) {
          part[ROWS * D + 2 * at] = m[n];
          part[ROWS * D + 2 * at + 1] = sum;
        }
      } else {
        const int32_t i = row / p.group;
        const int64_t row_t = seq.q0 + i, hh = head * p.group + row - i * p.group;
        const float inv = sum == 0.0f ? 0.0f : 4.0f / sum;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + row_t * p.o_st + hh * p.o_sh + 4 * h;
#pragma unroll
        for (int d = 0; d < kDims; d++)
          *reinterpret_cast<u32x2*>(dst + 16 * d) =
              u32x2{pack_out<DT>(o[n][d][0] * inv, o[n][d][1] * inv), pack_out<DT>(o[n][d][2] * inv, o[n][d][3] * inv)};
        if (p.lse && h == 0)
          p.lse[row_t * p.l_st + hh] = sum == 0.0f ? kNegInf : (m[n] + __builtin_amdgcn_logf(sum)) * kLn2;
      }
    }
  }
}

// Joins the pieces of query rows, WAVES waves for each: they take the pieces in turn, every
// lane D / 64 elements.
template <int D, int DT, int ROWS, int WAVES>
__global__ __launch_bounds__(64 * kJoinWaves) void kv4_join_kernel(Kv4AttnParams p) {
  constexpr int kPer = D / 64;
  constexpr int kStepF = ROWS * (D + 2);  // floats of a piece
  __shared__ float lds_o[WAVES][D], lds_l[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int32_t row = blockIdx.x * (kJoinWaves / WAVES) + (WAVES == 1 ? wave : 0);  // of T * Hq
  if (row >= static_cast<int32_t>(p.T) * p.Hq) return;
  const int32_t t = row / p.Hq, qh = row - t * p.Hq;
  int32_t b = t;
  if (p.q_indptr) {  // the sequence that holds row t: the last one whose clamped start is not after it
    int32_t lo = 0, hi = static_cast<int32_t>(p.B);
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (clamp32(read_int(p.q_indptr, mid), p.T) <= t) lo = mid; else hi = mid;
    }
    b = lo;
  }
  const Seq seq = sequence(p, b);
  const int32_t total = p.plan[p.B] * p.Hkv;
  if (t < seq.q0 || t >= seq.q0 + seq.q_len || total == 0) return;
  const int32_t head = qh / p.group, spans = spans_of(p, seq);
  const int32_t idx = (t - seq.q0) * p.group + qh - head * p.group;
  const int32_t unit = idx / ROWS * p.Hkv + head, at = idx % ROWS;
  // the runs that hold a part of this unit
  const int32_t run = run_length(total, p.blocks), from = p.plan[b] * p.Hkv + unit * spans;
  const int32_t run0 = from / run, pieces = (from + spans - 1) / run - run0 + 1;
  if (pieces == 1) return;
  const float* base = p.parts + static_cast<int64_t>(run0 + p.plan[p.B + 1 + b] * p.Hkv + unit) * kStepF;
  const float* ml = base + ROWS * D + 2 * at;

  float top = kNegInf;
  for (int32_t c = lane; c < pieces; c += 64) top = fmaxf(top, ml[static_cast<int64_t>(c) * kStepF]);
  top = wave_max(top);
  const float ts = top == kNegInf ? 0.0f : top;
  float acc[kPer], l = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; i++) acc[i] = 0.0f;
#pragma unroll 4
  for (int32_t c = WAVES == 1 ? 0 : wave; c < pieces; c += WAVES) {
    const int64_t off = static_cast<int64_t>(c) * kStepF;
    const float f = exp2_fast(ml[off] - ts);
    l += ml[off + 1] * f;
#pragma unroll
    for (int i = 0; i < kPer; i++) acc[i] += base[off + at * D + kPer * lane + i] * f;
  }
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int i = 0; i < kPer; i++) lds_o[wave][kPer * lane + i] = acc[i];
    if (lane == 0) lds_l[wave] = l;
    __syncthreads();
    if (wave != 0) return;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; i++) acc[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
      l += lds_l[w];
#pragma unroll
      for (int i = 0; i < kPer; i++) acc[i] += lds_o[w][kPer * lane + i];
    }
  }
  const float inv = l == 0.0f ? 0.0f : 4.0f / l;
  uint16_t* dst = static_cast<uint16_t*>(p.out) + t * p.o_st + qh * p.o_sh + kPer * lane;
  if constexpr (kPer == 1) {
    *dst = static_cast<uint16_t>(pack_out<DT>(acc[0] * inv, 0.0f));
  } else {
#pragma unroll
    for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack_out<DT>(acc[i] * inv, acc[i + 1] * inv);
  }
  if (p.lse && lane == 0) p.lse[t * p.l_st + qh] = l == 0.0f ? kNegInf : (ts + __builtin_amdgcn_logf(l)) * kLn2;
}

// ------------------------------------------------------------------ launch
struct Launch {
  const Kv4AttnParams& p;
  bool split;
  int page;  // kByToken, kBy16, kByStep
  const AttnShape& shape;
  unsigned grid;
  hipStream_t stream;

  template <int D, int DT, int ROWS, bool SPLIT, int PAGE>
  void run() const {
    const size_t lds = 2 * (p.B + 1) * sizeof(int32_t);
    if constexpr (ROWS == kRows) {
      // the plan of a tall call: at most one sequence per CU
      static_assert(tall_waves(DT, D) * (32 * (D + kPadV) * 2 + 2 * kRows * 4 + 16) + 8 * 1024 <= 160 * 1024, "LDS of a CU");
      if (!SPLIT && shape.tall)
        hipLaunchKernelGGL((kv4_attention_kernel<D, DT, tall_waves(DT, D), 2, false, PAGE>), dim3(grid),
                           dim3(64 * tall_waves(DT, D)), lds, stream, p);
      else
        hipLaunchKernelGGL((kv4_attention_kernel<D, DT, kNarrowWaves, narrow_halves(DT, D), SPLIT, PAGE>), dim3(grid),
                           dim3(64 * kNarrowWaves), lds, stream, p);
    } else {
      hipLaunchKernelGGL((kv4_attention_wide_kernel<D, DT, ROWS / 64, SPLIT, PAGE>), dim3(grid),
                         dim3(64 * kWideWaves), lds, stream, p);
    }
    if constexpr (SPLIT) {
      const int64_t rows = p.T * p.Hq;
      // a wave per row, or where the units are cut into many pieces a block
      if (shape.blocks < 8 * shape.units)
        hipLaunchKernelGGL((kv4_join_kernel<D, DT, ROWS, 1>), dim3(static_cast<unsigned>((rows + kJoinWaves - 1) / kJoinWaves)),
                           dim3(64 * kJoinWaves), 0, stream, p);
      else
        hipLaunchKernelGGL((kv4_join_kernel<D, DT, ROWS, kJoinWaves>), dim3(static_cast<unsigned>(rows)),
                           dim3(64 * kJoinWaves), 0, stream, p);
    }
  }
  template <int D, int DT, int ROWS, bool SPLIT>
  void by_page() const {
    if (page == kByStep) run<D, DT, ROWS, SPLIT, kByStep>();
    else if (page == kBy16) run<D, DT, ROWS, SPLIT, kBy16>();
    else run<D, DT, ROWS, SPLIT, kByToken>();
  }
  template <int D, int DT, int ROWS>
  void by_kind() const {
    split ? by_page<D, DT, ROWS, true>() : by_page<D, DT, ROWS, false>();
  }
  template <int D, int DT>
  void by_rows() const {
    if (shape.rows == kRows) by_kind<D, DT, kRows>();
    else if (shape.rows == 64) by_kind<D, DT, 64>();
    else if constexpr (widest(DT, D) == 128) by_kind<D, DT, 128>();
  }
  template <int D>
  void by_type(int dtype) const {
    if (dtype == FP8Q_DTYPE_BF16) by_rows<D, FP8Q_DTYPE_BF16>();
    else by_rows<D, FP8Q_DTYPE_F16>();
  }
};

}  // namespace

int64_t kv4_attention_workspace(int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_tokens) {
  return attention_shape(current_device_shape().cus, dtype, B, T, Hq, Hkv, D, max_tokens).bytes;
}

int launch_kv4_attention(int dtype, int64_t D, Kv4AttnParams p, void* ws, int64_t ws_bytes, hipStream_t stream) {
  const AttnShape s = attention_shape(current_device_shape().cus, dtype, p.B, p.T, p.Hq, p.Hkv, D, p.max_tokens);
  const bool split = s.bytes > 0 && ws && ws_bytes >= s.bytes;
  p.max_units = s.units;
  p.span_shift = s.span_shift;
  if (split) {
    p.blocks = static_cast<int32_t>(s.blocks);
    p.plan = static_cast<int32_t*>(ws);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + s.plan_bytes);
  }
  // Uniform pages where their offsets can be computed in 32 bits.
  const int64_t most = int64_t(1) << 32, most_row = most >> p.c.page_shift;
  const bool fits = p.c.c_sp < most && p.c.s_sp < most && p.c.c_st < most_row && p.c.s_st < most_row;
  const int step = s.rows != kRows ? kStepW : s.tall ? 32 : static_cast<int>(16 * narrow_halves(dtype, D));
  const int page = !fits || p.c.page_shift < 4 ? kByToken : (1 << p.c.page_shift) < step ? kBy16 : kByStep;
  // unsplit: blocks walk the units in turn
  const unsigned grid = static_cast<unsigned>(split ? s.blocks : std::min<int64_t>(s.units, int64_t(1) << 20));
  const Launch run{p, split, page, s, grid, stream};
  if (D == 64) run.by_type<64>(dtype);
  else if (D == 128) run.by_type<128>(dtype);
  else run.by_type<256>(dtype);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("kv4 attention launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace fp8q
