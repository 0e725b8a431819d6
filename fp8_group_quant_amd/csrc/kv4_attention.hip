// kv4_attention.hip — attention over the paged 4-bit cache.
//
//   out[t][h] = sum_j p_j v_j, p = softmax_j(scale * q[t][h] . k_j) over the cached tokens j that
//   query t sees (all of its sequence's, or with `causal` those up to its own place).
//
// One pass over the cache with a running maximum and sum per query row (fp32, base 2). Query
// heads that share a cached head are rows of one tile, so the cache is read once for all.
//
// Tiles. Work is an item: 16 query rows (tokens x heads of the group) of one cached head
// against a chunk of the cached tokens. The waves of a block take 32 tokens at a time in turn,
// each with its own running softmax; their results meet in LDS at the item's end.
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
constexpr int32_t kWhole = 1 << 30;  // spans per chunk: one chunk
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
__device__ __forceinline__ int32_t spans_of(const Seq& s) { return (s.kv_len + kSpan - 1) / kSpan; }
__device__ __forceinline__ int32_t chunks_of(int32_t spans, int32_t per_chunk) {
  return max((spans + per_chunk - 1) / per_chunk, 1);
}

// ------------------------------------------------------------------ work items
// Sum over the block's threads; every thread gets it. `lds` holds one value per wave.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  T s = 0;
#pragma unroll
  for (int i = 0; i < kWaves; i++) s += lds[i];
  return s;
}

// Fills pref[0 .. B] with the exclusive prefix over the sequences of (query tiles x chunks) and
// returns the cached spans of a chunk: the smallest chunk with which all of the work makes at
// most `target` items beside one per tile, so a long sequence is cut into as many pieces as the
// chip needs and short ones stay whole. Every block computes the same from the lengths.
template <bool SPLIT>
__device__ int32_t make_plan(const Kv4AttnParams& p, int32_t* pref) {
  __shared__ unsigned long long sums[kWaves];
  __shared__ int32_t wave_tot[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t B = static_cast<int32_t>(p.B);
  const int32_t per = (B + kThreads - 1) / kThreads;
  const int32_t beg = min(tid * per, B), end = min(beg + per, B);
  int32_t per_chunk = kWhole;
  unsigned long long all_tiles = 0, all_spans = 0;
  for (int32_t b = beg; b < end; b++) {
    const Seq s = sequence(p, b);
    all_tiles += tiles_of(p, s);
    all_spans += static_cast<unsigned long long>(tiles_of(p, s)) * spans_of(s);
  }
  const bool fits = block_sum(all_tiles, sums) * p.Hkv <= static_cast<unsigned long long>(p.max_base);
  if (SPLIT && fits) {
    const unsigned long long total = block_sum(all_spans, sums) * p.Hkv;
    per_chunk = static_cast<int32_t>(max((total + p.target - 1) / p.target, 1ull));
  }
  if (!fits) {  // q_indptr does not ascend: its ranges overlap. Nothing is run
    for (int32_t b = tid; b <= B; b += kThreads) pref[b] = 0;
    __syncthreads();
    return per_chunk;
  }
  int32_t local = 0;
  for (int32_t b = beg; b < end; b++) {
    const Seq s = sequence(p, b);
    local += tiles_of(p, s) * chunks_of(spans_of(s), per_chunk);
  }
  int32_t inc = local;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t up = __shfl_up(inc, off, 64);
    if (lane >= off) inc += up;
  }
  if (lane == 63) wave_tot[wave] = inc;
  __syncthreads();
  int32_t run = inc - local;
#pragma unroll
  for (int w = 0; w < kWaves; w++) run += w < wave ? wave_tot[w] : 0;
  for (int32_t b = beg; b < end; b++) {
    pref[b] = run;
    const Seq s = sequence(p, b);
    run += tiles_of(p, s) * chunks_of(spans_of(s), per_chunk);
  }
  if (tid == kThreads - 1) pref[B] = run;
  __syncthreads();
  return per_chunk;
}

// The sequence b with pref[b] <= u < pref[b + 1].
__device__ __forceinline__ int32_t find_seq(const int32_t* pref, int32_t B, int32_t u) {
  int32_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (pref[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
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

// The 32 tokens of one step of a wave.
template <int D>
struct Step {
  Codes<D> k[2], v[2];
  uint32_t there;  // bit i: token i is inside the range and its page is in the cache
};

template <int D>
__device__ __forceinline__ void load_step(const Kv4AttnParams& p, const int32_t* table, int32_t head, int32_t t,
                                          int32_t t_end, Step<D>& st) {
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  st.there = 0;
#pragma unroll
  for (int s = 0; s < 2; s++) {
    const int32_t tok = t + 16 * s + r;
    bool ok = tok < t_end;
    int32_t page = 0;
    if (ok) {
      page = table[tok >> p.c.page_shift];
      ok = page >= 0 && page < p.c.pages;
    }
    zero_codes<D>(st.k[s]);
    zero_codes<D>(st.v[s]);
    if (ok) {
      const int64_t in = tok & ((1 << p.c.page_shift) - 1);
      const int64_t c = page * p.c.c_sp + in * p.c.c_st + head * p.c.c_sh;
      const int64_t b = page * p.c.s_sp + in * p.c.s_st + head * p.c.s_sh;
      load_codes<D>(p.c.k + c, p.c.ks + b, h, st.k[s]);
      load_codes<D>(p.c.v + c, p.c.vs + b, h, st.v[s]);
    }
    st.there |= static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(ok) & 0xFFFFu) << (16 * s);
  }
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

template <int D, int DT, bool SPLIT>
__global__ __launch_bounds__(kThreads) void kv4_attention_kernel(Kv4AttnParams p) {
  constexpr int PARTS = DT == FP8Q_DTYPE_F16 ? 2 : 1;
  constexpr int kSteps = D / 32;   // contraction steps of S^T
  constexpr int kDims = D / 16;    // dim tiles of O^T
  constexpr int kRowV = D + kPadV;  // LDS row of V (bf16 elements)
  constexpr int kRowO = D + 4;      // LDS row of the joined output (floats)
  static_assert(kRows * kRowO * 4 <= kTile * kRowV * 2, "the joined output reuses V's LDS");
  __shared__ __align__(16) uint16_t lds_v[kWaves][kTile * kRowV];
  __shared__ float lds_m[kWaves][kRows], lds_l[kWaves][kRows];
  extern __shared__ int32_t pref[];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int r = lane & 15, h = lane >> 4;

  // one item per sequence and cached head unless something is split or has several tiles
  const bool direct = !SPLIT && p.q_indptr == nullptr && p.group <= kRows;
  int32_t per_chunk = kWhole;
  if (!direct) per_chunk = make_plan<SPLIT>(p, pref);
  const int32_t units = direct ? static_cast<int32_t>(p.B) : pref[p.B];
  if (SPLIT && blockIdx.x == 0) {
    for (int32_t b = tid; b <= p.B; b += kThreads) p.plan[b] = pref[b];
    if (tid == 0) p.plan[p.B + 1] = per_chunk;
  }
  const int32_t items = units * p.Hkv;

  for (int32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int32_t u = item / p.Hkv, head = item - u * p.Hkv;
    const int32_t b = direct ? u : find_seq(pref, static_cast<int32_t>(p.B), u);
    const Seq seq = sequence(p, b);
    int32_t tile = 0, chunk = 0, chunks = 1;
    if (!direct) {
      const int32_t tiles = tiles_of(p, seq), at = u - pref[b];
      chunks = chunks_of(spans_of(seq), per_chunk);
      chunk = at / tiles;
      tile = at - chunk * tiles;
    }
    const int32_t spans = spans_of(seq);
    const int32_t t0 = static_cast<int32_t>(static_cast<int64_t>(spans) * chunk / chunks) * kSpan;
    const int32_t t1 = min(static_cast<int32_t>(static_cast<int64_t>(spans) * (chunk + 1) / chunks) * kSpan, seq.kv_len);

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
    const int32_t t_end = min(t1, high);

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

    const int32_t* table = p.table + b * p.table_sb;
    uint16_t* vt = lds_v[wave];
    f32x4 o[kDims];
#pragma unroll
    for (int d = 0; d < kDims; d++) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = kNegInf, l = 0.0f;  // l: this lane's share of the row's sum

    Step<D> cur;
    int32_t t = t0 + kTile * wave;
    if (t < t_end) load_step<D>(p, table, head, t, t_end, cur);
    for (; t < t_end; t += kSpan) {
      Step<D> nxt;
      if (t + kSpan < t_end) load_step<D>(p, table, head, t + kSpan, t_end, nxt);

      f32x4 s[2];
#pragma unroll
      for (int c = 0; c < 2; c++) {
        s[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kSteps; j++) {
          const bf16x8 k = widen_codes<D>(cur.k[c], j);
#pragma unroll
          for (int a = 0; a < PARTS; a++) s[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[a][j], s[c], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kSteps; j++)
          *reinterpret_cast<bf16x8*>(vt + (16 * c + r) * kRowV + D / 4 * h + 8 * j) = widen_codes<D>(cur.v[c], j);
      }

      float x[2][4], mx = kNegInf;
#pragma unroll
      for (int c = 0; c < 2; c++)
#pragma unroll
        for (int i = 0; i < 4; i++) x[c][i] = s[c][i] * p.scale_log2;
      if (cur.there != 0xFFFFFFFFu || t + kTile > low) {  // wave-uniform
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int at = 16 * c + 4 * h + i;
            if (((cur.there >> at) & 1u) == 0u || t + at >= limit) x[c][i] = kNegInf;
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
        const uint16_t* at = vt + (4 * h + (r >> 2)) * kRowV + 16 * d + 4 * (r & 3);
        const s16x4 a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at));
        const s16x4 a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * kRowV));
        const auto av = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int a = 0; a < PARTS; a++)
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av), pr[a], o[d], 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      cur = nxt;
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
      if (SPLIT && chunks > 1) {
        float* part = p.parts + static_cast<int64_t>(item) * (kRows * (D + 2));
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
        const int64_t at = seq.q0 + i, hh = head * p.group + static_cast<int32_t>(ri - static_cast<int64_t>(i) * p.group);
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] = pack16<DT>(v[2 * j] * inv, v[2 * j + 1] * inv);
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out) + at * p.o_st + hh * p.o_sh + col) = w;
        if (p.lse && col == 0)
          p.lse[at * p.l_st + hh] = ll > 0.0f ? (mm + __builtin_amdgcn_logf(ll)) * 0.6931471805599453f : kNegInf;
      }
    }
    __syncthreads();
  }
}

// Joins the chunks of one query row: a block per (token, query head). The waves take the chunks
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
  const int32_t tiles = tiles_of(p, seq);
  const int32_t chunks = chunks_of(spans_of(seq), p.plan[p.B + 1]);
  if (chunks <= 1) return;
  const int32_t head = qh / p.group;
  const int64_t idx = static_cast<int64_t>(t - seq.q0) * p.group + (qh - head * p.group);
  const int32_t tile = static_cast<int32_t>(idx / kRows), row = static_cast<int32_t>(idx % kRows);
  const int64_t step = static_cast<int64_t>(tiles) * p.Hkv * (kRows * (D + 2));
  const float* base = p.parts + (static_cast<int64_t>(p.plan[b] + tile) * p.Hkv + head) * (kRows * (D + 2));

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
  int64_t base;    // items without splitting, at most
  int64_t target;  // items wanted when splitting
  int64_t plan_bytes, bytes;
};

Shape shape_of(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  Shape s;
  s.base = Hkv * ((T * (Hq / Hkv) + kRows - 1) / kRows + B);
  s.target = static_cast<int64_t>(current_device_shape().cus) * 4;
  s.plan_bytes = ((B + 2) * 4 + 255) / 256 * 256;
  s.bytes = s.plan_bytes + (s.base + s.target) * (kRows * (D + 2)) * 4;
  return s;
}

template <int D, int DT>
void launch_d(const Kv4AttnParams& p, bool split, unsigned grid, hipStream_t stream) {
  const size_t lds = (p.B + 1) * sizeof(int32_t);
  if (split) {
    hipLaunchKernelGGL((kv4_attention_kernel<D, DT, true>), dim3(grid), dim3(kThreads), lds, stream, p);
    hipLaunchKernelGGL((kv4_join_kernel<D, DT>), dim3(static_cast<unsigned>(p.T * p.Hq)), dim3(kThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL((kv4_attention_kernel<D, DT, false>), dim3(grid), dim3(kThreads), lds, stream, p);
  }
}

template <int D>
void launch_dt(int dtype, const Kv4AttnParams& p, bool split, unsigned grid, hipStream_t stream) {
  if (dtype == FP8Q_DTYPE_BF16) launch_d<D, FP8Q_DTYPE_BF16>(p, split, grid, stream);
  else launch_d<D, FP8Q_DTYPE_F16>(p, split, grid, stream);
}

}  // namespace

int64_t kv4_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_tokens) {
  const Shape s = shape_of(B, T, Hq, Hkv, D);
  if (max_tokens <= kSpan || s.base >= 4 * s.target) return 0;
  return s.bytes;
}

int launch_kv4_attention(int dtype, int64_t D, Kv4AttnParams p, void* ws, int64_t ws_bytes, hipStream_t stream) {
  const Shape s = shape_of(p.B, p.T, p.Hq, p.Hkv, D);
  const int64_t need = kv4_attention_workspace(p.B, p.T, p.Hq, p.Hkv, D, p.max_tokens);
  const bool split = need > 0 && ws && ws_bytes >= need;
  p.max_base = s.base;
  if (split) {
    p.target = static_cast<int32_t>(s.target);
    p.plan = static_cast<int32_t*>(ws);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + s.plan_bytes);
  }
  // blocks walk the items in turn
  const int64_t most = split ? s.base + s.target : s.base;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(most, static_cast<int64_t>(current_device_shape().cus) * 8));
  if (D == 64) launch_dt<64>(dtype, p, split, grid, stream);
  else if (D == 128) launch_dt<128>(dtype, p, split, grid, stream);
  else launch_dt<256>(dtype, p, split, grid, stream);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("kv4 attention launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace fp8q
