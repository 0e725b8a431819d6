// gemm_mxfp4.hip — Y = A B^T of two matrices of e2m1 codes with one UE8M0 scale per 32 elements of a row
// (MXFP4), rounded to bf16 once:
//   Y[m][n] = bf16( sum_k 2^(ea(m, k/32) - 127) A[m][k] * 2^(eb(n, k/32) - 127) B[n][k] )
//
// A product of two codes and scales is exact; the sums are the matrix cores' fp32, in the order of K within a range, and
// the rounding to bf16 is the only other one.
//
// Tiles. A block owns a tile of 256 x 256, 128 x 128 or 64 x 128 outputs and takes K in steps that four
// stages of LDS hold, loaded straight there by the asynchronous loads, three steps ahead, so that the matrix cores are fed
// without a pause also from one tile to the next: blocks are persistent, and the loads run on into the next tile while the
// last one's outputs are stored. Between the products of a quarter step lie the LDS reads of the next one and the loads' issue.
// Rows are swizzled in LDS so that no reads collide. The outputs go through LDS, 32 rows x 64 columns of a wave at a
// time, so that every store writes whole lines (past the caches they are slower).
//
// What bounds it. 8192^3, tiles of 256 x 256: 281 to 312 us back to back (by the clock that the power allows; 3.5 to 3.9
// PFLOP/s), 260 in calls with pauses between them. The matrix pipe is busy in 58 % of the cycles of a clock that the power holds at 1.7 GHz (products
// alone, without loads, reach 6.3 to 6.9 PFLOP/s on random codes and 8.6 to 9.2 on zeros). The loads come next: 31
// clocks of a CU for each 1 KB, so that 32 of a step's 34 KB take 992 clocks next to 1024 of products. Scale words by
// 16-byte loads, four in the place of eight of the 40 instructions: 2 to 4 % less on column-major words, but no other
// layout; not done. 8 waves to a block, or tiles in groups of 2 or 8 rows instead of 4: no faster. 4096^2 x 7168 67 us (3.6
// PFLOP/s), 2048 x 4096 x 7168 44 (2.7), 1024 x 4096 x 7168 22.7 (2.6), 333 x 4104 x 2176 9.4, 1024^3 6.5.
#include <algorithm>
#include <type_traits>

#include "mxfp4.h"
#include "mxfp4_shape.h"

namespace fp8q {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Outputs, whose rows may begin at any element (vector stores to global memory need no alignment here).
typedef u32x2 __attribute__((aligned(2))) u32x2_any;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

constexpr int kFp4 = 4;     // operand format of the matrix instruction
constexpr int kStepK = 128;  // K is split, and scale words are counted, in units of 128 elements
constexpr int kUnit = kStepK / 2;  // their bytes

// A block's tile: BM x BN outputs by WAVES_M x WAVES_N waves, in steps of QUARTERS * 64 elements of K, STAGES of them in
// LDS, BLOCKS of a CU.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int QUARTERS_, int STAGES_, int BLOCKS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, QUARTERS = QUARTERS_, STAGES = STAGES_;
  static constexpr int kBlocks = BLOCKS_;
  static constexpr bool kSplit = false;  // whether K is split
  static constexpr int kWaves = WAVES_M * WAVES_N, kThreads = 64 * kWaves;
  static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N, SM = WTM / 32, SN = WTN / 32;
  static constexpr int kRow = 32 * QUARTERS, kWords = kRow / kUnit;  // bytes and scale words of a row and step
  // one stage: rows of A and B, then their scale words [kWords][BM], [kWords][BN]
  static constexpr int kB = BM * kRow, kSA = kB + BN * kRow, kSB = kSA + 4 * kWords * BM, kStage = kSB + 4 * kWords * BN;
  static constexpr int kLds = STAGES * kStage;
  // loads of a wave and step: 1 KB pieces of kPiece rows, and 64 scale words each
  static constexpr int kPiece = 1024 / kRow, kLA = BM / kPiece / kWaves, kLB = BN / kPiece / kWaves;
  static constexpr int kGroups = (BM + BN) / 64, kPer = (kGroups + kWaves - 1) / kWaves;  // groups of 64 scale rows
  static constexpr int kLoads = kLA + kLB + kPer * kWords, kMma = SM * SN;
  static constexpr int kFirst = kLoads / 2;  // that go out in a step's last quarter, the others in the next one's first
  static_assert(QUARTERS == 2 || QUARTERS == 4, "64 or 128 bytes");
  static_assert(kLA * kWaves * kPiece == BM && kLB * kWaves * kPiece == BN && BM % 64 == 0 && BN % 64 == 0, "load split");
  static_assert(kRow == 64 || (kLA % 2 == 0 && kLB % 2 == 0), "a wave's pieces alternate from an even one on");
  static_assert(SN % 2 == 0, "outputs go through LDS in pairs of subtiles");
  static_assert(kBlocks * (kLds + kWaves * 32 * 144) <= 160 * 1024, "LDS");

  // Rows that the same lanes of a fragment read lie in all banks: 16-byte chunk c of a row is at c ^ swizzle(row).
  static __device__ __forceinline__ int swizzle(int row) { return kRow == 64 ? (row >> 2) & 3 : (row >> 1) & 7; }
};

template <class T>
struct Splitting : T {
  static constexpr bool kSplit = true;
};

typedef __attribute__((address_space(3))) uint8_t lds_u8;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8*)p));
}
typedef int v4i __attribute__((ext_vector_type(4)));
// A load to LDS that reads M0 needs a wait state after the scalar instruction that writes it; in an asm statement the
// compiler puts none.
// lane l: LDS [lds + 16 l, + 16) <- buffer [voff, + 16), all of the offset in the register that the bounds check looks at
__device__ __forceinline__ void dma16(uint32_t lds, v4i buffer, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(buffer)
               : "memory", "m0");
}
// lane l: LDS [lds + 4 l, + 4) <- global [base + voff, + 4)
__device__ __forceinline__ void dma4(uint32_t lds, const uint8_t* base, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ v8i operand(u32x4 w) {
  return v8i{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3]), 0, 0, 0, 0};
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(a))) |
         static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(b))) << 16;
}

constexpr int kGroupM = 4;

// The kernel's arguments, read again where they are used, so that they hold no registers in the loop.
typedef const __attribute__((address_space(4))) Mxfp4GemmParams* Args;
__device__ __forceinline__ Args arguments() {
  Args a = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}

__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Unit t of the work: a tile and one of p->splits ranges of K (units first .. first + units - 1). The host makes sure
// that there are fewer than 2^31.
struct Place {
  int64_t m0, n0;
  int split, first, units;
};
template <class C>
__device__ __forceinline__ Place place_of(Args p, int32_t t) {
  const int32_t tiles_m = static_cast<int32_t>((p->M + C::BM - 1) / C::BM), tiles_n = static_cast<int32_t>((p->N + C::BN - 1) / C::BN);
  const int32_t split = C::kSplit ? uniform(t / (tiles_m * tiles_n)) : 0;
  t -= split * tiles_m * tiles_n;
  const int32_t first = uniform(t / tiles_n / kGroupM) * kGroupM;  // rows of tiles are taken kGroupM at a time
  const int32_t rows = min(tiles_m - first, kGroupM), at = t - first * tiles_n, n = uniform(at / rows);
  const int32_t all = static_cast<int32_t>(p->K / kStepK);  // splits * all < 2^31
  const int32_t k0 = C::kSplit ? uniform(all * split / p->splits) : 0, k1 = C::kSplit ? uniform(all * (split + 1) / p->splits) : all;
  return Place{int64_t(first + at - n * rows) * C::BM, int64_t(n) * C::BN, split, k0, k1 - k0};
}

// What a block's loads of one tile start from: the operands' rows as buffers (what lies past the last row's end is not
// read), and the scale words of the lanes' rows.
template <class C>
struct Source {
  v4i a, b;
  const uint8_t* s_base[C::kPer];
  uint32_t s_off[C::kPer];

  // Of scale group q of a wave: whether it is A's, and its first row. (Where the groups do not divide, some are loaded twice.)
  static __device__ __forceinline__ int group(int q, int wave) { return (q * C::kWaves + wave) % C::kGroups; }
  static __device__ __forceinline__ bool of_a(int q, int wave) { return group(q, wave) < C::BM / 64; }
  static __device__ __forceinline__ int first(int q, int wave) { return (group(q, wave) - (of_a(q, wave) ? 0 : C::BM / 64)) * 64; }
  static __device__ __forceinline__ v4i buffer(const uint8_t* base, int64_t rows, int64_t ld, int64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    const uint32_t size = static_cast<uint32_t>(min((rows - 1) * ld + bytes, int64_t(0xFFFFFFFF)));
    return v4i{static_cast<int32_t>(at), static_cast<int32_t>(at >> 32), static_cast<int32_t>(size), 0x00020000};
  }
  __device__ __forceinline__ void enter(int32_t tile, int lane, int wave) {
    const Args p = arguments();
    const Place at = place_of<C>(p, tile);
    const int64_t skip = int64_t(at.first) * kUnit, bytes = p->K / 2 - skip;
    a = buffer(p->a + at.m0 * p->lda + skip, p->M - at.m0, p->lda, bytes);
    b = buffer(p->b + at.n0 * p->ldb + skip, p->N - at.n0, p->ldb, bytes);
#pragma unroll
    for (int q = 0; q < C::kPer; q++) {
      const bool is_a = of_a(q, wave);
      const int64_t sm = is_a ? p->sa_sm : p->sb_sn, rows = is_a ? p->M - 1 - at.m0 : p->N - 1 - at.n0;
      s_base[q] = (is_a ? p->sa + at.m0 * sm * 4 : p->sb + at.n0 * sm * 4) + at.first * (is_a ? p->sa_sk : p->sb_sk) * 4;
      s_off[q] = static_cast<uint32_t>(min(int64_t(first(q, wave) + lane), rows) * sm * 4);
    }
  }
};

// The loads of a block's steps, one after the other through its tiles; past the last tile its steps again, so that every
// step issues the same loads. Rows past an operand's end bring anything: their products are not stored. Where a step holds
// two units of K, the last one may hold only one: the other's bytes are the next row's (or nothing), and not used.
template <class C>
struct Loader {
  const uint32_t lds;
  const int lane, wave, units, steps;  // units of K, steps
  const int32_t stride, stop;          // of the tiles
  const uint32_t lda_piece, ldb_piece;  // bytes of a piece's rows
  uint32_t a_off[2], b_off[2];          // the lane's part: even and odd pieces
  int64_t s_step[C::kPer];              // bytes between the words of two units
  int32_t tile;
  int step;
  uint32_t stage;  // its offset
  Source<C> now, next;

  __device__ __forceinline__ Loader(const TileSpan& s, uint32_t lds_at, int lane_, int wave_, int units_)
      : lds(lds_at), lane(lane_), wave(wave_), units(units_), steps((units_ + C::kWords - 1) / C::kWords),
        stride(static_cast<int32_t>(s.stride)), stop(static_cast<int32_t>(s.end)),
        lda_piece(static_cast<uint32_t>(C::kPiece * arguments()->lda)), ldb_piece(static_cast<uint32_t>(C::kPiece * arguments()->ldb)),
        tile(static_cast<int32_t>(s.beg)), step(0), stage(0) {
    constexpr int kChunks = C::kRow / 16;
    const int row = lane / kChunks;
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const uint32_t chunk = 16 * ((lane % kChunks) ^ C::swizzle(C::kPiece * q + row));
      a_off[q] = row * (lda_piece / C::kPiece) + chunk;
      b_off[q] = row * (ldb_piece / C::kPiece) + chunk;
    }
#pragma unroll
    for (int q = 0; q < C::kPer; q++) s_step[q] = 4 * (Source<C>::of_a(q, wave) ? arguments()->sa_sk : arguments()->sb_sk);
    now.enter(tile, lane, wave);
  }
  // Looks up the tile after the loads' present one, once per tile that is computed: every tile has one step at which the
  // loads go on to the next.
  __device__ __forceinline__ void look_ahead() {
    if (tile + stride < stop) tile += stride;
    next.enter(tile, lane, wave);
  }
  // Load number n of the step: pieces of A and B, then scale words.
  __device__ __forceinline__ void issue(int n) {
    const uint32_t at = lds + stage;
    if (n < C::kLA) {
      dma16(at + (wave * C::kLA + n) * 1024, now.a, a_off[n & 1] + ((wave * C::kLA + n) * lda_piece + step * C::kRow));
    } else if (n < C::kLA + C::kLB) {
      const int q = n - C::kLA;
      dma16(at + C::kB + (wave * C::kLB + q) * 1024, now.b, b_off[q & 1] + ((wave * C::kLB + q) * ldb_piece + step * C::kRow));
    } else {
      const int q = (n - C::kLA - C::kLB) / C::kWords, word = (n - C::kLA - C::kLB) % C::kWords;
      const bool is_a = Source<C>::of_a(q, wave), there = word == 0 || C::kWords * step + word < units;
      dma4(at + (is_a ? C::kSA + 4 * word * C::BM : C::kSB + 4 * word * C::BN) + 4 * Source<C>::first(q, wave),
           now.s_base[q] + (word > 0 && there ? s_step[q] : 0), now.s_off[q]);
    }
  }
  // On to the next step (without a branch, across which products could be moved).
  __device__ __forceinline__ void advance() {
    stage = stage + C::kStage == C::kLds ? 0 : stage + C::kStage;
    const bool last = step + 1 == steps;
    step = last ? 0 : step + 1;
#pragma unroll
    for (int i = 0; i < 3; i++) {
      now.a[i] = last ? next.a[i] : now.a[i];
      now.b[i] = last ? next.b[i] : now.b[i];
    }
#pragma unroll
    for (int q = 0; q < C::kPer; q++) {
      now.s_base[q] = last ? next.s_base[q] : now.s_base[q] + C::kWords * s_step[q];
      now.s_off[q] = last ? next.s_off[q] : now.s_off[q];
    }
  }
  __device__ __forceinline__ void issue_all() {
#pragma unroll
    for (int n = 0; n < C::kLoads; n++) issue(n);
    advance();
  }
};

// v_mfma_scale_f32_32x32x64: lane (r, h) of an operand holds row r's 32 elements of K block h and that block's scale byte.
template <class C>
struct Compute {
  const uint8_t* smem;
  uint32_t a_at[C::QUARTERS], b_at[C::QUARTERS];  // LDS offsets of the lane's first subtile for each quarter of a step
  uint32_t sa_at, sb_at, pick;
  u32x4 fa[2][C::SM], fb[2][C::SN];
  uint32_t wa[C::kWords][C::SM], wb[C::kWords][C::SN];  // scale words of the next step
  uint32_t ea[C::SM], eb[C::SN];                        // scale bytes of this step's quarters
  v16f acc[C::SM][C::SN];

  __device__ __forceinline__ Compute(const uint8_t* s, int lane, int wm, int wn) : smem(s) {
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int k = 0; k < C::QUARTERS; k++) {
      const int chunk = 16 * ((2 * k + h) ^ C::swizzle(r));
      a_at[k] = (wm * C::WTM + r) * C::kRow + chunk;
      b_at[k] = C::kB + (wn * C::WTN + r) * C::kRow + chunk;
    }
    sa_at = C::kSA + 4 * (wm * C::WTM + r);
    sb_at = C::kSB + 4 * (wn * C::WTN + r);
    pick = C::kWords == 1 ? 8 * h : h ? 0x07050301u : 0x06040200u;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < C::SM; i++)
#pragma unroll
      for (int j = 0; j < C::SN; j++) acc[i][j] = v16f{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  }
  static constexpr int kReads = C::SM + C::SN, kReads0 = (1 + C::kWords) * kReads;
  // Read number n of quarter K of the stage at offset `st`: operands of A and B, then (K = 0) the scale words.
  template <int K>
  __device__ __forceinline__ void read(int n, uint32_t st) {
    if (n < C::SM) {
      fa[K & 1][n] = *reinterpret_cast<const u32x4*>(smem + st + a_at[K] + n * 32 * C::kRow);
    } else if (n < kReads) {
      fb[K & 1][n - C::SM] = *reinterpret_cast<const u32x4*>(smem + st + b_at[K] + (n - C::SM) * 32 * C::kRow);
    } else if (K == 0 && n < kReads0) {
      const int i = (n - kReads) / C::kWords, w = (n - kReads) % C::kWords;
      if (i < C::SM) wa[w][i] = *reinterpret_cast<const uint32_t*>(smem + st + sa_at + 4 * w * C::BM + 128 * i);
      else wb[w][i - C::SM] = *reinterpret_cast<const uint32_t*>(smem + st + sb_at + 4 * w * C::BN + 128 * (i - C::SM));
    }
  }
  // The lane's bytes of the step that was read: of quarter k byte k (two units), or 2 k.
  __device__ __forceinline__ void scales() {
#pragma unroll
    for (int i = 0; i < C::SM; i++) ea[i] = C::kWords == 1 ? wa[0][i] >> pick : __builtin_amdgcn_perm(wa[C::kWords - 1][i], wa[0][i], pick);
#pragma unroll
    for (int j = 0; j < C::SN; j++) eb[j] = C::kWords == 1 ? wb[0][j] >> pick : __builtin_amdgcn_perm(wb[C::kWords - 1][j], wb[0][j], pick);
  }
  // The products of quarter K, between them the reads of quarter NEXT from the stage at `st` and `more` of each one.
  template <int K, int NEXT, class F>
  __device__ __forceinline__ void quarter(uint32_t st, F more) {
    constexpr int kN = NEXT == 0 ? kReads0 : kReads, kByte = C::kWords == 1 ? 2 * K : K;
    int done = 0;
#pragma unroll
    for (int t = 0; t < C::kMma; t++) {
      const int i = t / C::SN, j = t % C::SN;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[K & 1][j]), operand(fa[K & 1][i]), acc[i][j], kFp4, kFp4,
                                                                  kByte, static_cast<int>(eb[j]), kByte, static_cast<int>(ea[i]));
#pragma unroll
      for (; done < (t + 1) * kN / C::kMma; done++) read<NEXT>(done, st);
      more(t);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The wave's outputs, 32 rows x 64 columns at a time through LDS, so that every store writes whole lines (a lane has 4
// columns of its row in each group of 8).
constexpr int kOutRow = 128 + 16;       // LDS bytes of a row of 64 columns
constexpr int kOutWave = 32 * kOutRow;  // of a wave

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The sums of one range of K, [split][M][N4] fp32 with rows of N4 = N rounded up to 4: a subtile of 32 x 32 at a time.
template <class C>
__device__ __forceinline__ void store_part(uint8_t* lds, Args p, const Place& at, const Compute<C>& c, int lane, int wm, int wn) {
  const int64_t n4 = (p->N + 3) & ~int64_t(3), m0 = at.m0 + wm * C::WTM, n0 = at.n0 + wn * C::WTN;
  uint8_t* const put = lds + (lane & 31) * kOutRow + 16 * (lane >> 5);
  const uint8_t* const get = lds + (lane >> 3) * kOutRow + 16 * (lane & 7);
  float* row = p->ws + (at.split * p->M + m0 + (lane >> 3)) * n4 + n0 + 4 * (lane & 7);
  const int rows = static_cast<int>(min(p->M - m0, int64_t(C::WTM))) - (lane >> 3);
  const int cols = static_cast<int>(min(n4 - n0, int64_t(C::WTN))) - 4 * (lane & 7);
#pragma unroll
  for (int i = 0; i < C::SM; i++) {
#pragma unroll
    for (int j = 0; j < C::SN; j++) {
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const v16f& v = c.acc[i][j];
        *reinterpret_cast<v4f*>(put + 32 * g) = v4f{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
      }
      wave_fence();
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const v4f w = *reinterpret_cast<const v4f*>(get + 8 * k * kOutRow);
        if (32 * i + 8 * k < rows && 32 * j < cols) *reinterpret_cast<v4f*>(row + 8 * k * n4 + 32 * j) = w;
      }
      wave_fence();
      __builtin_amdgcn_sched_barrier(0);
    }
    row += 32 * n4;
  }
}

template <class C>
__device__ __forceinline__ void store_tile(uint8_t* lds, int32_t tile, const Compute<C>& c, int lane, int wm, int wn) {
  const Args p = arguments();
  const Place at = place_of<C>(p, tile);
  if constexpr (C::kSplit) {
    store_part<C>(lds, p, at, c, lane, wm, wn);
    return;
  }
  const int64_t m0 = at.m0 + wm * C::WTM, n0 = at.n0 + wn * C::WTN, ldy = p->ldy;
  uint8_t* const put = lds + (lane & 31) * kOutRow + 8 * (lane >> 5);
  const uint8_t* const get = lds + (lane >> 3) * kOutRow + 16 * (lane & 7);
  uint16_t* row = p->y + (m0 + (lane >> 3)) * ldy + n0 + 8 * (lane & 7);
  const bool whole = m0 + C::WTM <= p->M && n0 + C::WTN <= p->N;
  const int rows = static_cast<int>(min(p->M - m0, int64_t(C::WTM))) - (lane >> 3);
  const int cols = static_cast<int>(min(p->N - n0, int64_t(C::WTN))) - 8 * (lane & 7);
#pragma unroll
  for (int i = 0; i < C::SM; i++) {
#pragma unroll
    for (int j = 0; j < C::SN; j += 2) {
#pragma unroll
      for (int q = 0; q < 2; q++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
          const v16f& v = c.acc[i][j + q];
          *reinterpret_cast<u32x2*>(put + 64 * q + 16 * g) = u32x2{bf16_pair(v[4 * g], v[4 * g + 1]), bf16_pair(v[4 * g + 2], v[4 * g + 3])};
        }
      wave_fence();
      u32x4 w[4];
#pragma unroll
      for (int k = 0; k < 4; k++) w[k] = *reinterpret_cast<const u32x4*>(get + 8 * k * kOutRow);
      if (whole) {
#pragma unroll
        for (int k = 0; k < 4; k++) *reinterpret_cast<u32x4_any*>(row + 8 * k * ldy + 32 * j) = w[k];
      } else {
        const int left = cols - 32 * j;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          if (32 * i + 8 * k < rows) {
            uint16_t* const to = row + 8 * k * ldy + 32 * j;
            if (left >= 8) {
              *reinterpret_cast<u32x4_any*>(to) = w[k];
            } else {
#pragma unroll
              for (int q = 0; q < 7; q++)
                if (q < left) to[q] = static_cast<uint16_t>(w[k][q >> 1] >> (16 * (q & 1)));
            }
          }
        }
      }
      wave_fence();
      __builtin_amdgcn_sched_barrier(0);
    }
    row += 32 * ldy;
  }
}

template <class C>
__global__ __launch_bounds__(C::kThreads, C::kBlocks) void gemm_mxfp4_kernel(Mxfp4GemmParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::kLds + C::kWaves * kOutWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % C::WAVES_M, wn = wave / C::WAVES_M;
  const int64_t tiles = ((p.M + C::BM - 1) / C::BM) * ((p.N + C::BN - 1) / C::BN) * (C::kSplit ? p.splits : 1);
  const TileSpan span = tile_span(tiles, blockIdx.x, gridDim.x, p.xcds);
  if (span.beg >= span.end) return;
  // (a call that splits K has a tile for each block, so that all of a block's tiles have as many steps)
  const int units = C::kSplit ? place_of<C>(arguments(), static_cast<int32_t>(span.beg)).units : static_cast<int>(p.K / kStepK);
  const int whole = units / C::kWords;
  Loader<C> load(span, lds_addr(smem), lane, wave, units);
  Compute<C> c(smem, lane, wm, wn);
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; s++) {
    if (load.step == 0) load.look_ahead();
    load.issue_all();
  }
  if (load.step == 0) load.look_ahead();
#pragma unroll
  for (int n = 0; n < C::kFirst; n++) load.issue(n);
  wait_vmcnt<(C::STAGES - 2) * C::kLoads + C::kFirst>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int n = 0; n < Compute<C>::kReads0; n++) c.template read<0>(n, 0);
  uint32_t st = 0;
  for (int32_t t = static_cast<int32_t>(span.beg); t < static_cast<int32_t>(span.end); t += static_cast<int32_t>(span.stride)) {
    c.clear();
    // what ends a step: its successor's loads have landed (they are older than those of the steps after it; a tile's stores,
    // younger than some of these, only make the wait longer), everyone has read its stage, which is filled anew
    auto turn = [&]() {
      wait_vmcnt<(C::STAGES - 2) * C::kLoads>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      st = st + C::kStage == C::kLds ? 0 : st + C::kStage;
    };
    auto none = [](int) {};
    // a step's first loads go out after the turn that frees their stage, the others in the next step's first quarter
    auto loads_first = [&](int n) {
#pragma unroll
      for (int i = n * C::kFirst / C::kMma; i < (n + 1) * C::kFirst / C::kMma; i++) load.issue(i);
    };
    auto loads_rest = [&](int n) {
      constexpr int kRest = C::kLoads - C::kFirst;
#pragma unroll
      for (int i = n * kRest / C::kMma; i < (n + 1) * kRest / C::kMma; i++) load.issue(C::kFirst + i);
    };
    for (int s = 0; s < whole; s++) {
      c.scales();
      c.template quarter<0, 1>(st, loads_rest);
      load.advance();
      if constexpr (C::QUARTERS == 4) {
        c.template quarter<1, 2>(st, none);
        c.template quarter<2, 3>(st, none);
      }
      turn();
      c.template quarter<C::QUARTERS - 1, 0>(st, loads_first);
    }
    if constexpr (C::QUARTERS == 4) {
      if (units % C::kWords != 0) {  // a last step of one unit
        c.scales();
        c.template quarter<0, 1>(st, loads_rest);
        load.advance();
        turn();
        c.template quarter<1, 0>(st, loads_first);
      }
    }
    store_tile<C>(smem + C::kLds + wave * kOutWave, t, c, lane, wm, wn);
    load.look_ahead();
  }
  wait_vmcnt<0>();  // nothing is under way into LDS when the block ends
}

// 256 x 256 outputs of 4 waves hold 512 registers a lane, with the loop free of scratch; the others leave half of them.
using Large = Tile<256, 256, 2, 2, 2, 4, 1>;
using Deep = Tile<128, 128, 2, 2, 4, 4, 1>;
using Flat = Tile<64, 128, 2, 2, 4, 4, 1>;

// Y = bf16( the splits' sums added in their order, so that results do not change from call to call ): four columns per
// thread.
__global__ __launch_bounds__(256) void gemm_mxfp4_join_kernel(Mxfp4GemmParams p) {
  const int64_t quads = (p.N + 3) / 4, total = p.M * quads, plane = p.M * quads;
  for (int64_t t = blockIdx.x * int64_t(256) + threadIdx.x; t < total; t += gridDim.x * int64_t(256)) {
    const v4f* src = reinterpret_cast<const v4f*>(p.ws) + t;
    v4f v[kMxfp4MostSplits];
#pragma unroll
    for (int s = 0; s < kMxfp4MostSplits; s++)
      if (s < p.splits) v[s] = src[s * plane];
    v4f sum = v[0];
#pragma unroll
    for (int s = 1; s < kMxfp4MostSplits; s++)
      if (s < p.splits) {
#pragma unroll
        for (int q = 0; q < 4; q++) sum[q] += v[s][q];
      }
    const int64_t m = t / quads, n = (t - m * quads) * 4;
    uint16_t* y = p.y + m * p.ldy + n;
    const u32x2 w = {bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
    if (n + 4 <= p.N) {
      *reinterpret_cast<u32x2_any*>(y) = w;
    } else {
#pragma unroll
      for (int q = 0; q < 3; q++)
        if (n + q < p.N) y[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
    }
  }
}

// Y of an empty K.
__global__ __launch_bounds__(256) void gemm_mxfp4_zero_kernel(uint16_t* y, int64_t M, int64_t N, int64_t ldy) {
  for (int64_t t = blockIdx.x * int64_t(256) + threadIdx.x; t < M * N; t += gridDim.x * int64_t(256)) y[t / N * ldy + t % N] = 0;
}

// ------------------------------------------------------------------ few rows
// Up to 16 SM rows of A: a block has 16 rows of B and all of K, its W waves contiguous ranges of it; operands go from
// memory straight to registers, P units of 128 elements at a time, and the waves' sums meet in LDS, added in their
// order. (v_mfma_scale_f32_16x16x128: lane (r, h) holds row r, the 32 elements of K block h, and its scale byte.) A lane
// loads the scale word of one row for one of four units (lane group h the h-th), which the others get by exchanges.
//
// The weights' bytes bound it, for one row N x K (launch included): 4096 x 7168, 15.6 MB, 5.6 us; 16384 x 4096, 35.7 MB, 8.9
// (4.0 TB/s); 28672 x 8192, 125 MB, 25.3 (4.9). A range that is not whole in P ends in a step of four units or of P with
// clamped loads (steps of P only: 16384 x 4096, of 4 units to a wave, 12.9). Blocks are of 8 waves while no CU has two,
// else of 4, which then have more loads each under way: us for 4 and 8, one row, 4096 x 7168 6.0 and 5.7, 16384 x 4096 8.8 and
// 10.1, 28672 x 8192 25.7 and 29.8; 32 rows, 4096 x 7168 8.5 and 7.7, 8192 x 8192 15.4 and 15.9; 64 rows, 4096 x 7168 13.9 and
// 11.3, 8192 x 8192 23.9 and 23.6.

// The words that lane groups 0 .. 3 hold for row r, for every lane of it.
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&all)[4]) {
  const auto x = __builtin_amdgcn_permlane16_swap(w, w, false, false);  // groups 0 0 2 2, 1 1 3 3
  const auto a = __builtin_amdgcn_permlane32_swap(x[0], x[0], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(x[1], x[1], false, false);
  all[0] = a[0];
  all[2] = a[1];
  all[1] = b[0];
  all[3] = b[1];
}

template <int SM, int W>
__global__ __launch_bounds__(64 * W, 1) void gemm_mxfp4_few_kernel(Mxfp4GemmParams p) {
  constexpr int P = SM == 4 ? 4 : 8;
  static_assert(SM <= W, "a wave adds up a row of subtiles");
  __shared__ v4f red[W][SM][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, h = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * 16;
  const int all = static_cast<int>(p.K / 128), beg = static_cast<int>(int64_t(all) * wave / W), end = static_cast<int>(int64_t(all) * (wave + 1) / W);
  const uint8_t* const b = p.b + min(n0 + r, p.N - 1) * p.ldb + 16 * h;
  const uint8_t* const sb = p.sb + min(n0 + r, p.N - 1) * p.sb_sn * 4;
  const uint8_t* a[SM];
  const uint8_t* sa[SM];
#pragma unroll
  for (int i = 0; i < SM; i++) {
    const int64_t m = min(int64_t(16 * i + r), p.M - 1);
    a[i] = p.a + m * p.lda + 16 * h;
    sa[i] = p.sa + m * p.sa_sm * 4;
  }
  v4f acc[SM];
#pragma unroll
  for (int i = 0; i < SM; i++) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  // units k .. k + U - 1 (a multiple of four); where they may pass the range's end, its last one again, which is not used
  auto step = [&](auto count, auto past, int k) {
    constexpr int U = decltype(count)::value;
    constexpr bool kPast = decltype(past)::value;
    u32x4 fb[U], fa[U][SM];
    uint32_t wb[U / 4], wa[U / 4][SM];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t at = int64_t(kPast ? min(k + u, end - 1) : k + u) * kUnit;
      fb[u] = *reinterpret_cast<const u32x4*>(b + at);
#pragma unroll
      for (int i = 0; i < SM; i++) fa[u][i] = *reinterpret_cast<const u32x4*>(a[i] + at);
    }
#pragma unroll
    for (int g = 0; g < U / 4; g++) {
      const int64_t at = kPast ? min(k + 4 * g + h, end - 1) : k + 4 * g + h;
      wb[g] = *reinterpret_cast<const uint32_t*>(sb + at * p.sb_sk * 4);
#pragma unroll
      for (int i = 0; i < SM; i++) wa[g][i] = *reinterpret_cast<const uint32_t*>(sa[i] + at * p.sa_sk * 4);
    }
#pragma unroll
    for (int g = 0; g < U / 4; g++) {
      uint32_t eb[4], ea[SM][4];
      spread(wb[g], eb);
#pragma unroll
      for (int i = 0; i < SM; i++) spread(wa[g][i], ea[i]);
#pragma unroll
      for (int u = 0; u < 4; u++) {
        if (!kPast || k + 4 * g + u < end) {
#pragma unroll
          for (int i = 0; i < SM; i++)
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(fb[4 * g + u]), operand(fa[4 * g + u][i]), acc[i], kFp4, kFp4, 0,
                                                                      static_cast<int>(eb[u] >> (8 * h)), 0,
                                                                      static_cast<int>(ea[i][u] >> (8 * h)));
        }
      }
    }
  };
  int k = beg;
  for (; k + P <= end; k += P) step(std::integral_constant<int, P>{}, std::false_type{}, k);
  if (end - k > 4) step(std::integral_constant<int, P>{}, std::true_type{}, k);
  else if (k < end) step(std::integral_constant<int, 4>{}, std::true_type{}, k);
#pragma unroll
  for (int i = 0; i < SM; i++) red[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave >= SM) return;
  v4f sum = red[0][wave][lane];
#pragma unroll
  for (int w = 1; w < W; w++) {
    const v4f o = red[w][wave][lane];
#pragma unroll
    for (int q = 0; q < 4; q++) sum[q] += o[q];
  }
  const int64_t m = 16 * wave + r, n = n0 + 4 * h;
  if (m >= p.M) return;
  uint16_t* y = p.y + m * p.ldy + n;
  const u32x2 w = {bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3])};
  if (n + 4 <= p.N) {
    *reinterpret_cast<u32x2_any*>(y) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 3; q++)
      if (n + q < p.N) y[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
  }
}

// ------------------------------------------------------------------ launch
template <class C>
void launch(const Mxfp4GemmParams& p, const DeviceShape& ds, hipStream_t stream) {
  const int64_t units = mxfp4_tiles(p.M, p.N, C::BM, C::BN) * p.splits;
  int64_t grid = std::min<int64_t>(units, int64_t(ds.cus) * C::kBlocks);
  grid = std::max<int64_t>((grid + ds.xcds - 1) / ds.xcds * ds.xcds, ds.xcds);
  hipLaunchKernelGGL((gemm_mxfp4_kernel<C>), dim3(static_cast<unsigned>(grid)), dim3(C::kThreads), 0, stream, p);
}

template <int W>
void launch_few(const Mxfp4GemmParams& p, int64_t blocks, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * W);
  if (p.M <= 16) hipLaunchKernelGGL((gemm_mxfp4_few_kernel<1, W>), grid, block, 0, stream, p);
  else if (p.M <= 32) hipLaunchKernelGGL((gemm_mxfp4_few_kernel<2, W>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((gemm_mxfp4_few_kernel<4, W>), grid, block, 0, stream, p);
}

int finish() {
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("mxfp4 product launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace

int64_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) { return mxfp4_shape(M, N, K, current_device_shape().cus).ws; }

int launch_mxfp4_gemm(const Mxfp4GemmParams& p_in, hipStream_t stream) {
  const DeviceShape ds = current_device_shape();
  Mxfp4GemmParams p = p_in;
  p.xcds = ds.xcds;
  Mxfp4Shape s = mxfp4_shape(p.M, p.N, p.K, ds.cus);
  if (s.ws > 0 && (p.ws == nullptr || p.ws_bytes < s.ws)) s.splits = 1;
  p.splits = s.splits;
  switch (s.kind) {
    case Mxfp4Kind::kFew: {
      const int64_t blocks = (p.N + 15) / 16;
      blocks > ds.cus ? launch_few<4>(p, blocks, stream) : launch_few<8>(p, blocks, stream);
      break;
    }
    case Mxfp4Kind::kLarge: launch<Large>(p, ds, stream); break;
    case Mxfp4Kind::kDeep: p.splits > 1 ? launch<Splitting<Deep>>(p, ds, stream) : launch<Deep>(p, ds, stream); break;
    case Mxfp4Kind::kFlat: p.splits > 1 ? launch<Splitting<Flat>>(p, ds, stream) : launch<Flat>(p, ds, stream); break;
  }
  if (p.splits > 1) {
    const int64_t quads = p.M * ((p.N + 3) / 4);
    hipLaunchKernelGGL(gemm_mxfp4_join_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((quads + 255) / 256, 4096))), dim3(256), 0, stream, p);
  }
  return finish();
}

int launch_mxfp4_zero(const Mxfp4GemmParams& p, hipStream_t stream) {
  const int64_t blocks = std::min<int64_t>((p.M * p.N + 255) / 256, 4096);
  hipLaunchKernelGGL(gemm_mxfp4_zero_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p.y, p.M, p.N, p.ldy);
  return finish();
}

}  // namespace fp8q
