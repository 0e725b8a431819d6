// gemm_mxfp4.hip — Y = A B^T of two matrices of e2m1 codes with one UE8M0 scale per 32 elements of a row
// (MXFP4), rounded to bf16 once:
//   Y[m][n] = bf16( sum_k 2^(ea(m, k/32) - 127) A[m][k] * 2^(eb(n, k/32) - 127) B[n][k] )
#include <algorithm>

#include "mxfp4.h"

namespace fp8q {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;     // operand format of the matrix instruction
constexpr int kStepK = 256;  // elements of K per step
constexpr int kRowBytes = kStepK / 2;

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, int BLOCKS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
  static constexpr int kBlocks = BLOCKS_;  // of a CU
  static constexpr int kWaves = WAVES_M * WAVES_N, kThreads = 64 * kWaves;
  static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N, SM = WTM / 32, SN = WTN / 32;
  // one stage: rows of A and B, then their scale words [2][BM], [2][BN]
  static constexpr int kB = BM * kRowBytes, kSA = kB + BN * kRowBytes, kSB = kSA + 8 * BM, kStage = kSB + 8 * BN;
  static constexpr int kLds = STAGES * kStage;
  // loads of a wave and step: 1 KB pieces of 8 rows, and 64 scale words each
  static constexpr int kLA = BM / 8 / kWaves, kLB = BN / 8 / kWaves, kLS = (BM + BN) / 32 / kWaves;
  static constexpr int kLoads = kLA + kLB + kLS;
  static_assert(kLA * kWaves * 8 == BM && kLB * kWaves * 8 == BN && kLS * kWaves * 32 == BM + BN && kLS % 2 == 0 && kLA % 2 == 0 && kLB % 2 == 0, "load split");
  static_assert(kBlocks * kLds <= 160 * 1024, "LDS");
};

typedef __attribute__((address_space(3))) uint8_t lds_u8;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8*)p));
}
typedef int v4i __attribute__((ext_vector_type(4)));
// lane l: LDS [lds + 16 l, + 16) <- buffer [voff + soff, + 16)
__device__ __forceinline__ void dma16(uint32_t lds, v4i buffer, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff), "s"(buffer), "s"(soff) : "memory");
}
// lane l: LDS [lds + 4 l, + 4) <- global [base + voff, + 4)
__device__ __forceinline__ void dma4(uint32_t lds, const uint8_t* base, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory");
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

__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

constexpr int kGroupM = 4;

struct Place {
  int64_t m0, n0;
};
// The host makes sure that there are fewer than 2^31 tiles.
template <class C>
__device__ __forceinline__ Place place_of(const Mxfp4GemmParams& p, int32_t t) {
  const int32_t tiles_m = static_cast<int32_t>((p.M + C::BM - 1) / C::BM), tiles_n = static_cast<int32_t>((p.N + C::BN - 1) / C::BN);
  const int32_t group = t / tiles_n / kGroupM;  // of kGroupM rows of tiles
  const int32_t first = group * kGroupM, rows = min(tiles_m - first, kGroupM), at = t - first * tiles_n;
  const int32_t n = at / rows;
  return Place{int64_t(first + at - n * rows) * C::BM, int64_t(n) * C::BN};
}

// Rows of an operand from `base` on as a buffer: what lies past the last row's end is not read.
__device__ __forceinline__ v4i rows_buffer(const uint8_t* base, int64_t rows, int64_t ld, int64_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  const uint32_t size = static_cast<uint32_t>(min((rows - 1) * ld + bytes, int64_t(0xFFFFFFFF)));
  return v4i{__builtin_amdgcn_readfirstlane(static_cast<int32_t>(at)), __builtin_amdgcn_readfirstlane(static_cast<int32_t>(at >> 32)),
             __builtin_amdgcn_readfirstlane(static_cast<int32_t>(size)), 0x00020000};
}

// The loads of a block's steps, one after the other through its tiles; past the last step the last one again, so that
// every step issues the same loads. Rows past an operand's end bring anything: their products are not stored. The
// last step of an odd number of K halves brings bytes of the next row (or nothing), which are not used.
template <class C>
struct Loader {
  static constexpr int kGroups = (C::BM + C::BN) / 64, kPer = kGroups / C::kWaves;  // of 64 scale rows
  const Mxfp4GemmParams& p;
  const TileSpan span;
  const uint32_t lds;
  const int lane, wave, steps;
  const uint32_t lda8, ldb8;  // bytes of 8 rows
  int32_t tile;
  int step;
  uint32_t stage;             // its offset
  v4i a, b;
  uint32_t a_off[2], b_off[2];  // the lane's part: pieces of 8 rows, even and odd ones
  const uint8_t* s_base[kPer];  // scale words of the lanes' rows at this step
  uint32_t s_off[kPer];

  __device__ __forceinline__ Loader(const Mxfp4GemmParams& params, const TileSpan& s, uint32_t lds_at, int lane_, int wave_, int n)
      : p(params), span(s), lds(lds_at), lane(lane_), wave(wave_), steps(n), lda8(static_cast<uint32_t>(8 * params.lda)),
        ldb8(static_cast<uint32_t>(8 * params.ldb)), tile(static_cast<int32_t>(s.beg)), step(0), stage(0) {
    const int sub = lane >> 3;
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const uint32_t chunk = 16 * ((lane & 7) ^ swizzle(8 * q + sub));
      a_off[q] = static_cast<uint32_t>(sub * p.lda) + chunk;
      b_off[q] = static_cast<uint32_t>(sub * p.ldb) + chunk;
    }
    enter();
  }
  // Of scale group q of this wave: whether it is A's, and its first row.
  __device__ __forceinline__ bool of_a(int q) const { return q * C::kWaves + wave < C::BM / 64; }
  __device__ __forceinline__ int first(int q) const { return (q * C::kWaves + wave - (of_a(q) ? 0 : C::BM / 64)) * 64; }
  __device__ __forceinline__ void enter() {
    const Place at = place_of<C>(p, tile);
    a = rows_buffer(p.a + at.m0 * p.lda, p.M - at.m0, p.lda, p.K / 2);
    b = rows_buffer(p.b + at.n0 * p.ldb, p.N - at.n0, p.ldb, p.K / 2);
#pragma unroll
    for (int q = 0; q < kPer; q++) {
      const int64_t sm = of_a(q) ? p.sa_sm : p.sb_sn, rows = of_a(q) ? p.M - 1 - at.m0 : p.N - 1 - at.n0;
      s_base[q] = of_a(q) ? p.sa + at.m0 * sm * 4 : p.sb + at.n0 * sm * 4;
      s_off[q] = static_cast<uint32_t>(min(int64_t(first(q) + lane), rows) * sm * 4);
    }
  }
  __device__ __forceinline__ void issue_a() {
    const uint32_t at = lds + stage + wave * (C::kLA * 1024), from = wave * C::kLA * lda8 + step * kRowBytes;
#pragma unroll
    for (int q = 0; q < C::kLA; q++) dma16(at + q * 1024, a, a_off[q & 1], from + q * lda8);
    const bool more = 2 * step + 1 < p.K / 128;
#pragma unroll
    for (int q = 0; q < kPer; q++) {
      const int64_t sk = of_a(q) ? p.sa_sk : p.sb_sk;
      const uint32_t to = lds + stage + (of_a(q) ? C::kSA : C::kSB) + 4 * first(q);
      dma4(to, s_base[q], s_off[q]);
      dma4(to + 4 * (of_a(q) ? C::BM : C::BN), s_base[q] + (more ? 4 * sk : 0), s_off[q]);
    }
  }
  __device__ __forceinline__ void issue_b() {
    const uint32_t at = lds + stage + C::kB + wave * (C::kLB * 1024), from = wave * C::kLB * ldb8 + step * kRowBytes;
#pragma unroll
    for (int q = 0; q < C::kLB; q++) dma16(at + q * 1024, b, b_off[q & 1], from + q * ldb8);
    stage = stage + C::kStage == C::kLds ? 0 : stage + C::kStage;
    if (step + 1 < steps) {
      step++;
#pragma unroll
      for (int q = 0; q < kPer; q++) s_base[q] += 8 * (of_a(q) ? p.sa_sk : p.sb_sk);
    } else if (tile + span.stride < span.end) {
      tile += static_cast<int32_t>(span.stride);
      step = 0;
      enter();
    }
  }
};

template <class C>
struct Compute {
  const uint8_t* smem;
  uint32_t a_at[4], b_at[4];  // LDS offsets of the lane's first subtile for each quarter of a step
  uint32_t sa_at, sb_at, select;
  u32x4 fa[2][C::SM], fb[2][C::SN];
  uint32_t wa[2][C::SM], wb[2][C::SN];  // scale words of the next step
  uint32_t ea[C::SM], eb[C::SN];        // scale bytes of this step's quarters
  v16f acc[C::SM][C::SN];

  __device__ __forceinline__ Compute(const uint8_t* s, int lane, int wm, int wn) : smem(s) {
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int chunk = 16 * ((2 * k + h) ^ swizzle(r));
      a_at[k] = (wm * C::WTM + r) * kRowBytes + chunk;
      b_at[k] = C::kB + (wn * C::WTN + r) * kRowBytes + chunk;
    }
    sa_at = C::kSA + 4 * (wm * C::WTM + r);
    sb_at = C::kSB + 4 * (wn * C::WTN + r);
    select = h ? 0x07050301u : 0x06040200u;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < C::SM; i++)
#pragma unroll
      for (int j = 0; j < C::SN; j++) acc[i][j] = v16f{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  }
  // Read number n of quarter K of the stage at offset `st`: operands of A and B, then (K = 0) the scale words.
  template <int K>
  __device__ __forceinline__ void read(int n, uint32_t st) {
    if (n < C::SM) {
      fa[K & 1][n] = *reinterpret_cast<const u32x4*>(smem + st + a_at[K] + n * 32 * kRowBytes);
    } else if (n < C::SM + C::SN) {
      fb[K & 1][n - C::SM] = *reinterpret_cast<const u32x4*>(smem + st + b_at[K] + (n - C::SM) * 32 * kRowBytes);
    } else if (K == 0 && n < 3 * C::SM + C::SN) {
      const int i = n - C::SM - C::SN;
      wa[i & 1][i >> 1] = *reinterpret_cast<const uint32_t*>(smem + st + sa_at + 4 * (i & 1) * C::BM + 128 * (i >> 1));
    } else if (K == 0 && n < 3 * (C::SM + C::SN)) {
      const int i = n - 3 * C::SM - C::SN;
      wb[i & 1][i >> 1] = *reinterpret_cast<const uint32_t*>(smem + st + sb_at + 4 * (i & 1) * C::BN + 128 * (i >> 1));
    }
  }
  static constexpr int kReads = C::SM + C::SN, kReads0 = 3 * kReads;

  __device__ __forceinline__ void scales() {
#pragma unroll
    for (int i = 0; i < C::SM; i++) ea[i] = __builtin_amdgcn_perm(wa[1][i], wa[0][i], select);
#pragma unroll
    for (int j = 0; j < C::SN; j++) eb[j] = __builtin_amdgcn_perm(wb[1][j], wb[0][j], select);
  }

  // The products of quarter K, between them the reads of quarter NEXT from the stage at `st`.
  template <int K, int NEXT>
  __device__ __forceinline__ void quarter(uint32_t st) {
    constexpr int kMma = C::SM * C::SN, kN = NEXT == 0 ? kReads0 : kReads;
    int done = 0;
#pragma unroll
    for (int t = 0; t < kMma; t++) {
      const int i = t / C::SN, j = t % C::SN;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[K & 1][j]), operand(fa[K & 1][i]), acc[i][j], kFp4, kFp4, K,
                                                                  static_cast<int>(eb[j]), K, static_cast<int>(ea[i]));
#pragma unroll
      for (; done < (t + 1) * kN / kMma; done++) read<NEXT>(done, st);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// Lanes of the lower half store the 8 columns of an even group of the result's rows, those of the upper half of the odd
// one after it.
template <class C>
__device__ __forceinline__ void store_tile(const Mxfp4GemmParams& p, const Place& at, const Compute<C>& c, int lane, int wm, int wn) {
  const int r = lane & 31, h = lane >> 5;
  const bool wide = p.ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
  const int64_t first = at.m0 + wm * C::WTM;
  const int rows = static_cast<int>(min(p.M - first, int64_t(C::WTM))) - r;
  const int64_t n0 = at.n0 + wn * C::WTN;
  const int cols = static_cast<int>(min(p.N - n0, int64_t(C::WTN))) - 8 * h;
  uint16_t* row = p.y + (first + r) * p.ldy + n0 + 8 * h;
#pragma unroll
  for (int i = 0; i < C::SM; i++) {
    if (32 * i < rows) {
#pragma unroll
      for (int j = 0; j < C::SN; j++) {
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
          const v16f& v = c.acc[i][j];
          uint32_t x[2], y[2];
#pragma unroll
          for (int q = 0; q < 2; q++) {
            x[q] = bf16_pair(v[4 * g + 2 * q], v[4 * g + 2 * q + 1]);
            y[q] = bf16_pair(v[4 * g + 4 + 2 * q], v[4 * g + 4 + 2 * q + 1]);
          }
          const auto s0 = __builtin_amdgcn_permlane32_swap(x[0], y[0], false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(x[1], y[1], false, false);
          const u32x4 w = {s0[0], s1[0], s0[1], s1[1]};
          const int n = 32 * j + 8 * g;
          if (wide && n + 8 <= cols) {
            *reinterpret_cast<u32x4*>(row + n) = w;
          } else {
#pragma unroll
            for (int q = 0; q < 8; q++)
              if (n + q < cols) row[n + q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    row += 32 * p.ldy;
  }
}

template <class C>
__global__ __launch_bounds__(C::kThreads, C::kBlocks) void gemm_mxfp4_kernel(Mxfp4GemmParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % C::WAVES_M, wn = wave / C::WAVES_M;
  const int64_t tiles = ((p.M + C::BM - 1) / C::BM) * ((p.N + C::BN - 1) / C::BN);
  const TileSpan span = tile_span(tiles, blockIdx.x, gridDim.x, p.xcds);
  if (span.beg >= span.end) return;
  const int steps = static_cast<int>((p.K + kStepK - 1) / kStepK);
  const bool odd = (p.K & 128) != 0;
  Loader<C> load(p, span, lds_addr(smem), lane, wave, steps);
  Compute<C> c(smem, lane, wm, wn);
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; s++) {
    load.issue_a();
    load.issue_b();
  }
  load.issue_a();
  wait_vmcnt<(C::STAGES - 2) * C::kLoads + C::kLA + C::kLS>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int n = 0; n < Compute<C>::kReads0; n++) c.template read<0>(n, 0);
  uint32_t st = 0;
  for (int64_t t = span.beg; t < span.end; t += span.stride) {
    c.clear();
    bool fresh = true;  // stores may be under way
    // what ends a step: its loads have landed, everyone has read its stage, which is filled anew
    auto turn = [&]() {
      if (fresh) wait_vmcnt<0>();
      else wait_vmcnt<(C::STAGES - 2) * C::kLoads>();
      fresh = false;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      load.issue_a();
      st = st + C::kStage == C::kLds ? 0 : st + C::kStage;
    };
    const int whole = odd ? steps - 1 : steps;
    for (int s = 0; s < whole; s++) {
      c.scales();
      load.issue_b();
      c.template quarter<0, 1>(st);
      c.template quarter<1, 2>(st);
      c.template quarter<2, 3>(st);
      turn();
      c.template quarter<3, 0>(st);
    }
    if (odd) {
      c.scales();
      load.issue_b();
      c.template quarter<0, 1>(st);
      turn();
      c.template quarter<1, 0>(st);
    }
    store_tile<C>(p, place_of<C>(p, static_cast<int32_t>(t)), c, lane, wm, wn);
  }
  wait_vmcnt<0>();  // nothing is under way into LDS when the block ends
}

using Large = Tile<256, 256, 2, 2, 2, 1>;
using Medium = Tile<128, 128, 2, 2, 2, 2>;

template <class C>
void launch(const Mxfp4GemmParams& p, const DeviceShape& ds, hipStream_t stream) {
  const int64_t tiles = ((p.M + C::BM - 1) / C::BM) * ((p.N + C::BN - 1) / C::BN);
  int64_t grid = std::min<int64_t>(tiles, int64_t(ds.cus) * C::kBlocks);
  grid = std::max<int64_t>((grid + ds.xcds - 1) / ds.xcds * ds.xcds, ds.xcds);
  hipLaunchKernelGGL((gemm_mxfp4_kernel<C>), dim3(static_cast<unsigned>(grid)), dim3(C::kThreads), 0, stream, p);
}

}  // namespace

int64_t mxfp4_gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

int launch_mxfp4_gemm(const Mxfp4GemmParams& p_in, hipStream_t stream) {
  const DeviceShape ds = current_device_shape();
  Mxfp4GemmParams p = p_in;
  p.xcds = ds.xcds;
  const int64_t large = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  if (large >= ds.cus) launch<Large>(p, ds, stream);
  else launch<Medium>(p, ds, stream);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("mxfp4 product launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace fp8q
