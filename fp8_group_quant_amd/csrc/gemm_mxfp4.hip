// gemm_mxfp4.hip — Y = A B^T of two matrices of e2m1 codes with one UE8M0 scale per 32 elements of a row
// (MXFP4), rounded to bf16 once:
//   Y[m][n] = bf16( sum_k 2^(ea(m, k/32) - 127) A[m][k] * 2^(eb(n, k/32) - 127) B[n][k] )
#include <algorithm>

#include "mxfp4.h"

namespace fp8q {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;     // operand format of the matrix instruction
constexpr int kStepK = 128;  // elements of K per step
constexpr int kRowBytes = kStepK / 2;

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, int BLOCKS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, STAGES = STAGES_;
  static constexpr int kBlocks = BLOCKS_;  // of a CU
  static constexpr int kWaves = WAVES_M * WAVES_N, kThreads = 64 * kWaves;
  static constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N, SM = WTM / 32, SN = WTN / 32;
  // one stage: rows of A and B, then their scale words
  static constexpr int kB = BM * kRowBytes, kSA = kB + BN * kRowBytes, kSB = kSA + 4 * BM, kStage = kSB + 4 * BN;
  static constexpr int kLds = STAGES * kStage;
  // loads of a wave and step: 1 KB pieces of 8 rows, and 64 scale words each
  static constexpr int kLA = BM / 16 / kWaves, kLB = BN / 16 / kWaves, kLS = (BM + BN) / 64 / kWaves;
  static constexpr int kLoads = kLA + kLB + kLS, kMma = SM * SN, kFirst = kLoads / 2;
  static_assert(kLA * kWaves * 16 == BM && kLB * kWaves * 16 == BN && kLS * kWaves * 64 == BM + BN, "load split");
  static_assert(kBlocks * (kLds + kWaves * 32 * 144) <= 160 * 1024, "LDS");
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

__device__ __forceinline__ int swizzle(int row) { return (row >> 2) & 3; }

constexpr int kGroupM = 4;

// The kernel's arguments, read again where they are used, so that they hold no registers in the loop.
typedef const __attribute__((address_space(4))) Mxfp4GemmParams* Args;
__device__ __forceinline__ Args arguments() {
  Args a = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}

struct Place {
  int64_t m0, n0;
};
// The host makes sure that there are fewer than 2^31 tiles.
template <class C>
__device__ __forceinline__ Place place_of(Args p, int32_t t) {
  const int32_t tiles_m = static_cast<int32_t>((p->M + C::BM - 1) / C::BM), tiles_n = static_cast<int32_t>((p->N + C::BN - 1) / C::BN);
  const int32_t group = t / tiles_n / kGroupM;  // of kGroupM rows of tiles
  const int32_t first = group * kGroupM, rows = min(tiles_m - first, kGroupM), at = t - first * tiles_n;
  const int32_t n = at / rows;
  return Place{int64_t(first + at - n * rows) * C::BM, int64_t(n) * C::BN};
}

// What a block's loads of one tile start from: the operands' rows as buffers (what lies past the last row's end is not
// read), and the scale words of the lanes' rows.
template <class C>
struct Source {
  static constexpr int kPer = (C::BM + C::BN) / 64 / C::kWaves;  // groups of 64 scale rows per wave
  v4i a, b;
  const uint8_t* s_base[kPer];
  uint32_t s_off[kPer];

  // Of scale group q of a wave: whether it is A's, and its first row.
  static __device__ __forceinline__ bool of_a(int q, int wave) { return q * C::kWaves + wave < C::BM / 64; }
  static __device__ __forceinline__ int first(int q, int wave) { return (q * C::kWaves + wave - (of_a(q, wave) ? 0 : C::BM / 64)) * 64; }
  static __device__ __forceinline__ v4i buffer(const uint8_t* base, int64_t rows, int64_t ld, int64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    const uint32_t size = static_cast<uint32_t>(min((rows - 1) * ld + bytes, int64_t(0xFFFFFFFF)));
    return v4i{static_cast<int32_t>(at), static_cast<int32_t>(at >> 32), static_cast<int32_t>(size), 0x00020000};
  }
  __device__ __forceinline__ void enter(int32_t tile, int lane, int wave) {
    const Args p = arguments();
    const Place at = place_of<C>(p, tile);
    a = buffer(p->a + at.m0 * p->lda, p->M - at.m0, p->lda, p->K / 2);
    b = buffer(p->b + at.n0 * p->ldb, p->N - at.n0, p->ldb, p->K / 2);
#pragma unroll
    for (int q = 0; q < kPer; q++) {
      const bool is_a = of_a(q, wave);
      const int64_t sm = is_a ? p->sa_sm : p->sb_sn, rows = is_a ? p->M - 1 - at.m0 : p->N - 1 - at.n0;
      s_base[q] = is_a ? p->sa + at.m0 * sm * 4 : p->sb + at.n0 * sm * 4;
      s_off[q] = static_cast<uint32_t>(min(int64_t(first(q, wave) + lane), rows) * sm * 4);
    }
  }
};

// The loads of a block's steps, one after the other through its tiles; past the last tile its steps again, so that every
// step issues the same loads. Rows past an operand's end bring anything: their products are not stored. The
// last step of an odd number of K halves brings bytes of the next row (or nothing), which are not used.
template <class C>
struct Loader {
  static constexpr int kPer = Source<C>::kPer;
  const uint32_t lds;
  const int lane, wave, steps;
  const int32_t stride, stop;   // of the tiles
  const uint32_t lda16, ldb16;    // bytes of 8 rows
  uint32_t a_off, b_off;  // the lane's part: pieces of 8 rows, even and odd ones
  int64_t s_step[kPer];         // bytes between the words of two K halves
  const bool odd;
  int32_t tile;
  int step;
  uint32_t stage;  // its offset
  Source<C> now, next;

  __device__ __forceinline__ Loader(const TileSpan& s, uint32_t lds_at, int lane_, int wave_, int n, bool odd_)
      : lds(lds_at), lane(lane_), wave(wave_), steps(n), stride(static_cast<int32_t>(s.stride)), stop(static_cast<int32_t>(s.end)),
        lda16(static_cast<uint32_t>(16 * arguments()->lda)), ldb16(static_cast<uint32_t>(16 * arguments()->ldb)), odd(odd_),
        tile(static_cast<int32_t>(s.beg)), step(0), stage(0) {
    const int row = lane >> 2;
    const uint32_t chunk = 16 * ((lane & 3) ^ swizzle(row));
    a_off = row * (lda16 >> 4) + chunk;
    b_off = row * (ldb16 >> 4) + chunk;
#pragma unroll
    for (int q = 0; q < kPer; q++) s_step[q] = 4 * (Source<C>::of_a(q, wave) ? arguments()->sa_sk : arguments()->sb_sk);
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
      dma16(at + (wave * C::kLA + n) * 1024, now.a, a_off, (wave * C::kLA + n) * lda16 + step * kRowBytes);
    } else if (n < C::kLA + C::kLB) {
      const int q = n - C::kLA;
      dma16(at + C::kB + (wave * C::kLB + q) * 1024, now.b, b_off, (wave * C::kLB + q) * ldb16 + step * kRowBytes);
    } else {
      const int q = n - C::kLA - C::kLB;
      const bool is_a = Source<C>::of_a(q, wave);
      dma4(at + (is_a ? C::kSA : C::kSB) + 4 * Source<C>::first(q, wave), now.s_base[q], now.s_off[q]);
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
    for (int q = 0; q < kPer; q++) {
      now.s_base[q] = last ? next.s_base[q] : now.s_base[q] + s_step[q];
      now.s_off[q] = last ? next.s_off[q] : now.s_off[q];
    }
  }
  __device__ __forceinline__ void issue_all() {
#pragma unroll
    for (int n = 0; n < C::kLoads; n++) issue(n);
    advance();
  }
};

template <class C>
struct Compute {
  const uint8_t* smem;
  uint32_t a_at[2], b_at[2];  // LDS offsets of the lane's first subtile for each half of a step
  uint32_t sa_at, sb_at, shift;
  u32x4 fa[2][C::SM], fb[2][C::SN];
  uint32_t wa[C::SM], wb[C::SN];  // scale words of the next step
  uint32_t ea[C::SM], eb[C::SN];  // of this one: its halves' bytes are 0 and 2
  v16f acc[C::SM][C::SN];

  __device__ __forceinline__ Compute(const uint8_t* s, int lane, int wm, int wn) : smem(s) {
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int chunk = 16 * ((2 * k + h) ^ swizzle(r));
      a_at[k] = (wm * C::WTM + r) * kRowBytes + chunk;
      b_at[k] = C::kB + (wn * C::WTN + r) * kRowBytes + chunk;
    }
    sa_at = C::kSA + 4 * (wm * C::WTM + r);
    sb_at = C::kSB + 4 * (wn * C::WTN + r);
    shift = 8 * h;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < C::SM; i++)
#pragma unroll
      for (int j = 0; j < C::SN; j++) acc[i][j] = v16f{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  }
  // Read number n of half K of the stage at offset `st`: operands of A and B, then (K = 0) the scale words.
  template <int K>
  __device__ __forceinline__ void read(int n, uint32_t st) {
    if (n < C::SM) {
      fa[K][n] = *reinterpret_cast<const u32x4*>(smem + st + a_at[K] + n * 32 * kRowBytes);
    } else if (n < C::SM + C::SN) {
      fb[K][n - C::SM] = *reinterpret_cast<const u32x4*>(smem + st + b_at[K] + (n - C::SM) * 32 * kRowBytes);
    } else if (K == 0 && n < 2 * C::SM + C::SN) {
      wa[n - C::SM - C::SN] = *reinterpret_cast<const uint32_t*>(smem + st + sa_at + 128 * (n - C::SM - C::SN));
    } else if (K == 0 && n < 2 * (C::SM + C::SN)) {
      wb[n - 2 * C::SM - C::SN] = *reinterpret_cast<const uint32_t*>(smem + st + sb_at + 128 * (n - 2 * C::SM - C::SN));
    }
  }
  static constexpr int kReads = C::SM + C::SN, kReads0 = 2 * kReads;

  __device__ __forceinline__ void scales() {
#pragma unroll
    for (int i = 0; i < C::SM; i++) ea[i] = wa[i] >> shift;
#pragma unroll
    for (int j = 0; j < C::SN; j++) eb[j] = wb[j] >> shift;
  }

  // The products of half K, between them the reads of half NEXT from the stage at `st`.
  template <int K, int NEXT, class F>
  __device__ __forceinline__ void half(uint32_t st, F extra) {
    constexpr int kMma = C::SM * C::SN, kN = NEXT == 0 ? kReads0 : kReads;
    int done = 0;
#pragma unroll
    for (int t = 0; t < kMma; t++) {
      const int i = t / C::SN, j = t % C::SN;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[K][j]), operand(fa[K][i]), acc[i][j], kFp4, kFp4, 2 * K,
                                                                  static_cast<int>(eb[j]), 2 * K, static_cast<int>(ea[i]));
#pragma unroll
      for (; done < (t + 1) * kN / kMma; done++) read<NEXT>(done, st);
      extra(t);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The wave's outputs, 32 rows x 64 columns at a time through LDS, so that every store writes whole lines (a lane has 4
// columns of its row in each group of 8).
constexpr int kOutRow = 128 + 16;       // LDS bytes of a row of 64 columns
constexpr int kOutWave = 32 * kOutRow;  // of a wave

template <class C>
__device__ __forceinline__ void store_tile(uint8_t* lds, int32_t tile, const Compute<C>& c, int lane, int wm, int wn) {
  const Args p = arguments();
  const Place at = place_of<C>(p, tile);
  const int64_t m0 = at.m0 + wm * C::WTM, n0 = at.n0 + wn * C::WTN, ldy = p->ldy;
  uint8_t* const put = lds + (lane & 31) * kOutRow + 8 * (lane >> 5);
  const uint8_t* const get = lds + (lane >> 3) * kOutRow + 16 * (lane & 7);
  uint16_t* row = p->y + (m0 + (lane >> 3)) * ldy + n0 + 8 * (lane & 7);
  const bool whole = m0 + C::WTM <= p->M && n0 + C::WTN <= p->N && ldy % 8 == 0 && (reinterpret_cast<uintptr_t>(p->y) & 15) == 0;
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
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      u32x4 w[4];
#pragma unroll
      for (int k = 0; k < 4; k++) w[k] = *reinterpret_cast<const u32x4*>(get + 8 * k * kOutRow);
      if (whole) {
#pragma unroll
        for (int k = 0; k < 4; k++) *reinterpret_cast<u32x4*>(row + 8 * k * ldy + 32 * j) = w[k];
      } else {
        const int left = cols - 32 * j;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          if (32 * i + 8 * k < rows) {
#pragma unroll
            for (int q = 0; q < 8; q++)
              if (q < left) row[8 * k * ldy + 32 * j + q] = static_cast<uint16_t>(w[k][q >> 1] >> (16 * (q & 1)));
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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
  const int64_t tiles = ((p.M + C::BM - 1) / C::BM) * ((p.N + C::BN - 1) / C::BN);
  const TileSpan span = tile_span(tiles, blockIdx.x, gridDim.x, p.xcds);
  if (span.beg >= span.end) return;
  const int steps = static_cast<int>((p.K + kStepK - 1) / kStepK);
  const bool odd = (p.K & 128) != 0;
  Loader<C> load(span, lds_addr(smem), lane, wave, steps, odd);
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
    auto loads3 = [&](int n) {
#pragma unroll
      for (int i = n * C::kFirst / C::kMma; i < (n + 1) * C::kFirst / C::kMma; i++) load.issue(i);
    };
    auto loads0 = [&](int n) {
      constexpr int kRest = C::kLoads - C::kFirst;
#pragma unroll
      for (int i = n * kRest / C::kMma; i < (n + 1) * kRest / C::kMma; i++) load.issue(C::kFirst + i);
    };
    for (int s = 0; s < steps; s++) {
      c.scales();
      c.template half<0, 1>(st, loads0);
      load.advance();
      turn();
      c.template half<1, 0>(st, loads3);
    }
    store_tile<C>(smem + C::kLds + wave * kOutWave, t, c, lane, wm, wn);
    load.look_ahead();
  }
  wait_vmcnt<0>();  // nothing is under way into LDS when the block ends
}

using Large = Tile<256, 256, 2, 2, 4, 1>;
using Medium = Tile<128, 128, 2, 2, 3, 2>;

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
