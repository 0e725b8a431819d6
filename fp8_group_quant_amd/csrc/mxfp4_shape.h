// mxfp4_shape.h — which kernel, tile and ranges of K a 4-bit product takes, from its sizes alone.
//
// Plain C++ (no HIP types) so that the host tests can check the choice directly.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace fp8q {

constexpr int kMxfp4MostSplits = 16;  // ranges of K

enum class Mxfp4Kind { kFew, kLarge, kDeep, kFlat };
struct Mxfp4Shape {
  Mxfp4Kind kind;
  int splits;
  int64_t ws;  // bytes
};

inline int64_t mxfp4_tiles(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

// The kernel, tile and ranges of K with the least estimated time: rounds of tiles over the CUs, each its steps of 256
// elements and a part for its outputs, and a part for the call; not less than the bytes take. Splitting adds a launch and
// the partial sums' way to memory and back. us by replayed graphs, calls back to back on quantized normal values, each
// kernel where it was forced (* with K split, where that was the better), the chosen one marked; where two are given, the
// clock that the power allows decides:
//   M x N x K             256 x 256   128 x 128   64 x 128
//   8192 x 8192 x 8192    > 281-312      343         456
//   4096 x 4096 x 7168    >  67           82         111
//   2048 x 8192 x 2048    >  29.8         32.9        41.1
//   2048 x 4096 x 7168       53        >  44          58
//   1024 x 4096 x 7168       45        >  22.7        29.0
//   3000 x 3000 x  512       18.7      >  14.7        16.0
//   1993 x 5920 x  256       18.4      >  14.2        16.8
//    512 x 4096 x 7168       43.9         19.8      > 16.9
//    128 x 4096 x 7168       41.2         17.8 *    > 14.8
//     65 x 4096 x 7168       41.6         15.8 *    > 14.2 *
//    333 x 4104 x 2176       23.8         11.4      >  9.4
//    300 x  300 x 8192       50.2         12.1 *    > 11.8 * (16.7 unsplit)
// Up to 64 rows, without staging and with tiles of 64 x 128: B goes through the registers of every 16 rows, which is
// the shorter way while there are few of them or few rounds.
//   64 x  4096 x 7168   > 11.6   13.8 *      32 x  4096 x 7168   >  8.0   12.7 *
//   64 x  8192 x 8192     23.4 > 18.5        32 x 14336 x 4096     14.6 > 11.6
//   64 x 14336 x 4096     21.6 > 12.0        32 x 28672 x 8192     50.8 > 31-34
//   64 x 28672 x 8192     80.9 > 32-35       16 x 28672 x 8192     37.4 > 30-32
//   64 x  2048 x 4096   >  7.4   10.7        16 x  8192 x 8192   > 11.9   14.5 *
//                                            16 x 14336 x 4096     10.4 > 11.2
inline Mxfp4Shape mxfp4_shape(int64_t M, int64_t N, int64_t K, int cus) {
  struct Model {
    Mxfp4Kind kind;
    int bm, bn;
    double step, round, call;  // us
    bool split;
  };
  const Model models[] = {{Mxfp4Kind::kFew, 64, 16, M <= 16 ? 0.08 + 0.003 * M : M <= 32 ? 0.165 : 0.30, 0.4, 3.4, false},
                          {Mxfp4Kind::kLarge, 256, 256, 1.85, 7.0, 7.0, false},
                          {Mxfp4Kind::kDeep, 128, 128, 0.58, 2.5, 4.0, true},
                          {Mxfp4Kind::kFlat, 64, 128, 0.38, 2.0, 4.0, true}};
  const double steps = static_cast<double>(K) / 256;
  const double least_time = 4.0 + (static_cast<double>(M + N) * K * 17 / 32 + 2.0 * M * N) / 4.5e6;
  const int64_t n4 = (N + 3) / 4 * 4;
  Mxfp4Shape best{Mxfp4Kind::kLarge, 1, 0};
  double least = 1e300;
  for (const Model& m : models) {
    if (m.kind == Mxfp4Kind::kFew && M > m.bm) continue;
    const int64_t tiles = mxfp4_tiles(M, N, m.bm, m.bn);
    const int64_t most = m.split ? std::max<int64_t>(1, std::min<int64_t>({cus / tiles, K / 1024, kMxfp4MostSplits})) : 1;
    for (int64_t s = 1; s <= most; s++) {
      const double rounds = static_cast<double>((tiles * s + cus - 1) / cus), bytes = static_cast<double>(s * M * n4 * 4);
      const double join = s > 1 ? 4.0 + 2 * bytes / 3e6 : 0.0;
      const double time = std::max(m.call + rounds * (steps / s * m.step + m.round) + join, least_time);
      if (time < least || (time == least && m.kind == best.kind)) {  // (of equal ones the most ranges: more CUs load)
        least = time;
        best = {m.kind, static_cast<int>(s), s > 1 ? s * M * n4 * 4 : 0};
      }
    }
  }
  return best;
}

}  // namespace fp8q
