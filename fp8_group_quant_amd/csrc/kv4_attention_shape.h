// kv4_attention_shape.h — how a call of the attention over the 4-bit cache is cut: rows of a tile, units,
// spans and workspace, from sizes alone.
//
// Plain C++ (no HIP types) so that the host tests can check the sizes directly.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "fp8q.h"

namespace fp8q {

// Which tokens up to its limit a row sees: all; the last `window` and the first `sinks`; of the drafted ones those that its
// mask names.
enum Mask { kAll = 0, kWindow = 1, kTree = 2 };

constexpr int kRows = 16;   // query rows of a tile of the kernel for few rows
constexpr int kMinRun = 2;  // spans of a block's run at least
constexpr int kStepW = 64;  // tokens of a step of the kernel for many rows

// Waves per SIMD that the registers are kept to (O^T and Q take D / 4 + D / 8 of them per lane, a
// step's codes N D / 16).
constexpr int waves_per_simd(int64_t D, int DT, int N) {
  if (D == 256 || (D == 128 && N == 4)) return 2;
  return N == 4 || (DT == FP8Q_DTYPE_F16 && D == 128) ? 3 : 4;
}

// Rows of the widest tile whose queries and outputs the registers hold (in fp16, as two parts, all but up
// to 24 of them).
constexpr int widest(int dtype, int64_t D) { return D * (dtype == FP8Q_DTYPE_F16 ? 2 : 1) <= 128 ? 128 : 64; }

constexpr int kMostWideSteps = 32;  // of a unit that the wide kernel does not split

// Query rows of a tile. Up to two tiles of 16 rows per sequence (of mean length) and cached head
// take the kernel whose waves share the tokens; more take the one whose waves share the rows. 16
// sequences of 4096 tokens, 8 cached heads of 128, with 16, 64 and 128 rows to a tile: 32 rows 33,
// 41 and 53 us; 36 rows 47, 41 and 54; 64 rows 50, 45 and 58; 96 rows 76, 73 and 63. The widest
// tile shares each conversion of K and V among the most rows; where caches are short and there is no second
// block for a CU anyway, 64 rows use more CUs and have the shorter steps (512 queries, 4 heads
// to each of 8 cached: over 512 tokens 16.1 us, 20.6 with 128 rows, over 2000 43.2 and 46.3,
// over 4000, split, 74 and 64).
inline int tile_rows(int cus, int dtype, int64_t B, int64_t rows_each, int64_t Hkv, int64_t D, int64_t max_tokens) {
  if (rows_each <= 2 * kRows) return kRows;
  const bool one_each = Hkv * B * ((rows_each + 63) / 64) <= cus;
  return rows_each <= 64 || (one_each && max_tokens <= kMostWideSteps * kStepW) ? 64 : widest(dtype, D);
}

// The narrow kernel's split and general form: 16 N tokens per wave and step (64, but 32 where V's
// rows in LDS and the codes' registers leave no room), in blocks of 4 waves.
constexpr int narrow_halves(int DT, int64_t D) { return D == 256 || (D == 128 && DT == FP8Q_DTYPE_F16) ? 2 : 4; }
constexpr int kNarrowWaves = 4;
constexpr int narrow_blocks(int DT, int64_t D) { return waves_per_simd(D, DT, narrow_halves(DT, D)) * 4 / kNarrowWaves; }

// Blocks for short caches: all the waves that a CU holds, so that a unit needs no second block and
// no join.
constexpr int tall_waves(int DT, int64_t D) { return waves_per_simd(D, DT, 2) * 4; }

// How the narrow kernel's calls are cut: every unit whole, in a block of 4 waves or a tall one, or the
// line split. The split has a plan, pieces in the workspace and a second launch, which cost about 6 us
// more than the others' 5 us, but its time does not depend on how even the lengths are; the others
// take as long as their longest unit, 1.3 us for each of a block's steps (tall: 1.65). So whole units
// have a bounded number of steps (the longest unit then takes about twice the split's fixed time), and
// those of tall blocks, up to one per CU, not more than three times the steps of the split's blocks. us
// for whole, tall and split of B sequences and at most L tokens, 8 cached heads of 128:
//   1 x  500  7.1  8.0 10.4    16 x  700  9.0  9.1 17.0    64 x  300 10.5 15.9 19.6
//   1 x 2000 15   13.6 12.1    16 x 1500 15   12.4 19.2    64 x 1500 20.3 25.3 31.9
//   2 x 4000 25   19.1 11.5    32 x 5000      33   39.6    64 x 3000 38.9 41.7 47
// Trees stay whole for two steps more, up to 1024 tokens of the table's width (heads of 128 in bf16). us whole, tall and split:
//   one of 25 over 1000  13.1 14.3 13.5    4 of 25 over 1000  13.9 15.4 19.1    16 of 4 over 1000  13.6 15.0 17.6
//                  1280  14.6 15.1 15.2                 1250  15.5 16.4 21.2                 1250  15.1 15.9 22.4
//                  1536  16.2 16.4 15.9                 1500  17.3 17.8 21.8                 1500  16.8 17.2 19.9
//                  2000  19.0 18.4 16.5                 2000  20.4 20.0 29.6                 2000  20.7 20.2 21.4
// (five and six steps are within 5 % either way; 8 single tokens with windows of 700 9.7 and 10.0).
enum class Cut { kWhole, kTall, kSplit };
constexpr int kMostSteps = 16, kMostTallSteps = 12;

inline Cut narrow_cut(int cus, int dtype, int64_t D, int64_t units, int64_t max_tokens, int64_t blocks, Mask mask = kAll) {
  const int64_t step = 16 * narrow_halves(dtype, D) * kNarrowWaves, tall_step = 32 * tall_waves(dtype, D);
  const int64_t whole = (max_tokens + step - 1) / step, tall = (max_tokens + tall_step - 1) / tall_step;
  if (whole <= (mask == kTree ? 4 : 2) || units >= 8 * blocks) return Cut::kWhole;
  if (units > cus) return whole <= kMostSteps ? Cut::kWhole : Cut::kSplit;
  return tall <= kMostTallSteps && tall <= 3 * (units * max_tokens / (blocks * step) + 1) ? Cut::kTall : Cut::kSplit;
}

// The wide kernel's calls, by the same weighing: a step of a whole unit takes 1.4 us while its CU has one
// block, the split about 9 steps more than its blocks' own, two of which share a CU. us whole and split,
// 8 cached heads of 128, 4 query heads to each; sequences x queries of tokens:
//   1 x 128 of 512  19.8 24.6    4 x 128 of 300   16.3 35.3    16 x 64 of  512  24.0 48.5
//   1 x 128 of 1000 31.4 27.1    4 x 128 of 1000  33.4 38.4    16 x 64 of 2000  60.3 75.4
//   8 x  17 of 1000 31.0 22.9    4 x 128 of 2000  56.7 46.9    16 x 64 of 8000 194  191
inline Cut wide_cut(int64_t units, int64_t max_tokens, int64_t blocks) {
  const int64_t steps = (max_tokens + kStepW - 1) / kStepW;
  if (units >= blocks) return Cut::kWhole;
  return steps <= kMostWideSteps && steps <= 9 + 2 * units * steps / blocks ? Cut::kWhole : Cut::kSplit;
}

// The sinks' stretch of a window call: steps of 64 tokens (the longest step of any kernel).
inline int64_t sink_stretch(int64_t sinks) { return (sinks + 63) / 64 * 64; }

// The most tokens that a unit of a window call reads: both stretches, the windows of its queries (at most 128)
// reaching one token further for each after the first, and their start rounded down to a step.
inline int64_t window_tokens(int64_t max_tokens, int64_t window, int64_t sinks) {
  return std::min(max_tokens, sink_stretch(sinks) + window + 128 - 1 + 64 - 1);
}

// Tiles of a window or tree call: 16 rows while there are few of them, which then use more of the device than tiles of 64
// (us for 16 and 64 rows, each cut as it is best, 32 heads on 8 cached ones of 128: a tree of 25 over 1000 tokens 13.1 and
// 16.7, of 60 over 4000 24 and 30, 4 trees of 25 over 2000 20 and 28, 256 queries with a window of 512 16.3 and 21.5; 8 trees of
// 60 over 1000, which have 960 tiles of 16 rows, 34 and 30).
inline bool few_narrow_tiles(int cus, int64_t B, int64_t rows_each, int64_t Hkv) {
  return Hkv * B * ((rows_each + kRows - 1) / kRows) <= 2 * static_cast<int64_t>(cus);
}

struct AttnShape {
  int rows;        // of a tile
  bool tall;
  int64_t units;   // at most
  int64_t blocks;  // that a split call's work is cut for: those that run at once
  int span_shift;
  int64_t plan_bytes, bytes;  // workspace; 0: no split
};

// T * Hq < 2^31 and Hkv divides Hq. The units stay below 2^31: a tile has a row of its own, and only the
// last tile of a sequence that has queries is not full. A split call has few of them (its mean-length
// units are fewer than 8 * blocks, the bound at most twice as many), so the line of spans always finds a
// span short enough.
inline AttnShape attention_shape(int cus, int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                 int64_t max_tokens, Mask mask = kAll) {
  AttnShape s;
  // rows and units of sequences of mean length
  const int64_t group = Hq / Hkv, rows_each = (T * group + B - 1) / B;
  s.rows = mask != kAll && few_narrow_tiles(cus, B, rows_each, Hkv) ? kRows : tile_rows(cus, dtype, B, rows_each, Hkv, D, max_tokens);
  const int64_t units = Hkv * B * ((rows_each + s.rows - 1) / s.rows);
  s.units = Hkv * std::min((T * group + s.rows - 1) / s.rows + std::min(B, T), T * group);
  const bool narrow = s.rows == kRows;
  s.blocks = static_cast<int64_t>(cus) * (narrow ? narrow_blocks(dtype, D) : 2);
  // Windows are about equally long, so that nothing is gained by cutting them once every CU has two units (64 single tokens
  // with windows of 4096, 8 cached heads of 128: 59 us whole, 66 split).
  const Cut cut = narrow && mask == kWindow && units >= 2 * static_cast<int64_t>(cus) ? Cut::kWhole
                  : narrow ? narrow_cut(cus, dtype, D, units, max_tokens, s.blocks, mask) : wide_cut(units, max_tokens, s.blocks);
  s.tall = cut == Cut::kTall;
  // spans of 128 tokens, or longer ones where a split call's line could have 2^31 places
  s.span_shift = 7;
  if (cut == Cut::kSplit)
    while (s.units * ((max_tokens >> s.span_shift) + 1) >= (int64_t(1) << 31)) s.span_shift++;
  s.plan_bytes = (2 * (B + 1) * 4 + 255) / 256 * 256;
  const bool split = cut == Cut::kSplit && max_tokens > (int64_t(kMinRun) << s.span_shift);
  s.bytes = split ? s.plan_bytes + (s.units + s.blocks) * (s.rows * (D + 2)) * 4 : 0;
  return s;
}

}  // namespace fp8q
