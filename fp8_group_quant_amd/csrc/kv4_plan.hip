// kv4_plan.hip — one serving step's page bookkeeping, from the requests' lengths.
//
// Sequence b holds l_b cached tokens and gets n_b new ones, packed one sequence after the other. With pages of
// P tokens it needs the pages ceil(l_b / P) .. ceil((l_b + n_b) / P) - 1 of its table row, which are taken from
// the free pages in the order of the sequences: two prefixes, over n_b and over the page counts. Token i of b
// has position l_b + i, and its slot follows from that position's page, which is either held already (the
// last, partly filled one) or a new one, found in the free pages and not in the table, so that no block reads
// what another writes.
//
// One launch. Every block brings the lengths to LDS (at most 4096 sequences), forms both prefixes there and does
// 256 of the tokens, each found in the prefix by bisection; the first token of a new page writes its table
// entry. What it takes is the launch and a chain of three loads from memory: lengths, free pages or table, stores. More
// tokens to a block would form the prefixes less often but go through that chain again for each 256: us for 256, 512 and 1024
// tokens, B sequences with n new tokens each:
//   256 x 1024, ragged  5.1  5.8  7.3      1 x 16384  6.1 7.0 9.0      1000 x 30  4.1 4.7 5.8
//   4096 x 1 (many sequences, few tokens)  11.0 12.3 14.9    4096 x 40  12.1 12.7 15.2    64 x 1  3.8
#include <algorithm>

#include "serving.h"

namespace fp8q {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;  // a thread for each of a block's tokens

// Inclusive sum over the block's threads; `lds` holds one value per wave.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* lds, int64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t up = __shfl_up(v, off, 64);
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

__device__ __forceinline__ int64_t clamped(int64_t v, int64_t hi) { return v < 0 ? 0 : v > hi ? hi : v; }

__global__ __launch_bounds__(kThreads) void kv4_plan_kernel(Kv4PlanParams p) {
  __shared__ int64_t sum[2][kWaves];
  extern __shared__ int32_t lds[];
  const int32_t B = static_cast<int32_t>(p.B), tid = threadIdx.x;
  int32_t* const ends = lds;              // [B + 1] new tokens before each sequence
  int32_t* const taken = lds + B + 1;     // [B] new pages before each sequence
  int32_t* const lens = taken + B;        // [B] cached tokens
  const int32_t per = ((B + kThreads - 1) / kThreads) | 1;  // (odd: the threads' parts begin in all LDS banks)
  const int32_t beg = min(tid * per, B), end = min(beg + per, B);

#pragma unroll 4
  for (int32_t b = tid; b < B; b += kThreads) {
    ends[b] = max(p.q_lens[b], 0);
    lens[b] = static_cast<int32_t>(clamped(p.kv_lens[b], p.max_tokens));
  }
  __syncthreads();
  int64_t mine = 0, total;
  for (int32_t b = beg; b < end; b++) mine += ends[b];
  int64_t at = block_scan(mine, sum[0], total) - mine;
  for (int32_t b = beg; b < end; b++) {
    const int32_t n = ends[b];
    ends[b] = static_cast<int32_t>(min(at, p.T));
    at += n;
  }
  if (tid == 0) ends[B] = static_cast<int32_t>(min(total, p.T));
  __syncthreads();

  const int32_t round = (1 << p.page_shift) - 1;
  // tokens that sequence b holds afterwards, and its new pages
  auto after = [&](int32_t b, int64_t len) { return min(len + ends[b + 1] - ends[b], p.max_tokens); };
  auto pages_of = [&](int64_t len) { return static_cast<int32_t>((len + round) >> p.page_shift); };
  mine = 0;
  for (int32_t b = beg; b < end; b++) mine += pages_of(after(b, lens[b])) - pages_of(lens[b]);
  at = block_scan(mine, sum[1], total) - mine;
  for (int32_t b = beg; b < end; b++) {
    const int64_t len = lens[b], now = after(b, len);
    taken[b] = static_cast<int32_t>(at);
    at += pages_of(now) - pages_of(len);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int32_t b = tid; b <= B; b += kThreads) {
      p.q_indptr[b] = ends[b];
      if (b < B) p.new_lens[b] = static_cast<int32_t>(after(b, lens[b]));
    }
    if (tid == 0) *p.pages_taken = static_cast<int32_t>(total);
  }

  const int32_t t = blockIdx.x * kThreads + tid;
  if (t >= p.T) return;
  int64_t slot = -1, place = -1;
  if (t < ends[B]) {
    int32_t lo = 0, hi = B;  // the last sequence that begins at or before t
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (ends[mid] <= t) lo = mid; else hi = mid;
    }
    const int64_t len = lens[lo];
    place = len + t - ends[lo];
    if (place < p.max_tokens) {
      const int32_t first = pages_of(len), page = static_cast<int32_t>(place >> p.page_shift);
      int32_t* const entry = p.table + lo * p.table_sb + page;
      int64_t number = -1;
      if (page < first) {
        number = *entry;
      } else {
        const int64_t j = static_cast<int64_t>(taken[lo]) + page - first;
        if (j < p.F) number = p.free_pages[j];
      }
      if (number < 0 || number >= p.pages) number = -1;
      if (page >= first && (place & round) == 0) *entry = static_cast<int32_t>(number);
      if (number >= 0) slot = (number << p.page_shift) + (place & round);
    }
  }
  p.slots[t] = static_cast<int32_t>(slot);
  if (p.positions) p.positions[t] = static_cast<int32_t>(place);
}

}  // namespace

int launch_kv4_plan(const Kv4PlanParams& p, hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(std::max<int64_t>(1, (p.T + kThreads - 1) / kThreads));
  hipLaunchKernelGGL(kv4_plan_kernel, dim3(blocks), dim3(kThreads), (3 * p.B + 1) * sizeof(int32_t), stream, p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(FP8Q_ELAUNCH, std::string("kv4 plan launch: ") + hipGetErrorString(err));
  return FP8Q_OK;
}

}  // namespace fp8q
