"""How calls of the attention over the 4-bit cache are cut (fp8_group_quant_amd/csrc/kv4_attention_shape.h),
compiled for the host: for all sizes that the entry point accepts, the units, the places of the line of
spans and their number per sequence stay in the 32 bits that the kernels count them in."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <algorithm>
#include <cstdio>
#include "kv4_attention_shape.h"
using namespace fp8q;
static long bad = 0, cases = 0, splits = 0;

// The most units that any lengths of B sequences with T queries in all can have: one row of each tile
// that is not full.
static int64_t most_units(int64_t B, int64_t T, int64_t group, int64_t Hkv, int rows) {
  const int64_t seqs = std::min(B, T);  // that have a query
  int64_t most = 0;
  for (int64_t n : {int64_t(1), seqs}) {  // the others one query, the last the rest
    const int64_t one = (group + rows - 1) / rows, rest = ((T - (n - 1)) * group + rows - 1) / rows;
    most = std::max(most, (n - 1) * one + rest);
  }
  return most * Hkv;
}

static void check(int dtype, int64_t B, int64_t T, int64_t Hkv, int64_t group, int64_t D, int64_t tokens) {
  const int64_t limit = int64_t(1) << 31, Hq = Hkv * group;
  if (Hq > (1 << 20) || T * Hq >= limit) return;  // refused
  const AttnShape s = attention_shape(256, dtype, B, T, Hq, Hkv, D, tokens);
  cases++;
  const int64_t spans = std::max<int64_t>((tokens + (int64_t(1) << s.span_shift) - 1) >> s.span_shift, 1);
  bool ok = s.span_shift >= 7 && s.span_shift <= 30 && s.units < limit && s.units >= most_units(B, T, group, Hkv, s.rows);
  if (s.bytes > 0) {
    splits++;
    ok = ok && s.units * spans < limit && s.bytes >= s.plan_bytes + (s.units + s.blocks) * s.rows * (D + 2) * 4 &&
         s.plan_bytes >= 2 * (B + 1) * 4;
  }
  if (!ok) {
    bad++;
    std::printf("B %ld T %ld Hkv %ld group %ld D %ld tokens %ld: units %ld shift %d\n", B, T, Hkv, group, D, tokens, s.units, s.span_shift);
  }
}

int main() {
  const int64_t seqs[] = {1, 2, 17, 64, 255, 1000, 2048, 4095, 4096};
  const int64_t queries[] = {1, 2, 5, 17, 64, 300, 2047, 4096, 65536, (int64_t(1) << 31) - 1};
  const int64_t heads[] = {1, 3, 8, 64, 255, 4096, 1 << 17, 1 << 18, 1 << 19, (1 << 19) + 1, 1 << 20};
  const int64_t groups[] = {1, 4, 5, 16, 100, 1 << 12, 1 << 20};
  const int64_t lengths[] = {0, 1, 128, 300, 2048, 5000, 262144, 1 << 27, (1 << 30) - 1, 1 << 30};
  for (int dtype : {FP8Q_DTYPE_BF16, FP8Q_DTYPE_F16})
    for (int64_t D : {64, 128, 256})
      for (int64_t B : seqs)
        for (int64_t T : queries)
          for (int64_t Hkv : heads)
            for (int64_t group : groups)
              for (int64_t tokens : lengths) check(dtype, B, T, Hkv, group, D, tokens);
  std::printf("%ld %ld %ld\n", cases, splits, bad);
  return bad != 0;
}
"""


def test_every_accepted_size_is_cut(tmp_path):
    src, exe = tmp_path / "drv.cpp", tmp_path / "drv"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "fp8_group_quant_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout[-2000:]
    cases, splits, bad = map(int, r.stdout.split())
    assert cases > 50000 and splits > 5000 and bad == 0
