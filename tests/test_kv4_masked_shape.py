"""How window and tree calls of the attention over the 4-bit cache are cut: the checks of test_kv4_attention_shape.py with
each mask, blocks of 16 waves only with a sequence to a CU at most (their plan's LDS), and what a window's unit reads."""
import os
import subprocess

import pytest
from test_kv4_attention_shape import DRIVER, ROOT


def compiled(tmp_path, source):
    src, exe = tmp_path / "drv.cpp", tmp_path / "drv"
    src.write_text(source)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "fp8_group_quant_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)


@pytest.mark.parametrize("mask", ["kWindow", "kTree"])
def test_every_accepted_size_is_cut(tmp_path, mask):
    call = "attention_shape(256, dtype, B, T, Hq, Hkv, D, tokens);"
    assert DRIVER.count(call) == 1
    source = DRIVER.replace(call, f"attention_shape(256, dtype, B, T, Hq, Hkv, D, tokens, {mask});\n"
                                  "  if (s.tall && (s.rows != kRows || B > 256)) bad++;")
    r = compiled(tmp_path, source)
    assert r.returncode == 0, r.stdout[-2000:]
    cases, splits, bad = map(int, r.stdout.split())
    assert cases > 50000 and splits > 2000 and bad == 0


WINDOW = r"""
#include <cstdio>
#include "kv4_attention_shape.h"
using namespace fp8q;
// Tokens, none past the last query's, of the steps of 64 in which a unit of n consecutive queries, the last at place `last`,
// has some to see, counted.
static int64_t seen(int64_t last, int64_t n, int64_t window, int64_t sinks) {
  int64_t steps = 0;
  for (int64_t s = 0; s <= last / 64; s++) {
    bool any = false;
    for (int64_t j = 64 * s; j < 64 * s + 64 && j <= last && !any; j++)
      for (int64_t p = last - n + 1; p <= last && !any; p++) any = p >= 0 && j <= p && (j > p - window || j < sinks);
    steps += any;
  }
  return steps * 64 - (63 - last % 64);
}
int main() {
  long bad = 0;
  for (int64_t last : {0, 1, 63, 64, 200, 700, 1000})
    for (int64_t n : {1, 2, 32, 128})
      for (int64_t window : {1, 2, 63, 64, 65, 300, 2000})
        for (int64_t sinks : {0, 1, 64, 65, 100, 2000}) {
          if (window_tokens(int64_t(1) << 30, window, sinks) < seen(last, n, window, sinks)) bad++;
          if (window_tokens(last + 1, window, sinks) > last + 1) bad++;
        }
  if (window_tokens(int64_t(1) << 30, int64_t(1) << 40, int64_t(1) << 40) != int64_t(1) << 30) bad++;
  std::printf("%ld\n", bad);
  return bad != 0;
}
"""


def test_window_tokens_hold_what_a_unit_sees(tmp_path):
    r = compiled(tmp_path, WINDOW)
    assert r.returncode == 0, r.stdout
