"""Which kernel the 4-bit product takes (fp8_group_quant_amd/csrc/mxfp4_shape.h), compiled for the host: the GPU tests'
sizes reach every kernel, and for all sizes that the entry point accepts the ranges of K and the workspace are sound."""
import os
import subprocess

from test_gpu_mxfp4_kernels import SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "mxfp4_shape.h"
using namespace fp8q;
static const char* const kName[] = {"few", "large", "deep", "flat"};

int main(int n, char** v) {
  for (int i = 1; i + 2 < n; i += 3) {
    const Mxfp4Shape s = mxfp4_shape(atoll(v[i]), atoll(v[i + 1]), atoll(v[i + 2]), 256);
    std::printf("%s %d\n", kName[static_cast<int>(s.kind)], s.splits);
  }
  if (n > 1) return 0;
  const int64_t rows[] = {1, 2, 16, 17, 32, 33, 64, 65, 100, 128, 129, 256, 300, 513, 1000, 2048, 4097, 8192, 20000, 100000, 1 << 20, 1 << 26};
  const int64_t units[] = {1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 33, 56, 64, 103, 211, 1000, 4097, (1 << 18) - 1};
  long cases = 0, split = 0, bad = 0;
  for (int cus : {1, 32, 80, 256, 304})
    for (int64_t M : rows)
      for (int64_t N : rows)
        for (int64_t u : units) {
          if (M * N > (int64_t(1) << 40)) continue;
          const int64_t K = 128 * u;
          const Mxfp4Shape s = mxfp4_shape(M, N, K, cus);
          const int bm[] = {64, 256, 128, 64}, bn[] = {16, 256, 128, 128};
          const int kind = static_cast<int>(s.kind);
          const int64_t tiles = mxfp4_tiles(M, N, bm[kind], bn[kind]);
          cases++;
          bool ok = s.splits >= 1 && s.splits <= kMxfp4MostSplits && tiles < (int64_t(1) << 31);
          ok = ok && (s.kind != Mxfp4Kind::kFew || M <= 64);
          ok = ok && s.ws == (s.splits > 1 ? s.splits * M * ((N + 3) / 4 * 4) * 4 : 0);
          if (s.splits > 1) {  // a block for every tile and range, every range of 8 units of K at least
            split++;
            ok = ok && tiles * s.splits <= cus && u / s.splits >= 8 && (s.kind == Mxfp4Kind::kDeep || s.kind == Mxfp4Kind::kFlat);
          }
          if (!ok) {
            bad++;
            std::printf("%ld x %ld x %ld on %d: %s, %d ranges\n", M, N, K, cus, kName[kind], s.splits);
          }
        }
  std::printf("%ld %ld %ld\n", cases, split, bad);
  return bad != 0;
}
"""


def compiled(tmp_path):
    src, exe = tmp_path / "drv.cpp", tmp_path / "drv"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "fp8_group_quant_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    return str(exe)


def test_the_gpu_tests_reach_every_kernel(tmp_path):
    sizes = [str(x) for s in SHAPES for x in s[:3]]
    r = subprocess.run([compiled(tmp_path), *sizes], capture_output=True, text=True, check=True)
    took = [(kind, int(splits)) for kind, splits in (line.split() for line in r.stdout.splitlines())]
    assert took == [s[3:] for s in SHAPES]
    assert {("few", False), ("large", False), ("deep", False), ("deep", True), ("flat", False), ("flat", True)} == \
        {(kind, splits > 1) for kind, splits in took}


def test_every_accepted_size_has_a_sound_shape(tmp_path):
    r = subprocess.run([compiled(tmp_path)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-2000:]
    cases, split, bad = map(int, r.stdout.split()[-3:])
    assert cases > 20000 and split > 500 and bad == 0
