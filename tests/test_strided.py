"""Host check of the exact overlap test of strided tensors (no GPU): the header is compiled with g++
into a program that compares it with marking every byte, for many small tensors, and answers for the
layouts that callers use."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "deepseek_v4_engram_gb300", "csrc")

PROGRAM = r"""
#include "strided.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using namespace engram;

static long mark(const Strided& a, std::vector<int>& bytes, bool& twice) {
  long n = 0;
  for (int64_t i = 0; i < a.n[0]; ++i)
    for (int64_t j = 0; j < a.n[1]; ++j)
      for (int64_t k = 0; k < a.n[2]; ++k)
        for (int64_t w = 0; w < a.width; ++w, ++n)
          if (bytes[a.lo + (a.n[0] > 1 ? i * a.stride[0] : 0) + (a.n[1] > 1 ? j * a.stride[1] : 0) +
                    (a.n[2] > 1 ? k * a.stride[2] : 0) + w]++) twice = true;
  return n;
}

static Strided any() {
  auto n = [] { return rand() % 3 ? 1 + rand() % 6 : 1; };
  auto s = [] { return rand() % 2 ? 1 + rand() % 12 : 8 * (1 + rand() % 12); };
  return Strided(reinterpret_cast<void*>(uintptr_t(rand() % 200)), 1 + rand() % 9, n(), s(), n(), s(), n(), s());
}

int main() {
  srand(5);
  long bad = 0, shared = 0, self = 0;
  for (int rep = 0; rep < 200000; ++rep) {
    const Strided a = any();
    Strided b = any();
    if (rep % 2)   // the same layout, moved
      for (int k = 0; k < 3; ++k) b.n[k] = a.n[k], b.stride[k] = a.stride[k];
    std::vector<int> ba(4000, 0), bb(4000, 0);
    bool ta = false, tb = false, both = false;
    mark(a, ba, ta);
    mark(b, bb, tb);
    for (int i = 0; i < 4000; ++i) both |= ba[i] && bb[i];
    bad += shares_memory(a, b) != both || shares_memory(b, a) != both;
    bad += rows_share_memory(a) != ta || rows_share_memory(b) != tb;
    shared += both;
    self += ta;
  }
  // nothing overflows at the largest strides and counts, and rows of single elements
  const int64_t big = int64_t(1) << 39, n = int64_t(1) << 17;
  const Strided x(reinterpret_cast<void*>(16), 256, n, big, 1 << 10, 1 << 12);
  const Strided y(reinterpret_cast<void*>(16 + 256), 256, n, big, 1 << 10, 1 << 12);
  const Strided z(reinterpret_cast<void*>(16 + 255), 1, n, big, 1 << 10, 1 << 12);
  bad += shares_memory(x, y) || !shares_memory(x, z) || shares_memory(y, z) || rows_share_memory(x);
  // strides that do not nest end in a bounded number of steps
  const Strided u(reinterpret_cast<void*>(0), 16, 1 << 24, 1048576 + 16, 1 << 20, 1048576 + 48);
  const Strided v(reinterpret_cast<void*>(8), 8, 1 << 24, 1048576 + 32, 1 << 20, 1048576 + 80);
  (void)shares_memory(u, v);
  printf("shared=%ld self=%ld bad=%ld\n", shared, self, bad);
  return bad != 0 || shared < 10000 || self < 10000;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_overlap_is_exact(tmp_path):
    src = tmp_path / "check.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-I", CSRC, str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stdout + r.stderr
