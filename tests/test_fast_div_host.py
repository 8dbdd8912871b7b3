"""Division by a fixed divisor (csrc/intdiv.h, FastDiv) against integer division, on the host (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r"""
#define __host__
#define __device__
#include "intdiv.h"
#include <cstdio>
#include <random>

int main() {
  std::mt19937 rng(7);
  auto check = [](const attn::FastDiv& f, unsigned x) {
    if (x <= 0x7fffffffu && f.div(x) != x / f.d) {
      std::printf("%u / %u\n", x, f.d);
      return false;
    }
    return true;
  };
  for (unsigned long long d = 1; d < (1ull << 31); d += d < 3000 ? 1 : d / 97) {
    const attn::FastDiv f = attn::make_fast_div((unsigned)d);
    for (unsigned x : {0u, 1u, (unsigned)d - 1, (unsigned)d, (unsigned)d + 1, 0x40000000u, 0x7ffffffeu, 0x7fffffffu})
      if (!check(f, x)) return 1;
    for (int i = 0; i < 200; ++i) {
      const unsigned x = rng() & 0x7fffffffu, y = x / (unsigned)d * (unsigned)d;
      if (!check(f, x) || !check(f, y) || (y > 0 && !check(f, y - 1))) return 1;
    }
  }
  std::printf("ok\n");
  return 0;
}
"""


def test_fast_div_is_exact(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src = tmp_path / "fast_div.cpp"
    src.write_text(SRC)
    exe = str(tmp_path / "fast_div")
    subprocess.run([gxx, "-std=c++17", "-O2", "-I", os.path.join(ROOT, "attention_attn_fwd_06_gb300", "csrc"), str(src), "-o",
                    exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
