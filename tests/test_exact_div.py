"""The attention schedule's integer quotients (csrc/exact_div.hpp), compiled for the host: every reciprocal
within two steps of fp32 must give the exact quotient."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rotation_lloyd_max_amd", "csrc")
PROGRAM = r"""
#include "exact_div.hpp"
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>

static int64_t tried = 0;
static bool check(int64_t x, int64_t d) {
  if (x < 1 || x > (1 << 27) || d < 1 || d > (1 << 27)) return true;
  const int want = static_cast<int>((x + d - 1) / d);
  float r = 1.f / static_cast<float>(d);
  r = std::nextafterf(std::nextafterf(r, 0.f), 0.f);
  for (int k = 0; k < 5; ++k, r = std::nextafterf(r, 2.f)) {
    ++tried;
    const int got = tq::ceil_div_by(static_cast<int>(x), static_cast<int>(d), r);
    if (got != want) {
      std::printf("ceil(%lld / %lld) = %d, got %d (step %d)\n", (long long)x, (long long)d, want, got, k - 2);
      return false;
    }
  }
  return true;
}

int main() {
  static_assert(tq::ceil_div_by(7, 2, 0.5f) == 4, "");
  // quotients that one step of correction left wrong
  bool ok = check(25434587, 1) && check(65511726, 2) && check(1 << 27, 1) && check(1, 1 << 27) && check(1 << 27, 1 << 27);
  for (int64_t d = 1; ok && d <= 800; ++d)
    for (int64_t q = 1; ok && q <= 64; ++q)
      for (int64_t e = -2; ok && e <= 2; ++e)
        ok = check(d * q + e, d) && check((((1ll << 27) / d) - q) * d + e, d) && check((1ll << 27) - q * 1000003 % (1 << 20) + e, d);
  std::mt19937_64 g(1);
  for (int i = 0; ok && i < 4000000; ++i) {
    const int64_t x = 1 + static_cast<int64_t>(g() >> (37 + g() % 27)) % (1 << 27), d = 1 + static_cast<int64_t>(g() >> (37 + g() % 27)) % (1 << 27);
    ok = check(x, d) && check(x / d * d, d) && check(x / d * d + 1, d) && check(x / d * d + d - 1, d);
  }
  std::printf("%s %lld\n", ok ? "ok" : "failed", (long long)tried);
  return ok ? 0 : 1;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_ceil_div_is_exact_for_every_reciprocal_within_two_steps(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
    assert out.stdout.startswith("ok")
