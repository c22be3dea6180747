"""The arithmetic behind the FP8 product's bounded waits, compiled for the host
and run on the CPU: no kernel has to run out of time for it."""

import os
import subprocess

import pytest

from quantized_rl_fine_b200 import build


def run_on_host(tmp_path, body):
    """Compiles `body` (a main function) with the kernel's own header for the CPU and runs it; 0 is success."""
    src, exe = tmp_path / "main.cu", tmp_path / "main"
    src.write_text('#include <cstdint>\n#include <cstdio>\n#include <cstdlib>\n#include "fp8_wait.cuh"\nusing namespace moeq;\n' + body)
    subprocess.run([build._nvcc(), "-std=c++17", "-O1", "-I", build.CSRC, "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


BUDGET = r"""
static int bad = 0;
static void expect(bool v, bool want, const char* what, long long budget, long long t0) {
  if (v != want) { std::printf("%s: budget %lld begun at %lld\n", what, budget, t0); bad = 1; }
}
int main() {
  const long long top = 1ll << 41;
  const long long budgets[] = {1, 200, 1023, 1024, 5000, 2000000000ll, (1ll << 32) - 1, 1ll << 32, (1ll << 32) + 77,
                               1ll << 36, top - 1, top, top + 1, 1ll << 50, 0x7fffffffffffffffll};
  const long long starts[] = {0, 1, 1023, 1024, (1ll << 32) - 5, (1ll << 42) - 1000, (1ll << 42) - 1, 1ll << 42, (1ll << 52) + 12345};
  for (long long b : budgets)
    for (long long t0 : starts) {
      const long long end = b < top ? b : top;
      const uint32_t u0 = wait_units(t0);
      for (long long e : {0ll, end / 2, end - 1, end})
        expect(wait_spent(u0, wait_units(t0 + e), b), false, "too early", b, t0);
      for (long long e : {end + 3 * 1024, end + 1000000, end + (1ll << 33), top + (1ll << 40)})   // looked at late
        if (e > end) expect(wait_spent(u0, wait_units(t0 + e), b), true, "not at all", b, t0);
    }
  return bad;
}
"""


def test_every_budget_ends_a_wait_and_none_too_early(tmp_path):
    """Budgets past 32 bits among them: the longest a wait can take is 2^41 cycles, whatever was set."""
    run_on_host(tmp_path, BUDGET)
