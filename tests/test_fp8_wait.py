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


CLOSE = r"""
// Barriers as the hardware counts them: a phase completes when its arrivals and its bytes are all there.
struct Barrier {
  int pending = 1, phase = 0;
  long long tx = 0;
  void settle() { if (pending == 0 && tx == 0) { pending = 1; ++phase; } }
  void arrive(long long bytes) { tx += bytes; --pending; settle(); }
  void bytes(long long n) { tx -= n; settle(); }
};
constexpr int kBytes = 32768;
static int bad = 0;
struct Model {
  uint32_t S;
  Barrier bar[8];
  int in_flight[8] = {0};          // copies that have not landed, by stage
  void land(uint32_t s) { if (in_flight[s] > 0) { --in_flight[s]; bar[s].bytes(kBytes); } }
  void add_bytes(uint32_t s) { bar[s].bytes(kBytes); }
  void arrive(uint32_t s) { bar[s].arrive(kBytes); }
  bool done(uint32_t s, uint32_t parity) const { return (bar[s].phase & 1) != (int)parity; }
  void wait(uint32_t s, uint32_t parity) {
    while (in_flight[s] > 0) {
      if (done(s, parity)) { std::printf("over before the copies\n"); bad = 1; return; }
      land(s);
    }
    if (!done(s, parity)) { std::printf("never over\n"); bad = 1; }
  }
};
// A pair (or a CTA alone) stopped at a random point: `used` fills were consumed, the even CTA has begun n0 and the
// odd one n1 of them, and some of the copies that are not consumed have landed.
static void stopped(uint32_t S, uint32_t used, uint32_t n0, uint32_t n1, bool pair) {
  Model m;
  m.S = S;
  const uint32_t end = n0 > n1 ? n0 : n1;
  for (uint32_t g = 0; g < end; ++g) {
    Barrier& b = m.bar[g % S];
    const int even = g < n0, odd = pair && g < n1;
    const bool odd_first = std::rand() & 1;
    if (odd && odd_first) { if (g < used || (std::rand() & 1)) b.bytes(kBytes); else ++m.in_flight[g % S]; }
    if (even) {
      b.arrive(pair ? 2 * kBytes : kBytes);
      if (g < used || (std::rand() & 1)) b.bytes(kBytes); else ++m.in_flight[g % S];
    }
    if (odd && !odd_first) { if (g < used || (std::rand() & 1)) b.bytes(kBytes); else ++m.in_flight[g % S]; }
  }
  close_fills(n0, pair ? n1 : n0, S, m);
  for (uint32_t s = 0; s < S; ++s)
    if (m.in_flight[s]) { std::printf("copies left: S %u used %u begun %u %u\n", S, used, n0, n1); bad = 1; }
}
int main() {
  for (uint32_t S = 3; S <= 5; ++S)
    for (uint32_t used = 0; used < 14; ++used)
      for (uint32_t a = 0; a <= S; ++a)
        for (uint32_t b = 0; b <= S; ++b)
          for (int pair = 0; pair < 2; ++pair)
            for (int i = 0; i < 20; ++i) stopped(S, used, used + a, pair ? used + b : used + a, pair);
  return bad;
}
"""


def test_a_stopped_product_waits_for_every_copy_that_was_begun(tmp_path):
    """Wherever the copying warps of a CTA or of a pair's two stopped, against barriers counted in a model: no wait
    is over before the stage's copies have landed, and none lasts for ever."""
    run_on_host(tmp_path, CLOSE)
