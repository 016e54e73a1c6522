"""The limit of the waits inside the attention kernels, on the host: time in which the context was suspended does not
use it up, time in which the thread ran does."""
import os
import shutil
import subprocess

from transformer_rope_positional_gb300 import build as B

PROGRAM = r"""
#include "serving/wait_clock.h"
#include <initializer_list>

int main() {
  const uint64_t ms = 1000000ull, s = 1000 * ms;  // of the clock, of which the lower 32 bits are seen
  for (uint64_t start : {uint64_t(0), 5 * s, uint64_t(0xfffffffe)}) {
    {  // suspended for an hour, then again for ten seconds, within one wait
      rope::WaitClock c(start);
      if (c.expired(start + 3600 * s)) return 1;
      if (c.expired(start + 3610 * s)) return 2;
      if (c.expired(start + 3610 * s + 1 * ms)) return 3;
    }
    for (uint64_t step : {uint64_t(1000), ms, 40 * ms}) {  // never suspended: after 2 s, not before
      rope::WaitClock c(start);
      uint64_t t = 0;
      while (!c.expired(start + (t += step)))
        if (t > 2 * s) return 4;
      if (t <= 2 * s || t > 2 * s + step) return 5;
    }
    {  // looks that are far apart end the wait too
      rope::WaitClock c(start);
      int looks = 0;
      while (!c.expired(start + 10 * s * ++looks))
        if (looks > 100) return 6;
      if (looks < 40) return 7;
    }
    rope::WaitClock c(start);  // a clock that stands still
    for (int i = 0; i < 1000; ++i)
      if (c.expired(start)) return 8;
  }
  return 0;
}
"""


def test_time_suspended_does_not_use_up_a_wait(tmp_path):
    src, exe = tmp_path / "clock.cpp", tmp_path / "clock"
    src.write_text(PROGRAM)
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", B.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
