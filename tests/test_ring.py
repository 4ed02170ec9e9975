"""Loads on their way when a wait gives up (CPU): the waits at a kernel's end, of
csrc/ring.h, against barriers that are played step by step."""
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "ring.h"

// A barrier with one load a phase: a wait for a parity passes when the phase
// of that parity is over, which is what the hardware's wait tells.
struct Barrier {
  int phase = 0;
  bool passes(unsigned parity) const { return (phase & 1) != (int)parity; }
};

int main() {
  long checked = 0, bad = 0;
  for (int stages = 1; stages <= 8; ++stages)
    for (int tiles = 1; tiles <= 40; ++tiles)
      for (int fail = 0; fail < tiles; ++fail)
        // the consumer waited for loads 0 .. fail - 1 and gave up at load `fail`;
        // of the pending ones a later one may have landed before an earlier one
        for (unsigned landed = 0; landed < (1u << stages); ++landed) {
          std::vector<Barrier> bar(stages);
          int issued = 0;
          auto issue = [&] { if (issued < tiles) ++issued; };
          for (int i = 0; i < stages; ++i) issue();
          for (int i = 0; i < fail; ++i) {
            ++bar[i % stages].phase;
            issue();
          }
          std::vector<bool> pending(tiles, false);
          for (int i = fail; i < issued; ++i) {
            if ((landed >> (i % stages)) & 1u) ++bar[i % stages].phase;
            else pending[i] = true;
          }
          for (int64_t i = mxg::ring_pending(issued, stages); i < issued; ++i) {
            Barrier &b = bar[i % stages];
            const unsigned parity = mxg::ring_parity(i, stages);
            ++checked;
            if (b.passes(parity) == pending[i]) ++bad;  // passes while its load is on its way, or waits for none
            if (pending[i]) {                           // it lands
              ++b.phase;
              pending[i] = false;
              if (!b.passes(parity)) ++bad;
            }
          }
          for (int i = 0; i < tiles; ++i) bad += pending[i];  // landed after the end
        }
  for (unsigned long long ns : {1ull, 1000ull, 1999999999ull})  // a short limit is not one for what is on its way
    bad += mxg::landing_limit(ns) != 2000000000ull;
  bad += mxg::landing_limit(5000000000ull) != 5000000000ull;
  printf("%ld %ld\n", checked, bad);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_every_load_on_its_way_is_waited_for(tmp_path):
    (tmp_path / "ring.cpp").write_text(PROGRAM)
    exe = tmp_path / "ring"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", str(ROOT / "block_scaled_gemm_gb300" / "csrc"), "-o", str(exe),
                    str(tmp_path / "ring.cpp")], check=True)
    checked, bad = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert checked > 100000 and bad == 0
