"""Index arithmetic of the fused and grouped linears, on the host: a small program over the functions that the
kernels call."""
import os
import subprocess

import pytest

from tests.conftest import ROOT
from ternary_weight_quantized_q2_amd import build_lib

PROGRAM = r"""
#include <cstdio>
#include "q2_fused.h"
using namespace q2dev;
// Every piece that a kernel may ask for lies inside its row, and every piece of the row is where it belongs.
int main() {
  for (int per = 1; per <= 2; ++per)
    for (int blocks = 4; blocks <= 130; ++blocks) {
      const long row = blocks * (per == 2 ? 32L : 64L);
      for (int u = 0; u <= last_unit(blocks, per) + 24; ++u)
        for (int p = 0; p < 4; ++p) {
          const long at = (long)unit_start(u, blocks, per) + 16 * p - unit_back(u, blocks, per, p);
          const long want = 64L * u + 16 * p;
          if (at < 0 || at + 16 > row || (want + 16 <= row && at != want)) {
            printf("per %d blocks %d unit %d piece %d: %ld of %ld\n", per, blocks, u, p, at, row);
            return 1;
          }
        }
    }
  puts("bounds ok");
}
"""


def run_program(tmp_path, text):
    if not os.path.exists(build_lib.HIPCC):
        pytest.fail("hipcc is needed to build the program")
    src, exe = tmp_path / "program.hip", str(tmp_path / "program")
    src.write_text(text)
    r = subprocess.run([build_lib.HIPCC, *build_lib.FLAGS, str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=60, env=dict(os.environ, HIP_VISIBLE_DEVICES=""))


def test_code_prefetches_stay_in_the_row(tmp_path):
    r = run_program(tmp_path, PROGRAM)
    assert r.returncode == 0 and "bounds ok" in r.stdout, r.stdout + r.stderr
