"""Host-only: a role that leaves a kernel waits for the last copy that it armed, wherever it leaves.

The barrier is modelled as it is defined: a wait on a parity returns once the phase of that parity has
completed, which includes the phase before the current one.  The count is the kernels' own
(tc::ArmedLoads), compiled for the host."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SOURCE = r"""
#include <cstdio>
#include "tc.cuh"
struct Barrier {                       // one arrival a phase
  int armed = 0, landed = 0;           // phases armed; phases complete
  bool wait_returns(unsigned parity) const { return ((unsigned)landed & 1u) != parity; }
};
int main() {
  // a role arms a load per segment and waits for it; it may leave before it armed segment `leave`'s
  // (the wait for the free buffer gave up) or after, with that load in flight or landed
  for (int leave = 0; leave < 9; ++leave)
    for (int how = 0; how < 3; ++how) {
      Barrier bar;
      csa::tc::ArmedLoads loads;
      for (int n = 0; n <= leave; ++n) {
        if (n == leave && how == 0) break;
        loads.arm();
        ++bar.armed;
        if (n == leave && how == 1) break;
        ++bar.landed;
      }
      if (loads.any() != (bar.armed > 0)) { std::printf("any %d %d\n", leave, how); return 1; }
      if (!loads.any()) continue;
      if (bar.wait_returns(loads.last()) != (bar.landed == bar.armed)) { std::printf("wait %d %d\n", leave, how); return 1; }
      bar.landed = bar.armed;
      if (!bar.wait_returns(loads.last())) { std::printf("landed %d %d\n", leave, how); return 1; }
    }
  std::printf("ok\n");
  return 0;
}
"""


@pytest.mark.skipif(not (os.path.exists(NVCC) or shutil.which(NVCC)), reason="needs nvcc")
def test_the_last_armed_load_is_waited_for(tmp_path):
    src, exe = tmp_path / "loads.cu", tmp_path / "loads"
    src.write_text(SOURCE)
    r = subprocess.run([NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I",
                        os.path.join(ROOT, "compressed_sparse_long_csa_b200", "csrc"), str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.stdout.strip() == "ok", r.stdout


def test_the_rule_before_would_not_have_waited():
    """Leaving after the load of segment n was armed and counted (n + 1 armed), the parity of the phase
    after it was waited on: that returns while the load is in flight."""
    armed, landed = 3, 2
    assert (landed & 1) != (armed & 1)                  # the phase not armed: returns at once
    assert (landed & 1) == ((armed - 1) & 1)            # the last armed: waits
