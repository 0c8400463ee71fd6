"""The number of clusters that share out the rows of a layer norm backward pass, where a device holds few of them: a
small C++ program prints late_clusters for a table of arguments."""

import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = """
#include <cstdio>
#include <initializer_list>
#include "ra_layernorm_plan.h"
int main() {
  for (int phases : {1, 4, 8})
    for (int fit = 0; fit <= 76; ++fit)
      for (int rows = 1; rows <= 200; ++rows)
        std::printf("%d %d %d %d\\n", phases, fit, rows, (int)ra::late_clusters(fit, rows, phases));
}
"""


def test_clusters_for_rows(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "plan.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "plan")
    csrc = os.path.join(ROOT, "ring_all_reduce_02_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", f"-I{csrc}", str(tmp_path / "plan.cpp"), "-o", exe], check=True)
    table = [tuple(map(int, line.split())) for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()]
    assert len(table) == 3 * 77 * 200
    for phases, fit, rows, n in table:
        assert 0 <= n <= min(fit, rows)
        # a cluster's rows r, r + n, r + 2 n, ... share a phase
        assert n == 0 or rows <= n or n % phases == 0
        # none only where no number of clusters would do
        assert (n == 0) == (rows > fit and fit < phases)
        # and as many as there can be
        assert n in (0, rows) or n + phases > fit
