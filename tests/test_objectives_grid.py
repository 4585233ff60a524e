"""The number of workgroups that the objectives' launches over rows take, on the host (csrc/objectives_grid.h)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "second_order_optimizer_amd", "csrc", "objectives_grid.h")
ROWS = [0, 1, 2, 3, 4, 5, 255, 256, 257, 511, 512, 513, 2047, 2048, 2049, 100003, (1 << 31) - 1, 1 << 31, (1 << 40) + 1]
PROGRAM = """
#include <stdio.h>
#include <stdlib.h>
#include "%s"
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3)
    printf("%%d\\n", kfac::grid_of(atoll(argv[i]), atoi(argv[i + 1]), atoi(argv[i + 2])));
  return 0;
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="g++ not installed")
def test_workgroups_of_any_number_of_rows(tmp_path):
    """None for no rows; else at least one, no more than are resident or have a row, and every row is walked to."""
    src, exe = tmp_path / "grid.cpp", tmp_path / "grid"
    src.write_text(PROGRAM % HEADER)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    cases = [(rows, teams, per_cu) for rows in ROWS for teams in (1, 4) for per_cu in (1, 2, 4, 5, 6, 8)]
    r = subprocess.run([str(exe)] + [str(v) for c in cases for v in c], capture_output=True, text=True)
    assert r.returncode == 0, r.returncode
    got = [int(v) for v in r.stdout.split()]
    assert len(got) == len(cases)
    for (rows, teams, per_cu), grid in zip(cases, got):
        need, most = -(-rows // teams), 256 * per_cu
        assert (grid == 0) if rows == 0 else (1 <= grid <= min(need, most)), (rows, teams, per_cu, grid)
        if rows and teams == 1:        # equal rounds: no more of them than full residency takes
            assert grid * -(-need // most) >= need, (rows, teams, per_cu, grid)
