"""The sizes of tests/int8_tiles.py take the kernels that they are listed for."""
import os
import shutil
import subprocess

import pytest

import int8_tiles

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dense_fp32_matrix_03_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
STAGES = {"64/2": 2, "64/3": 3, "64/4": 4, "128": 4, "128x256": 3, "256": 2}


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_cases_take_every_kernel(tmp_path):
    exe = tmp_path / "int8_tile_check"
    subprocess.run([HIPCC, "-std=c++17", "-O2", "--cuda-host-only", "-x", "hip", "-I", CSRC,
                    os.path.join(HERE, "int8_tile_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, timeout=300)
    every = [(name, case) for table in (int8_tiles.CASES, int8_tiles.GROUPED)
             for name, cases in table.items() for case in cases]
    out = subprocess.run([str(exe)] + [str(v) for _, case in every for v in case], check=True,
                         capture_output=True, text=True).stdout.split()
    assert [(n, c) for (n, c), got in zip(every, out) if got != n] == []
    assert len(out) == len(every)


def test_slices_leave_every_remainder_over_the_stages():
    for name, cases in int8_tiles.CASES.items():
        left = {-(-K // 128) % STAGES[name] for _, _, _, K in cases}
        assert left == set(range(STAGES[name])), name
