"""What tests/orthogonalize_pieces.py allows sees the loss of any part of the arithmetic; and the
cases of tests/test_gpu_orthogonalize_tiles.py take every tile there is."""
import os
import shutil
import subprocess

import numpy as np
import pytest

import orthogonalize_model as om
import orthogonalize_pieces as op

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dense_fp32_matrix_03_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
S_Z, SS_Z = (0.0, 1.0, 0.0), (0.0, 0.0, 1.0)


def _forms(x, steps, coefficients):
    unit = x.astype(np.float64) / np.linalg.norm(x.astype(np.float64))
    c = op.singles(coefficients)
    single = op.formula(unit, steps, [np.float32(v) for v in c], np.matmul,
                        lambda v: v.astype(np.float32))
    return c, op.formula(unit, steps, c, np.matmul, lambda v: v), single.astype(np.float64)


@pytest.mark.parametrize("shape", [(65, 130), (128, 256), (257, 300), (150, 90), (129, 1050)])
@pytest.mark.parametrize("coefficients,steps", [(S_Z, 1), (SS_Z, 1), (om.STEP, 5)])
def test_a_lost_product_of_pieces_is_seen(shape, coefficients, steps):
    x = np.random.default_rng(sum(shape)).standard_normal(shape).astype(np.float32)
    c, want, single = _forms(x, steps, coefficients)
    op.check(op.in_pieces(x, steps, c).astype(np.float64), want, single)
    for dropped in ("high low", "low high"):
        with pytest.raises(AssertionError, match="off by"):
            op.check(op.in_pieces(x, steps, c, (dropped,)).astype(np.float64), want, single)


# Rows and columns both: an element is held to 2^-40 of the smaller of its row's and its column's
# range, which is not small against it any more once its row has grown by 2^15.
@pytest.mark.parametrize("kind,steps", [("rows", 5), ("rows", 20), ("columns", 5), ("columns", 20),
                                        ("graded", 5), ("graded", 20), ("both", 5), ("both", 8),
                                        ("few", 5), ("few", 8)])
@pytest.mark.parametrize("shape", [(96, 200), (200, 96), (100, 100)])
def test_rows_and_columns_of_unequal_size(shape, kind, steps):
    x = op.unequal(kind, shape, 1e-6, 5)
    c, want, single = _forms(x, steps, om.STEP)
    op.check(op.in_pieces(x, steps, c).astype(np.float64), want, single)


def test_what_p_is_held_to_at_least():
    """Many rows: the singular values are far below 1, and S S further still."""
    x = np.random.default_rng(1).standard_normal((500, 900)).astype(np.float32)
    c, want, single = _forms(x, 1, SS_Z)
    least = op.least_of_p(x.astype(np.float64) / np.linalg.norm(x.astype(np.float64)))
    op.check(op.in_pieces(x, 1, c).astype(np.float64), want, single, least)
    for dropped in ("high low", "low high"):
        with pytest.raises(AssertionError, match="off by"):
            op.check(op.in_pieces(x, 1, c, (dropped,)).astype(np.float64), want, single, least)


def test_one_power_of_two_for_a_matrix_is_seen():
    for kind, steps in (("rows", 1), ("rows", 5), ("columns", 5), ("columns", 20)):
        x = op.unequal(kind, (96, 200), 1e-8, 5)
        c, want, single = _forms(x, steps, om.STEP)
        with pytest.raises(AssertionError, match="off by"):
            op.check(op.in_pieces(x, steps, c, by_rows=False).astype(np.float64), want, single)


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_cases_take_every_tile(tmp_path):
    exe = tmp_path / "ortho_tile_check"
    subprocess.run([HIPCC, "-std=c++17", "-O2", "--cuda-host-only", "-x", "hip", "-I", CSRC,
                    os.path.join(HERE, "ortho_tile_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, timeout=300)
    args = [str(v) for b, M, N in op.TILE_CASES for v in (b, min(M, N), max(M, N))]
    out = subprocess.run([str(exe), *args], check=True, capture_output=True, text=True).stdout
    lines = [line.split() for line in out.splitlines()]
    s, p, last = zip(*lines)
    assert set(s) == {"64x64", "128x128"} and set(p) == {"64x64", "128x128"}
    wide = {t for t, (_, M, N) in zip(last, op.TILE_CASES) if M < N}
    tall = {t for t, (_, M, N) in zip(last, op.TILE_CASES) if M > N}
    assert wide >= {"128x128", "128x256"} and tall >= {"128x128", "128x256"}
    assert {t for t, (b, _, _) in zip(last, op.TILE_CASES) if b > 1} >= {"64x64", "128x256"}, out
