"""sgemm_orthogonalize: argument checks, which precede any runtime call, and the model of the tests
(no GPU needed)."""
import ctypes

import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import orthogonalize_model as om

INVALID, LARGE, READY = ("SGEMM_ERR_INVALID_VALUE", "SGEMM_ERR_TOO_LARGE",
                         "SGEMM_ERR_NOT_INITIALIZED")
ARGS = dict(batch=2, M=5, N=7, steps=5, sets=1, coefficients=om.STEP, eps=1e-7, alpha=1.0, typeX=0,
            X=16, ldx=7, strideX=35, typeY=0, Y=16, ldy=7, strideY=35, workspace=256,
            workspace_bytes=1 << 40)


def _status(**over):
    a = dict(ARGS)
    a.update(over)
    c = a["coefficients"]
    a["coefficients"] = None if c is None else (ctypes.c_float * len(c))(*c)
    return sg.sgemm_status_string(sg.load_library().sgemm_orthogonalize(*a.values(), None))


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(batch=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID),
    (dict(steps=0), INVALID), (dict(steps=65), INVALID), (dict(sets=0), INVALID),
    (dict(sets=2), INVALID), (dict(sets=5, coefficients=om.STEP * 5), READY),
    (dict(coefficients=None), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=0.0), READY), (dict(alpha=float("inf")), INVALID),
    (dict(alpha=float("nan")), INVALID), (dict(alpha=0.0), READY), (dict(typeX=2), INVALID),
    (dict(typeY=3), INVALID), (dict(X=None), INVALID), (dict(Y=None), INVALID),
    (dict(X=18), INVALID), (dict(X=18, typeX=1), READY), (dict(Y=18), INVALID),
    (dict(Y=18, typeY=1), READY), (dict(ldx=6), INVALID), (dict(ldy=6), INVALID),
    (dict(strideX=-1), INVALID), (dict(strideX=0), READY), (dict(strideY=34), INVALID),
    (dict(strideY=0, batch=1), READY), (dict(workspace=None), INVALID),
    (dict(workspace=264), INVALID),
    (dict(batch=0, X=None, Y=None, workspace=None), READY),
    (dict(M=0, X=None, Y=None, workspace=None), READY),
    (dict(ldx=2 ** 31), LARGE), (dict(ldy=2 ** 31, strideY=2 ** 40), LARGE),
    (dict(M=2 ** 20 + 1, strideY=2 ** 40), LARGE), (dict(batch=65536), LARGE),
    (dict(M=2 ** 18, N=2 ** 18, ldx=2 ** 18, ldy=2 ** 18, strideY=2 ** 40), LARGE),
    # polynomials that run away, or are not finite
    (dict(coefficients=(10.0, 10.0, 10.0)), INVALID), (dict(coefficients=(3.0, 0.0, 0.0), steps=10), READY),
    (dict(coefficients=(3.0, 0.0, 0.0), steps=11), INVALID),
    (dict(coefficients=(1.5, -0.5, 0.0), steps=64), READY),
    (dict(coefficients=om.STEP, steps=64), READY),
    (dict(coefficients=(1.0, float("nan"), 1.0)), INVALID),
    (dict(coefficients=(0.0, 0.0, 0.0)), READY),
])
def test_checks(over, status):
    assert _status(**over) == status


def test_workspace():
    size = sg.sgemm_orthogonalize_workspace_size
    assert size(0, 5, 5) == 0 and size(3, 0, 5) == 0
    # Z, twice its transpose, S and P with 32 columns a block of 128 bytes; parts of a norm
    assert size(1, 65, 70) == 65 * 3 * 128 + 2 * 70 * 3 * 128 + 2 * 65 * 3 * 128 + 8 * 5
    assert size(7, 70, 65) == 7 * (65 * 3 * 128 + 2 * 70 * 3 * 128 + 2 * 65 * 3 * 128 + 8 * 5)
    # up to 64 rows or columns: Z and S's parts of 64 columns twice, in single precision
    assert size(1, 40, 70) == 2 * 4 * (40 * 70 + 2 * 40 * 40) + 8 * 3
    assert size(7, 70, 64) == 7 * (2 * 4 * (64 * 70 + 2 * 64 * 64) + 8 * 5)
    need = size(2, 5, 7)
    assert _status(workspace_bytes=need) == READY and _status(workspace_bytes=need - 1) == INVALID
    with pytest.raises(sg.SgemmError):
        size(1, -1, 4)


def test_binding_counts_coefficients():
    with pytest.raises(ValueError, match="3 or 3 \\* steps = 15"):
        sg.sgemm_orthogonalize(1, 2, 2, 5, (1.0, 2.0), 0.0, 1.0, "f32", 16, 2, 4, "f32", 16, 2, 4,
                               stream=0)


def test_model_is_the_polynomial_of_singular_values():
    g = np.random.default_rng(1)
    for shape in ((4, 9), (9, 4), (6, 6), (1, 5)):
        x = g.standard_normal(shape)
        y, _ = om.orthogonalize(x, 5, om.STEP, 1e-7, 2.0)
        u, s, v = np.linalg.svd(x / (np.linalg.norm(x) + 1e-7), full_matrices=False)
        a, b, c = (float(np.float32(k)) for k in om.STEP)
        for _ in range(5):
            s = a * s + b * s ** 3 + c * s ** 5
        assert np.abs(2 * (u * s) @ v - y).max() < 1e-12


def test_bound_holds_for_single_precision():
    """The bound with 24-bit operands covers a plain single-precision computation."""
    g = np.random.default_rng(2)
    for m, n in ((30, 50), (64, 64), (100, 300)):
        x = g.standard_normal((m, n)).astype(np.float32)
        z = x / np.float32(np.linalg.norm(x) + 1e-7)
        for _ in range(5):
            s = z @ z.T
            z = np.float32(om.STEP[0]) * z + (np.float32(om.STEP[1]) * s
                                              + np.float32(om.STEP[2]) * (s @ s)) @ z
        y, off = om.orthogonalize(x, 5, om.STEP, 1e-7, 1.0, bits=24)
        assert np.linalg.norm(z - y) <= off
        assert off < 0.02 * np.linalg.norm(y)  # and says something
