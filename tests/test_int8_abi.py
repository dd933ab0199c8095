"""8-bit integer operands: argument checks, which precede any runtime call (no GPU needed)."""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import int8_model as i8

INVALID, LARGE, READY = ("SGEMM_ERR_INVALID_VALUE", "SGEMM_ERR_TOO_LARGE",
                         "SGEMM_ERR_NOT_INITIALIZED")


def _name(rc):
    return sg.sgemm_status_string(rc)


def test_sizes():
    assert sg.sgemm_int8_codes_size(3, 1) == 3 * 128
    assert sg.sgemm_int8_codes_size(3, 128) == 3 * 128
    assert sg.sgemm_int8_codes_size(3, 129) == 3 * 256
    assert sg.sgemm_int8_codes_size(0, 5) == 0 and sg.sgemm_int8_codes_size(5, 0) == 0
    assert sg.sgemm_int8_workspace_size("int8", 100, 100) == 0
    assert sg.sgemm_int8_workspace_size("f32", 100, 100) == 100 * (128 + 4)
    lib = sg.load_library()
    assert _name(lib.sgemm_int8_codes_size(-1, 5)) == INVALID
    assert _name(lib.sgemm_int8_codes_size(5, 2 ** 17)) == LARGE
    assert _name(lib.sgemm_int8_workspace_size(2, 5, 5)) == INVALID
    assert _name(lib.sgemm_int8_workspace_size(0, 2 ** 31, 5)) == LARGE
    with pytest.raises(sg.SgemmError):
        sg.sgemm_int8_codes_size(-1, 5)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(trans=2), INVALID), (dict(type=2), INVALID), (dict(type=3), INVALID),
    (dict(rows=-1), INVALID), (dict(K=-1), INVALID), (dict(ldx=6), INVALID),
    (dict(trans=1, ldx=7), INVALID), (dict(trans=1, ldx=8), READY), (dict(ldq=127), INVALID),
    (dict(ldq=136), INVALID), (dict(ldq=144), READY), (dict(K=129, ldx=129), INVALID),
    (dict(X=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(codes=24), INVALID), (dict(scales=18), INVALID), (dict(X=18), INVALID),
    (dict(X=18, type=1), READY), (dict(X=17, type=1), INVALID),
    (dict(rows=0, X=None, codes=None, scales=None), READY),
    (dict(K=2 ** 17, ldx=2 ** 17, ldq=2 ** 17), LARGE),
    (dict(K=2 ** 17 - 1, ldx=2 ** 17, ldq=2 ** 17), READY),
    (dict(ldx=2 ** 31), LARGE), (dict(ldq=2 ** 31), LARGE), (dict(rows=2 ** 24), LARGE),
    (dict(rows=2 ** 24 - 1), READY),
])
def test_cast_checks(over, status):
    a = dict(trans=0, rows=8, K=7, type=0, X=16, ldx=7, codes=16, ldq=128, scales=16)
    a.update(over)
    assert _name(sg.load_library().sgemm_int8_quantize(*a.values(), None)) == status


PRODUCT = dict(M=8, N=5, K=7, alpha=1.0, typeA=0, A=16, lda=7, scalesA=None, B=16, ldb=128,
               scalesB=16, beta=0.0, typeC=0, C=16, ldc=5)
WORKSPACE = dict(workspace=256, workspace_bytes=8 * 132)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(typeA=2), INVALID), (dict(typeA=4), INVALID), (dict(typeC=3), INVALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(lda=6), INVALID),
    (dict(ldc=4), INVALID), (dict(ldb=112), INVALID), (dict(ldb=130), INVALID),
    (dict(ldb=144), READY), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(scalesB=None), INVALID), (dict(C=None), INVALID), (dict(B=24), INVALID),
    (dict(scalesB=18), INVALID), (dict(C=18), INVALID), (dict(C=18, typeC=1), READY),
    (dict(A=18), INVALID), (dict(A=18, typeA=1), READY),
    (dict(workspace=None), INVALID), (dict(workspace=264), INVALID),
    (dict(workspace_bytes=8 * 132 - 1), INVALID),
    # held A: lda is the codes' leading dimension, no workspace
    (dict(typeA=3, lda=128, scalesA=16, workspace=None, workspace_bytes=0), READY),
    (dict(typeA=3, lda=112, scalesA=16), INVALID), (dict(typeA=3, lda=136, scalesA=16), INVALID),
    (dict(typeA=3, lda=128), INVALID), (dict(typeA=3, lda=128, scalesA=16, A=24), INVALID),
    (dict(typeA=3, lda=128, scalesA=18), INVALID),
    (dict(typeA=3, lda=2 ** 22, scalesA=16), LARGE), (dict(ldb=2 ** 22), LARGE),
    # nothing is read: alpha or K is zero
    (dict(alpha=0.0, A=None, B=None, scalesB=None, workspace=None), READY),
    (dict(K=0, A=None, B=None, scalesB=None, workspace=None, ldb=0), READY),
    (dict(M=0, A=None, B=None, scalesB=None, C=None, workspace=None), READY),
    (dict(K=2 ** 17, lda=2 ** 18, ldb=2 ** 18), LARGE), (dict(M=2 ** 31), LARGE),
    (dict(N=2 ** 31, ldc=2 ** 31), LARGE), (dict(lda=2 ** 31), LARGE), (dict(ldc=2 ** 27), LARGE),
    (dict(M=2 ** 24, workspace_bytes=2 ** 50), LARGE),
    (dict(M=16 * 2 ** 12, N=16 * 2 ** 12, ldc=2 ** 26, workspace_bytes=2 ** 50), LARGE),
])
def test_product_checks(over, status):
    lib = sg.load_library()
    a = dict(PRODUCT, **WORKSPACE)
    a.update(over)
    assert _name(lib.sgemm_run_int8(*a.values(), None)) == status
    if a["M"] > 1000 or a["N"] > 1000:  # the grouped form counts a few more rows of tiles
        return
    ws, nbytes = a.pop("workspace"), a.pop("workspace_bytes")
    run = lib.sgemm_run_int8_grouped
    assert _name(run(3, *a.values(), 16, ws, nbytes, None)) == status
    if status == READY:
        assert _name(run(-1, *a.values(), 16, ws, nbytes, None)) == INVALID
        assert _name(run(0, *a.values(), None, ws, nbytes, None)) == READY
        if a["M"]:
            assert _name(run(3, *a.values(), None, ws, nbytes, None)) == INVALID
            assert _name(run(3, *a.values(), 12, ws, nbytes, None)) == INVALID
        assert _name(run(4096, *a.values(), 16, ws, nbytes, None)) == READY
        assert _name(run(4097, *a.values(), 16, ws, nbytes, None)) == LARGE


def test_model_of_the_cast():
    """The numpy model against the definition taken word by word, in exact fractions."""
    from fractions import Fraction
    g = np.random.default_rng(1)
    x = g.standard_normal((20, 50)).astype(np.float32)
    x[:10] = np.rint(x[:10] * 64) / 2
    x[:10, 0] = 127
    codes, scales = i8.quantize(x)
    for row, q, s in zip(x, codes, scales):
        assert s == np.float32(np.abs(row).max()) / np.float32(127)
        for v, c in zip(row, q):
            assert round(Fraction(float(v)) / Fraction(float(s))) == c  # round: halves to even
    assert (codes[:, 50:] == 0).all()
