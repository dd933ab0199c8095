"""Entry points for products grouped by expert and for microscaled 4-bit
operands: argument checks, which precede any runtime call (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

import dense_fp32_matrix_03_amd as sg

INVALID, LARGE, READY = ("SGEMM_ERR_INVALID_VALUE", "SGEMM_ERR_TOO_LARGE",
                         "SGEMM_ERR_NOT_INITIALIZED")


def _name(rc):
    return sg.sgemm_status_string(rc)


def _grouped(**over):
    a = dict(transB=0, groups=3, M=8, N=5, K=7, alpha=1.0, A=16, lda=7, B=16, ldb=5, strideB=35,
             beta=0.0, C=16, ldc=5, offsets=16)
    a.update(over)
    return _name(sg.load_library().sgemm_run_grouped(*a.values(), None))


@pytest.mark.parametrize("over,status", [
    ({}, READY),
    (dict(transB=2), INVALID), (dict(groups=-1), INVALID), (dict(M=-1), INVALID),
    (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(lda=6), INVALID), (dict(ldb=4), INVALID), (dict(ldc=4), INVALID),
    (dict(transB=1, ldb=6), INVALID), (dict(transB=1, ldb=7), READY),
    (dict(strideB=-1), INVALID), (dict(strideB=0), READY),
    (dict(C=None), INVALID), (dict(offsets=None), INVALID), (dict(A=None), INVALID),
    (dict(B=None), INVALID), (dict(offsets=12), INVALID), (dict(C=18), INVALID),
    (dict(A=18), INVALID), (dict(B=18), INVALID),
    (dict(A=None, B=None, alpha=0.0), READY), (dict(A=None, B=None, K=0), READY),
    (dict(A=None, B=None, C=None, offsets=None, groups=0), READY),
    (dict(A=None, B=None, C=None, offsets=None, M=0), READY),
    (dict(groups=4096), READY), (dict(groups=4097), LARGE),
    (dict(M=2 ** 31), LARGE), (dict(lda=2 ** 22), LARGE), (dict(ldb=2 ** 22), LARGE),
    (dict(lda=2 ** 22, K=0), READY), (dict(ldc=2 ** 27), LARGE), (dict(ldc=2 ** 27 - 1), READY),
    # one 256-thread work-group per 16 x 64 block, and one more for each group
    (dict(M=2 ** 27, N=64, ldb=64, ldc=64), READY),
    (dict(M=2 ** 28, N=64, ldb=64, ldc=64), LARGE),
])
def test_grouped_checks(over, status):
    assert _grouped(**over) == status


def _grouped_k(**over):
    a = dict(groups=3, M=8, N=5, K=7, alpha=1.0, A=16, lda=8, B=16, ldb=5, beta=0.0, C=16, ldc=5,
             strideC=40, offsets=16)
    a.update(over)
    return _name(sg.load_library().sgemm_run_grouped_k(*a.values(), None))


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(groups=-1), INVALID), (dict(M=-1), INVALID), (dict(K=-1), INVALID),
    (dict(lda=7), INVALID), (dict(ldb=4), INVALID), (dict(ldc=4), INVALID),
    (dict(strideC=39), INVALID), (dict(strideC=0, groups=1), READY), (dict(strideC=-1), INVALID),
    (dict(C=None), INVALID), (dict(offsets=None), INVALID), (dict(A=None), INVALID),
    (dict(A=None, B=None, K=0), READY), (dict(A=None, B=None, alpha=0.0), READY),
    (dict(offsets=20), INVALID), (dict(groups=4097), LARGE), (dict(lda=2 ** 22), LARGE),
    (dict(ldc=2 ** 27, strideC=2 ** 30), LARGE), (dict(K=2 ** 30 + 1), LARGE),
    (dict(K=2 ** 30), READY),
    (dict(groups=1024, M=4096, N=4096, lda=4096, ldb=4096, ldc=4096, strideC=2 ** 24), LARGE),
    (dict(groups=512, M=4096, N=4096, lda=4096, ldb=4096, ldc=4096, strideC=2 ** 24), READY),
])
def test_grouped_k_checks(over, status):
    assert _grouped_k(**over) == status


def test_mxfp4_sizes():
    assert sg.sgemm_mxfp4_codes_size(3, 1) == 3 * 64
    assert sg.sgemm_mxfp4_codes_size(3, 128) == 3 * 64
    assert sg.sgemm_mxfp4_codes_size(3, 129) == 3 * 128
    assert sg.sgemm_mxfp4_scales_size(3, 129) == 3 * 8
    assert sg.sgemm_mxfp4_codes_size(0, 5) == 0 and sg.sgemm_mxfp4_codes_size(5, 0) == 0
    assert sg.sgemm_mxfp4_workspace_size("mxfp4", 100, 100) == 0
    assert sg.sgemm_mxfp4_workspace_size("f32", 100, 100) == 100 * (64 + 4)
    assert sg.sgemm_mxfp4_workspace_size("bf16", 100, 100) == 100 * (64 + 4)
    lib = sg.load_library()
    assert _name(lib.sgemm_mxfp4_codes_size(-1, 5)) == INVALID
    assert _name(lib.sgemm_mxfp4_scales_size(5, 2 ** 21 + 1)) == LARGE
    assert _name(lib.sgemm_mxfp4_workspace_size(3, 5, 5)) == INVALID
    assert _name(lib.sgemm_mxfp4_workspace_size(0, 2 ** 31, 5)) == LARGE
    with pytest.raises(sg.SgemmError):
        sg.sgemm_mxfp4_codes_size(-1, 5)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(trans=2), INVALID), (dict(type=2), INVALID), (dict(type=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(K=-1), INVALID), (dict(ldx=6), INVALID),
    (dict(trans=1, ldx=7), INVALID), (dict(trans=1, ldx=8), READY), (dict(lds=7), INVALID),
    (dict(X=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(codes=24), INVALID), (dict(scales=18), INVALID), (dict(X=18), INVALID),
    (dict(X=18, type=1), READY), (dict(X=17, type=1), INVALID),
    (dict(rows=0, X=None, codes=None, scales=None), READY),
    (dict(K=2 ** 21 + 1, ldx=2 ** 22), LARGE), (dict(lds=2 ** 31), LARGE),
    (dict(rows=2 ** 20, K=2 ** 21, ldx=2 ** 21, lds=2 ** 20), LARGE),
])
def test_mxfp4_cast_checks(over, status):
    a = dict(trans=0, rows=8, K=7, type=0, X=16, ldx=7, codes=16, scales=16, lds=8)
    a.update(over)
    lib = sg.load_library()
    assert _name(lib.sgemm_mxfp4_quantize(*a.values(), None)) == status
    t, r, k, ty, X, ldx, c, s, lds = a.values()
    assert _name(lib.sgemm_mxfp4_dequantize(t, r, k, c, s, lds, ty, X, ldx, None)) == status


PRODUCT = dict(M=8, N=5, K=7, alpha=1.0, typeA=0, A=16, lda=7, scalesA=None, B=16, scalesB=16,
               ldsb=15, beta=0.0, typeC=0, C=16, ldc=5)
WORKSPACE = dict(workspace=256, workspace_bytes=8 * 68)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(typeA=3), INVALID), (dict(typeC=2), INVALID), (dict(M=-1), INVALID),
    (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(lda=6), INVALID), (dict(ldc=4), INVALID),
    (dict(ldsb=4), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(scalesB=None), INVALID), (dict(C=None), INVALID), (dict(B=24), INVALID),
    (dict(scalesB=18), INVALID), (dict(C=18), INVALID), (dict(C=18, typeC=1), READY),
    (dict(A=18), INVALID), (dict(A=18, typeA=1), READY),
    (dict(workspace=None), INVALID), (dict(workspace=264), INVALID),
    (dict(workspace_bytes=8 * 68 - 1), INVALID),
    # held A: lda is the scales' leading dimension, no workspace
    (dict(typeA=2, lda=8, scalesA=16, workspace=None, workspace_bytes=0), READY),
    (dict(typeA=2, lda=7, scalesA=16), INVALID), (dict(typeA=2, lda=8), INVALID),
    (dict(typeA=2, lda=8, scalesA=16, A=24), INVALID),
    (dict(typeA=2, lda=8, scalesA=18), INVALID),
    # nothing is read: alpha or K is zero
    (dict(alpha=0.0, A=None, B=None, scalesB=None, workspace=None), READY),
    (dict(K=0, A=None, B=None, scalesB=None, workspace=None), READY),
    (dict(M=0, A=None, B=None, scalesB=None, C=None, workspace=None), READY),
    (dict(K=2 ** 21 + 1, lda=2 ** 22), LARGE), (dict(M=2 ** 31), LARGE),
    (dict(ldsb=2 ** 31), LARGE), (dict(ldc=2 ** 27), LARGE),
])
def test_mxfp4_product_checks(over, status):
    lib = sg.load_library()
    a = dict(PRODUCT, **WORKSPACE)
    a.update(over)
    assert _name(lib.sgemm_run_mxfp4(*a.values(), None)) == status
    ws, nbytes = a.pop("workspace"), a.pop("workspace_bytes")
    if a["ldsb"] == 15:  # enough for three groups of five rows
        run = lib.sgemm_run_mxfp4_grouped
        assert _name(run(3, *a.values(), 16, ws, nbytes, None)) == status
        if status == READY:
            assert _name(run(-1, *a.values(), 16, ws, nbytes, None)) == INVALID
            assert _name(run(0, *a.values(), None, ws, nbytes, None)) == READY
            few = dict(a, ldsb=14)
            assert _name(run(3, *few.values(), 16, ws, nbytes, None)) == INVALID
            if a["M"]:
                assert _name(run(3, *a.values(), None, ws, nbytes, None)) == INVALID
                assert _name(run(3, *a.values(), 12, ws, nbytes, None)) == INVALID
            many = dict(a, ldsb=4097 * 5)
            assert _name(run(4097, *many.values(), 16, ws, nbytes, None)) == LARGE


def test_binding_checks_offsets():
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError, match="int64"):
        sg._offsets(torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        sg._offsets(torch.zeros(8, dtype=torch.int64)[::2])
    assert sg._offsets(4096) == 4096


# ------------------------------------------------------ the map of work-groups
def _ranges(offsets, M):
    """The rows of each group as the kernels clamp them."""
    out = []
    for s, e in zip(offsets, offsets[1:]):
        first = min(max(s, 0), M)
        out.append((first, first if e < first else min(e, M)))
    return out


HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dense_fp32_matrix_03_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_map_of_tiles_inside_groups(tmp_path):
    """tests/group_map_check.cpp, compiled for the host only: every tile of a
    group is reached once, the divisions are exact, and the launched rows of
    tiles cover any way to divide the rows."""
    exe = tmp_path / "group_map_check"
    subprocess.run([HIPCC, "-std=c++17", "-O2", "--cuda-host-only", "-x", "hip", "-I", CSRC,
                    os.path.join(HERE, "group_map_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "failures 0" in r.stdout


def test_clamped_groups_stay_inside():
    import random
    rng = random.Random(8)
    for _ in range(2000):
        M = rng.randrange(1, 50)
        at = [rng.choice([-2 ** 63, -1, 0, rng.randrange(-60, 120), M, 2 ** 62]) for _ in range(9)]
        for s, e in _ranges(at, M):
            assert 0 <= s <= e <= M


@pytest.mark.parametrize("over,status", [
    # up to 16 rows over more than 2048 k: 512 work-items for 16 columns, so 2^23 blocks are 2^32
    (dict(K=2049), LARGE), (dict(K=2 ** 21), LARGE), (dict(M=1, K=2049), LARGE),
    (dict(K=2049, typeA=2, lda=16, scalesA=16), LARGE),
    (dict(K=2049, N=2 ** 27 - 16), READY), (dict(K=2048), READY), (dict(K=2049, alpha=0.0), READY),
])
def test_mxfp4_work_items_of_few_rows(over, status):
    a = dict(PRODUCT, workspace=256, workspace_bytes=2 ** 40, M=16, N=2 ** 27 - 15,
             ldsb=2 ** 27 - 1, ldc=2 ** 27 - 1, lda=2 ** 21)
    a.update(over)
    assert _name(sg.load_library().sgemm_run_mxfp4(*a.values(), None)) == status


def test_binding_checks_the_number_of_offsets():
    """The kernels read groups + 1 values whatever the tensor holds."""
    torch = pytest.importorskip("torch")
    at = torch.zeros(4, dtype=torch.int64)
    for groups in (4, 5, 4096):
        with pytest.raises(ValueError, match=f"offsets must hold groups \\+ 1 = {groups + 1} values"):
            sg._offsets(at, groups)
        with pytest.raises(ValueError, match="groups"):
            sg.sgemm_run_grouped(0, groups, 8, 5, 7, 1.0, 16, 7, 16, 5, 35, 0.0, 16, 5, at, 0)
        with pytest.raises(ValueError, match="groups"):
            sg.sgemm_run_grouped_k(groups, 8, 5, 7, 1.0, 16, 8, 16, 5, 0.0, 16, 5, 40, at, 0)
        with pytest.raises(ValueError, match="groups"):
            sg.sgemm_run_mxfp4_grouped(groups, 8, 5, 7, 1.0, "f32", 16, 7, None, 16, 16, 5 * groups,
                                       0.0, "f32", 16, 5, at, 256, 8 * 68, 0)
    for groups in (0, 1, 3):  # enough: the next check is the device's
        with pytest.raises(ValueError, match="GPU"):
            sg._offsets(at, groups)
    assert sg._offsets(None, 0) is None and sg._offsets(4096, 4096) == 4096


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_the_kernels_clamp_of_group_rows(tmp_path):
    """tests/group_range_check.cpp, compiled for the host only."""
    exe = tmp_path / "group_range_check"
    subprocess.run([HIPCC, "-std=c++17", "-O2", "--cuda-host-only", "-x", "hip", "-I", CSRC,
                    os.path.join(HERE, "group_range_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "failures 0" in r.stdout
