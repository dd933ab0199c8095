"""sgemm_orthogonalize on every tile it has, and on matrices whose rows and columns are of unequal
size, held to the formula in 64 bits by what the formula in single precision is off by
(tests/orthogonalize_pieces.py)."""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import orthogonalize_model as om
import orthogonalize_pieces as op

pytestmark = pytest.mark.gpu
S_Z, SS_Z, ONLY_Z = (0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (1.5, 0.0, 0.0)


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


def _type(kind):
    import torch
    return torch.float32 if kind == "f32" else torch.bfloat16


def _run(x, steps, coefficients, kind="f32", out="f32", pad=0, in_place=False, alpha=1.0):
    """x, a tensor of matrices, through the library, rows and matrices `pad` apart; what lies
    between them has to stay."""
    import torch
    B, M, N = x.shape
    ld = N + pad
    stride = M * ld + 3 * pad
    X = torch.full((B * stride,), float("nan"), dtype=_type(kind), device="cuda")
    inside = torch.zeros_like(X, dtype=torch.bool)

    def body(t):
        return t.as_strided((B, M, N), (stride, ld, 1))

    body(X)[:] = x
    body(inside)[:] = True
    Y = X if in_place else torch.full((B * stride,), 7.0, dtype=_type(out), device="cuda")
    before = Y.clone()
    need = sg.sgemm_orthogonalize_workspace_size(B, M, N)
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    sg.sgemm_orthogonalize(B, M, N, steps, coefficients, 0.0, alpha, kind, X, ld, stride, out, Y,
                           ld, stride, ws, need)
    assert (ws[need:] == 0xFF).all()
    same = (Y == before) | (Y.isnan() & before.isnan())
    assert same[~inside].all()
    return body(Y).clone()


def _check(x, y, steps, coefficients):
    """Each matrix of y against the formula on x, both forms on the GPU."""
    import torch
    c = op.singles(coefficients)

    def matmul(a, b):
        return torch.matmul(a.contiguous(), b.contiguous())

    for one, got in zip(x, y):
        unit = one.double() / one.double().norm()
        want = op.formula(unit, steps, c, matmul, lambda v: v)
        single = op.formula(unit, steps, c, matmul, lambda v: v.float()).double()
        least = op.least_of_p(unit.cpu().numpy()) if coefficients == SS_Z else 0.0
        op.check(got.double().cpu().numpy(), want.cpu().numpy(), single.cpu().numpy(), least)


def _values(shape, kind="f32", seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return x.to(_type(kind)).float()


@pytest.mark.parametrize("coefficients,steps", [(om.STEP, 5), (ONLY_Z, 1), (S_Z, 1), (SS_Z, 1)])
@pytest.mark.parametrize("case", op.TILE_CASES)
def test_every_tile(case, coefficients, steps):
    x = _values(case)
    _check(x, _run(x, steps, coefficients), steps, coefficients)


@pytest.mark.parametrize("case", [(3, 65, 130), (2, 130, 65), (2, 257, 300), (1, 129, 2050)])
@pytest.mark.parametrize("coefficients,steps", [(om.STEP, 5), (ONLY_Z, 1), (S_Z, 1), (SS_Z, 1)])
def test_small_ones(case, coefficients, steps):
    test_every_tile(case, coefficients, steps)


@pytest.mark.parametrize("case", op.TILE_CASES + [(2, 90, 141), (2, 141, 90), (3, 40, 70)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_strides_types_and_in_place(case, kind):
    """A bfloat16 result is the single-precision one, rounded; in place the bits are the same."""
    import torch
    x = _values(case, kind, 1)
    plain = _run(x, 5, om.STEP, kind)
    _check(x, plain, 5, om.STEP)
    for pad in (1, 8):
        assert torch.equal(_run(x, 5, om.STEP, kind, pad=pad), plain)
    assert torch.equal(_run(x, 5, om.STEP, kind, "bf16", pad=3), plain.bfloat16())
    want = _run(x, 5, om.STEP, kind, kind, alpha=0.25)
    assert torch.equal(want, (plain * 0.25).to(_type(kind)))
    assert torch.equal(_run(x, 5, om.STEP, kind, kind, pad=5, in_place=True, alpha=0.25), want)


@pytest.mark.parametrize("size", [1e-3, 1e-6, 1e-8])
@pytest.mark.parametrize("kind", ["rows", "columns", "both", "graded", "few"])
@pytest.mark.parametrize("shape", [(2, 96, 200), (2, 200, 96), (1, 100, 100), (1, 700, 515),
                                   (2, 33, 90), (2, 300, 64)])
def test_rows_and_columns_of_unequal_size(shape, kind, size):
    import torch
    x = torch.from_numpy(op.unequal(kind, shape, size, 3)).cuda()
    for steps in (1, 5):
        _check(x, _run(x, steps, om.STEP), steps, om.STEP)


# Past 8 steps the sizes are looked at again, at 8, 16, 24 ...
@pytest.mark.parametrize("coefficients,steps", [
    (om.STEP, 9), (om.STEP, 20), ((1.875, -1.25, 0.375), 40), ((1.5, -0.5, 0.0), 64),
    (om.STEP * 12 + (1.875, -1.25, 0.375) * 5, 17)])
@pytest.mark.parametrize("kind", ["rows", "columns"])
@pytest.mark.parametrize("shape", [(2, 96, 200), (2, 200, 96), (3, 130, 1403)])
def test_many_steps(shape, kind, coefficients, steps):
    import torch
    x = torch.from_numpy(op.unequal(kind, shape, 1e-6, 4)).cuda()
    _check(x, _run(x, steps, coefficients), steps, coefficients)


@pytest.mark.parametrize("kind", ["both", "few"])
@pytest.mark.parametrize("shape", [(2, 96, 200), (2, 200, 96), (3, 130, 1403)])
def test_eight_steps_of_unequal_rows_and_columns(shape, kind):
    test_many_steps(shape, kind, om.STEP, 8)


def test_a_long_matrix_whose_columns_share_exponents():
    """More columns than the exponents have room for: 2 of them have one."""
    import torch
    for shape in ((1, 65, 13001), (1, 13001, 65), (1, 70, 40003)):
        x = _values(shape, seed=8)
        x[:, ::2] *= 1e-5 if shape[1] < shape[2] else 1.0
        for steps in (1, 5, 10):
            _check(x, _run(x, steps, om.STEP), steps, om.STEP)
        assert torch.equal(_run(x.repeat(2, 1, 1), 5, om.STEP)[1], _run(x, 5, om.STEP)[0])


def test_zero_rows_and_columns():
    import torch
    for shape in ((1, 100, 230), (1, 230, 100), (1, 1001, 1203)):
        x = _values(shape, seed=6)
        x[:, 5], x[:, :, 17] = 0, 0
        y = _run(x, 5, om.STEP)
        assert (y[:, 5] == 0).all() and (y[:, :, 17] == 0).all()
        _check(x[:, 6:, 18:], _run(x[:, 6:, 18:].contiguous(), 5, om.STEP), 5, om.STEP)
        keep_r = torch.arange(shape[1], device="cuda") != 5
        keep_c = torch.arange(shape[2], device="cuda") != 17
        _check(x[:, keep_r][:, :, keep_c], y[:, keep_r][:, :, keep_c], 5, om.STEP)


@pytest.mark.parametrize("shape,steps", [((2, 90, 141), 18), ((4, 1000, 1000), 9), ((1, 1501, 2203), 5)])
def test_replayed_with_other_matrices(shape, steps):
    """A captured call, its sizes looked at again on the way, replayed with rows of other sizes and a
    workspace that something else has used in between."""
    import torch
    B, M, N = shape
    X, Y = _values(shape, seed=9), torch.empty(shape, device="cuda")
    need = sg.sgemm_orthogonalize_workspace_size(B, M, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def body():
        sg.sgemm_orthogonalize(B, M, N, steps, om.STEP, 0.0, 1.0, "f32", X, N, M * N, "f32", Y, N,
                               M * N, ws, need)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for r in range(4):
        X[:, r::3] *= 1e-4
        X[:, :, r::5] *= 30
        body()
        torch.cuda.synchronize()
        want = Y.clone()
        Y.fill_(9)
        ws.fill_(255 - 85 * r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own, beside a batch of broadcast matrices."""
    import torch
    shapes = [(3, 130, 1403), (1, 700, 515)]
    xs = [_values(s, seed=i) for i, s in enumerate(shapes)]
    want = [_run(x, 10, om.STEP) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            B, M, N = x.shape
            with torch.cuda.stream(s):
                Y = torch.empty_like(x)
                need = sg.sgemm_orthogonalize_workspace_size(B, M, N)
                ws = torch.empty(need, dtype=torch.uint8, device="cuda")
                sg.sgemm_orthogonalize(B, M, N, 10, om.STEP, 0.0, 1.0, "f32", x, N, M * N, "f32", Y,
                                       N, M * N, ws, need)
            got.append((Y, ws))
        torch.cuda.synchronize()
        for (Y, _), w in zip(got, want):
            assert torch.equal(Y, w)
    x = xs[1]
    B, M, N = 4, x.shape[1], x.shape[2]
    Y = torch.empty(B, M, N, device="cuda")
    need = sg.sgemm_orthogonalize_workspace_size(B, M, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    sg.sgemm_orthogonalize(B, M, N, 10, om.STEP, 0.0, 1.0, "f32", x, N, 0, "f32", Y, N, M * N, ws, need)
    for y in Y:
        assert torch.equal(y, want[1][0])
