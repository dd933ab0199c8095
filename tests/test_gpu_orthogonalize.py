"""sgemm_orthogonalize against the formula in 64 bits.  The tolerance is the model's bound on the
Frobenius norm (tests/orthogonalize_model.py), which counts the roundings of the operands and sums
and follows them through the steps; a bfloat16 result is off by 2^-8 of its value more."""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import orthogonalize_model as om

pytestmark = pytest.mark.gpu
TYPES = ("f32", "bf16")


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


def _torch_type(kind):
    import torch
    return torch.float32 if kind == "f32" else torch.bfloat16


def _run(x, kind="f32", out="f32", steps=5, coefficients=om.STEP, eps=1e-7, alpha=1.0, pad=0,
         in_place=False):
    """x (batch, M, N) through the library; rows, matrices and the workspace are padded with values
    that must stay as they are.  Returns (Y, X as held) in float32."""
    import torch
    B, M, N = x.shape
    ld = N + pad
    stride = M * ld + 3 * pad
    X = torch.full((B * stride + 8,), float("nan"), dtype=_torch_type(kind), device="cuda")
    view = X[:B * stride].view(B, stride)[:, :M * ld].view(B, M, ld)
    view[:, :, :N] = torch.from_numpy(x).cuda().to(X.dtype)
    held = view[:, :, :N].float().cpu().numpy()
    Y = X if in_place else torch.full((B * stride + 8,), 7.0, dtype=_torch_type(out), device="cuda")
    before = Y.clone()
    need = sg.sgemm_orthogonalize_workspace_size(B, M, N)
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every format
    sg.sgemm_orthogonalize(B, M, N, steps, coefficients, eps, alpha, kind, X, ld, stride, out, Y, ld,
                           stride, ws, need)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xFF).all()
    got = Y[:B * stride].view(B, stride)[:, :M * ld].view(B, M, ld)[:, :, :N].clone()
    keep = torch.ones_like(Y, dtype=torch.bool)
    keep[:B * stride].view(B, stride)[:, :M * ld].view(B, M, ld)[:, :, :N] = False
    same = (Y == before) | (Y.isnan() & before.isnan())
    assert same[keep].all()
    return got.float().cpu().numpy(), held


def _check(y, held, out="f32", steps=5, coefficients=om.STEP, eps=1e-7, alpha=1.0):
    for got, x in zip(y, held):
        want, off = om.orthogonalize(x, steps, coefficients, float(np.float32(eps)), alpha)
        tol = off + (2.0 ** -8 * np.linalg.norm(want) if out == "bf16" else 0)
        err = np.linalg.norm(got - want)
        assert err <= tol, f"off by {err:.3g}, {err / tol:.3g} of the bound"


def _values(seed, shape):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape)
    x += 2 * g.standard_normal(shape[:-1] + (1,)) * g.standard_normal(shape[:-2] + (1, shape[-1]))
    return (x * 1e-3).astype(np.float32)


SHAPES = [(1, 1, 1), (2, 1, 5), (2, 5, 1), (3, 2, 3), (2, 31, 33), (1, 64, 64), (3, 65, 130),
          (2, 130, 65), (1, 33, 1000), (1, 1000, 33), (2, 257, 300), (1, 256, 512), (1, 500, 700),
          (40, 20, 24), (1, 129, 2050)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_formula(shape, kind, out):
    y, held = _run(_values(sum(shape), shape), kind, out)
    _check(y, held, out)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", [(3, 40, 70), (3, 70, 41), (1, 200, 300), (1, 5, 2000)])
@pytest.mark.parametrize("pad", [1, 8])
def test_strides_and_in_place(shape, kind, pad):
    x = _values(3, shape)
    y, held = _run(x, kind, kind, pad=pad, alpha=0.3)
    _check(y, held, kind, alpha=0.3)
    again, _ = _run(x, kind, kind, pad=pad, alpha=0.3, in_place=True)
    assert np.array_equal(y, again)


@pytest.mark.parametrize("shape", [(2, 64, 100), (1, 150, 90), (1, 300, 310)])
@pytest.mark.parametrize("coefficients,steps", [
    ((1.5, -0.5, 0.0), 1), ((1.5, -0.5, 0.0), 12), (om.STEP, 1), ((1.875, -1.25, 0.375), 8),
    (om.STEP * 3 + (1.875, -1.25, 0.375) * 2, 5), ((0.0, 0.0, 0.0), 2), ((3.0, 0.0, 0.0), 9),
    ((0.01, 0.0, 0.0), 7), ((0.0, 0.0, -2.0), 2), ((40.0, -100.0, 70.0), 1)])
def test_other_polynomials(shape, coefficients, steps):
    y, held = _run(_values(9, shape), steps=steps, coefficients=coefficients, alpha=-2.0)
    _check(y, held, steps=steps, coefficients=coefficients, alpha=-2.0)


@pytest.mark.parametrize("shape", [(1, 60, 80), (1, 200, 130)])
@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-7, 1.0, 1e30, 1e37])
def test_sizes_of_values(shape, size):
    x = (_values(4, shape).astype(np.float64) * 1e3 * size).astype(np.float32)
    y, held = _run(x, eps=0.0)
    _check(y, held, eps=0.0)
    y, held = _run(x, eps=1e-3)
    _check(y, held, eps=1e-3)


def test_zeros_and_matrices_beside_them():
    x = _values(5, (4, 70, 90))
    alone, _ = _run(x[3:])
    x[0] = 0
    x[1, 5, 5] = np.nan
    for eps in (0.0, 1e-7):
        y, held = _run(x, eps=eps)
        assert (y[0] == 0).all() and np.isnan(y[1]).any()
        _check(y[2:], held[2:], eps=eps)
    assert np.array_equal(y[3], alone[0])  # the same bits whatever is around


def test_rank_one_and_orthogonal():
    g = np.random.default_rng(6)
    x = (g.standard_normal((1, 90, 1)) * g.standard_normal((1, 1, 120))).astype(np.float32)
    y, held = _run(x)
    _check(y, held)
    q = np.linalg.qr(g.standard_normal((90, 90)))[0].astype(np.float32)[None]
    y, held = _run(q, steps=3)
    _check(y, held, steps=3)
    one = np.zeros((1, 70, 70), np.float32)
    one[0, 3, 69] = 2.0  # all of the norm in one element: the largest a held matrix has
    y, held = _run(one)
    _check(y, held)


def test_in_a_graph_and_on_another_stream():
    import torch
    B, M, N = 3, 90, 140
    X = torch.from_numpy(_values(7, (B, M, N))).cuda()
    Y = torch.empty_like(X)
    need = sg.sgemm_orthogonalize_workspace_size(B, M, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def body():
        sg.sgemm_orthogonalize(B, M, N, 5, om.STEP, 1e-7, 1.0, "f32", X, N, M * N, "f32", Y, N,
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
        X.mul_(1.5).add_(1e-4 * r)
        body()
        torch.cuda.synchronize()
        want = Y.clone()
        Y.fill_(9)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


@pytest.mark.parametrize("shape", [(1, 1, 1 << 20), (1, 1 << 20, 2), (1, 3, 300001)])
def test_longest_rows(shape):
    y, held = _run(_values(11, shape))
    _check(y, held)


def test_largest_batch():
    shape = (65535, 2, 3)
    y, held = _run(_values(12, shape))
    some = np.r_[0:20, 32760:32780, 65515:65535]
    _check(y[some], held[some])
    # All: values stay below 1.3 and a step's slope below 3.5.  A step adds the errors of three
    # products, each off by 3 2^-22 of its terms (S's and P's by |b| + 2 |c| |S| + |c| |S|^2 < 13
    # of it on the way to Z), below 40 2^-22; five steps' are at most 3.5^5 / 2.5 times that.
    z = held.astype(np.float64)
    z /= np.sqrt((z * z).sum((1, 2), keepdims=True)) + float(np.float32(1e-7))
    a, b, c = (float(np.float32(v)) for v in om.STEP)
    for _ in range(5):
        s = z @ z.transpose(0, 2, 1)
        z = a * z + (b * s + c * s @ s) @ z
    assert np.abs(y - z).max() <= 40 * 3.5 ** 5 * 2.0 ** -22


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", [(2, 64, 65), (2, 65, 64), (1, 64, 1024), (1, 1025, 63),
                                   (3, 33, 2100), (1, 64, 8192), (1, 8193, 40)])
def test_short_matrices(shape, kind, out):
    """A side of at most 64: one slab of columns and several, of one block and several."""
    y, held = _run(_values(21, shape), kind, out, pad=3)
    _check(y, held, out)
