"""sgemm_route, sgemm_route_backward, sgemm_route_plan and the calls that move rows, against numpy
in 64 bits (tests/route_model.py).

Whole numbers are compared exactly.  Tolerances count roundings, u = 2^-24 each relative to the
value, for range = the spread of a row's logits:
  scores     an exponential's argument is rounded (range u) and expf is off by at most 4 u; a sum of
             up to 16 values a lane and six exchanges (22 u); a quotient and a product (2 u): a
             weight is off by at most (2 range + 40) u of itself.
  gradients  the same twice, with the sum over picks (6 exchanges) and two more products: (4 range
             + 100) u of the sum of the magnitudes of what is added.
A bfloat16 result is off by 2^-8 of its value more.
"""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import mxfp4_model as mx
import route_model as rm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


def _cuda(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _typed(x, kind, ld=None, shift=0):
    """x (float32, 2-D) on the GPU as `kind`, rows ld apart, `shift` elements into a buffer of
    NaN; and the float32 values it holds."""
    import torch
    ld = x.shape[1] if ld is None else ld
    t = torch.float32 if kind == "f32" else torch.bfloat16
    buf = torch.full((shift + x.shape[0] * ld + 8,), float("nan"), dtype=t, device="cuda")
    body = buf[shift:shift + x.shape[0] * ld].view(x.shape[0], ld)
    body[:, :x.shape[1]] = _cuda(x).to(t)
    return buf[shift:], body[:, :x.shape[1]].float().cpu().numpy()


def _range(l):
    f = np.where(np.isfinite(l), l, np.nan).astype(np.float64)
    with np.errstate(all="ignore"):
        return np.nan_to_num(np.nanmax(np.abs(f), 1, keepdims=True)) * 2


def _route(l, topk, kind="f32", score="softmax", bias=None, groups=1, keep=1, top=1, norm=False,
           scale=1.0, pad=0, shift=0):
    import torch
    tokens, experts = l.shape
    d, held = _typed(l, kind, experts + pad, shift)
    picks = torch.full((tokens + 1, topk), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((tokens + 1, topk), 7.0, device="cuda")
    sg.sgemm_route(tokens, experts, topk, score, kind, d, experts + pad,
                   None if bias is None else _cuda(bias), groups, keep, top, norm, scale, picks,
                   weights)
    torch.cuda.synchronize()
    assert (picks[tokens] == 77).all() and (weights[tokens] == 7).all()
    picks, weights = picks[:tokens].cpu().numpy(), weights[:tokens].cpu().numpy()
    want, w = rm.route(score, held, topk, bias, groups, keep, top, norm, scale)
    assert np.array_equal(picks, want), np.argwhere(picks != want)[:5]
    tol = (2 * _range(held) + 40) * U * np.abs(w) + 1e-37
    assert (np.abs(weights - w) <= tol).all(), np.max(np.abs(weights - w) / tol)
    return picks, weights


def _logits(seed, tokens, experts, masked=0):
    g = np.random.default_rng(seed)
    x = (g.standard_normal((tokens, experts)) * 1.5).astype(np.float32)
    x[:, g.permutation(experts)[:masked]] = -np.inf
    return x


SHAPES = [(1, 1, 1), (1, 64, 8), (3, 8, 8), (5, 60, 4), (17, 65, 2), (9, 128, 6), (6, 160, 7),
          (33, 256, 8), (4, 257, 16), (3, 512, 10), (2, 1000, 64), (2, 1024, 1)]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,experts,topk", SHAPES)
def test_route(tokens, experts, topk, kind, score, norm):
    l = _logits(experts, tokens, experts)
    _route(l, topk, kind, score, norm=norm, scale=2.5)
    bias = np.random.default_rng(1).standard_normal(experts).astype(np.float32) * np.float32(0.05)
    _route(l, topk, kind, score, bias, norm=norm, pad=3, shift=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,keep,top,topk", [
    (256, 8, 4, 2, 8), (60, 5, 2, 2, 6), (64, 64, 7, 1, 7), (64, 64, 9, 2, 9), (160, 8, 3, 1, 6),
    (24, 2, 1, 2, 12), (1024, 32, 5, 2, 20), (8, 8, 8, 1, 8), (130, 13, 4, 2, 5)])
def test_route_groups(experts, groups, keep, top, topk, score):
    bias = np.random.default_rng(1).standard_normal(experts).astype(np.float32) * np.float32(0.05)
    for masked in (0, experts // 3, experts - 3):
        l = _logits(experts + groups, 21, experts, masked)
        _route(l, topk, "f32", score, None, groups, keep, top, norm=True)
        _route(l, topk, "bf16", score, bias, groups, keep, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(score):
    g = np.random.default_rng(4)
    l = g.integers(-2, 3, (40, 100)).astype(np.float32)
    l[:5] = 1.0
    b = g.integers(0, 2, 100).astype(np.float32)
    for bias in (None, b, np.zeros(100, np.float32)):
        _route(l, 12, "f32", score, bias)
        _route(l, 12, "bf16", score, bias, groups=10, keep=3, top=2)
    zeros = np.where(np.arange(100) % 2 == 0, np.float32(0.0), np.float32(-0.0))
    _route(np.tile(zeros, (3, 1)), 12, "f32", score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
def test_choices_that_single_precision_cannot_make(score, groups, keep):
    """Biases that undo the scores up to their rounding: the values compared are 1e-8 apart."""
    l = _logits(8, 1, 128)
    for t in range(12):
        one = l + np.float32(0.01 * t)
        bias = (0.75 - rm.scores(score, one[0])).astype(np.float32)
        _route(one, 8, "f32", score, bias, groups, keep, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_disabled_experts(score):
    l = _logits(5, 20, 70, masked=66)
    l[3] = -np.inf
    l[4, :] = -np.inf
    l[4, 69] = 2.0
    for norm in (False, True):
        for bias in (None, np.linspace(-1, 1, 70).astype(np.float32)):
            _route(l, 6, "f32", score, bias, norm=norm)
            _route(l, 6, "f32", score, bias, 7, 2, 2, norm=norm)
    picks, w = _route(np.full((3, 64), -np.inf, np.float32), 8, score=score, norm=True)
    assert (picks == -1).all() and (w == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_apart_logits(score):
    l = _logits(6, 10, 64) * np.float32(40)
    _route(l, 5, "f32", score, norm=True)
    l[:, 7] = 3e38
    l[:, 9] = -3e38
    _route(l, 64, "f32", score, norm=score == "softmax")


def test_rows_with_nan_or_infinity_stay_inside():
    import torch
    l = _logits(7, 12, 60)
    l[:6, 11] = np.nan
    l[6:, 20] = np.inf
    d = _cuda(l)
    picks = torch.empty(12, 5, dtype=torch.int32, device="cuda")
    w = torch.empty(12, 5, device="cuda")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(60, device="cuda")):
            for groups in (1, 6):
                sg.sgemm_route(12, 60, 5, score, "f32", d, 60, bias, groups, min(groups, 2), 2, 1,
                               1.0, picks, w)
                p = picks.cpu().numpy()
                assert ((p >= -1) & (p < 60)).all()
                for row in p:
                    assert len(set(row[row >= 0])) == (row >= 0).sum()
                assert not torch.isfinite(w[:6]).all(1).any()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,experts,topk", SHAPES)
def test_route_backward(tokens, experts, topk, kind, score, norm):
    import torch
    g = np.random.default_rng(tokens)
    for masked, pad in ((0, 0), (min(experts // 3, experts - 1), 5)):
        l = _logits(experts + 1, tokens, experts, masked)
        d, held = _typed(l, kind, experts + pad, pad % 2)
        picks = np.stack([g.permutation(experts)[:topk] for _ in range(tokens)]).astype(np.int32)
        picks[g.random(picks.shape) < 0.1] = -1
        dw = g.standard_normal((tokens, topk)).astype(np.float32)
        want, mag = rm.route_backward(score, held, picks, dw, norm, 2.5)
        dw[picks < 0] = np.nan
        t = torch.float32 if kind == "f32" else torch.bfloat16
        out = torch.full((tokens, experts + pad), 9.0, dtype=t, device="cuda")
        sg.sgemm_route_backward(tokens, experts, topk, score, kind, d, experts + pad, norm, 2.5,
                                _cuda(picks), _cuda(dw), out, experts + pad)
        torch.cuda.synchronize()
        assert (out[:, experts:] == 9).all()
        got = out[:, :experts].float().cpu().numpy()
        tol = (4 * _range(held) + 100) * U * mag + (2.0 ** -8 * np.abs(want) if kind == "bf16" else 0)
        err = np.abs(got - want)
        assert (err <= tol * 1.001 + 1e-37).all(), np.max(err / (tol + 1e-37))


# ------------------------------------------------------------------ the plan
def _plan(picks, first, groups):
    import torch
    pairs = picks.size
    need = sg.sgemm_route_plan_workspace_size(pairs, groups)
    ws = torch.full((need + 16,), 0xCD, dtype=torch.uint8, device="cuda")
    offsets = torch.full((groups + 2,), -7, dtype=torch.int64, device="cuda")
    sources = torch.full((pairs + 1,), -7, dtype=torch.int32, device="cuda")
    places = torch.full((pairs + 1,), -7, dtype=torch.int32, device="cuda")
    sg.sgemm_route_plan(pairs, first, groups, _cuda(picks.reshape(-1)) if pairs else None, offsets,
                        sources, places, ws, need)
    torch.cuda.synchronize()
    assert offsets[-1] == -7 and sources[-1] == -7 and places[-1] == -7
    assert (ws[need:] == 0xCD).all()
    want = rm.plan(picks, first, groups)
    for got, ref in zip((offsets[:-1], sources[:-1], places[:-1]), want):
        assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("groups", [0, 1, 2, 7, 64, 256, 511, 513, 4096])
@pytest.mark.parametrize("pairs", [0, 1, 63, 64, 65, 300, 4095, 4096, 4097, 20000])
def test_plan(pairs, groups):
    g = np.random.default_rng(pairs + groups)
    picks = g.integers(-1, groups + 2, pairs).astype(np.int32)
    _plan(picks, 0, groups)
    _plan(np.minimum(picks, groups // 3), 0, groups)
    _plan(picks, 2, max(groups - 3, 0))


def test_plan_extremes():
    _plan(np.zeros(70000, np.int32), 0, 5)
    _plan(np.full(9000, 4, np.int32), 0, 5)
    _plan(np.full(9000, -1, np.int32), 0, 5)
    g = np.random.default_rng(1)
    _plan(g.choice([-2 ** 31, -1, 0, 1, 2 ** 31 - 1], 5000).astype(np.int32), 0, 4096)
    _plan(g.choice([-2 ** 31, -1, 0, 2 ** 31 - 2, 2 ** 31 - 1], 5000).astype(np.int32),
          2 ** 31 - 3, 4)
    _plan((g.random(2 ** 21 + 5) ** 3 * 256).astype(np.int32), 0, 256)


# ------------------------------------------------------------------ rows
def _rows(seed, shape, kind, ld=None, shift=0):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    return _typed(x, kind, ld, shift)


def _held(x, kind):
    return mx.bf16_floats(mx.bf16_bits(x)) if kind == "bf16" else x


ROWS = [(1, 1, 1), (5, 2, 3), (24, 2, 2048), (7, 6, 777), (64, 3, 64), (3, 8, 8200), (2, 1, 5000),
        (300, 4, 130)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,topk,N", ROWS)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_gather(tokens, topk, N, kind, pad, shift):
    import torch
    g = np.random.default_rng(N)
    pairs = tokens * topk
    rows = pairs + 2
    sources = np.concatenate([g.permutation(pairs), [0, pairs - 1]]).astype(np.int32)
    sources[g.random(rows) < 0.2] = g.choice([-1, pairs, 2 ** 31 - 1, -2 ** 31])
    X, x = _rows(N, (tokens, N), kind, N + pad, shift)
    w = g.standard_normal(pairs).astype(np.float32)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    for weights in (None, w):
        Y = torch.full((rows, N + pad), 5.0, dtype=t, device="cuda")
        sg.sgemm_rows_gather(rows, pairs, topk, N, kind, X, N + pad, _cuda(sources),
                             None if weights is None else _cuda(w), Y, N + pad)
        torch.cuda.synchronize()
        want = np.full((rows, N + pad), 5.0, np.float32)
        ok = (sources >= 0) & (sources < pairs)
        rows_of = x[sources[ok] // topk]
        want[ok, :N] = rows_of if weights is None else _held(w[sources[ok], None] * rows_of, kind)
        assert np.array_equal(Y.float().cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,topk,N", ROWS)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_combine_and_its_gradient(tokens, topk, N, kind, pad, shift):
    import torch
    g = np.random.default_rng(N + 1)
    pairs = tokens * topk
    rows = pairs + 3
    places = g.permutation(rows)[:pairs].astype(np.int32).reshape(tokens, topk)
    places[g.random(places.shape) < 0.2] = g.choice([-1, rows, 2 ** 31 - 1, -2 ** 31])
    places[0] = -1
    here = (places >= 0) & (places < rows)
    X, x = _rows(N, (rows, N), kind, N + pad, shift)
    w = g.standard_normal((tokens, topk)).astype(np.float32)
    w[~here] = np.nan
    safe = np.where(here, places, 0)
    t = torch.float32 if kind == "f32" else torch.bfloat16
    for weights in (None, w):
        ww = np.where(here, 1.0 if weights is None else w, 0.0).astype(np.float64)
        terms = ww[:, :, None] * x[safe]
        want, mag = terms.sum(1), np.abs(terms).sum(1)
        Y = torch.full((tokens, N + pad), 5.0, dtype=t, device="cuda")
        dw_in = None if weights is None else _cuda(w)
        sg.sgemm_rows_combine(tokens, topk, rows, N, kind, X, N + pad, _cuda(places), dw_in, Y,
                              N + pad)
        torch.cuda.synchronize()
        got = Y.float().cpu().numpy()
        assert (got[:, N:] == 5).all() and (got[0, :N] == 0).all()
        # topk fused multiply-adds, then the type's rounding
        tol = topk * U * mag + (2.0 ** -8 * np.abs(want) if kind == "bf16" else 0)
        assert (np.abs(got[:, :N] - want) <= tol * 1.01).all()

        dY, dy = _rows(N + 2, (tokens, N), kind, N + pad, shift)
        dX = torch.full((rows, N + pad), 5.0, dtype=t, device="cuda")
        dw = torch.full((pairs + 1,), 5.0, device="cuda")
        args = (tokens, topk, rows, N, kind)
        sg.sgemm_rows_combine_backward(*args, X, N + pad, dY, N + pad, _cuda(places), dw_in, dX,
                                       N + pad, dw)
        torch.cuda.synchronize()
        want_dx = np.full((rows, N + pad), 5.0, np.float32)
        product = np.repeat(dy[:, None], topk, 1)[here]
        if weights is not None:
            product = _held(w[here][:, None] * product, kind)
        want_dx[places[here], :N] = product
        assert np.array_equal(dX.float().cpu().numpy(), want_dx)
        products = np.where(here[:, :, None], x[safe].astype(np.float64) * dy[:, None], 0.0)
        want_dw, mag_dw = products.sum(2), np.abs(products).sum(2)
        got_dw = dw[:pairs].cpu().numpy().reshape(tokens, topk)
        # a lane's chain of N / 64 products, rounded up to whole loads of 8, and six exchanges
        tol = (N / 64 + 8 + 6) * U * mag_dw
        assert dw[pairs] == 5 and (np.abs(got_dw - want_dw) <= tol * 1.01).all()
        assert (got_dw[~here] == 0).all()

        alone = torch.full_like(dX, 5.0)
        sg.sgemm_rows_combine_backward(*args, None, 0, dY, N + pad, _cuda(places), dw_in, alone,
                                       N + pad, None)
        only = torch.full_like(dw, 5.0)
        sg.sgemm_rows_combine_backward(*args, X, N + pad, dY, N + pad, _cuda(places), dw_in, None,
                                       0, only)
        assert torch.equal(alone, dX) and torch.equal(only, dw)


def test_rows_past_4_gib():
    """Rows of more than 2^32 bytes in all, read and written at their end."""
    import torch
    N = ld = 1 << 20
    rows = 2100
    X = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = (torch.arange(rows, device="cuda") % 100).bfloat16()
    X[:, N - 1] = (torch.arange(rows, device="cuda") % 90).bfloat16()
    at = torch.tensor([rows - 1, 5, rows - 2], dtype=torch.int32, device="cuda")
    Y = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device="cuda")
    sg.sgemm_rows_gather(3, rows, 1, N, "bf16", X, ld, at, None, Y, ld)
    assert torch.equal(Y[:3], X[at.long()]) and (Y[3] == 3).all()
    sg.sgemm_rows_combine(3, 1, rows, N, "bf16", X, ld, at, None, Y, ld)
    assert torch.equal(Y[:3], X[at.long()])
    sg.sgemm_rows_combine_backward(3, 1, rows, N, "bf16", None, 0, X, ld, at, None, Y, ld, None)
    assert torch.equal(Y[at.long()], X[:3]) and (Y[6] == 3).all()


def test_a_row_of_the_largest_length():
    """2^31 - 1 columns: the last piece ends one element before the index would overflow.  Sums
    of small whole numbers are exact."""
    import torch
    N = (1 << 31) - 1
    X = torch.zeros(N, dtype=torch.bfloat16, device="cuda")
    X[0], X[N - 1025], X[N - 1] = 3, 5, 7
    Y = torch.full((N + 8,), 2.0, dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sgemm_rows_gather(1, 1, 1, N, "bf16", X, N, at, None, Y, N)
    assert torch.equal(Y[:N], X) and (Y[N:] == 2).all()
    Y.fill_(2)
    sg.sgemm_rows_combine(1, 1, 1, N, "bf16", X, N, at, None, Y, N)
    assert torch.equal(Y[:N], X) and (Y[N:] == 2).all()
    Y.fill_(2)
    dw = torch.full((1,), 9.0, device="cuda")
    sg.sgemm_rows_combine_backward(1, 1, 1, N, "bf16", X, N, X, N, at, None, Y, N, dw)
    assert torch.equal(Y[:N], X) and (Y[N:] == 2).all() and dw.item() == 9 + 25 + 49


@pytest.mark.parametrize("scale", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scales_that_are_not_finite_leave_missing_picks_at_0(score, scale):
    import torch
    l = np.full((2, 8), -np.inf, np.float32)
    l[0, :2] = 1, 2
    picks, weights = torch.empty(2, 4, dtype=torch.int32, device="cuda"), torch.empty(
        2, 4, device="cuda")
    sg.sgemm_route(2, 8, 4, score, "f32", _cuda(l), 8, None, 1, 1, 1, True, scale, picks, weights)
    weights = weights.cpu().numpy()
    assert picks.cpu().numpy().tolist() == [[1, 0, -1, -1], [-1] * 4]
    assert not weights[0, 2:].any() and not weights[1].any()
    assert np.array_equal(weights[0, :2], np.full(2, scale, np.float32), equal_nan=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
def test_bias_of_infinity(score, groups, keep):
    """-infinity: never picked, like a disabled logit; +infinity: picked first."""
    l = _logits(8, 40, 32)
    b = (np.random.default_rng(9).standard_normal(32) * 0.1).astype(np.float32)
    b[[3, 17]], b[[9, 30]] = -np.inf, np.inf
    picks, _ = _route(l, 6, "f32", score, b, groups, keep, 1)
    assert not np.isin(picks, [3, 17]).any()
    assert (picks[:, :2] == [9, 30]).all()


@pytest.mark.parametrize("pairs,groups", [(2048, 30), (2049, 30), (524288, 7), (700001, 100),
                                          (700001, 4000)])
def test_plan_of_many_pairs(pairs, groups):
    """One chunk and two; all chunks in one step each, and in several."""
    import torch
    picks = np.random.default_rng(pairs).integers(-1, groups + 2, pairs).astype(np.int32)
    need = sg.sgemm_route_plan_workspace_size(pairs, groups)
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    off = torch.full((groups + 2,), -5, dtype=torch.int64, device="cuda")
    sources, places = (torch.full((pairs + 1,), -5, dtype=torch.int32, device="cuda")
                       for _ in range(2))
    sg.sgemm_route_plan(pairs, 0, groups, _cuda(picks), off, sources, places, ws, need)
    torch.cuda.synchronize()
    for got, want, rest in zip((off, sources, places), rm.plan(picks, 0, groups), (-5, -5, -5)):
        got = got.cpu().numpy()
        assert np.array_equal(got[:-1], want) and got[-1] == rest
    assert (ws[need:] == 0xFF).all()


def test_a_million_tokens():
    """Distinct logits, so that the picks are those of a sort."""
    import torch
    tokens, experts, topk = (1 << 20) + 3, 9, 2
    l = torch.rand(tokens, experts, device="cuda").argsort(1).float()
    picks = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
    weights = torch.empty(tokens, topk, device="cuda")
    sg.sgemm_route(tokens, experts, topk, "softmax", "f32", l, experts, None, 1, 1, 1, True, 1.0,
                   picks, weights)
    best, at = l.topk(topk, 1)
    assert torch.equal(picks.long(), at)
    want = best.double().softmax(1)
    assert ((weights - want).abs() <= (2 * 16 + 40) * U * want).all()
    dw = torch.randn(tokens, topk, device="cuda")
    dl = torch.full((tokens, experts), 5.0, device="cuda")
    sg.sgemm_route_backward(tokens, experts, topk, "softmax", "f32", l, experts, True, 1.0, picks, dw,
                            dl, experts)
    d = want * (dw - (dw * want).sum(1, keepdim=True))
    full = torch.zeros(tokens, experts, dtype=torch.float64, device="cuda").scatter_(1, at, d)
    mag = want * (dw.abs() + (dw.abs() * want).sum(1, keepdim=True))
    tol = torch.zeros_like(full).scatter_(1, at, (4 * 16 + 100) * U * mag)
    assert ((dl - full).abs() <= tol).all()
