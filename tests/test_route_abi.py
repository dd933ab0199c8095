"""Routing and the movement of rows: argument checks, which precede any runtime call, and the
model of the tests (no GPU needed)."""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import route_model as rm

INVALID, LARGE, READY = ("SGEMM_ERR_INVALID_VALUE", "SGEMM_ERR_TOO_LARGE",
                         "SGEMM_ERR_NOT_INITIALIZED")


def _call(fn, defaults, over):
    a = dict(defaults)
    a.update(over)
    return sg.sgemm_status_string(getattr(sg.load_library(), fn)(*a.values(), None))


ROUTE = dict(tokens=5, experts=12, topk=3, score=0, type=0, logits=16, ldl=12, bias=None, groups=1,
             topk_groups=1, group_top=1, renormalize=0, scale=1.0, picks=16, weights=16)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(score=2), INVALID), (dict(type=2), INVALID), (dict(renormalize=2), INVALID),
    (dict(tokens=-1), INVALID), (dict(experts=0), INVALID), (dict(topk=0), INVALID),
    (dict(topk=13), INVALID), (dict(topk=12), READY), (dict(ldl=11), INVALID),
    (dict(groups=0), INVALID), (dict(groups=5), INVALID), (dict(groups=24), INVALID),
    (dict(groups=4, topk_groups=4), READY), (dict(groups=4, topk_groups=5), INVALID),
    (dict(topk_groups=0), INVALID), (dict(group_top=0), INVALID), (dict(group_top=3), INVALID),
    (dict(experts=1024, ldl=1024, topk=64), READY), (dict(experts=1024, ldl=1024, topk=65), INVALID),
    (dict(experts=1025, ldl=1025), LARGE), (dict(ldl=2 ** 31), LARGE),
    (dict(tokens=2 ** 26), LARGE), (dict(tokens=2 ** 26 - 8), READY),
    (dict(tokens=2 ** 26 - 8, experts=64, ldl=64, topk=33), LARGE),
    (dict(experts=128, ldl=128, groups=128), LARGE), (dict(experts=128, ldl=128, groups=64), READY),
    (dict(logits=None), INVALID), (dict(picks=None), INVALID), (dict(weights=None), INVALID),
    (dict(logits=18), INVALID), (dict(logits=18, type=1), READY), (dict(logits=17, type=1), INVALID),
    (dict(bias=18), INVALID), (dict(bias=20), READY), (dict(picks=18), INVALID),
    (dict(weights=18), INVALID), (dict(tokens=0, logits=None, picks=None, weights=None), READY),
])
def test_route_checks(over, status):
    assert _call("sgemm_route", ROUTE, over) == status


BACK = dict(tokens=5, experts=12, topk=3, score=0, type=0, logits=16, ldl=12, renormalize=0,
            scale=1.0, picks=16, dweights=16, dlogits=16, ldd=12)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(score=-1), INVALID), (dict(type=2), INVALID), (dict(renormalize=-1), INVALID),
    (dict(tokens=-1), INVALID), (dict(topk=13), INVALID), (dict(ldl=11), INVALID),
    (dict(ldd=11), INVALID), (dict(ldd=2 ** 31), LARGE), (dict(experts=1025, ldl=2000, ldd=2000), LARGE),
    (dict(logits=None), INVALID), (dict(picks=None), INVALID), (dict(dweights=None), INVALID),
    (dict(dlogits=None), INVALID), (dict(dlogits=18), INVALID), (dict(dlogits=18, type=1), READY),
    (dict(tokens=0, logits=None, picks=None, dweights=None, dlogits=None), READY),
])
def test_route_backward_checks(over, status):
    assert _call("sgemm_route_backward", BACK, over) == status


PLAN = dict(pairs=10000, first=0, groups=8, picks=16, offsets=16, sources=16, places=16,
            workspace=16, workspace_bytes=1 << 30)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(pairs=-1), INVALID), (dict(first=-1), INVALID), (dict(groups=-1), INVALID),
    (dict(pairs=2 ** 31), LARGE), (dict(groups=4097), LARGE), (dict(first=2 ** 31), LARGE),
    (dict(picks=None), INVALID), (dict(offsets=None), INVALID), (dict(offsets=12), INVALID),
    (dict(sources=None), INVALID), (dict(places=18), INVALID), (dict(workspace=None), INVALID),
    (dict(workspace=24), INVALID), (dict(workspace_bytes=8 * 4 * 5 - 1), INVALID),
    (dict(workspace_bytes=8 * 4 * 5), READY),
    (dict(pairs=2048, workspace=None, workspace_bytes=0), READY),
    (dict(pairs=0, picks=None, sources=None, places=None, workspace=None), READY),
])
def test_plan_checks(over, status):
    assert _call("sgemm_route_plan", PLAN, over) == status


def test_plan_workspace():
    assert sg.sgemm_route_plan_workspace_size(2048, 8) == 0
    assert sg.sgemm_route_plan_workspace_size(2049, 8) == 2 * 8 * 4
    assert sg.sgemm_route_plan_workspace_size(2 ** 31 - 1, 4096) <= 256 * 4096 * 4
    with pytest.raises(sg.SgemmError):
        sg.sgemm_route_plan_workspace_size(5, 4097)


GATHER = dict(rows=9, pairs=12, topk=3, N=7, type=0, X=16, ldx=7, sources=16, weights=None, Y=16,
              ldy=7)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(rows=-1), INVALID), (dict(pairs=-3), INVALID), (dict(topk=0), INVALID),
    (dict(pairs=13), INVALID), (dict(N=-1), INVALID), (dict(type=2), INVALID),
    (dict(ldx=6), INVALID), (dict(ldy=6), INVALID), (dict(X=None), INVALID), (dict(Y=None), INVALID),
    (dict(sources=None), INVALID), (dict(weights=18), INVALID), (dict(X=18), INVALID),
    (dict(X=18, Y=18, type=1), READY), (dict(rows=0, X=None, Y=None, sources=None), READY),
    (dict(N=0, X=None, Y=None, sources=None), READY), (dict(pairs=0, X=None), READY),
    (dict(rows=2 ** 31), LARGE), (dict(pairs=3 * 2 ** 30), LARGE), (dict(ldx=2 ** 31), LARGE),
    (dict(ldy=2 ** 31), LARGE), (dict(rows=2 ** 26), LARGE), (dict(rows=2 ** 26 - 8), READY),
    (dict(rows=2 ** 25, N=1025, ldx=1025, ldy=1025), LARGE),
])
def test_gather_checks(over, status):
    assert _call("sgemm_rows_gather", GATHER, over) == status


COMBINE = dict(tokens=4, topk=3, rows=9, N=7, type=0, X=16, ldx=7, places=16, weights=None, Y=16,
               ldy=7)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(tokens=-1), INVALID), (dict(rows=-1), INVALID), (dict(topk=0), INVALID),
    (dict(N=-1), INVALID), (dict(type=3), INVALID), (dict(ldx=6), INVALID), (dict(ldy=6), INVALID),
    (dict(X=None), INVALID), (dict(rows=0, X=None), READY), (dict(Y=None), INVALID),
    (dict(places=None), INVALID), (dict(weights=18), INVALID),
    (dict(tokens=0, X=None, Y=None, places=None), READY),
    (dict(rows=2 ** 31), LARGE), (dict(topk=2 ** 30), LARGE), (dict(tokens=2 ** 26), LARGE),
])
def test_combine_checks(over, status):
    assert _call("sgemm_rows_combine", COMBINE, over) == status


COMBINE_BACK = dict(tokens=4, topk=3, rows=9, N=7, type=0, X=16, ldx=7, dY=16, lddy=7, places=16,
                    weights=None, dX=16, lddx=7, dweights=16)


@pytest.mark.parametrize("over,status", [
    ({}, READY), (dict(tokens=-1), INVALID), (dict(rows=-1), INVALID), (dict(topk=0), INVALID),
    (dict(N=-1), INVALID), (dict(type=3), INVALID), (dict(ldx=6), INVALID), (dict(lddy=6), INVALID),
    (dict(lddx=6), INVALID), (dict(dX=None, lddx=0), READY),
    (dict(dweights=None, X=None, ldx=0), READY), (dict(X=None), INVALID), (dict(dY=None), INVALID),
    (dict(places=None), INVALID), (dict(dX=18), INVALID), (dict(dweights=18), INVALID),
    (dict(dX=None, dweights=None, X=None, dY=None, places=None), READY),
    (dict(tokens=2 ** 26), LARGE), (dict(topk=2 ** 30), LARGE), (dict(lddx=2 ** 31), LARGE),
])
def test_combine_backward_checks(over, status):
    assert _call("sgemm_rows_combine_backward", COMBINE_BACK, over) == status


def test_binding_checks_types_and_lengths():
    torch = pytest.importorskip("torch")
    i32, f32 = torch.zeros(12, dtype=torch.int32), torch.zeros(12)
    with pytest.raises(TypeError, match="picks must be int32"):
        sg.sgemm_route_plan(12, 0, 4, torch.zeros(12, dtype=torch.int64), 16, 16, 16, stream=0)
    with pytest.raises(ValueError, match="picks must hold 13 values, not 12"):
        sg.sgemm_route_plan(13, 0, 4, i32, 16, 16, 16, stream=0)
    with pytest.raises(TypeError, match="weights must be float32"):
        sg.sgemm_rows_combine(4, 3, 9, 7, "f32", 16, 7, 16, f32.double(), 16, 7, 0)
    with pytest.raises(ValueError, match="contiguous"):
        sg.sgemm_rows_combine(2, 3, 9, 7, "f32", 16, 7, 16, f32[::2], 16, 7, 0)
    with pytest.raises(ValueError, match="scalesB must hold 20 values"):
        sg.sgemm_run_int8(4, 20, 8, 1.0, "f32", 16, 8, None, 16, 128, f32, 0.0, "f32", 16, 20,
                          stream=0)


# ------------------------------------------------ the model against torch and by differences
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_model_gradient_by_differences(kind, renormalize):
    g = np.random.default_rng(3)
    l, dw = g.standard_normal((4, 10)), g.standard_normal((4, 3))
    picks, _ = rm.route(kind, l, 3)
    d, _ = rm.route_backward(kind, l, picks, dw, renormalize, 1.7)

    def loss(x):
        total = 0.0
        for t in range(4):
            s = rm.scores(kind, x[t])[picks[t]]
            total += 1.7 * (dw[t] * (s / s.sum() if renormalize else s)).sum()
        return total

    for t in range(4):
        for e in range(10):
            h = np.zeros_like(l)
            h[t, e] = 1e-5
            assert abs((loss(l + h) - loss(l - h)) / 2e-5 - d[t, e]) < 1e-9


def test_model_of_groups_and_disabled_experts():
    l = np.array([[0.0, 3.0, -np.inf, 2.0, 1.0, -np.inf]])
    picks, w = rm.route("softmax", l, 4)
    assert picks.tolist() == [[1, 3, 4, 0]]
    picks, w = rm.route("softmax", l, 4, groups=3, keep=1, group_top=2, renormalize=True)
    assert picks.tolist() == [[1, 0, -1, -1]] and abs(w.sum() - 1) < 1e-15 and (w[0, 2:] == 0).all()
    picks, w = rm.route("sigmoid", np.full((1, 6), -np.inf), 2)
    assert (picks == -1).all() and (w == 0).all()
