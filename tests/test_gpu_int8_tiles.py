"""sgemm_run_int8 and sgemm_run_int8_grouped on every kernel that they have, bit for bit.

The sum of the codes' products is exact, in 64-bit products on the GPU too, and each step after it
is an IEEE operation on single precision that torch repeats; with alpha = 1/2 and beta = 2 the
products alpha v and beta C are exact, so that the fused multiply-add is a sum.
"""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import int8_model as i8
import int8_tiles

pytestmark = pytest.mark.gpu
CASES = [(n, c) for t in (int8_tiles.CASES, int8_tiles.GROUPED) for n, cs in t.items() for c in cs]


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


def _type(kind):
    import torch
    return torch.float32 if kind == "f32" else torch.bfloat16


def _held(x, pad=0):
    """(codes with ldq = padded K + pad, scales) of x, by the library's cast, which other tests
    compare with the format."""
    import torch
    rows, K = x.shape
    codes = torch.full((rows, i8.padded(K) + pad), 77, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, device="cuda")
    sg.sgemm_int8_quantize(0, rows, K, "f32", x, K, codes, codes.shape[1], scales)
    return codes, scales


def _lengths(groups, rows, seed):
    """Unequal, one of them empty where there are three or more; a few rows belong to none."""
    g = np.random.default_rng(seed)
    share = g.random(groups) + 0.2
    if groups > 2:
        share[groups // 2] = 0
    at = np.concatenate([[0], np.cumsum(share) / share.sum() * (rows - 3)]).astype(np.int64)
    return at + 2  # rows 0, 1 and the last


@pytest.mark.parametrize("name,case", CASES)
def test_bits(name, case):
    import torch
    groups, M, N, K = case
    G = max(groups, 1)
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda") * torch.exp2(
        torch.randint(-9, 9, (M, 1), generator=g, device="cuda").float())
    w = torch.randn(G * N, K, generator=g, device="cuda")
    x16 = x.bfloat16()
    at = _lengths(groups, M, M) if groups else np.array([0, M])
    offsets = torch.from_numpy(at).cuda()
    cw, sw = _held(w, 16)
    forms = {}
    for kind, values in (("f32", x), ("bf16", x16.float())):
        c, s = _held(values)
        total = torch.empty(M, N, dtype=torch.float64, device="cuda")
        unit = torch.ones(M, N, device="cuda")
        for i, (a, b) in enumerate(zip(at, at[1:])):
            rows = slice(i * N, (i + 1) * N)
            total[a:b] = c[a:b, :K].double() @ cw[rows, :K].double().T.contiguous()
            unit[a:b] = sw[rows]
        forms[kind] = (total.float() * s[:, None]) * unit
    ca, sa = _held(x, 32)
    inside = torch.zeros(M, 1, dtype=torch.bool, device="cuda")
    inside[at[0]:at[-1]] = True
    for kind, A, lda, scales in (("int8", ca, ca.shape[1], sa), ("f32", x, K, None),
                                 ("bf16", x16, K, None)):
        need = sg.sgemm_int8_workspace_size(kind, M, K)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        for out, alpha, beta, pad in (("f32", 1.0, 0.0, 0), ("bf16", 1.0, 0.0, 3),
                                      ("f32", 0.5, 2.0, 1), ("bf16", 0.5, 2.0, 0)):
            C = torch.randn(M, N + pad, generator=g, device="cuda").to(_type(out))
            before = C.clone()
            args = (M, N, K, alpha, kind, A, lda, scales, cw, cw.shape[1], sw, beta, out, C, N + pad)
            if groups:
                sg.sgemm_run_int8_grouped(groups, *args, offsets, ws, need)
            else:
                sg.sgemm_run_int8(*args, ws, need)
            v = forms["bf16" if kind == "bf16" else "f32"]
            want = v if beta == 0 else alpha * v + beta * before[:, :N].float()
            want = torch.where(inside, want.to(C.dtype), before[:, :N])
            assert torch.equal(C[:, :N], want), (
                f"A {kind}, C {out}, beta {beta}: {(C[:, :N] != want).sum()} of {C.numel()} differ")
            assert torch.equal(C[:, N:], before[:, N:])
