"""Products whose rows fall into groups (sgemm_run_grouped, sgemm_run_grouped_k)
against sums in 64 bits.

Tolerance: the library's contract, |C - exact| <= 1e-5 sum |products| + 1e-6,
where the sum takes in |beta c|.  Summing K <= 1100 products in single
precision one after the other is off by at most (K + 1) 2^-24 sum |products|,
6.6e-5 in the worst case and near sqrt(K) 2^-24 = 2e-6 for independent
roundings; sums of integers below 2^24 are exact.
"""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
from dense_fp32_matrix_03_amd import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


def _dev(x, shift=0):
    """x on the GPU; shift: floats by which its start is moved off 16-byte alignment."""
    import torch
    flat = torch.from_numpy(np.ascontiguousarray(x).reshape(-1)).cuda()
    out = torch.full((flat.numel() + shift + 8,), float("nan"), device="cuda")[shift:]
    out = out[:flat.numel()]
    out.copy_(flat)
    return out


def _offsets(lengths, first=0):
    import torch
    at = np.cumsum([first] + list(lengths)).astype(np.int64)
    return at, torch.from_numpy(at).cuda()


def _check(C, ref, mag):
    err = np.abs(C.astype(np.float64) - ref)
    bad = ~(err <= 1e-5 * mag + 1e-6)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}, "
                           f"worst {np.nanmax(err / (1e-5 * mag + 1e-6)):.3g}")


# lengths, rows before the first group, rows after the last
GROUPS = {
    "one row": ([1], 0, 0),
    "one group": ([70], 0, 0),
    "empty ones": ([0, 5, 0, 0, 17, 1, 0], 0, 0),
    "all empty": ([0, 0, 0], 3, 4),
    "rows outside": ([16, 33, 2], 5, 9),
    "one large": ([3, 300, 1, 2], 0, 1),
    "two hundred": ([(7 * g) % 5 for g in range(200)], 1, 1),
    "several tiles": ([260, 131, 0, 129], 0, 0),
}


def _lengths(groups, mean, seed):
    """Unequal lengths, some of them zero, around `mean`."""
    g = np.random.default_rng(seed)
    n = (g.exponential(mean, groups) * (g.random(groups) > 0.1)).astype(int)
    return [int(v) for v in n]


# Enough rows and groups for each of the tiles through LDS.
LARGE = {
    "short groups": (_lengths(45, 30, 1), 3, 2),
    "long groups": (_lengths(8, 330, 2), 1, 5),
    "very long groups": (_lengths(5, 3600, 3), 0, 7),
}
GROUPS_AND_LARGE = {**GROUPS, **LARGE}


def _run_rows(groups, N, K, tb, alpha=1.0, beta=0.0, pads=(0, 0, 0), shift=0, dist="uniform",
              share=False, seed=0):
    import torch
    lengths, before, after = GROUPS_AND_LARGE[groups]
    G = len(lengths)
    at, d_at = _offsets(lengths, before)
    M = int(at[-1]) + after
    g = np.random.default_rng(seed + N + K + M)
    lda, ldb, ldc = K + pads[0], (K if tb else N) + pads[1], N + pads[2]
    A = inputs.padded(inputs.draw(g, dist, (M, K)), max(lda, 1))
    nb = 1 if share else G
    rows_b, cols_b = (N, K) if tb else (K, N)
    B = np.full((nb, rows_b + 1, max(ldb, 1)), np.nan, np.float32)  # a row between matrices
    B[:, :rows_b, :cols_b] = inputs.draw(g, dist, (nb, rows_b, cols_b))
    C0 = inputs.draw(g, dist, (M, ldc))
    dA, dB, dC = _dev(A, shift), _dev(B, shift), _dev(C0, shift)
    sg.sgemm_run_grouped(tb, G, M, N, K, alpha, dA, max(lda, 1), dB, max(ldb, 1),
                         0 if share else (rows_b + 1) * max(ldb, 1), beta, dC, ldc, d_at)
    torch.cuda.synchronize()
    C = dC.cpu().numpy().reshape(M, ldc)
    ref = C0.astype(np.float64)
    mag = np.abs(ref)
    for n in range(G):
        a = A[at[n]:at[n + 1], :K].astype(np.float64)
        b = B[0 if share else n, :rows_b, :cols_b].astype(np.float64)
        b = b.T if tb else b
        c0 = C0[at[n]:at[n + 1], :N].astype(np.float64)
        ref[at[n]:at[n + 1], :N] = alpha * (a @ b) + beta * c0
        mag[at[n]:at[n + 1], :N] = abs(alpha) * (np.abs(a) @ np.abs(b)) + np.abs(beta * c0)
    # rows of no group and columns past N keep their bits
    inside = np.zeros(C.shape, bool)
    inside[at[0]:at[-1], :N] = True
    assert np.array_equal(C.view(np.uint32)[~inside], C0.view(np.uint32)[~inside])
    return C[inside], ref[inside], mag[inside]


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N,K", [(64, 64), (1, 1), (33, 45), (130, 77), (256, 512), (100, 1100)])
def test_rows(groups, N, K, tb):
    _check(*_run_rows(groups, N, K, tb))


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups", ["rows outside", "several tiles", "empty ones"])
@pytest.mark.parametrize("alpha,beta", [(-1.5, 0.0), (0.5, 2.0), (1.0, -1.0), (0.0, 0.5),
                                        (0.0, 0.0)])
def test_rows_alpha_beta(groups, alpha, beta, tb):
    _check(*_run_rows(groups, 131, 70, tb, alpha, beta))


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups", ["rows outside", "several tiles"])
@pytest.mark.parametrize("pads,shift", [((1, 3, 2), 1), ((4, 8, 4), 0), ((0, 0, 0), 2),
                                        ((5, 0, 1), 3)])
@pytest.mark.parametrize("N,K", [(96, 128), (67, 100)])
def test_rows_strides_and_alignment(groups, N, K, pads, shift, tb):
    _check(*_run_rows(groups, N, K, tb, 1.0, 0.0, pads, shift))


@pytest.mark.parametrize("tb", [0, 1])
def test_rows_no_k_and_shared_b(tb):
    C, ref, _ = _run_rows("rows outside", 40, 0, tb, 1.0, 0.0)
    assert not C.any()
    C, ref, mag = _run_rows("rows outside", 40, 0, tb, 2.0, -0.5)
    _check(C, ref, mag)
    _check(*_run_rows("several tiles", 65, 50, tb, share=True))


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups", ["several tiles", "two hundred"])
def test_rows_exact_on_integers(groups, tb):
    C, ref, _ = _run_rows(groups, 150, 333, tb, dist="int8range")
    assert np.array_equal(C, ref)


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups,N", [("short groups", 1000), ("short groups", 1001),
                                      ("long groups", 1032), ("long groups", 1029),
                                      ("very long groups", 2052), ("very long groups", 2049)])
@pytest.mark.parametrize("K,alpha,beta,pads,shift", [
    (64, 1.0, 0.0, (0, 0, 0), 0), (101, -0.5, 0.0, (0, 0, 0), 0), (3, 1.0, 0.0, (1, 3, 2), 1),
    (130, 0.5, 2.0, (5, 1, 3), 3), (36, 1.0, 0.0, (0, 4, 0), 2)])
def test_rows_of_many_tiles(groups, N, tb, K, alpha, beta, pads, shift):
    _check(*_run_rows(groups, N, K, tb, alpha, beta, pads, shift))


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups,N", [("short groups", 1000), ("long groups", 1029),
                                      ("very long groups", 2052)])
def test_rows_of_many_tiles_exact_on_integers(groups, N, tb):
    C, ref, _ = _run_rows(groups, N, 77, tb, dist="int8range")
    assert np.array_equal(C, ref)


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups", ["one group", "several tiles", "two hundred", "short groups"])
@pytest.mark.parametrize("K", [15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 255, 257,
                               384, 385])
def test_rows_around_whole_turns_of_the_sets(groups, K, tb):
    """Sets of waves take slices of k in turn: a last turn of 1 to all of them,
    whole and partial slices."""
    _check(*_run_rows(groups, 1001 if groups == "short groups" else 90, K, tb))


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("groups,N", [("one group", 256), ("several tiles", 255),
                                      ("two hundred", 300), ("short groups", 1001),
                                      ("long groups", 1032)])
@pytest.mark.parametrize("K,alpha,beta,pads,shift", [
    (4100, 1.0, 0.0, (0, 0, 0), 0), (2047, -0.5, 2.0, (1, 3, 2), 1), (1030, 1.0, 1.0, (2, 2, 0), 2)])
def test_rows_of_long_sums(groups, N, tb, K, alpha, beta, pads, shift):
    _check(*_run_rows(groups, N, K, tb, alpha, beta, pads, shift))


@pytest.mark.parametrize("N", [1, 2, 3, 5, 6, 7, 9, 34, 63])
@pytest.mark.parametrize("K", [1, 31, 32, 64, 65, 300])
@pytest.mark.parametrize("groups", ["rows outside", "two hundred", "long groups"])
def test_rows_of_widths_that_are_no_multiple_of_four(groups, N, K):
    """The last row of each B_g is the end of its buffer (no padding)."""
    _check(*_run_rows(groups, N, K, 0))


def _run_k(groups, M, N, alpha=1.0, beta=0.0, pads=(0, 0, 0), shift=0, dist="uniform", seed=0):
    import torch
    lengths, before, after = GROUPS_AND_LARGE[groups]
    G = len(lengths)
    at, d_at = _offsets(lengths, before)
    K = int(at[-1]) + after
    g = np.random.default_rng(seed + N + K + M)
    lda, ldb, ldc = M + pads[0], N + pads[1], N + pads[2]
    A = inputs.padded(inputs.draw(g, dist, (K, M)), lda)
    B = inputs.padded(inputs.draw(g, dist, (K, N)), ldb)
    A[:at[0]] = A[at[-1]:] = B[:at[0]] = B[at[-1]:] = np.nan  # rows of no group
    C0 = inputs.draw(g, dist, (G, M + 1, ldc))
    dA, dB, dC = _dev(A, shift), _dev(B, shift), _dev(C0, shift)
    sg.sgemm_run_grouped_k(G, M, N, K, alpha, dA, lda, dB, ldb, beta, dC, ldc, (M + 1) * ldc, d_at)
    torch.cuda.synchronize()
    C = dC.cpu().numpy().reshape(C0.shape)
    inside = np.zeros(C.shape, bool)
    inside[:, :M, :N] = True
    assert np.array_equal(C.view(np.uint32)[~inside], C0.view(np.uint32)[~inside])
    ref, mag = np.empty((G, M, N)), np.empty((G, M, N))
    for n in range(G):
        a = A[at[n]:at[n + 1], :M].astype(np.float64)
        b = B[at[n]:at[n + 1], :N].astype(np.float64)
        c0 = C0[n, :M, :N].astype(np.float64)
        ref[n] = alpha * (a.T @ b) + beta * c0
        mag[n] = abs(alpha) * (np.abs(a).T @ np.abs(b)) + np.abs(beta * c0)
    return C[:, :M, :N], ref, mag


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("M,N", [(64, 64), (1, 1), (33, 45), (200, 130), (257, 300)])
def test_k(groups, M, N):
    _check(*_run_k(groups, M, N))


@pytest.mark.parametrize("groups", ["rows outside", "several tiles", "all empty"])
@pytest.mark.parametrize("alpha,beta", [(-1.5, 0.0), (0.5, 2.0), (1.0, 1.0), (0.0, 0.5),
                                        (0.0, 0.0)])
def test_k_alpha_beta(groups, alpha, beta):
    _check(*_run_k(groups, 70, 131, alpha, beta))


@pytest.mark.parametrize("groups", ["rows outside", "several tiles"])
@pytest.mark.parametrize("pads,shift", [((1, 3, 2), 1), ((4, 8, 4), 0), ((0, 0, 0), 2),
                                        ((5, 0, 1), 3)])
@pytest.mark.parametrize("M,N", [(96, 128), (67, 101)])
def test_k_strides_and_alignment(groups, M, N, pads, shift):
    _check(*_run_k(groups, M, N, 1.0, 0.0, pads, shift))


@pytest.mark.parametrize("groups", ["several tiles", "two hundred"])
def test_k_exact_on_integers(groups):
    C, ref, _ = _run_k(groups, 150, 133, dist="int8range")
    assert np.array_equal(C, ref)


@pytest.mark.parametrize("M,N", [(500, 520), (501, 520), (500, 517), (501, 517), (129, 640)])
@pytest.mark.parametrize("alpha,beta,pads,shift", [(1.0, 0.0, (0, 0, 0), 0), (0.5, 2.0, (1, 3, 2), 1),
                                                   (-1.0, 0.0, (4, 0, 1), 3)])
@pytest.mark.parametrize("groups", ["short groups", "long groups"])
def test_k_of_many_tiles(groups, M, N, alpha, beta, pads, shift):
    _check(*_run_k(groups, M, N, alpha, beta, pads, shift))


@pytest.mark.parametrize("M,N", [(500, 520), (600, 640)])
def test_k_of_many_tiles_exact_on_integers(M, N):
    C, ref, _ = _run_k("short groups", M, N, dist="int8range")
    assert np.array_equal(C, ref)


@pytest.mark.parametrize("groups", ["long groups", "very long groups"])
@pytest.mark.parametrize("M,N", [(64, 64), (1, 1), (33, 45), (130, 68), (36, 131)])
@pytest.mark.parametrize("alpha,beta,pads,shift", [(1.0, 0.0, (0, 0, 0), 0), (0.5, 2.0, (1, 3, 2), 1)])
def test_k_of_few_tiles_and_long_groups(groups, M, N, alpha, beta, pads, shift):
    _check(*_run_k(groups, M, N, alpha, beta, pads, shift))


@pytest.mark.parametrize("M,N", [(1, 5), (5, 1), (2, 2), (3, 3), (5, 6), (7, 9), (34, 65), (1, 64),
                                 (64, 1), (2, 68), (66, 4)])
@pytest.mark.parametrize("groups", ["one row", "one group", "empty ones", "rows outside",
                                    "long groups"])
def test_k_of_widths_that_are_no_multiple_of_four(groups, M, N):
    _check(*_run_k(groups, M, N))


def test_k_of_few_tiles_exact_on_integers():
    C, ref, _ = _run_k("long groups", 70, 45, dist="int8range")
    assert np.array_equal(C, ref)


@pytest.mark.parametrize("alpha,beta,pads,shift", [(1.0, 0.0, (0, 0, 0), 0), (0.5, 2.0, (4, 3, 2), 1)])
def test_k_of_large_tiles(alpha, beta, pads, shift):
    _check(*_run_k("short groups", 600, 640, alpha, beta, pads, shift))


@pytest.mark.parametrize("at", [[0, 40, 20, 50], [-7, 10, 60, 90], [50, 0, 50, 0],
                                [2 ** 62, 3, -2 ** 63, 50]])
def test_offsets_out_of_range_write_nothing_outside(at):
    """Ranges are clamped to the operands: every access stays in C's rows, and
    rows of C beyond M keep their bits."""
    import torch
    M, N, K, G = 50, 40, 36, 3
    d_at = torch.tensor(at, dtype=torch.int64, device="cuda")
    A = torch.randn(M, K, device="cuda")
    B = torch.randn(G, K, N, device="cuda")
    C = torch.full((M + 40, N), 7.0, device="cuda")
    sg.sgemm_run_grouped(0, G, M, N, K, 1.0, A, K, B, N, K * N, 0.0, C[20:], N, d_at)
    D = torch.full((G + 2, K, N), 7.0, device="cuda")
    E = torch.randn(M, N, device="cuda")
    sg.sgemm_run_grouped_k(G, K, N, M, 1.0, A, K, E, N, 0.0, D[1:], N, K * N, d_at)
    torch.cuda.synchronize()
    assert (C[:20] == 7).all() and (C[20 + M:] == 7).all()
    assert (D[0] == 7).all() and (D[-1] == 7).all()
    assert torch.isfinite(C).all() and torch.isfinite(D).all()


@pytest.mark.parametrize("tb", [0, 1])
def test_offsets_out_of_range_with_many_tiles(tb):
    import torch
    M, N, K, G = 1200, 1000, 40, 40
    g = np.random.default_rng(6)
    at = np.sort(g.integers(0, M + 1, G + 1))
    at[5], at[11], at[20], at[30], at[40] = -3, 2 ** 40, 7, M + 9, 900
    d_at = torch.from_numpy(at).cuda()
    A = torch.randn(M, K, device="cuda")
    B = torch.randn(G, K * N, device="cuda")
    C = torch.full((M + 40, N), 7.0, device="cuda")
    sg.sgemm_run_grouped(tb, G, M, N, K, 1.0, A, K, B, K if tb else N, K * N, 0.0, C[20:], N, d_at)
    torch.cuda.synchronize()
    assert (C[:20] == 7).all() and (C[20 + M:] == 7).all() and torch.isfinite(C).all()


def test_empty_sums_do_not_multiply_alpha():
    """An empty group's sum, or one over no k, is 0 even where alpha is infinite."""
    import torch
    at, d_at = _offsets([0, 3, 0])
    A, B = torch.ones(3, 6, device="cuda"), torch.ones(3, 5, device="cuda")
    D = torch.full((3, 6, 5), 2.0, device="cuda")
    sg.sgemm_run_grouped_k(3, 6, 5, 3, float("inf"), A, 6, B, 5, 0.5, D, 5, 30, d_at)
    assert (D[0] == 1).all() and (D[2] == 1).all() and torch.isinf(D[1]).all()
    C = torch.full((3, 5), 2.0, device="cuda")
    sg.sgemm_run_grouped(0, 3, 3, 5, 0, float("inf"), None, 1, None, 5, 0, 0.5, C, 5, d_at)
    assert (C == 1).all()


def test_rows_far_apart():
    """Offsets into A and C pass 2^31 elements: 1100 rows 2^21 floats apart."""
    import torch
    M, N, K, ld = 1100, 40, 24, 2 ** 21
    at, d_at = _offsets([500, 0, 600])
    g = np.random.default_rng(5)
    A, B = inputs.uniform(g, (M, K)), inputs.uniform(g, (3, K, N))
    big = torch.empty(M * ld, device="cuda")
    big.as_strided((M, K), (ld, 1)).copy_(torch.from_numpy(A))
    c = big[ld // 2:]
    sg.sgemm_run_grouped(0, 3, M, N, K, 1.0, big, ld, _dev(B), N, K * N, 0.0, c, ld, d_at)
    C = c.as_strided((M, N), (ld, 1)).cpu().numpy()
    ref, mag = np.empty((M, N)), np.empty((M, N))
    for n in range(3):
        a, b = A[at[n]:at[n + 1]].astype(np.float64), B[n].astype(np.float64)
        ref[at[n]:at[n + 1]], mag[at[n]:at[n + 1]] = a @ b, np.abs(a) @ np.abs(b)
    _check(C, ref, mag)


def test_repeated_calls_give_the_same_bits():
    a, _, _ = _run_rows("several tiles", 130, 500, 0)
    b, _, _ = _run_rows("several tiles", 130, 500, 0)
    assert a.tobytes() == b.tobytes()
    a, _, _ = _run_k("several tiles", 130, 100)
    b, _, _ = _run_k("several tiles", 130, 100)
    assert a.tobytes() == b.tobytes()


def _layer(x, w1, w2, at, dy):
    """y = (x w1_g) w2_g by group; returns y and the gradients of x, w1 and w2."""
    import torch
    M, K = x.shape
    G, _, H = w1.shape
    N = w2.shape[2]
    new = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    h, y, dh, dx = new(M, H), new(M, N), new(M, H), new(M, K)
    dw1, dw2 = new(G, K, H), new(G, H, N)
    sg.sgemm_run_grouped(0, G, M, H, K, 1.0, x, K, w1, H, K * H, 0.0, h, H, at)
    sg.sgemm_run_grouped(0, G, M, N, H, 1.0, h, H, w2, N, H * N, 0.0, y, N, at)
    sg.sgemm_run_grouped(1, G, M, H, N, 1.0, dy, N, w2, N, H * N, 0.0, dh, H, at)
    sg.sgemm_run_grouped_k(G, H, N, M, 1.0, h, H, dy, N, 0.0, dw2, N, H * N, at)
    sg.sgemm_run_grouped(1, G, M, K, H, 1.0, dh, H, w1, H, K * H, 0.0, dx, K, at)
    sg.sgemm_run_grouped_k(G, K, H, M, 1.0, x, K, dh, H, 0.0, dw1, H, K * H, at)
    return y, dx, dw1, dw2


def test_a_layer_of_experts_forward_and_backward():
    """Two products of a layer of experts and all their gradients, against the
    formulas in 64 bits and against differences of the loss sum(y dy)."""
    import torch
    M, K, H, N, lengths = 150, 40, 72, 36, [60, 0, 1, 89]
    G = len(lengths)
    at, d_at = _offsets(lengths)
    g = np.random.default_rng(11)
    X, W1 = inputs.uniform(g, (M, K)), inputs.uniform(g, (G, K, H))
    W2, DY = inputs.uniform(g, (G, H, N)), inputs.uniform(g, (M, N))
    t = [torch.from_numpy(v).cuda() for v in (X, W1, W2)]
    got = [v.cpu().numpy() for v in _layer(*t, d_at, torch.from_numpy(DY).cuda())]

    def loss(x, w1, w2):
        return sum(float((x[i:j] @ w1[n] @ w2[n] * DY[i:j]).sum())
                   for n, (i, j) in enumerate(zip(at, at[1:])))

    x, w1, w2, dy = (v.astype(np.float64) for v in (X, W1, W2, DY))
    ref = [np.zeros((M, N)), np.zeros((M, K)), np.zeros((G, K, H)), np.zeros((G, H, N))]
    mag = [v.copy() for v in ref]
    for out, f in ((ref, lambda v: v), (mag, np.abs)):
        for n, (i, j) in enumerate(zip(at, at[1:])):
            a, b, c, d = f(x[i:j]), f(w1[n]), f(w2[n]), f(dy[i:j])
            out[0][i:j] = a @ b @ c
            out[1][i:j] = d @ c.T @ b.T
            out[2][n] = a.T @ (d @ c.T)
            out[3][n] = (a @ b).T @ d
    # two products in a row: each is within the contract of its own inputs, and
    # the first one's error passes through the second
    for v, r, m in zip(got, ref, mag):
        assert (np.abs(v - r) <= 2.1e-5 * m + 2e-6 * H).all()
    # central differences in 64 bits: the loss is linear in each argument, so
    # they are exact but for rounding
    for arg, grad, places in ((0, got[1], [(0, 3), (60, 7), (149, 39)]),
                              (1, got[2], [(0, 5, 6), (1, 2, 3), (2, 0, 71), (3, 39, 0)]),
                              (2, got[3], [(0, 71, 35), (1, 0, 0), (3, 8, 9)])):
        for place in places:
            args = [x.copy(), w1.copy(), w2.copy()]
            args[arg][place] += 0.5
            up = loss(*args)
            args[arg][place] -= 1.0
            assert abs(grad[place] - (up - loss(*args))) <= 2.1e-5 * mag[arg + 1][place] + 2e-4


def test_in_a_graph_with_other_lengths_on_each_replay():
    """The lengths are read when the graph runs: one captured call serves any."""
    import torch
    G, M, N, K = 5, 120, 70, 50
    g = np.random.default_rng(3)
    A, B = inputs.uniform(g, (M, K)), inputs.uniform(g, (G, K, N))
    dA, dB = torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda()
    dE = torch.from_numpy(inputs.uniform(g, (M, N))).cuda()
    C, D = torch.empty(M, N, device="cuda"), torch.empty(G, K, N, device="cuda")
    d_at = torch.zeros(G + 1, dtype=torch.int64, device="cuda")

    def body():
        sg.sgemm_run_grouped(0, G, M, N, K, 1.0, dA, K, dB, N, K * N, 0.0, C, N, d_at)
        sg.sgemm_run_grouped_k(G, K, N, M, 1.0, dA, K, dE, N, 0.0, D, N, K * N, d_at)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        body()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for lengths in ([120, 0, 0, 0, 0], [24] * 5, [0, 1, 2, 3, 114], [0, 0, 0, 0, 7], [40, 40, 40, 0, 0]):
        at = np.cumsum([0] + lengths).astype(np.int64)
        d_at.copy_(torch.from_numpy(at))
        C.fill_(5.0)
        D.fill_(5.0)
        body()
        torch.cuda.synchronize()
        want = C.cpu().numpy().tobytes(), D.cpu().numpy().tobytes()
        C.fill_(5.0)
        D.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (C.cpu().numpy().tobytes(), D.cpu().numpy().tobytes()) == want
        c = C.cpu().numpy()
        for n in range(G):
            i, j = at[n], at[n + 1]
            a, b = A[i:j].astype(np.float64), B[n].astype(np.float64)
            _check(c[i:j], a @ b, np.abs(a) @ np.abs(b)) if j > i else None
        assert (c[at[-1]:] == 5).all()


def test_on_another_stream():
    import torch
    M, N, K, G = 200, 96, 64, 4
    at, d_at = _offsets([50, 0, 100, 50])
    g = np.random.default_rng(9)
    A, B = inputs.uniform(g, (M, K)), inputs.uniform(g, (G, K, N))
    dA, dB = torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda()
    C = torch.empty(M, N, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sg.sgemm_run_grouped(0, G, M, N, K, 1.0, dA, K, dB, N, K * N, 0.0, C, N, d_at, stream=s)
    s.synchronize()
    for n in range(G):
        a, b = A[at[n]:at[n + 1]].astype(np.float64), B[n].astype(np.float64)
        if len(a):
            _check(C.cpu().numpy()[at[n]:at[n + 1]], a @ b, np.abs(a) @ np.abs(b))


@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("K,N,lengths", [(50, 45, [17, 20, 33]), (1100, 34, [40, 1, 90]),
                                         (33, 1001, [700, 350, 900])])
def test_what_is_not_finite_stays_in_its_row(K, N, lengths, tb):
    """One row of A is NaN and one B_g infinite: the other groups' rows, and the
    NaN row's neighbours, are what they are without them."""
    import torch
    at, d_at = _offsets(lengths)
    M, G = int(at[-1]), len(lengths)
    g = np.random.default_rng(K + N)
    A, B = inputs.uniform(g, (M, K)), inputs.uniform(g, (G, N, K) if tb else (G, K, N))
    out = []
    for spoilt in (False, True):
        if spoilt:
            A[at[1]] = np.nan        # the first row of the second group
            B[2] = np.inf
        C = torch.full((M, N), 3.0, device="cuda")
        sg.sgemm_run_grouped(tb, G, M, N, K, 1.0, _dev(A), K, _dev(B), K if tb else N, K * N, 0.0,
                             C, N, d_at)
        out.append(C.cpu().numpy())
    same = np.ones(M, bool)
    same[at[1]] = same[at[2]:] = False
    assert np.array_equal(out[0][same], out[1][same])
    assert np.isnan(out[1][at[1]]).all() and not np.isfinite(out[1][at[2]:]).any()


@pytest.mark.parametrize("M,N,lengths", [(37, 45, [17, 20, 33]), (64, 130, [300, 500, 700]),
                                         (601, 999, [30, 2, 64] + [9] * 20)])
def test_what_is_not_finite_stays_in_its_group(M, N, lengths):
    import torch
    at, d_at = _offsets(lengths)
    K, G = int(at[-1]), len(lengths)
    g = np.random.default_rng(M + N)
    A, B = inputs.uniform(g, (K, M)), inputs.uniform(g, (K, N))
    out = []
    for spoilt in (False, True):
        if spoilt:
            A[at[1]:at[2]] = np.nan
            B[at[1]:at[2]] = np.inf
        C = torch.full((G, M, N), 3.0, device="cuda")
        sg.sgemm_run_grouped_k(G, M, N, K, 1.0, _dev(A), M, _dev(B), N, 0.0, C, N, M * N, d_at)
        out.append(C.cpu().numpy())
    others = [n for n in range(G) if n != 1]
    assert np.array_equal(out[0][others], out[1][others]) and np.isnan(out[1][1]).all()


def test_the_most_groups():
    """4096 groups, most of them empty or of one row; the last one long."""
    import torch
    lengths = [(n * 7) % 3 // 2 for n in range(4095)] + [300]
    at, d_at = _offsets(lengths)
    M, G, K, N = int(at[-1]), 4096, 24, 20
    g = np.random.default_rng(2)
    A, B = inputs.uniform(g, (M, K)), inputs.uniform(g, (G, K, N))
    E = inputs.uniform(g, (M, N))
    C, D = torch.empty(M, N, device="cuda"), torch.empty(G, K, N, device="cuda")
    sg.sgemm_run_grouped(0, G, M, N, K, 1.0, _dev(A), K, _dev(B), N, K * N, 0.0, C, N, d_at)
    sg.sgemm_run_grouped_k(G, K, N, M, 1.0, _dev(A), K, _dev(E), N, 0.0, D, N, K * N, d_at)
    of = np.repeat(np.arange(G), lengths)
    a, b, e = A.astype(np.float64), B.astype(np.float64)[of], E.astype(np.float64)
    _check(C.cpu().numpy(), np.einsum("mk,mkn->mn", a, b),
           np.einsum("mk,mkn->mn", np.abs(a), np.abs(b)))
    ref, mag = np.zeros((G, K, N)), np.zeros((G, K, N))
    np.add.at(ref, of, a[:, :, None] * e[:, None, :])
    np.add.at(mag, of, np.abs(a[:, :, None] * e[:, None, :]))
    _check(D.cpu().numpy(), ref, mag)


def test_two_streams_at_once():
    """Two calls in flight share nothing."""
    import torch
    G, M, N, K = 6, 900, 500, 400
    g = np.random.default_rng(4)
    at, d_at = _offsets([100, 250, 0, 300, 50, 200])
    A = [_dev(inputs.uniform(g, (M, K))) for _ in range(2)]
    B = [_dev(inputs.uniform(g, (G, K, N))) for _ in range(2)]
    C = [torch.zeros(M, N, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            sg.sgemm_run_grouped(0, G, M, N, K, 1.0, A[i], K, B[i], N, K * N, 0.0, C[i], N, d_at,
                                 stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        alone = torch.zeros(M, N, device="cuda")
        sg.sgemm_run_grouped(0, G, M, N, K, 1.0, A[i], K, B[i], N, K * N, 0.0, alone, N, d_at)
        assert torch.equal(alone, C[i])


@pytest.mark.parametrize("N,pads,shift", [(512, (0, 0, 0), 0), (512, (0, 0, 0), 8), (528, (0, 0, 0), 16),
                                          (512, (0, 0, 8), 0), (513, (0, 0, 15), 0), (517, (0, 0, 0), 3)])
@pytest.mark.parametrize("alpha,beta", [(1.0, 0.0), (0.5, 2.0)])
def test_k_of_short_groups_on_lines_of_c_and_off_them(N, pads, shift, alpha, beta):
    _run_k("short groups", 500, N, alpha, beta, pads, shift)
