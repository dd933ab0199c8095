"""Products of grouped rows over long sums whose products have one sign, where
roundings of a single-precision chain add up instead of cancelling, against sums
in 64 bits.

Tolerance: the contract, |C - exact| <= 1e-5 sum |products| + 1e-6, whatever
the operands.  With u = 2^-24 a chain of n fused multiply-adds is off by up to
n u sum |products|, so one chain for a sum passes 1e-5 from n = 168 on: 6e-5 at
2048 constant products, 1/2 at 2^25 ones, where it stands still at 2^24.
Chains of 128, up to 32 of them added (31 u; the first addition is exact), and
up to four sets of waves (3 u) make 162 u = 9.7e-6.  More chains are added
with the rounding of each addition carried into the next chain: 128 u for the
chains, 2 u for additions and carries, 4 u at the end, and K u^2 for the
roundings of the carried parts: 8.0e-6 at K = 2^25.
"""
import pytest

import dense_fp32_matrix_03_amd as sg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


KINDS = ["constant", "positive", "first large"]


def _operands(kind, a_shape, b_shape, seed):
    import torch
    if kind == "positive":
        g = torch.Generator(device="cuda").manual_seed(seed)
        return (torch.rand(a_shape, generator=g, device="cuda"),
                torch.rand(b_shape, generator=g, device="cuda"))
    A = torch.full(a_shape, 0.1 if kind == "constant" else 1.0, device="cuda")
    B = torch.full(b_shape, 0.1 if kind == "constant" else 2.0 ** -25, device="cuda")
    return A, B


def _check(C, ref, what):
    """All products are positive: the sum of their magnitudes is the reference itself."""
    err = (C.double() - ref).abs()
    worst = (err / (1e-5 * ref + 1e-6)).max().item()
    rel = (err / ref.clamp(min=1e-300)).max().item()
    assert worst <= 1, f"{what}: {worst:.3g} of the tolerance, relative error {rel:.3g}"


# Few tiles (four sets of waves), tiles of 64 x 64, tiles of 64 x 128; M or N = 1.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,lengths", [
    (64, 64, [4096]), (64, 64, [16384, 700]), (33, 70, [1 << 20]), (1, 3, [16385, 40000]),
    (3, 1, [1 << 20]), (1024, 1024, [5000, 9001]), (1024, 1024, [2048, 900, 4097, 97, 1, 3000, 96, 193]),
    (1021, 1023, [2048, 900, 4097, 97, 1, 3000, 96, 193])])
def test_k(M, N, lengths, kind):
    import torch
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    K, G = at[-1], len(lengths)
    A, B = _operands(kind, (K, M), (K, N), K + M)
    if kind == "first large":
        for i in at[:-1]:
            B[i] = 1.0
    C = torch.full((G, M, N), float("nan"), device="cuda")
    offsets = torch.tensor(at, device="cuda")
    sg.sgemm_run_grouped_k(G, M, N, K, 1.0, A, M, B, N, 0.0, C, N, M * N, offsets)
    for g in range(G):
        i, j = at[g], at[g + 1]
        _check(C[g], A[i:j].double().t().contiguous() @ B[i:j].double(), f"group {g}")


# Few tiles, short groups, groups of 16 to 191 rows, long groups.
@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,K,lengths", [
    (40, 4096, [40]), (45, 100001, [3, 40]), (33, (1 << 20) + 1, [5]), (1, 20000, [9, 50]),
    (640, 8200, [0, 3, 1, 0, 2, 2, 0, 1, 5, 1, 1, 0, 2, 3, 2, 1]),
    (1030, 4099, [64, 20, 100, 70, 30, 65, 90, 1, 64, 64, 70, 65, 80, 33, 120, 64]),
    (2048, 8192, [2048]), (2047, 2050, [1000, 1100])])
def test_rows(N, K, lengths, kind, tb):
    import torch
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    M, G = at[-1], len(lengths)
    A, B = _operands(kind, (M, K), (G, N, K) if tb else (G, K, N), K + N)
    if kind == "first large":
        (B[:, :, 0] if tb else B[:, 0]).fill_(1.0)
    C = torch.full((M, N), float("nan"), device="cuda")
    offsets = torch.tensor(at, device="cuda")
    sg.sgemm_run_grouped(tb, G, M, N, K, 1.0, A, K, B, K if tb else N, K * N, 0.0, C, N, offsets)
    for g in range(G):
        i, j = at[g], at[g + 1]
        if i < j:
            b = B[g].double().t().contiguous() if tb else B[g].double()
            _check(C[i:j], A[i:j].double() @ b, f"group {g}")


def test_a_count_past_two_to_the_24():
    """2^25 + 3 ones: the column sums of a gradient's ones column."""
    import torch
    K = (1 << 25) + 3
    A = torch.ones(K, 2, device="cuda")
    B = torch.ones(K, 1, device="cuda")
    C = torch.empty(2, 1, device="cuda")
    sg.sgemm_run_grouped_k(1, 2, 1, K, 1.0, A, 2, B, 1, 0.0, C, 1, 2,
                           torch.tensor([0, K], device="cuda"))
    assert (C.double() - K).abs().max().item() <= 1e-5 * K


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("K", [97, 200, 1000, 5000])
def test_an_infinity_in_a_long_sum_stays_one(K, value):
    """Whichever k it is at; a later one of the other sign makes a NaN."""
    import torch
    for at in (0, 90, 96, K // 2, K - 1):
        A = torch.ones(K, 3, device="cuda")
        B = torch.ones(K, 5, device="cuda")
        A[min(at, K - 1), 1] = value
        A[0, 2], A[K - 1, 2] = value, -value
        C = torch.empty(3, 5, device="cuda")
        offsets = torch.tensor([0, K], device="cuda")
        sg.sgemm_run_grouped_k(1, 3, 5, K, 1.0, A, 3, B, 5, 0.0, C, 5, 15, offsets)
        D = torch.empty(3, 5, device="cuda")
        At = A.t().contiguous()
        sg.sgemm_run_grouped(0, 1, 3, 5, K, 1.0, At, K, B, 5, 0, 0.0, D, 5,
                             torch.tensor([0, 3], device="cuda"))
        for out in (C, D):
            assert (out[0] == K).all()
            assert (out[1] == value).all()
            assert out[2].isnan().all()
