"""8-bit integer operands (sgemm_int8_quantize, sgemm_run_int8, sgemm_run_int8_grouped) against
the format's definition.

The casts are compared bit for bit, and so are products with alpha = 1 and beta = 0: the sum of the
codes' products is exact, and the three steps after it (to single precision, times a scale, times
the other) are IEEE operations that numpy repeats; a bfloat16 C is rounded once more, to the nearest
even.  With alpha and beta the result is alpha v + beta C, off by at most 2^-24 of beta C, 2^-24 of
the result, and 2^-8 of it for bfloat16.
"""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import int8_model as i8
import mxfp4_model as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


def _cuda(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _typed(x, kind, ld=None, shift=0):
    """x (float32, 2-D) on the GPU as `kind` with leading dimension ld, its start moved by `shift`
    elements, NaN around it; and the float32 values it holds."""
    import torch
    bits = mx.bf16_bits(x) if kind == "bf16" else x.view(np.uint32)
    if kind == "bf16":
        bits[np.isnan(x)] = 0x7fc0
        bits[np.isinf(x)] = np.where(x[np.isinf(x)] > 0, 0x7f80, 0xff80)
    dt, fill = (np.int16, 0x7fc0) if kind == "bf16" else (np.int32, 0x7fc00000)
    ld = x.shape[1] if ld is None else ld
    buf = np.full(shift + x.shape[0] * ld + 8, fill, dt)
    buf[shift:shift + x.shape[0] * ld].reshape(x.shape[0], ld)[:, :x.shape[1]] = bits.view(dt)
    t = torch.from_numpy(buf).cuda()[shift:]
    t = t.view(torch.bfloat16 if kind == "bf16" else torch.float32)
    return t, (mx.bf16_floats(bits) if kind == "bf16" else x)


def _values(seed, shape, kind="normal"):
    g = np.random.default_rng(seed)
    if kind == "wide":  # rows of all magnitudes
        x = g.standard_normal(shape) * np.exp2(g.integers(-150, 126, (shape[0], 1)))
    elif kind == "ties":  # the largest is 127, so that scale is 1 and halves are ties
        x = g.integers(-252, 253, shape) / 2.0
        x[:, -1] = 127
        x = x * np.exp2(g.integers(-30, 31, (shape[0], 1)))
    elif kind == "sparse":
        x = g.standard_normal(shape) * (g.random(shape) < 0.02)
    elif kind == "tiny":  # subnormal rows, and rows whose scale is
        x = g.standard_normal(shape) * np.exp2(g.integers(-149, -118, (shape[0], 1)))
    elif kind == "special":
        x = g.standard_normal(shape)
        for v in (np.nan, np.inf, -np.inf):
            x[tuple(g.integers(0, n) for n in shape)] = v
    else:
        x = g.standard_normal(shape)
    with np.errstate(over="ignore", under="ignore"):
        x = x.astype(np.float32)
    return np.where(np.isinf(x) & (kind != "special"), np.float32(1), x)


def _quantize(x, kind, trans, ld_pad=0, ldq_pad=0, shift=0):
    import torch
    rows, K = x.shape
    stored = np.ascontiguousarray(x.T) if trans else x
    ld = stored.shape[1] + ld_pad
    dX, held = _typed(stored, kind, ld, shift)
    ldq = i8.padded(K) + ldq_pad
    codes = torch.full((rows, ldq), 0x55, dtype=torch.int8, device="cuda")
    scales = torch.full((rows + 4,), 9.0, device="cuda")
    sg.sgemm_int8_quantize(trans, rows, K, kind, dX, ld, codes, ldq, scales)
    torch.cuda.synchronize()
    assert (codes[:, i8.padded(K):] == 0x55).all() and (scales[rows:] == 9).all()
    return (codes[:, :i8.padded(K)].cpu().numpy(), scales[:rows].cpu().numpy(),
            held.T if trans else held)


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("values", ["normal", "wide", "ties", "sparse", "tiny", "special"])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 32), (33, 128), (70, 300), (5, 1024), (6, 1025),
                                    (40, 8192), (3, 8201), (2, 20000)])
def test_quantize(rows, K, values, kind, trans):
    codes, scales, held = _quantize(_values(rows + K, (rows, K), values), kind, trans)
    want, want_s = i8.quantize(held)
    assert np.array_equal(scales, want_s, equal_nan=True)
    assert np.array_equal(codes, want)


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("ld_pad,ldq_pad,shift", [(1, 16, 1), (8, 128, 0), (5, 1024, 3)])
def test_quantize_strides(kind, trans, ld_pad, ldq_pad, shift):
    for rows, K in ((75, 333), (9, 1500)):
        codes, scales, held = _quantize(_values(5, (rows, K)), kind, trans, ld_pad, ldq_pad, shift)
        want, want_s = i8.quantize(held)
        assert np.array_equal(codes, want) and np.array_equal(scales, want_s)


def _bits(v, out):
    """v as a C of type `out` holds it, float32."""
    if out == "f32":
        return v
    bits = mx.bf16_bits(v)
    bits[np.isnan(v)] = 0x7fc0
    return mx.bf16_floats(bits)


def _product(M, N, K, kind, out, alpha=1.0, beta=0.0, pads=(0, 0, 0), shift=0, seed=0,
             lengths=None, before=0, values="normal"):
    """One product on the GPU, checked."""
    import torch
    G = 1 if lengths is None else len(lengths)
    x, w = _values(seed + M, (M, K), values), _values(seed + N + 1, (G * N, K))
    cw, sw = i8.quantize(w)
    ldb = i8.padded(K) + pads[1]
    dB = np.full((G * N, ldb), 77, np.int8)
    dB[:, :i8.padded(K)] = cw
    if kind == "int8":
        ca, sa = i8.quantize(x)
        lda = i8.padded(K) + pads[0] // 16 * 16
        codes = np.full((M, lda), 77, np.int8)
        codes[:, :i8.padded(K)] = ca
        dA, dsA, ws = _cuda(codes), _cuda(sa), None
    else:
        lda = max(K, 1) + pads[0]
        dA, held = _typed(x, kind, lda, shift) if K else (_cuda(np.zeros(8, np.float32)), x)
        dsA = None
        ca, sa = i8.quantize(held)
        ws = torch.full((sg.sgemm_int8_workspace_size(kind, M, K) + 16,), 0xFF, dtype=torch.uint8,
                        device="cuda")
    ldc = N + pads[2]
    dC, C0 = _typed(_values(seed + 3, (M, ldc)), out, ldc, shift)
    n = 0 if ws is None else ws.numel() - 16
    if lengths is None:
        at = np.array([0, M])
        sg.sgemm_run_int8(M, N, K, alpha, kind, dA, lda, dsA, _cuda(dB), ldb, _cuda(sw), beta, out,
                          dC, ldc, ws, n)
    else:
        at = np.cumsum([before] + list(lengths)).astype(np.int64)
        sg.sgemm_run_int8_grouped(G, M, N, K, alpha, kind, dA, lda, dsA, _cuda(dB), ldb, _cuda(sw),
                                  beta, out, dC, ldc, _cuda(at), ws, n)
    torch.cuda.synchronize()
    C = dC[:M * ldc].float().cpu().numpy().reshape(M, ldc)
    if ws is not None:
        assert (ws[n:] == 0xFF).all()
    inside = np.zeros((M, ldc), bool)
    for g, (i, j) in enumerate(zip(at, at[1:])):
        v, exact = i8.products(ca[i:j], sa[i:j], cw[g * N:(g + 1) * N], sw[g * N:(g + 1) * N])
        got = C[i:j, :N]
        inside[i:j, :N] = True
        if alpha == 1.0 and beta == 0.0:
            want = _bits(v, out)
            same = (got == want) | (np.isnan(got) & np.isnan(want))
            assert same.all(), (f"group {g}: {(~same).sum()} of {same.size} differ, first at "
                                f"{np.argwhere(~same)[0]}: {got[~same][0]} for {want[~same][0]}")
        else:
            bc = beta * C0[i:j, :N].astype(np.float64) if beta != 0 else 0.0
            ref = alpha * exact + bc
            tol = (2.0 ** -24 * (3 * np.abs(alpha * exact) + np.abs(bc) + np.abs(ref)) * 1.01
                   + (2.0 ** -8 * np.abs(ref) * 1.01 if out == "bf16" else 0) + 1e-37)
            err = np.abs(got - ref)
            assert (err <= tol).all(), f"group {g}: worst {np.max(err / tol):.3g}"
    assert np.array_equal(C[~inside], C0[~inside])


SIZES = [(1, 1, 1), (1, 64, 128), (5, 33, 45), (16, 128, 512), (17, 100, 700), (40, 129, 1000),
         (70, 257, 333), (130, 300, 2050), (300, 520, 640), (1, 130, 9000), (2, 77, 2600),
         (64, 64, 12000), (100, 70, 8000), (257, 300, 129), (513, 770, 260), (32, 1000, 4096)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "int8"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, kind, out):
    _product(M, N, K, kind, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "int8"])
@pytest.mark.parametrize("alpha,beta", [(1.0, 1.0), (-0.5, 2.0), (0.0, 3.0), (2.0, 0.0), (0.0, 0.0)])
@pytest.mark.parametrize("M,N,K", [(3, 70, 200), (100, 130, 300), (300, 260, 0)])
def test_alpha_beta_strides(M, N, K, alpha, beta, kind, out):
    _product(M, N, K, kind, out, alpha, beta, pads=(16, 32, 3), shift=1)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_rows_without_finite_values_or_zero(M):
    for kind in ("f32", "bf16", "int8"):
        _product(M, 90, 200, kind, "f32", values="special")
        _product(M, 90, 200, kind, "bf16", values="tiny")
        _product(M, 90, 200, kind, "f32", values="sparse")


def test_largest_sums_are_exact():
    """2^17 - 1 products of -128 and -128 stay below 2^31."""
    import torch
    K = 2 ** 17 - 1
    for M, N in ((1, 3), (20, 40), (70, 65)):
        a = torch.full((M, i8.padded(K)), -128, dtype=torch.int8, device="cuda")
        b = torch.full((N, i8.padded(K)), -128, dtype=torch.int8, device="cuda")
        a[:, K:] = 0
        sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        C = torch.empty(M, N, device="cuda")
        sg.sgemm_run_int8(M, N, K, 1.0, "int8", a, i8.padded(K), sa, b, i8.padded(K), sb, 0.0,
                          "f32", C, N)
        assert (C == float(K * 16384)).all()


GROUPS = [([5], 0), ([0, 3, 0, 1], 0), ([1] * 9, 2), ([70, 0, 130, 1], 5), ([300, 2, 64, 65], 0),
          ([0, 0, 0], 1), ([2] * 70, 3), ([33] * 66, 0), ([600, 200], 7)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "int8"])
@pytest.mark.parametrize("lengths,before", GROUPS)
def test_grouped(lengths, before, kind, out):
    M = sum(lengths) + before + 3
    _product(M, 100, 300, kind, out, lengths=lengths, before=before)
    _product(M, 65, 130, kind, out, 0.5, 2.0, pads=(16, 16, 1), lengths=lengths, before=before)


@pytest.mark.parametrize("rows,groups,N,K", [(48, 32, 512, 2048), (500, 100, 130, 700), (1, 64, 64, 64)])
def test_grouped_like_a_router(rows, groups, N, K):
    g = np.random.default_rng(rows)
    lengths = np.bincount(g.integers(0, groups, rows), minlength=groups)
    for kind in ("bf16", "int8"):
        _product(rows, N, K, kind, "bf16", lengths=list(lengths))


def test_offsets_out_of_range_write_nothing_outside():
    import torch
    M, N, K = 40, 64, 128
    a = torch.ones(M, K, dtype=torch.int8, device="cuda")
    b = torch.ones(3 * N, K, dtype=torch.int8, device="cuda")
    s = torch.ones(3 * N, device="cuda")
    for at in ([-5, 10, 1 << 40, 7], [30, 20, 10, 0], [50, 60, 70, 80], [0, 0, 0, 40]):
        C = torch.full((M + 2, N), 5.0, device="cuda")
        sg.sgemm_run_int8_grouped(3, M, N, K, 1.0, "int8", a, K, s, b, K, s, 0.0, "f32", C[1:], N,
                                  torch.tensor(at, device="cuda"))
        torch.cuda.synchronize()
        assert (C[0] == 5).all() and (C[M + 1] == 5).all()
        assert ((C == 5) | (C == K)).all()


def test_b_past_4_gib():
    """The last rows of a B of more than 2^32 bytes."""
    import torch
    K, ldb, N = 256, 1 << 21, 2100
    b = torch.zeros(N * ldb, dtype=torch.int8, device="cuda").view(N, ldb)
    b[:, :K] = torch.arange(N, device="cuda")[:, None] % 100
    s = torch.ones(N, device="cuda")
    for M in (1, 20, 100):
        a = torch.ones(M, K, dtype=torch.int8, device="cuda")
        C = torch.empty(M, N, device="cuda")
        sg.sgemm_run_int8(M, N, K, 1.0, "int8", a, K, s, b, ldb, s, 0.0, "f32", C, N)
        assert (C == (torch.arange(N, device="cuda") % 100 * K).float()).all()


def test_other_stream_and_graph():
    """Captured and replayed with other inputs; each replay against the eager result."""
    import torch
    M, N, K, G = 30, 200, 500, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    w = torch.randn(G * N, K, device="cuda", generator=g)
    codes = torch.empty(G * N, i8.padded(K), dtype=torch.int8, device="cuda")
    scales = torch.empty(G * N, device="cuda")
    offsets = torch.tensor([0, 7, 7, 20, 30], device="cuda")
    C, C2 = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    ws = torch.empty(sg.sgemm_int8_workspace_size("bf16", M, K), dtype=torch.uint8, device="cuda")

    def body():
        sg.sgemm_int8_quantize(0, G * N, K, "f32", w, K, codes, i8.padded(K), scales)
        sg.sgemm_run_int8_grouped(G, M, N, K, 1.0, "bf16", x, K, None, codes, i8.padded(K), scales,
                                  0.0, "f32", C, N, offsets, ws, ws.numel())
        sg.sgemm_run_int8(M, N, K, 1.0, "bf16", x, K, None, codes, i8.padded(K), scales, 0.0,
                          "f32", C2, N, ws, ws.numel())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for r in range(4):
        x.copy_(torch.randn(M, K, device="cuda", generator=g))
        offsets.copy_(torch.tensor([[0, 7, 7, 20, 30], [0, 0, 30, 30, 30], [1, 2, 3, 4, 5],
                                    [0, 10, 20, 29, 30]][r], device="cuda"))
        body()
        torch.cuda.synchronize()
        want, want2 = C.clone(), C2.clone()
        C.fill_(9), C2.fill_(9)
        lo, hi = int(offsets[0]), int(offsets[-1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C[lo:hi], want[lo:hi]) and torch.equal(C2, want2)


@pytest.mark.parametrize("M,N,K", [(1 << 19, 5, 33), (3, 1 << 18, 40), (200003, 17, 130)])
@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_very_many_rows_or_columns(M, N, K, kind):
    _product(M, N, K, kind, "f32", pads=(3, 0, 1))
