"""Microscaled 4-bit operands (sgemm_mxfp4_quantize, sgemm_mxfp4_dequantize,
sgemm_run_mxfp4, sgemm_run_mxfp4_grouped) against the format's definition and
sums in 64 bits.

The casts are compared bit for bit.  Products: |C - exact| <= 1e-5 sum
|products| + 1e-6 before C is rounded to its type (products of elements are
exact; the sum of K terms in single precision is off by about sqrt(K) 2^-24 of
it), and a bfloat16 C is off by 2^-8 of its value more.
"""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
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
    """x (float32, 2-D) on the GPU as `kind` with leading dimension ld, its
    start moved by `shift` elements; and the float32 values it holds."""
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
    held = mx.bf16_floats(bits) if kind == "bf16" else x
    return t, held


def _values(seed, shape, kind="normal"):
    g = np.random.default_rng(seed)
    if kind == "wide":  # magnitudes over the whole range of single precision
        x = g.standard_normal(shape) * np.exp2(g.integers(-150, 126, shape))
    elif kind == "ties":  # halfway points of the format among its values
        x = g.choice([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9], shape)
        x = x * g.choice([-1, 1], shape) * np.exp2(g.integers(-3, 4, (shape[0], 1)))
    elif kind == "sparse":
        x = g.standard_normal(shape) * (g.random(shape) < 0.02)
    elif kind == "special":
        x = g.standard_normal(shape)
        for v in (np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, 3.4e38, 1e-45):
            x[tuple(g.integers(0, n, 3) for n in shape)] = v
    else:
        x = g.standard_normal(shape)
    with np.errstate(over="ignore", under="ignore"):
        x = x.astype(np.float32)
    return np.where(np.isinf(x) & (kind != "special"), np.float32(1), x)


def _quantize(x, kind, trans, ld_pad=0, lds_pad=0, shift=0):
    import torch
    rows, K = x.shape
    stored = np.ascontiguousarray(x.T) if trans else x
    ld = stored.shape[1] + ld_pad
    dX, held = _typed(stored, kind, ld, shift)
    lds = rows + lds_pad
    codes = torch.full((rows, mx.padded(K) // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((mx.padded(K) // 128, lds, 4), 0xA5, dtype=torch.uint8, device="cuda")
    sg.sgemm_mxfp4_quantize(trans, rows, K, kind, dX, ld, codes, scales, lds)
    torch.cuda.synchronize()
    return codes, scales, held.T if trans else held


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("values", ["normal", "wide", "ties", "sparse", "special"])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 32), (33, 128), (70, 300), (130, 517), (257, 1024)])
def test_quantize(rows, K, values, kind, trans):
    codes, scales, held = _quantize(_values(rows + K, (rows, K), values), kind, trans)
    want, want_s = mx.quantize(held)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("ld_pad,lds_pad,shift", [(1, 3, 1), (8, 1, 0), (5, 64, 3), (0, 0, 2)])
def test_quantize_strides(kind, trans, ld_pad, lds_pad, shift):
    rows, K = 75, 333
    codes, scales, held = _quantize(_values(5, (rows, K)), kind, trans, ld_pad, lds_pad, shift)
    want, want_s = mx.quantize(held)
    assert np.array_equal(codes.cpu().numpy(), want)
    s = scales.cpu().numpy()
    assert np.array_equal(s[:, :rows], want_s)
    assert (s[:, rows:] == 0xA5).all()


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_dequantize_every_scale_and_code(kind, trans):
    """256 scales by 16 codes; values past the type's range are infinite."""
    import torch
    rows, K = 256, 70
    g = np.random.default_rng(2)
    packed = g.integers(0, 256, (rows, mx.padded(K) // 2)).astype(np.uint8)
    packed[:, :8] = np.arange(8, dtype=np.uint8) * 0x22 + 0x10  # all sixteen codes
    scales = g.integers(0, 256, (1, rows + 3, 4)).astype(np.uint8)
    scales[0, :rows, 0] = np.arange(256)
    want = mx.values(packed, scales, K)
    ld = (rows if trans else K) + 5
    shape = (K if trans else rows, ld)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    X = torch.full(shape, 9.0, dtype=t, device="cuda")
    sg.sgemm_mxfp4_dequantize(trans, rows, K, _cuda(packed), _cuda(scales), rows + 3, kind, X, ld)
    out = X.float().cpu().numpy()
    assert (out[:, ld - 5:] == 9).all()
    out = out[:, :ld - 5].T if trans else out[:, :ld - 5]
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)
    assert np.array_equal(out, want, equal_nan=True)
    assert np.array_equal(np.signbit(out), np.signbit(want)) or np.isnan(want).any()


def _held(x):
    """(codes, scales, values): x cast by the model."""
    packed, s = mx.quantize(x)
    return packed, s, mx.values(packed, s, x.shape[1])


def _check(C, ref, mag, out):
    err = np.abs(C.astype(np.float64) - ref)
    tol = 1e-5 * mag + 1e-6 + (2.0 ** -8 * np.abs(ref) if out == "bf16" else 0)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}, "
                           f"worst {np.nanmax(err / tol):.3g}")


def _product(M, N, K, kind, out, alpha=1.0, beta=0.0, pads=(0, 0, 0), shift=0, seed=0,
             lengths=None, before=0, values="normal"):
    """One product on the GPU, C as float32, and in 64 bits: C, ref, sum |products|."""
    import torch
    G = 1 if lengths is None else len(lengths)
    x, w = _values(seed + M, (M, K), values), _values(seed + N + 1, (G * N, K))
    pw, sw, w = _held(w)
    ldsb = G * N + pads[1]
    sB = np.full((sw.shape[0], ldsb, 4), 255, np.uint8)
    sB[:, :G * N] = sw
    if kind == "mxfp4":
        px, sx, xv = _held(x)
        lda = M + pads[0]
        sA = np.full((sx.shape[0], lda, 4), 255, np.uint8)
        sA[:, :M] = sx
        dA, dsA, ws = _cuda(px), _cuda(sA), None
    else:
        lda = max(K, 1) + pads[0]
        dA, held = _typed(x, kind, lda, shift) if K else (_cuda(np.zeros(8, np.float32)), x)
        dsA, xv = None, mx.values(*mx.quantize(held), K)
        ws = torch.full((sg.sgemm_mxfp4_workspace_size(kind, M, K) + 16,), 0xFF, dtype=torch.uint8,
                        device="cuda")
    ldc = N + pads[2]
    C0 = _values(seed + 3, (M, ldc))
    dC, C0 = _typed(C0, out, ldc, shift)
    n = 0 if ws is None else ws.numel() - 16
    if lengths is None:
        at = np.array([0, M])
        sg.sgemm_run_mxfp4(M, N, K, alpha, kind, dA, lda, dsA, _cuda(pw), _cuda(sB), ldsb, beta,
                           out, dC, ldc, ws, n)
    else:
        at = np.cumsum([before] + list(lengths)).astype(np.int64)
        sg.sgemm_run_mxfp4_grouped(G, M, N, K, alpha, kind, dA, lda, dsA, _cuda(pw), _cuda(sB),
                                   ldsb, beta, out, dC, ldc, _cuda(at), ws, n)
    torch.cuda.synchronize()
    C = dC[:M * ldc].float().cpu().numpy().reshape(M, ldc)
    if ws is not None:
        assert (ws[n:] == 0xFF).all()
    ref, mag = np.empty((M, N)), np.empty((M, N))
    inside = np.zeros((M, ldc), bool)
    for g, (i, j) in enumerate(zip(at, at[1:])):
        a, b = xv[i:j], w[g * N:(g + 1) * N]
        c0 = C0[i:j, :N].astype(np.float64)
        add = beta * c0 if beta != 0 else 0.0
        ref[i:j] = alpha * (a @ b.T) + add
        mag[i:j] = abs(alpha) * (np.abs(a) @ np.abs(b).T) + np.abs(add)
        inside[i:j, :N] = True
    assert np.array_equal(C[~inside], C0[~inside])
    keep = inside[:, :N]
    return C[:, :N][keep], ref[keep], mag[keep]


SIZES = [(1, 1, 1), (1, 64, 128), (5, 33, 45), (16, 128, 512), (17, 100, 700), (40, 129, 1000),
         (70, 257, 333), (130, 300, 2050), (300, 520, 640), (1, 130, 9000), (2, 77, 2600),
         (12, 200, 4500), (30, 333, 5000), (90, 200, 4200), (31, 65, 130)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "mxfp4"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, kind, out):
    _check(*_product(M, N, K, kind, out), out)


# Enough tiles of 128 x 128 for the 256 x 256 tile, ragged in all directions.
@pytest.mark.parametrize("K", [1, 129, 260, 640])
@pytest.mark.parametrize("kind,out,alpha,beta", [("f32", "f32", 1.0, 0.0), ("mxfp4", "bf16", 1.0, 0.0),
                                                 ("bf16", "f32", -0.5, 2.0)])
def test_product_of_many_tiles(K, kind, out, alpha, beta):
    _check(*_product(4120, 3990, K, kind, out, alpha, beta, pads=(3, 2, 1)), out)


@pytest.mark.parametrize("M,N,K", [(65, 130, 8320), (40, 129, 6150), (250, 8190, 6150),
                                   (33, 300, 20000)])
@pytest.mark.parametrize("kind,out,alpha,beta", [("f32", "f32", 1.0, 0.0), ("mxfp4", "bf16", 0.5, 2.0)])
def test_product_of_few_tiles_and_long_sums(M, N, K, kind, out, alpha, beta):
    _check(*_product(M, N, K, kind, out, alpha, beta, pads=(1, 2, 3)), out)


SPREAD = {"one each": [1, 0, 0, 2, 1, 0, 0, 1], "two tiles in one": [18] + [0] * 15,
          "all in the last": [0] * 7 + [13], "seventy": [(n * 3) % 4 // 3 for n in range(70)],
          "none": [0, 0]}


@pytest.mark.parametrize("groups", SPREAD)
@pytest.mark.parametrize("N,K", [(1, 32), (33, 129), (150, 700), (40, 2050)])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("mxfp4", "f32")])
def test_grouped_rows_spread_thin(groups, N, K, kind, out):
    _check(*_product(sum(SPREAD[groups]) + 3, N, K, kind, out, lengths=SPREAD[groups], before=1), out)


@pytest.mark.parametrize("kind", ["f32", "mxfp4"])
@pytest.mark.parametrize("alpha,beta,pads,shift", [(0.5, 2.0, (1, 2, 3), 1), (1.0, 1.0, (0, 0, 1), 0),
                                                   (0.0, 0.5, (0, 0, 0), 0)])
def test_grouped_rows_spread_thin_strides_alpha_beta(kind, alpha, beta, pads, shift):
    lengths = SPREAD["one each"]
    _check(*_product(sum(lengths), 75, 600, kind, "f32", alpha, beta, pads, shift, lengths=lengths),
           "f32")


@pytest.mark.parametrize("rows", [3, 90])
def test_rows_of_b_past_four_gigabytes(rows):
    """Two groups' B of 2.5 GB each: all zero but for the last rows of either."""
    import torch
    N, K, some = 150000, 32768, 40
    g = np.random.default_rng(rows)
    codes = torch.zeros(2 * N * (K // 2), dtype=torch.uint8, device="cuda").view(2 * N, K // 2)
    scales = torch.zeros(K // 128, 2 * N, 4, dtype=torch.uint8, device="cuda")
    pb, sb = mx.quantize(_values(rows, (2 * some, K)))
    pa, sa = mx.quantize(_values(rows + 1, (rows, K)))
    for n in (0, 1):
        end = (n + 1) * N
        codes[end - some:end] = _cuda(pb[n * some:(n + 1) * some])
        scales[:, end - some:end] = _cuda(np.ascontiguousarray(sb[:, n * some:(n + 1) * some]))
    at = np.array([0, rows // 3, rows], np.int64)
    C = torch.full((rows, N), 7.0, device="cuda")
    sg.sgemm_run_mxfp4_grouped(2, rows, N, K, 1.0, "mxfp4", _cuda(pa), rows, _cuda(sa), codes,
                               scales, 2 * N, 0.0, "f32", C, N, _cuda(at))
    assert (C[:, :N - some] == 0).all()
    a, b = mx.values(pa, sa, K), mx.values(pb, sb, K)
    for n in (0, 1):
        i, j, bn = at[n], at[n + 1], b[n * some:(n + 1) * some]
        _check(C[i:j, N - some:].cpu().numpy(), a[i:j] @ bn.T, np.abs(a[i:j]) @ np.abs(bn).T, "f32")
    # both groups' rows as one matrix, by the kernel for few rows
    few = min(rows, 20)
    D = torch.full((few, 2 * N), 7.0, device="cuda")
    sg.sgemm_run_mxfp4(few, 2 * N - 1, K, 1.0, "mxfp4", _cuda(pa), rows, _cuda(sa), codes, scales,
                       2 * N, 0.0, "f32", D, 2 * N)
    assert (D[:, 2 * N - 1] == 7).all() and (D[:, N:2 * N - some] == 0).all()
    _check(D[:, 2 * N - some:2 * N - 1].cpu().numpy(), a[:few] @ b[some:2 * some - 1].T,
           np.abs(a[:few]) @ np.abs(b[some:2 * some - 1]).T, "f32")


def test_product_exact_on_many_tiles():
    """Values of the format itself under one scale: every sum is exact."""
    import torch
    M, N, K = 3900, 4200, 384
    g = np.random.default_rng(8)
    pa, pb = (g.integers(0, 256, (r, K // 2)).astype(np.uint8) for r in (M, N))
    sa, sb = (np.full((K // 128, r, 4), 127, np.uint8) for r in (M, N))
    C = torch.empty(M, N, device="cuda")
    sg.sgemm_run_mxfp4(M, N, K, 1.0, "mxfp4", _cuda(pa), M, _cuda(sa), _cuda(pb), _cuda(sb), N,
                       0.0, "f32", C, N)
    ref = mx.values(pa, sa, K) @ mx.values(pb, sb, K).T
    assert np.array_equal(C.cpu().numpy(), ref)


def test_grouped_of_many_tiles():
    lengths = [1500, 0, 2700, 33, 1000]
    for kind, out in (("bf16", "bf16"), ("mxfp4", "f32")):
        _check(*_product(sum(lengths) + 10, 4000, 300, kind, out, lengths=lengths, before=4), out)


@pytest.mark.parametrize("M,N,K", [(3, 70, 300), (90, 140, 400), (257, 300, 513)])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("mxfp4", "f32")])
@pytest.mark.parametrize("alpha,beta", [(-1.5, 0.0), (0.5, 2.0), (1.0, -1.0), (0.0, 0.5),
                                        (0.0, 0.0)])
def test_product_alpha_beta(M, N, K, kind, out, alpha, beta):
    _check(*_product(M, N, K, kind, out, alpha, beta), out)


@pytest.mark.parametrize("M,N,K", [(2, 70, 300), (90, 141, 401), (257, 260, 256)])
@pytest.mark.parametrize("kind,out", [("f32", "bf16"), ("bf16", "f32"), ("mxfp4", "bf16")])
@pytest.mark.parametrize("pads,shift", [((1, 3, 1), 1), ((8, 0, 4), 2), ((0, 5, 0), 3)])
def test_product_strides(M, N, K, kind, out, pads, shift):
    _check(*_product(M, N, K, kind, out, pads=pads, shift=shift), out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product_without_k(out):
    C, ref, mag = _product(40, 50, 0, "f32", out)
    assert not C.any()
    _check(*_product(40, 50, 0, "f32", out, 1.0, -0.5), out)


def test_empty_sum_does_not_multiply_alpha():
    import torch
    for M in (3, 100):
        C = torch.full((M, 5), 2.0, device="cuda")
        sg.sgemm_run_mxfp4(M, 5, 0, float("inf"), "f32", None, 1, None, None, None, 5, 0.5, "f32",
                           C, 5)
        assert (C == 1).all()


@pytest.mark.parametrize("M,N,K", [(4, 80, 400), (3, 50, 5000), (16, 70, 3000), (30, 90, 2500),
                                   (100, 200, 300), (300, 300, 600), (70, 100, 4500)])
def test_casting_on_the_way_gives_the_bits_of_the_cast(M, N, K):
    import torch
    for kind in ("f32", "bf16"):
        x = _values(M, (M, K))
        codes, scales, _ = _quantize(x, kind, 0)
        pw, sw, _ = _held(_values(N, (N, K)))
        dw, dsw = _cuda(pw), _cuda(sw)
        a, b = (torch.empty(M, N, device="cuda") for _ in range(2))
        sg.sgemm_run_mxfp4(M, N, K, 1.0, "mxfp4", codes, M, scales, dw, dsw, N, 0.0, "f32", a, N)
        n = sg.sgemm_mxfp4_workspace_size(kind, M, K)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dX, _ = _typed(x, kind)
        sg.sgemm_run_mxfp4(M, N, K, 1.0, kind, dX, K, None, dw, dsw, N, 0.0, "f32", b, N, ws, n)
        assert a.cpu().numpy().tobytes() == b.cpu().numpy().tobytes()


@pytest.mark.parametrize("kind", ["f32", "mxfp4"])
@pytest.mark.parametrize("M", [5, 40, 260])
def test_nan_blocks_reach_their_rows_only(M, kind):
    import torch
    N, K = 290, 700
    x, w = _values(1, (M, K)), _values(2, (N, K))
    x[2, 650], x[4, 3], w[7, 40], w[270, 699] = np.nan, np.inf, -np.inf, np.nan
    px, sx, xv = _held(x)
    pw, sw, wv = _held(w)
    C = torch.empty(M, N, device="cuda")
    n = sg.sgemm_mxfp4_workspace_size(kind, M, K)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    if kind == "mxfp4":
        sg.sgemm_run_mxfp4(M, N, K, 1.0, kind, _cuda(px), M, _cuda(sx), _cuda(pw), _cuda(sw), N,
                           0.0, "f32", C, N)
    else:
        sg.sgemm_run_mxfp4(M, N, K, 1.0, kind, _cuda(x), K, None, _cuda(pw), _cuda(sw), N, 0.0,
                           "f32", C, N, ws, n)
    C = C.cpu().numpy()
    nan = np.zeros((M, N), bool)
    nan[[2, 4]] = True
    nan[:, [7, 270]] = True
    assert np.array_equal(np.isnan(C), nan)
    xv, wv = np.nan_to_num(xv), np.nan_to_num(wv)
    _check(C[~nan], (xv @ wv.T)[~nan], (np.abs(xv) @ np.abs(wv).T)[~nan], "f32")


def test_scales_of_opposite_ends():
    """2^-127 on one side and 2^127 on the other: the scales' product is formed
    with more range than single precision has."""
    import torch
    M, N, K = 40, 48, 256
    g = np.random.default_rng(4)
    pa, pb = (g.integers(0, 256, (r, K // 2)).astype(np.uint8) for r in (M, N))
    sa, sb = np.zeros((2, M, 4), np.uint8), np.full((2, N, 4), 254, np.uint8)
    C = torch.empty(M, N, device="cuda")
    sg.sgemm_run_mxfp4(M, N, K, 1.0, "mxfp4", _cuda(pa), M, _cuda(sa), _cuda(pb), _cuda(sb), N,
                       0.0, "f32", C, N)
    assert np.array_equal(C.cpu().numpy(), mx.values(pa, sa, K) @ mx.values(pb, sb, K).T)


GROUPS = {
    "one row": ([1], 0, 0),
    "empty ones": ([0, 5, 0, 0, 17, 1, 0], 0, 0),
    "all empty": ([0, 0, 0], 3, 4),
    "rows outside": ([16, 33, 2], 5, 9),
    "one large": ([3, 300, 1, 2], 0, 1),
    "two hundred": ([(7 * g) % 5 for g in range(200)], 1, 1),
    "several tiles": ([260, 131, 0, 129], 0, 0),
}


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("mxfp4", "f32")])
@pytest.mark.parametrize("N,K", [(1, 1), (64, 128), (45, 333), (300, 1030)])
def test_grouped(groups, N, K, kind, out):
    lengths, before, after = GROUPS[groups]
    M = before + sum(lengths) + after
    _check(*_product(M, N, K, kind, out, lengths=lengths, before=before), out)


@pytest.mark.parametrize("groups", ["rows outside", "several tiles"])
@pytest.mark.parametrize("pads,shift,alpha,beta", [((1, 3, 1), 1, 1.0, 0.0), ((8, 0, 4), 2, -0.5, 2.0),
                                                   ((0, 5, 0), 3, 0.0, 0.5)])
@pytest.mark.parametrize("kind,out", [("f32", "bf16"), ("bf16", "f32"), ("mxfp4", "bf16")])
def test_grouped_strides_alpha_beta(groups, kind, out, pads, shift, alpha, beta):
    lengths, before, after = GROUPS[groups]
    M = before + sum(lengths) + after
    _check(*_product(M, 141, 401, kind, out, alpha, beta, pads, shift, lengths=lengths,
                     before=before), out)


@pytest.mark.parametrize("at", [[0, 40, 20, 50], [-7, 10, 60, 90], [50, 0, 50, 0],
                                [2 ** 62, 3, -2 ** 63, 50]])
def test_offsets_out_of_range_write_nothing_outside(at):
    import torch
    M, N, K, G = 50, 40, 136, 3
    d_at = torch.tensor(at, dtype=torch.int64, device="cuda")
    A = torch.randn(M, K, device="cuda")
    pw, sw, _ = _held(_values(1, (G * N, K)))
    n = sg.sgemm_mxfp4_workspace_size("f32", M, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    C = torch.full((M + 40, N), 7.0, device="cuda")
    sg.sgemm_run_mxfp4_grouped(G, M, N, K, 1.0, "f32", A, K, None, _cuda(pw), _cuda(sw), G * N,
                               0.0, "f32", C[20:], N, d_at, ws, n)
    torch.cuda.synchronize()
    assert (C[:20] == 7).all() and (C[20 + M:] == 7).all() and torch.isfinite(C).all()


def test_rows_outside_the_groups_do_not_matter():
    """NaN in rows of A that belong to no group reaches nothing."""
    import torch
    M, N, K, G = 60, 50, 200, 2
    at = np.array([10, 30, 45], np.int64)
    x = _values(1, (M, K))
    x[:10] = x[45:] = np.nan
    pw, sw, w = _held(_values(2, (G * N, K)))
    n = sg.sgemm_mxfp4_workspace_size("f32", M, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    C = torch.full((M, N), 3.0, device="cuda")
    sg.sgemm_run_mxfp4_grouped(G, M, N, K, 1.0, "f32", _cuda(x), K, None, _cuda(pw), _cuda(sw),
                               G * N, 0.0, "f32", C, N, _cuda(at), ws, n)
    C = C.cpu().numpy()
    assert (C[:10] == 3).all() and (C[45:] == 3).all()
    xv = mx.values(*mx.quantize(np.nan_to_num(x)), K)
    for g in range(G):
        a, b = xv[at[g]:at[g + 1]], w[g * N:(g + 1) * N]
        _check(C[at[g]:at[g + 1]], a @ b.T, np.abs(a) @ np.abs(b).T, "f32")


@pytest.mark.parametrize("M", [3, 200])
def test_in_a_graph(M):
    """The cast of weights, a product and a grouped product, captured together
    and replayed on other activations and group lengths."""
    import torch
    N, K, G = 96, 260, 3
    w = torch.randn(G * N, K, device="cuda")
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(G * N, mx.padded(K) // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(mx.padded(K) // 128, G * N, 4, dtype=torch.uint8, device="cuda")
    n = sg.sgemm_mxfp4_workspace_size("bf16", M, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    C, D = (torch.empty(M, N, device="cuda") for _ in range(2))
    at = torch.zeros(G + 1, dtype=torch.int64, device="cuda")

    def body():
        sg.sgemm_mxfp4_quantize(0, G * N, K, "f32", w, K, codes, scales, G * N)
        sg.sgemm_run_mxfp4(M, N, K, 1.0, "bf16", x, K, None, codes[N:], scales[:, N:], G * N, 0.0,
                           "f32", C, N, ws, n)
        sg.sgemm_run_mxfp4_grouped(G, M, N, K, 1.0, "bf16", x, K, None, codes, scales, G * N, 0.0,
                                   "f32", D, N, at, ws, n)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        body()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for r in range(4):
        x.copy_(torch.randn(M, K, device="cuda"))
        w.copy_(torch.randn(G * N, K, device="cuda"))
        at.copy_(torch.tensor([0, M // (r + 1), M // (r + 1), M]))
        C.fill_(5.0), D.fill_(5.0)
        body()
        torch.cuda.synchronize()
        want = C.cpu().numpy().tobytes(), D.cpu().numpy().tobytes()
        C.fill_(6.0), D.fill_(6.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (C.cpu().numpy().tobytes(), D.cpu().numpy().tobytes()) == want
        xv = mx.values(*mx.quantize(x.float().cpu().numpy()), K)
        wv = mx.values(*mx.quantize(w.cpu().numpy()), K)[N:2 * N]
        _check(C.cpu().numpy(), xv @ wv.T, np.abs(xv) @ np.abs(wv).T, "f32")


def test_an_expert_layer_with_4_bit_weights():
    """Weights stored as sgemm_run takes them (K x N), cast transposed expert
    by expert, then the layer's two products; against the model."""
    import torch
    G, M, K, H, N = 3, 90, 200, 264, 130
    at = np.array([0, 40, 40, 90], np.int64)
    x, w1, w2 = _values(1, (M, K)), _values(2, (G, K, H)), _values(3, (G, H, N))

    def cast(w):
        _, k, n = w.shape
        codes = torch.empty(G * n, mx.padded(k) // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(mx.padded(k) // 128, G * n, 4, dtype=torch.uint8, device="cuda")
        d = _cuda(w)
        for g in range(G):
            sg.sgemm_mxfp4_quantize(1, n, k, "f32", d[g], n, codes[g * n:], scales[:, g * n:],
                                    G * n)
        return codes, scales

    (c1, s1), (c2, s2) = cast(w1), cast(w2)
    h = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(M, N, device="cuda")
    n = max(sg.sgemm_mxfp4_workspace_size("f32", M, K), sg.sgemm_mxfp4_workspace_size("bf16", M, H))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    sg.sgemm_run_mxfp4_grouped(G, M, H, K, 0.1, "f32", _cuda(x), K, None, c1, s1, G * H, 0.0,
                               "bf16", h, H, _cuda(at), ws, n)
    sg.sgemm_run_mxfp4_grouped(G, M, N, H, 1.0, "bf16", h, H, None, c2, s2, G * N, 0.0, "f32", y,
                               N, _cuda(at), ws, n)
    xv = mx.values(*mx.quantize(x), K)
    hidden = h.float().cpu().numpy()
    hv = mx.values(*mx.quantize(hidden), H)
    for g in range(G):
        i, j = at[g], at[g + 1]
        b1 = mx.values(*mx.quantize(np.ascontiguousarray(w1[g].T)), K).T
        b2 = mx.values(*mx.quantize(np.ascontiguousarray(w2[g].T)), H).T
        if j > i:
            _check(hidden[i:j], 0.1 * (xv[i:j] @ b1), 0.1 * (np.abs(xv[i:j]) @ np.abs(b1)), "bf16")
            _check(y.cpu().numpy()[i:j], hv[i:j] @ b2, np.abs(hv[i:j]) @ np.abs(b2), "f32")


def test_two_streams_with_a_workspace_each():
    import torch
    M, N, K = 70, 520, 900
    w = torch.randn(N, K, device="cuda")
    codes = torch.empty(N, mx.padded(K) // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(mx.padded(K) // 128, N, 4, dtype=torch.uint8, device="cuda")
    sg.sgemm_mxfp4_quantize(0, N, K, "f32", w, K, codes, scales, N)
    X = [torch.randn(M, K, device="cuda") for _ in range(2)]
    C = [torch.zeros(M, N, device="cuda") for _ in range(2)]
    n = sg.sgemm_mxfp4_workspace_size("f32", M, K)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            sg.sgemm_run_mxfp4(M, N, K, 1.0, "f32", X[i], K, None, codes, scales, N, 0.0, "f32",
                               C[i], N, ws[i], n, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        alone = torch.zeros(M, N, device="cuda")
        sg.sgemm_run_mxfp4(M, N, K, 1.0, "f32", X[i], K, None, codes, scales, N, 0.0, "f32", alone,
                           N, ws[0], n)
        assert torch.equal(alone, C[i])


def test_the_most_groups():
    lengths = [n % 5 // 4 for n in range(4095)] + [200]
    for kind, out in (("f32", "f32"), ("mxfp4", "bf16")):
        _check(*_product(sum(lengths), 33, 150, kind, out, lengths=lengths), out)


@pytest.mark.parametrize("M,N,K", [(5, 70, 300), (40, 70, 512), (200, 300, 256), (700, 8192, 256)])
def test_beta_c_is_rounded_before_it_is_added(M, N, K):
    """alpha sum + beta C is one fused multiply-add on beta C rounded to single
    precision, bit for bit (the sums are exact: small integers)."""
    import torch
    g = np.random.default_rng(M)
    a, b = (g.integers(-3, 4, (n, K)).astype(np.float32) for n in (M, N))
    a[:, ::32], b[:, ::32] = 4, 4  # scales of 1: the values are held as they are
    ca, sa, _ = _quantize(a, "f32", 0)
    cb, sb, _ = _quantize(b, "f32", 0)
    C0 = g.standard_normal((M, N)).astype(np.float32)
    alpha, beta = np.float32(0.7), np.float32(-1 / 3)
    C = _cuda(C0)
    sg.sgemm_run_mxfp4(M, N, K, float(alpha), "mxfp4", ca, M, sa, cb, sb, N, float(beta), "f32", C, N)
    sums = a.astype(np.float64) @ b.astype(np.float64).T
    # 24 + 24 bits and an addend near them: rounded in 64 bits only where the last bit of 53 decides
    want = (np.float64(alpha) * sums + (beta * C0).astype(np.float64)).astype(np.float32)
    got = C.cpu().numpy()
    assert np.array_equal(got, want)
    # The other reading, one rounding in all, differs where beta C's (2^-26) moves a result of
    # about 2^7 (spacing 2^-16) over a halfway point: in about M N / 2^9 places, too few at 5 x 70.
    if M > 5:
        once = (np.float64(alpha) * sums + np.float64(beta) * C0).astype(np.float32)
        assert not np.array_equal(got, once)
