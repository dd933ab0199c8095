"""How near sgemm_orthogonalize has to come to the formula, and its arithmetic in numpy.

A product of operands in two half-precision pieces rounds each of the two to 2^-22 of itself and
leaves out a product of pieces, 2^-22 again, where a single-precision product rounds a term once, to
2^-24: 12 times as much.  Sums are single precision in both.  So a result may be 12 times as far
from the formula in 64 bits as the formula in single precision is: as a whole, and in its worst row,
its worst column and its worst block of 32 x 32, each relative to its own size.
"""
import math

import numpy as np

FACTOR = 12
TILE_CASES = [  # batch, M, N: every tile, with remainders of rows and columns
    (4, 1000, 1000), (1, 1501, 2203), (1, 2203, 1501), (3, 1300, 1403), (3, 1403, 1300),
    (8, 700, 900), (17, 600, 523), (1, 2600, 2603)]


def unequal(kind, shape, size, seed):
    """Matrices whose rows and columns are of unequal size."""
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape)
    if kind in ("rows", "both"):
        x[..., ::2, :] *= size
    if kind in ("columns", "both"):
        x[..., :, 1::3] *= size
    if kind == "graded":
        x *= np.logspace(0, math.log10(size), shape[-2])[:, None]
    if kind == "few":  # one row and one column apart from the rest
        x[..., 3, :] *= size
        x[..., :, 7] *= size
    return x.astype(np.float32)


def formula(x, steps, coefficients, matmul, cast):
    """The formula in the type that `cast` gives, of x already divided by its norm."""
    z = cast(x)
    tall = x.shape[0] > x.shape[1]
    z = z.T if tall else z
    for k in range(steps):
        a, b, c = coefficients[3 * k % len(coefficients):][:3]
        s = matmul(z, z.T)
        z = a * z + matmul(b * s + c * matmul(s, s), z)
    return z.T if tall else z


def singles(coefficients):
    return [float(np.float32(v)) for v in coefficients]


def errors(got, want):
    """(as a whole, worst row, worst column, worst block), relative; numpy arrays in 64 bits."""
    d, w = (got - want) ** 2, want ** 2
    m, n = (-s % 32 for s in d.shape)

    def blocks(a):
        a = np.pad(a, ((0, m), (0, n)))
        return a.reshape(a.shape[0] // 32, 32, a.shape[1] // 32, 32).sum((1, 3))

    def worst(top, under):
        return math.sqrt(np.max(top / np.maximum(under, 1e-300)))

    return (math.sqrt(d.sum() / w.sum()), worst(d.sum(1), w.sum(1)), worst(d.sum(0), w.sum(0)),
            worst(blocks(d), blocks(w)))


def least_of_p(unit):
    """What S S Z of `unit` may be off by besides, for every element: where P = S S alone is far
    below its rows' bound, its elements are held to a least part of that.

    A row's bound is 2^e: Z's row as its largest magnitude and its length bound it, times the
    largest singular value there can be, 1 (exponents are taken with 2% of room).  An element below
    2^15 after 2^(15 - e) is rounded to half of half precision's least step of 2^-24 in its low
    piece at worst, so by 2^-25 2^(e - 15), and that is multiplied by a column of Z.
    """
    z = np.abs(unit.T if unit.shape[0] > unit.shape[1] else unit)
    e = np.minimum(_exponent(z.max(1)) + _exponent(math.sqrt(z.shape[1])), _exponent(1.0)) + _exponent(1.0)
    least = np.ldexp(1.0, e - 40)[:, None] * z.sum(0)[None, :]
    return least.T if unit.shape[0] > unit.shape[1] else least


def check(got, want, single, least=0.0):
    """`got` against the formula in 64 bits, by what the formula in single precision is off by; past
    `least`, if an element may be off by that."""
    got = want + np.sign(got - want) * np.maximum(np.abs(got - want) - least, 0)
    off, allowed = errors(got, want), errors(single, want)
    for name, o, a in zip(("as a whole", "a row", "a column", "a block"), off, allowed):
        assert o <= FACTOR * a, f"{name}: off by {o:.3g}, single precision by {a:.3g}"


# ---------------------------------------------------------------- the library's arithmetic
def _split(v):
    high = v.astype(np.float16)
    low = (v - high.astype(np.float32)).astype(np.float16)
    return high.astype(np.float64), low.astype(np.float64)


def _exponent(bound):
    with np.errstate(divide="ignore"):
        return np.where(bound > 0, np.frexp(np.asarray(bound, np.float64) * 1.02)[1], -1000)


def in_pieces(x, steps, coefficients, dropped=(), by_rows=True, look_again=8):
    """Newton-Schulz steps on x with products in pieces, rows held by their own sizes (or all by the
    whole matrix's); without the products of pieces in `dropped`: "high low", "low high"."""
    tall = x.shape[0] > x.shape[1]
    x = (x.T if tall else x).astype(np.float64)
    z = (x / np.linalg.norm(x)).astype(np.float32)
    m, n = z.shape

    def held(v, e):
        return _split(np.ldexp(v, (15 - e)[:, None]).astype(np.float32))

    def values(a, e):
        return np.ldexp((a[0] + a[1]).astype(np.float32), e[:, None] - 15)

    def nearer(a, ea, b, eb):
        """Elements held by their rows in a and, transposed, by their columns in b: as the smaller
        range has them."""
        return np.where(ea[:, None] < eb[None, :], values(a, ea), values(b, eb).T)

    def product(a, ea, b, eb):
        total = a[0] @ b[0].T
        if "high low" not in dropped:
            total += a[0] @ b[1].T
        if "low high" not in dropped:
            total += a[1] @ b[0].T
        return np.ldexp(total.astype(np.float32).astype(np.float64),
                        ea[:, None] + eb[None, :] - 30).astype(np.float32)

    def symmetric(a):
        return np.tril(a) + np.tril(a, -1).T

    def sizes(axis):
        top = np.abs(z).max(axis)
        return _exponent(top.astype(np.float64)) + _exponent(math.sqrt(z.shape[axis]))

    bound, growth, rows, columns = 1.0, 1.0, sizes(1), sizes(0)
    e, ec = (np.clip(v, -100, _exponent(bound)) for v in (rows, columns))
    for k in range(steps):
        a, b, c = coefficients[3 * k % len(coefficients):][:3]
        if not by_rows:
            e, ec = np.full(m, _exponent(bound)), np.full(n, _exponent(bound))
        now = np.clip(rows + _exponent(growth), -100, _exponent(bound)) if by_rows else e
        Z, Zt = held(z, e), held(z.T, ec)
        s = symmetric(product(Z, e, Z, e))
        es = np.maximum(now + _exponent(bound), -100)
        S = held(s, es)
        p = symmetric(np.float32(c) * product(S, es, S, es) + np.float32(b) * nearer(S, es, S, es))
        ep = np.maximum(now + _exponent(bound * (abs(b) + abs(c) * bound ** 2)), -100)
        z = np.float32(a) * nearer(Z, e, Zt, ec) + product(held(p, ep), ep, Zt, ec)
        t = np.linspace(0, bound, 4001)
        growth *= 1.001 * np.abs(a + b * t ** 2 + c * t ** 4).max()
        bound = 1.001 * np.abs(a * t + b * t ** 3 + c * t ** 5).max()
        e, ec = (np.clip(v + _exponent(growth), -100, _exponent(bound)) for v in (rows, columns))
        if (k + 1) % look_again == 0:
            rows, columns, growth = sizes(1), sizes(0), 1.0
    return z.T if tall else z
