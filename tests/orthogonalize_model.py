"""Newton-Schulz steps in numpy, in 64 bits, and what a computation in two half-precision pieces
may be off by."""
import math

import numpy as np

STEP = (3.4445, -4.7750, 2.0315)


def orthogonalize(x, steps, coefficients, eps, alpha, bits=22):
    """(Y, a bound on the Frobenius norm of what a computed Y is off by) for one matrix.

    With u = 2^-bits the rounding of an operand in pieces, F(.) a Frobenius norm and |.| the largest
    singular value, a product of A (rows by K) and B is off by (3 u) F(A) |B| for the two operands'
    roundings and the left out product of pieces, and by the roundings of a sum of 3 K / 16
    instructions: taken as independent, at four standard deviations, 4 sqrt(3 K / 16) 2^-24 F(A)
    |B|.  A result is rounded to pieces again: u F.  An error E of Z becomes at most L E in a step,
    L the largest slope of p(s) = a s + b s^3 + c s^5 up to |Z| (and of the chords between -|Z| and
    |Z|, which the slopes bound).  S's error reaches P = b S + c S S as |b| + 2 |c| |S| of it, P's
    reaches Z as |Z| of it.
    """
    u = 2.0 ** -bits
    x = x.astype(np.float64)
    norm = math.sqrt((x * x).sum()) + eps
    z = x / norm if norm > 0 else x
    tall = z.shape[0] > z.shape[1]
    z = z.T if tall else z
    m, n = z.shape
    F, top = np.linalg.norm, lambda a: np.linalg.norm(a, 2)

    def per(K):
        return 3 * u + 4 * math.sqrt(3 * (K + 31) / 16) * 2.0 ** -24

    off = 2 * u * F(z) + math.sqrt(m * n) * 2.0 ** -39
    for k in range(steps):
        a, b, c = coefficients[3 * (k if len(coefficients) > 3 else 0):][:3]
        a, b, c = (float(np.float32(v)) for v in (a, b, c))
        s = z @ z.T
        p = b * s + c * s @ s
        new = a * z + p @ z
        zz, ss = top(z), top(s)
        t = np.linspace(0, zz * 1.01 + 1e-30, 2000)
        slope = np.abs(a + 3 * b * t ** 2 + 5 * c * t ** 4).max()
        off_s = per(n) * F(z) * zz + u * F(s)
        off_p = (abs(b) + 2 * abs(c) * ss) * off_s + abs(c) * per(m) * F(s) * ss + u * F(p)
        off = slope * off + off_p * zz + per(m) * F(p) * zz + u * F(new)
        z = new
    z = alpha * (z.T if tall else z)
    return z, abs(alpha) * off * 1.01 + 2.0 ** -23 * F(z)
