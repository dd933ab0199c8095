"""8-bit integers with a scale for each row, in numpy: the cast, and the bits of a product."""
import numpy as np


def padded(K):
    return (K + 127) // 128 * 128


def quantize(x):
    """(codes [rows][padded K], scales) of float32 x."""
    rows, K = x.shape
    codes = np.zeros((rows, padded(K)), np.int8)
    top = np.abs(x).max(1) if K else np.zeros(rows, np.float32)  # NaN where a row has one
    scales = np.where(np.isfinite(top), top / np.float32(127), np.float32(np.nan))
    scales = scales.astype(np.float32)
    some = scales > 0
    q = np.rint(x[some].astype(np.float64) / scales[some, None].astype(np.float64))
    codes[some, :K] = np.clip(q, -127, 127)
    return codes, scales


def products(a, sa, b, sb):
    """((float)sum * scaleA) * scaleB, each step rounded to single precision; and the value in 64
    bits."""
    total = a.astype(np.int64) @ b.astype(np.int64).T
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        v = (total.astype(np.float32) * sa[:, None]) * sb[None, :]
        exact = total.astype(np.float64) * sa[:, None].astype(np.float64) * sb.astype(np.float64)
    return v, exact
