"""The microscaled 4-bit format in numpy, from its definition
(include/sgemm_mxfp4.h), in 64 bits."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def padded(K):
    return (K + 127) // 128 * 128


def quantize(x):
    """x (rows x K float32): codes [rows][Kp/2] and scales [Kp/128][rows][4], uint8."""
    rows, K = x.shape
    b = np.zeros((rows, padded(K)), np.float32)
    b[:, :K] = x
    b = b.reshape(rows, -1, 32)
    finite = np.isfinite(b).all(2)
    v = np.where(finite[:, :, None], b, 0).astype(np.float64)
    top = np.abs(v).max(2)
    # the biased exponent of the largest magnitude: 2^(E - 127) <= top, 0 below the normal range
    e = np.where(top >= 2.0 ** -126, np.frexp(top)[1] + 126, 0)
    s = np.maximum(e - 2, 0)
    m = np.minimum(np.abs(v) / np.exp2(s - 127.0)[:, :, None], 6.0)
    # the nearest grid value; of two equally near, the even index
    d = np.abs(m[..., None] - GRID)
    near = d.min(-1, keepdims=True)
    hit = d == near
    even = hit & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), hit.argmax(-1))
    code = (code + 8 * np.signbit(b)).astype(np.uint8)
    code[~finite] = 0
    s = np.where(finite, s, 255).astype(np.uint8)
    flat = code.reshape(rows, -1)
    packed = flat[:, 0::2] | flat[:, 1::2] << 4
    return packed, np.ascontiguousarray(s.reshape(rows, -1, 4).transpose(1, 0, 2))


def values(packed, scales, K):
    """What a held matrix stands for, rows x K doubles."""
    rows = packed.shape[0]
    code = np.stack([packed & 15, packed >> 4], 2).reshape(rows, -1, 32)
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    s = scales[:, :rows].transpose(1, 0, 2).reshape(rows, -1).astype(np.float64)
    unit = np.where(s == 255, np.nan, np.exp2(s - 127))
    return (v * unit[:, :, None]).reshape(rows, -1)[:, :K]


def bf16_bits(x):
    """float32 -> bfloat16 bits, to the nearest, ties to even (finite x)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + (u >> 16 & 1)) >> 16).astype(np.uint16)


def bf16_floats(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)
