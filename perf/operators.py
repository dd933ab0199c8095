"""Measured cases of the library's products for layers of experts and for 4-bit weights.

Five operators: products grouped by expert with ragged rows (``sgemm_run_grouped``), the
weights' gradient of such a product (``sgemm_run_grouped_k``), the cast to microscaled 4-bit
floats and back (``sgemm_mxfp4_quantize`` / ``sgemm_mxfp4_dequantize``), the product of
activations with weights held in that format (``sgemm_run_mxfp4``) and the same product
grouped by expert (``sgemm_run_mxfp4_grouped``).

``own`` false computes each operator in its plain form, elementary torch operations in 32
bits; true makes the library's calls.  ``exact`` is the definition in 64 bits.

The 4-bit format: rows of K values padded with zeros to Kp, a multiple of 128.  A block is 32
consecutive values of a row with one scale 2^(s - 127), s = max(E - 2, 0), where E is the
biased exponent of the block's largest magnitude; a value is held as the nearest of
+-{0, 0.5, 1, 1.5, 2, 3, 4, 6} to value / scale, ties to the even code, at most 6.  Codes are
[rows][Kp / 2] bytes, the even k in the low half; scales are [Kp / 128][rows][4] bytes.
"""
import math
import random

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # -- rows of A grouped by expert, weights in 32 bits
        # a decoding step: two dozen rows spread thin over sixteen experts, some without any
        dict(name="grouped decode", op="grouped", groups=16, rows=24, K=2048, N=2048,
             transB=False, sizes=3),
        # a layer's forward pass over a batch of 8192 rows, eight experts of unequal load
        dict(name="grouped forward", op="grouped", groups=8, rows=8192, K=1024, N=2048,
             transB=False, sizes=1),
        # the gradient of its input through transposed weights, many experts, odd widths
        dict(name="grouped odd, B transposed", op="grouped", groups=64, rows=4099, K=777, N=1000,
             transB=True, sizes=2),
        # -- the weights' gradient: rows of A and B summed over, group by group
        dict(name="grouped_k backward", op="grouped_k", groups=8, rows=8192, M=1024, N=2048,
             sizes=1),
        dict(name="grouped_k odd", op="grouped_k", groups=32, rows=1500, M=257, N=1000, sizes=5),
        # -- the cast: a weight matrix at load time; activations of odd width, k along the rows
        dict(name="cast weights", op="cast", rows=8192, K=8192, type="f32", trans=False),
        dict(name="cast odd, transposed", op="cast", rows=1500, K=777, type="bf16", trans=True),
        # -- the product with 4-bit weights
        # one token
        dict(name="mxfp4 one row", op="mxfp4", M=1, N=8192, K=2048, type="bf16", out="bf16"),
        # operands that are both laid out already, odd sizes
        dict(name="mxfp4 odd, laid out", op="mxfp4", M=1000, N=1500, K=777, type="mxfp4",
             out="f32"),
        # a prompt, or a batch in training
        dict(name="mxfp4 large", op="mxfp4", M=8192, N=8192, K=8192, type="bf16", out="bf16"),
        # -- the same grouped by expert: a decoding step, and a prompt
        dict(name="mxfp4_grouped decode", op="mxfp4_grouped", groups=32, rows=48, N=4096, K=2048,
             type="bf16", out="bf16", sizes=7),
        dict(name="mxfp4_grouped prompt", op="mxfp4_grouped", groups=16, rows=8192, N=2048,
             K=2048, type="f32", out="f32", sizes=8),
    ]


def _log(rng, low, high):
    """A whole number, its logarithm uniform over the range; every other one odd."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, n | 1 if rng.random() < 0.5 else n // 64 * 64 if n >= 128 else n))


def draw(rng):
    op = rng.choice(["grouped", "grouped_k", "cast", "mxfp4", "mxfp4_grouped"])
    while True:
        if op == "grouped":
            c = dict(op=op, groups=_log(rng, 1, 128), rows=_log(rng, 1, 16384),
                     K=_log(rng, 64, 4096), N=_log(rng, 64, 4096), transB=rng.random() < 0.5,
                     sizes=rng.randrange(1 << 30))
            if 4 * c["groups"] * c["K"] * c["N"] <= 1 << 30 and \
                    2 * c["rows"] * c["K"] * c["N"] <= 7e10:
                return c
        elif op == "grouped_k":
            c = dict(op=op, groups=_log(rng, 1, 64), rows=_log(rng, 1, 16384),
                     M=_log(rng, 64, 4096), N=_log(rng, 64, 4096), sizes=rng.randrange(1 << 30))
            if 4 * c["groups"] * c["M"] * c["N"] <= 1 << 29 and \
                    2 * c["rows"] * c["M"] * c["N"] <= 7e10:
                return c
        elif op == "cast":
            return dict(op=op, rows=_log(rng, 1, 8192), K=_log(rng, 16, 8192),
                        type=rng.choice(["f32", "bf16"]), trans=rng.random() < 0.5)
        elif op == "mxfp4":
            return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=_log(rng, 64, 8192),
                        type=rng.choice(["f32", "bf16", "mxfp4"]), out=rng.choice(["f32", "bf16"]))
        else:
            c = dict(op=op, groups=_log(rng, 1, 128), rows=_log(rng, 1, 16384),
                     N=_log(rng, 64, 4096), K=_log(rng, 64, 4096),
                     type=rng.choice(["f32", "bf16", "mxfp4"]), out=rng.choice(["f32", "bf16"]),
                     sizes=rng.randrange(1 << 30))
            if c["groups"] * c["N"] * c["K"] <= 1 << 28:
                return c


def _offsets(case):
    """Where each group's rows begin, and the end of the last: unequal shares, as a router gives
    them; with few rows many groups get none."""
    rng = random.Random(case["sizes"])
    load = [rng.expovariate(1.0) for _ in range(case["groups"])]
    at, total, sums = [0], sum(load), 0.0
    for x in load[:-1]:
        sums += x
        at.append(int(case["rows"] * sums / total))
    return at + [case["rows"]]


def _padded(K):
    return (K + 127) // 128 * 128


def _held(rows, K):
    """Bytes of rows x K in the 4-bit format."""
    return rows * (_padded(K) // 2 + _padded(K) // 32)


def work(case):
    op = case["op"]
    if op == "cast":
        n = case["rows"] * case["K"]
        size = 4 if case["type"] == "f32" else 2
        # values in, codes and scales out, values out
        return dict(bytes=2 * size * n + _held(case["rows"], case["K"]), flops=4 * n)
    if op == "mxfp4":
        M, N, K = case["M"], case["N"], case["K"]
        a = dict(f32=4 * M * K, bf16=2 * M * K, mxfp4=_held(M, K))[case["type"]]
        return dict(bytes=a + _held(N, K) + M * N * (4 if case["out"] == "f32" else 2),
                    flops=2 * M * N * K)
    at = _offsets(case)
    used = sum(b > a for a, b in zip(at, at[1:]))  # only groups with rows need their weights
    rows, N = case["rows"], case["N"]
    if op == "grouped":
        K = case["K"]
        return dict(bytes=4 * (rows * K + used * K * N + rows * N), flops=2 * rows * K * N)
    if op == "grouped_k":
        M = case["M"]
        return dict(bytes=4 * (rows * (M + N) + case["groups"] * M * N), flops=2 * rows * M * N)
    K = case["K"]
    a = dict(f32=4 * rows * K, bf16=2 * rows * K, mxfp4=_held(rows, K))[case["type"]]
    return dict(bytes=a + used * _held(N, K) + rows * N * (4 if case["out"] == "f32" else 2),
                flops=2 * rows * K * N)


# ------------------------------------------------- the 4-bit format, in 32 bits
def _blocks(x):
    """x (rows x K) as [rows][Kp / 32][32] floats, zeros past K."""
    rows, K = x.shape
    y = torch.zeros(rows, _padded(K), device=x.device)
    y[:, :K] = x
    return y.view(rows, -1, 32)


def _quantize(x):
    """(codes 0..15 as [rows][Kp / 32][32], scale bytes as [rows][Kp / 32])."""
    b = _blocks(x)
    top = b.abs().amax(2)
    s = (torch.frexp(top).exponent + 124).clamp(min=0)  # frexp: top = m 2^e with m < 1
    s = torch.where(top > 0, s, torch.zeros_like(s))
    y = torch.ldexp(b, (127 - s)[:, :, None])
    m = y.abs()
    n = (m > 0.25).to(torch.uint8)
    n += m >= 0.75
    n += m > 1.25
    n += m >= 1.75
    n += m > 2.5
    n += m >= 3.5
    n += m > 5.0
    n += 8 * torch.signbit(b)
    return n, s.to(torch.uint8)


def _pack(codes, s):
    """The bytes that hold codes and scales."""
    c = codes.reshape(codes.shape[0], -1, 2)
    packed = c[:, :, 0] | (c[:, :, 1] << 4)
    return packed.contiguous(), s.view(s.shape[0], -1, 4).transpose(0, 1).contiguous()


def _unpack(packed, s):
    codes = torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0], -1, 32)
    return codes, s.transpose(0, 1).reshape(packed.shape[0], -1)


def _values(codes, s, K):
    """What codes and scales stand for, rows x K, in 32 bits (exactly)."""
    n = codes & 7
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    v = grid[n.int()]
    v = torch.where(codes > 7, -v, v)
    v = torch.ldexp(v, (s.int() - 127)[:, :, None])
    return v.view(codes.shape[0], -1)[:, :K]


# ------------------------------------------------------------------ the inputs
def _activations(rows, K, g):
    """Normal values with a few channels of large ones, as layers see them."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    loud = torch.rand(K, generator=g, device="cuda") < 1.0 / 64
    return x * torch.where(loud, 8.0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, st = case["op"], dict(case)
    if op == "cast":
        rows, K, t = case["rows"], case["K"], TYPES[case["type"]]
        x = _activations(rows, K, g)
        st["X"] = (x.t() if case["trans"] else x).to(t).contiguous()
        st["Y"] = torch.empty_like(st["X"])
        st["codes"] = torch.empty(rows, _padded(K) // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(_padded(K) // 128, rows, 4, dtype=torch.uint8, device="cuda")
        return st
    rows = case["M"] if op == "mxfp4" else case["rows"]
    groups = 1 if op == "mxfp4" else case["groups"]
    N = case["N"]
    if op != "mxfp4":
        at = _offsets(case)
        st["offsets"] = torch.tensor(at, dtype=torch.int64, device="cuda")
        st["cap"] = max(1, max(b - a for a, b in zip(at, at[1:])))  # rows a plain batch keeps room for
    if op == "grouped":
        K = case["K"]
        st["A"] = _activations(rows, K, g)
        shape = (groups, N, K) if case["transB"] else (groups, K, N)
        st["B"] = torch.randn(shape, generator=g, device="cuda") / math.sqrt(K)
        st["C"] = torch.empty(rows, N, device="cuda")
        return st
    if op == "grouped_k":
        M = case["M"]
        st["A"] = _activations(rows, M, g)
        st["B"] = torch.randn(rows, N, generator=g, device="cuda") / 64
        st["C"] = torch.empty(groups, M, N, device="cuda")
        return st
    K = case["K"]
    x = _activations(rows, K, g)
    if case["type"] == "mxfp4":
        st["A"], st["scalesA"] = _pack(*_quantize(x))
    else:
        st["A"], st["scalesA"] = x.to(TYPES[case["type"]]), None
    st["B"], st["scalesB"] = _pack(*_quantize(
        torch.randn(groups * N, K, generator=g, device="cuda") / math.sqrt(K)))
    st["C"] = torch.empty(rows, N, dtype=TYPES[case["out"]], device="cuda")
    # what a program keeps for the activations in 4 bits
    st["workspace"] = torch.empty(_held(rows, K) + 64, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- the plain forms
def _places(st, rows):
    """For a batch of [groups][cap] rows: the row of each place, whether it is one, and for each
    row its group and place."""
    at, cap = st["offsets"], st["cap"]
    idx = at[:-1, None] + torch.arange(cap, device="cuda")
    inside = idx < at[1:, None]
    r = torch.arange(rows, device="cuda")
    group = torch.searchsorted(at, r, right=True) - 1
    return idx.clamp(max=rows - 1), inside, group, r - at[group]


def _by_group(st, A, Bt):
    """Each row of A times its group's Bt ([groups][K][N]), in 32 bits."""
    idx, inside, group, place = _places(st, A.shape[0])
    batch = A[idx] * inside[:, :, None]
    return torch.bmm(batch, Bt)[group, place]


def _plain(st):
    op = st["op"]
    if op == "grouped":
        B = st["B"].transpose(1, 2).contiguous() if st["transB"] else st["B"]
        return _by_group(st, st["A"], B)
    if op == "grouped_k":
        idx, inside, _, _ = _places(st, st["rows"])
        a = st["A"][idx] * inside[:, :, None]
        b = st["B"][idx] * inside[:, :, None]
        return torch.bmm(a.transpose(1, 2).contiguous(), b)
    if op == "cast":
        x = st["X"].float()
        y = _values(*_quantize(x.t() if st["trans"] else x), st["K"])
        return (y.t() if st["trans"] else y).to(TYPES[st["type"]])
    K, N = st["K"], st["N"]
    if st["type"] == "mxfp4":
        a = _values(*_unpack(st["A"], st["scalesA"]), K)
    else:
        a = _values(*_quantize(st["A"].float()), K)
    b = _values(*_unpack(st["B"], st["scalesB"]), K)
    if op == "mxfp4":
        c = a @ b.t()
    else:
        c = _by_group(st, a, b.view(-1, N, K).transpose(1, 2).contiguous())
    return c.to(TYPES[st["out"]])


# ---------------------------------------------------------- the library's calls
_sg = None


def _library():
    global _sg
    if _sg is None:
        import dense_fp32_matrix_03_amd as sg
        sg.sgemm_create()
        _sg = sg
    return _sg


def _calls(st):
    sg = _library()
    op = st["op"]
    if op == "grouped":
        G, M, N, K = st["groups"], st["rows"], st["N"], st["K"]
        sg.sgemm_run_grouped(st["transB"], G, M, N, K, 1.0, st["A"], K, st["B"],
                             K if st["transB"] else N, K * N, 0.0, st["C"], N, st["offsets"])
        return st["C"]
    if op == "grouped_k":
        G, M, N, K = st["groups"], st["M"], st["N"], st["rows"]
        sg.sgemm_run_grouped_k(G, M, N, K, 1.0, st["A"], M, st["B"], N, 0.0, st["C"], N, M * N,
                               st["offsets"])
        return st["C"]
    if op == "cast":
        rows, K = st["rows"], st["K"]
        ld = rows if st["trans"] else K
        sg.sgemm_mxfp4_quantize(st["trans"], rows, K, st["type"], st["X"], ld, st["codes"],
                                st["scales"], rows)
        sg.sgemm_mxfp4_dequantize(st["trans"], rows, K, st["codes"], st["scales"], rows,
                                  st["type"], st["Y"], ld)
        return st["Y"]
    N, K = st["N"], st["K"]
    M = st["M"] if op == "mxfp4" else st["rows"]
    lda = M if st["type"] == "mxfp4" else K
    ws = st["workspace"]
    if op == "mxfp4":
        sg.sgemm_run_mxfp4(M, N, K, 1.0, st["type"], st["A"], lda, st["scalesA"], st["B"],
                           st["scalesB"], N, 0.0, st["out"], st["C"], N, ws, ws.numel())
    else:
        G = st["groups"]
        sg.sgemm_run_mxfp4_grouped(G, M, N, K, 1.0, st["type"], st["A"], lda, st["scalesA"],
                                   st["B"], st["scalesB"], G * N, 0.0, st["out"], st["C"], N,
                                   st["offsets"], ws, ws.numel())
    return st["C"]


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------ the definitions, 64 bits
def _nearest(x):
    """The 4-bit format's value of each x: [rows][K] doubles."""
    rows, K = x.shape
    b = torch.zeros(rows, _padded(K), dtype=torch.float64, device=x.device)
    b[:, :K] = x
    b = b.view(rows, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.log2(top).floor() - 2
    unit = torch.exp2(torch.where(top > 0, e, torch.zeros_like(e)).clamp(min=-127))
    y = (b.abs() / unit).clamp(max=6)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    y = torch.round(y / step) * step  # round: halves to even
    return (torch.sign(b) * y * unit).view(rows, -1)[:, :K]


def _decoded(packed, s, K):
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    table = torch.tensor(grid + [-v for v in grid], dtype=torch.float64, device=packed.device)
    v = torch.empty(packed.shape[0], packed.shape[1], 2, dtype=torch.float64, device=packed.device)
    v[..., 0] = table[(packed % 16).long()]
    v[..., 1] = table[(packed // 16).long()]
    unit = torch.exp2(s.double() - 127).permute(1, 0, 2).reshape(packed.shape[0], -1, 1)
    return (v.view(packed.shape[0], -1, 32) * unit).view(packed.shape[0], -1)[:, :K]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "cast":
        x = st["X"].double()
        return _nearest(x.t()).t().contiguous() if case["trans"] else _nearest(x)
    if op in ("grouped", "grouped_k"):
        a, b = st["A"].double(), st["B"].double()
    else:
        a = _decoded(st["A"], st["scalesA"], case["K"]) if case["type"] == "mxfp4" else \
            _nearest(st["A"].double())
        b = _decoded(st["B"], st["scalesB"], case["K"])
        if op == "mxfp4":
            return a @ b.t()
        b = b.view(case["groups"], case["N"], case["K"])
    at = _offsets(case)
    if op == "grouped_k":
        return torch.stack([a[i:j].t() @ b[i:j] for i, j in zip(at, at[1:])])
    turned = op == "mxfp4_grouped" or case["transB"]
    return torch.cat([a[i:j] @ (b[n].t() if turned else b[n])
                      for n, (i, j) in enumerate(zip(at, at[1:]))])
