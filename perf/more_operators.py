"""Measured cases of the library's operators around the products of a layer of experts.

Four operators: routing rows (tokens) to experts and its gradient (``sgemm_route``,
``sgemm_route_backward``); taking rows to their experts and back, with the gradient
(``sgemm_route_plan``, ``sgemm_rows_gather``, ``sgemm_rows_combine``,
``sgemm_rows_combine_backward``); products in 8-bit integers with a scale for each row of either
operand, for one matrix and grouped by expert (``sgemm_int8_quantize``, ``sgemm_run_int8``,
``sgemm_run_int8_grouped``); and orthogonalising the update of one weight matrix or of a batch of
them (``sgemm_orthogonalize``).

``own`` false computes each operator in its plain form, elementary torch operations in 32 bits
(choices between experts in 64); true makes the library's calls.  ``exact`` is the definition in
64 bits.

Routing.  s = softmax(logits) or sigmoid(logits) over a token's experts, c = s + bias.  With
experts in groups, only those of the topk_groups groups with the highest sums of their group_top
highest c (of fewer, where fewer are enabled) can be picked.  The topk highest c are picked, in
falling order, ties to the lowest index; weight = scale s, or scale s / (sum of the picked s).  A
logit of -infinity disables an expert; where fewer than topk can be picked the last picks are -1
with weight 0.

8-bit integers.  A row's scale is its largest magnitude / 127, rounded to 32 bits; a code is the
nearest whole number to value / scale, halves to even.

Orthogonalising.  X / (|X| + eps), turned so that it is not taller than wide, then in each step
X <- a X + (b S + c S S) X with S = X X^T.
"""
import math
import random

import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
TYPES = {"f32": F32, "bf16": BF16}
STEP = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # -- routing: one token of a decoding step, latency alone
        dict(name="route one token", op="route", tokens=1, experts=64, topk=8, score="softmax",
             type="f32", bias=False, groups=1, keep=1, top=1, norm=True, scale=1.0, masked=0),
        # a prompt or a training batch: a bias that balances the load, experts in groups
        dict(name="route batch, groups", op="route", tokens=8192, experts=256, topk=8,
             score="sigmoid", type="bf16", bias=True, groups=8, keep=4, top=2, norm=True,
             scale=2.5, masked=0),
        # the gradient of a batch's logits, an odd number of experts, some of them disabled
        dict(name="route backward, odd", op="route_back", tokens=4099, experts=60, topk=4,
             score="softmax", type="f32", norm=False, scale=1.0, masked=3),
        # -- rows to their experts and back: a decoding step's rows, sorted and gathered
        dict(name="dispatch decode", op="dispatch", tokens=24, experts=16, topk=2, N=2048,
             type="bf16", first=0, groups=16),
        # a prompt's rows back to their tokens, weighted and added
        dict(name="combine prompt", op="combine", tokens=8192, experts=128, topk=8, N=2048,
             type="bf16", first=0, groups=128),
        # its gradient in training, rows of odd width; half of the experts are on this device
        dict(name="combine backward, odd", op="combine_back", tokens=1500, experts=64, topk=6,
             N=777, type="f32", first=32, groups=32),
        # -- 8-bit integers: one token through a layer
        dict(name="int8 one row", op="int8", M=1, N=8192, K=2048, type="bf16", out="bf16"),
        # a decoding step over many experts
        dict(name="int8_grouped decode", op="int8_grouped", groups=32, rows=48, N=4096, K=2048,
             type="bf16", out="bf16", sizes=7),
        # a prompt, or a batch
        dict(name="int8 large", op="int8", M=8192, N=8192, K=8192, type="bf16", out="bf16"),
        # -- the update of small weight matrices, one for each of sixteen experts
        dict(name="orthogonalize batch", op="orthogonalize", batch=16, M=256, N=512, type="f32",
             steps=5),
        # odd sizes, a tall matrix, the gradient in 16 bits
        dict(name="orthogonalize odd", op="orthogonalize", batch=1, M=1500, N=1001, type="bf16",
             steps=5),
        # a large layer's matrix
        dict(name="orthogonalize large", op="orthogonalize", batch=1, M=2048, N=4096, type="f32",
             steps=5),
    ]


def _log(rng, low, high):
    """A whole number, its logarithm uniform over the range; every other one odd."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, n | 1 if rng.random() < 0.5 else n // 64 * 64 if n >= 128 else n))


def draw(rng):
    op = rng.choice(["route", "route", "route_back", "dispatch", "combine", "combine_back", "int8",
                     "int8", "int8_grouped", "orthogonalize", "orthogonalize"])
    while True:
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            experts = groups * max(2, _log(rng, 8, 512) // groups)
            keep = rng.randint(1, groups)
            topk = rng.randint(1, min(16, experts // groups * keep))
            return dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, topk=topk,
                        score=rng.choice(["softmax", "sigmoid"]), type=rng.choice(["f32", "bf16"]),
                        bias=rng.random() < 0.5, groups=groups, keep=keep,
                        top=rng.choice([1, 2]), norm=rng.random() < 0.5,
                        scale=rng.choice([1.0, 2.5]), masked=rng.choice([0, 0, experts // 8]))
        if op == "route_back":
            experts = _log(rng, 8, 512)
            return dict(op=op, tokens=_log(rng, 1, 8192), experts=experts,
                        topk=rng.randint(1, min(16, experts)),
                        score=rng.choice(["softmax", "sigmoid"]), type=rng.choice(["f32", "bf16"]),
                        norm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                        masked=rng.choice([0, 0, experts // 8]))
        if op in ("dispatch", "combine", "combine_back"):
            experts = _log(rng, 8, 256)
            groups = rng.choice([experts, experts, max(1, experts // 2)])
            c = dict(op=op, tokens=_log(rng, 1, 16384), experts=experts,
                     topk=rng.randint(1, min(8, experts)), N=_log(rng, 64, 8192),
                     type=rng.choice(["f32", "bf16"]), first=experts - groups, groups=groups)
            if c["tokens"] * c["topk"] * c["N"] <= 1 << 27:
                return c
        elif op == "int8":
            return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=_log(rng, 64, 8192),
                        type=rng.choice(["f32", "bf16", "int8"]), out=rng.choice(["f32", "bf16"]))
        elif op == "int8_grouped":
            c = dict(op=op, groups=_log(rng, 1, 128), rows=_log(rng, 1, 16384),
                     N=_log(rng, 64, 4096), K=_log(rng, 64, 4096),
                     type=rng.choice(["f32", "bf16", "int8"]), out=rng.choice(["f32", "bf16"]),
                     sizes=rng.randrange(1 << 30))
            if c["groups"] * c["N"] * c["K"] <= 1 << 28:
                return c
        else:
            c = dict(op=op, batch=_log(rng, 1, 32), M=_log(rng, 16, 4096), N=_log(rng, 16, 4096),
                     type=rng.choice(["f32", "bf16"]), steps=5)
            if work(c)["flops"] <= 4.4e11:
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
    """Codes of a row, in bytes: zeros after the first K."""
    return (K + 127) // 128 * 128


def work(case):
    op = case["op"]
    if op in ("route", "route_back"):
        n, picks = case["tokens"] * case["experts"], case["tokens"] * case["topk"]
        size = 4 if case["type"] == "f32" else 2
        if op == "route":
            return dict(bytes=n * size + 8 * picks + (4 * case["experts"] if case["bias"] else 0),
                        flops=8 * n)
        # scores of experts that were not picked matter only where all of them share the gradient
        read = n if case["score"] == "softmax" and not case["norm"] else picks
        return dict(bytes=size * (read + n) + 8 * picks, flops=8 * read)
    if op in ("dispatch", "combine", "combine_back"):
        size = 4 if case["type"] == "f32" else 2
        pairs, N, share = case["tokens"] * case["topk"], case["N"], case["groups"] / case["experts"]
        there, tokens = int(pairs * share) * N * size, case["tokens"] * N * size
        if op == "dispatch":
            return dict(bytes=tokens + there + 12 * pairs, flops=0)
        if op == "combine":
            return dict(bytes=tokens + there + 8 * pairs, flops=2 * int(pairs * share) * N)
        return dict(bytes=tokens + 2 * there + 12 * pairs, flops=3 * int(pairs * share) * N)
    if op == "orthogonalize":
        m, n = min(case["M"], case["N"]), max(case["M"], case["N"])
        size = 4 if case["type"] == "f32" else 2
        # S and S S are symmetric: half of their elements
        return dict(bytes=2 * size * case["batch"] * m * n,
                    flops=case["steps"] * case["batch"] * (m * (m + 1) * (n + m) + 2 * m * m * n))
    N, K = case["N"], case["K"]
    if op == "int8":
        rows, used = case["M"], 1
    else:
        at = _offsets(case)
        rows, used = case["rows"], sum(b > a for a, b in zip(at, at[1:]))
    a = rows * K * dict(f32=4, bf16=2, int8=1)[case["type"]] + (4 * rows if case["type"] == "int8"
                                                                else 0)
    return dict(bytes=a + used * N * (K + 4) + rows * N * (4 if case["out"] == "f32" else 2),
                flops=2 * rows * N * K)


# ------------------------------------------------------------------ the inputs
def _activations(rows, K, g):
    """Normal values with a few channels of large ones, as layers see them."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    loud = torch.rand(K, generator=g, device="cuda") < 1.0 / 64
    return x * torch.where(loud, 8.0, 1.0)


def _logits(case, g):
    """Scores before softmax or sigmoid: some experts liked more than others, some disabled."""
    tokens, experts = case["tokens"], case["experts"]
    x = torch.randn(tokens, experts, generator=g, device="cuda") * 1.5
    x += torch.randn(experts, generator=g, device="cuda") * 0.5
    off = torch.rand(experts, generator=g, device="cuda").argsort()[:case["masked"]]
    x[:, off] = -math.inf
    return x.to(TYPES[case["type"]])


def _some_picks(case, g):
    """topk different experts of each token, some liked more than others."""
    tokens, experts = case["tokens"], case["experts"]
    x = torch.randn(tokens, experts, generator=g, device="cuda")
    x += torch.randn(experts, generator=g, device="cuda") * 0.5
    return x.argsort(1, descending=True)[:, :case["topk"]].to(torch.int32).contiguous()


def _sorted_pairs(picks, first, groups):
    """Pairs (token, pick) ordered by expert, among experts first .. first + groups - 1: offsets
    of the experts, the pair of each row and the row of each pair (-1: none)."""
    e = picks.reshape(-1).long() - first
    here = (e >= 0) & (e < groups)
    key = torch.where(here, e, torch.full_like(e, groups))
    order = key.argsort(stable=True)
    count = torch.zeros(groups + 1, dtype=torch.int64, device=e.device).index_add_(
        0, key, torch.ones_like(key))
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device=e.device)
    offsets[1:] = count[:groups].cumsum(0)
    row = torch.arange(e.numel(), device=e.device)
    inside = row < offsets[groups]
    places = torch.empty_like(row)
    places[order] = torch.where(inside, row, torch.full_like(row, -1))
    sources = torch.where(inside, order, torch.full_like(order, -1))
    return offsets, sources.to(torch.int32), places.to(torch.int32)


def _codes(x):
    """(codes as [rows][padded K] int8, scales) of x (rows x K)."""
    rows, K = x.shape
    scale = (x.abs().amax(1).double() / 127).float()
    unit = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    q = torch.zeros(rows, _padded(K), dtype=torch.int8, device=x.device)
    for i in range(0, rows, 8192):  # in parts: 64-bit copies of a large matrix take room
        part = torch.round(x[i:i + 8192].double() / unit[i:i + 8192, None])
        q[i:i + 8192, :K] = part.to(torch.int8)
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, st = case["op"], dict(case)
    if op in ("route", "route_back"):
        tokens, experts, topk = case["tokens"], case["experts"], case["topk"]
        st["logits"] = _logits(case, g)
        st["weights"] = torch.empty(tokens, topk, device="cuda")
        if op == "route":
            st["picks"] = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
            bias = torch.randn(experts, generator=g, device="cuda") * 0.02
            st["b"] = bias if case["bias"] else None
        else:
            st["picks"] = _route(st, st["logits"].double(), None, 1, 1, 1).to(torch.int32)
            st["dweights"] = torch.randn(tokens, topk, generator=g, device="cuda") / 64
            st["dlogits"] = torch.empty_like(st["logits"])
        return st
    if op in ("dispatch", "combine", "combine_back"):
        tokens, topk, N, t = case["tokens"], case["topk"], case["N"], TYPES[case["type"]]
        pairs = tokens * topk
        st["picks"] = _some_picks(case, g)
        if op == "dispatch":
            st["X"] = _activations(tokens, N, g).to(t)
            st["Y"] = torch.zeros(pairs, N, dtype=t, device="cuda")
            st["offsets"] = torch.empty(case["groups"] + 1, dtype=torch.int64, device="cuda")
            st["sources"] = torch.empty(pairs, dtype=torch.int32, device="cuda")
            st["places"] = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
            st["workspace"] = None
            return st
        _, _, places = _sorted_pairs(st["picks"], case["first"], case["groups"])
        st["places"] = places.view(tokens, topk)
        st["weights"] = torch.rand(tokens, topk, generator=g, device="cuda").softmax(1)
        st["X"] = torch.randn(pairs, N, generator=g, device="cuda").to(t)
        if op == "combine":
            st["Y"] = torch.empty(tokens, N, dtype=t, device="cuda")
        else:
            st["dY"] = (torch.randn(tokens, N, generator=g, device="cuda") / 64).to(t)
            st["dX"] = torch.zeros(pairs, N, dtype=t, device="cuda")
            st["dweights"] = torch.empty(tokens, topk, device="cuda")
        return st
    if op == "orthogonalize":
        # a gradient's momentum: a few strong directions over noise
        B, M, N = case["batch"], case["M"], case["N"]
        r = min(M, N, 16)
        u = torch.randn(B, M, r, generator=g, device="cuda")
        v = torch.randn(B, r, N, generator=g, device="cuda")
        x = torch.bmm(u, v) * 0.1 + torch.randn(B, M, N, generator=g, device="cuda")
        st["X"] = (x * 1e-3).to(TYPES[case["type"]])
        st["Y"] = torch.empty_like(st["X"])
        st["workspace"] = None
        return st
    rows = case["M"] if op == "int8" else case["rows"]
    groups = 1 if op == "int8" else case["groups"]
    N, K = case["N"], case["K"]
    if op == "int8_grouped":
        at = _offsets(case)
        st["offsets"] = torch.tensor(at, dtype=torch.int64, device="cuda")
        # rows that a plain batch keeps room for
        st["cap"] = max(1, max(b - a for a, b in zip(at, at[1:])))
    x = _activations(rows, K, g)
    if case["type"] == "int8":
        st["A"], st["scalesA"] = _codes(x)
    else:
        st["A"], st["scalesA"] = x.to(TYPES[case["type"]]), None
    st["B"], st["scalesB"] = _codes(torch.randn(groups * N, K, generator=g, device="cuda")
                                    / math.sqrt(K))
    st["C"] = torch.empty(rows, N, dtype=TYPES[case["out"]], device="cuda")
    # what a program keeps for the activations in 8 bits
    st["workspace"] = torch.empty(rows * (_padded(K) + 4) + 64, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- the plain forms
def _scores(kind, x):
    """softmax or sigmoid of x in its own type; rows without a finite logit give zeros."""
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp(min=torch.finfo(x.dtype).tiny)


def _route(st, x, bias, groups, keep, top):
    """Picks (-1: none), from scores in 64 bits: what is compared may differ by very little."""
    tokens, experts = x.shape
    c = _scores(st["score"], x)
    if bias is not None:
        c = c + bias.double()
    c = torch.where(x == -math.inf, torch.full_like(c, -math.inf), c)
    if groups > 1:
        best = c.view(tokens, groups, -1).sort(dim=2, descending=True)[0][:, :, :top]
        some = best[:, :, 0] > -math.inf
        total = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        total = torch.where(some, total, torch.full_like(total, -math.inf))
        order = total.sort(dim=1, descending=True, stable=True)[1][:, :keep]
        open_ = torch.zeros(tokens, groups, dtype=torch.bool, device=x.device)
        open_.scatter_(1, order, True)
        c = torch.where(open_.repeat_interleave(experts // groups, 1), c,
                        torch.full_like(c, -math.inf))
    c, order = c.sort(dim=1, descending=True, stable=True)
    topk = st["topk"]
    c, order = c[:, :topk], order[:, :topk]
    return torch.where(c > -math.inf, order, torch.full_like(order, -1))


def _picked(values, picks):
    """values at the picks, zeros where there is none."""
    got = values.gather(1, picks.long().clamp(min=0))
    return torch.where(picks >= 0, got, torch.zeros_like(got))


def _weights(st, s, picks):
    w = _picked(s, picks)
    if st["norm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=torch.finfo(s.dtype).tiny)
    return w * st["scale"]


def _route_back(st, x, dw):
    """The logits' gradient in x's type, from the weights'."""
    picks = st["picks"]
    s = _scores(st["score"], x)
    p = _picked(s, picks)
    dw = torch.where(picks >= 0, dw, torch.zeros_like(dw)) * st["scale"]
    if st["norm"]:
        total = p.sum(1, keepdim=True).clamp(min=torch.finfo(x.dtype).tiny)
        dw = (dw - (dw * p).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_add_(1, picks.long().clamp(min=0),
                                          torch.where(picks >= 0, dw, torch.zeros_like(dw)))
    if st["score"] == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdim=True))


def _taken(x, places):
    """Rows of x at the places of each token, [tokens][topk][N], zeros where there is none."""
    got = x[places.long().clamp(min=0)]
    return torch.where((places >= 0)[:, :, None], got, torch.zeros_like(got))


def _by_group(st, A, Bt):
    """Each row of A times its group's Bt ([groups][K][N])."""
    at, cap = st["offsets"], st["cap"]
    idx = at[:-1, None] + torch.arange(cap, device="cuda")
    inside = idx < at[1:, None]
    r = torch.arange(A.shape[0], device="cuda")
    group = torch.searchsorted(at, r, right=True) - 1
    batch = A[idx.clamp(max=A.shape[0] - 1)] * inside[:, :, None]
    return torch.bmm(batch, Bt)[group, r - at[group]]


def _plain(st):
    op = st["op"]
    if op == "route":
        picks = _route(st, st["logits"].double(), st["b"], st["groups"], st["keep"], st["top"])
        s = _scores(st["score"], st["logits"].float())
        return picks.to(torch.int32), _weights(st, s, picks)
    if op == "route_back":
        return _route_back(st, st["logits"].float(), st["dweights"]).to(TYPES[st["type"]])
    if op == "dispatch":
        offsets, sources, places = _sorted_pairs(st["picks"], st["first"], st["groups"])
        rows = st["X"][sources.long().clamp(min=0) // st["topk"]]
        rows = torch.where((sources >= 0)[:, None], rows, torch.zeros_like(rows))
        return offsets, sources, places.view(st["picks"].shape), rows
    if op == "combine":
        rows = _taken(st["X"], st["places"]).float()
        return (rows * st["weights"][:, :, None]).sum(1).to(TYPES[st["type"]])
    if op == "combine_back":
        rows, dy = _taken(st["X"], st["places"]).float(), st["dY"].float()
        dw = (rows * dy[:, None, :]).sum(2)
        dx = torch.zeros_like(st["dX"])
        here = st["places"] >= 0
        back = st["weights"][:, :, None] * dy[:, None, :]
        dx[st["places"][here].long()] = back[here].to(dx.dtype)
        return dx, dw
    if op == "orthogonalize":
        x = st["X"].float()
        x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + EPS)
        tall = x.shape[1] > x.shape[2]
        x = x.transpose(1, 2).contiguous() if tall else x
        a, b, c = STEP
        for _ in range(st["steps"]):
            s = torch.bmm(x, x.transpose(1, 2).contiguous())
            x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
        return (x.transpose(1, 2).contiguous() if tall else x).to(TYPES[st["type"]])
    K, N = st["K"], st["N"]
    q, scale = (st["A"], st["scalesA"]) if st["type"] == "int8" else _codes(st["A"].float())
    a, b = q[:, :K].float(), st["B"][:, :K].float()
    if op == "int8":
        c = (a @ b.t()) * scale[:, None] * st["scalesB"]
    else:
        b = b * st["scalesB"][:, None]
        c = _by_group(st, a * scale[:, None], b.view(-1, N, K).transpose(1, 2).contiguous())
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


def _room(st, nbytes):
    """The workspace that a program keeps for its calls."""
    if st["workspace"] is None:
        st["workspace"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _calls(st):
    sg = _library()
    op = st["op"]
    if op == "route":
        sg.sgemm_route(st["tokens"], st["experts"], st["topk"], st["score"], st["type"],
                       st["logits"], st["experts"], st["b"], st["groups"], st["keep"], st["top"],
                       st["norm"], st["scale"], st["picks"], st["weights"])
        return st["picks"], st["weights"]
    if op == "route_back":
        sg.sgemm_route_backward(st["tokens"], st["experts"], st["topk"], st["score"], st["type"],
                                st["logits"], st["experts"], st["norm"], st["scale"], st["picks"],
                                st["dweights"], st["dlogits"], st["experts"])
        return st["dlogits"]
    if op in ("dispatch", "combine", "combine_back"):
        tokens, topk, N, t = st["tokens"], st["topk"], st["N"], st["type"]
        pairs = tokens * topk
        if op == "dispatch":
            G = st["groups"]
            ws = _room(st, sg.sgemm_route_plan_workspace_size(pairs, G))
            sg.sgemm_route_plan(pairs, st["first"], G, st["picks"], st["offsets"], st["sources"],
                                st["places"], ws, ws.numel())
            sg.sgemm_rows_gather(pairs, pairs, topk, N, t, st["X"], N, st["sources"], None,
                                 st["Y"], N)
            return st["offsets"], st["sources"], st["places"], st["Y"]
        if op == "combine":
            sg.sgemm_rows_combine(tokens, topk, pairs, N, t, st["X"], N, st["places"],
                                  st["weights"], st["Y"], N)
            return st["Y"]
        sg.sgemm_rows_combine_backward(tokens, topk, pairs, N, t, st["X"], N, st["dY"], N,
                                       st["places"], st["weights"], st["dX"], N, st["dweights"])
        return st["dX"], st["dweights"]
    if op == "orthogonalize":
        B, M, N, t = st["batch"], st["M"], st["N"], st["type"]
        ws = _room(st, sg.sgemm_orthogonalize_workspace_size(B, M, N))
        sg.sgemm_orthogonalize(B, M, N, st["steps"], STEP, EPS, 1.0, t, st["X"], N, M * N, t,
                               st["Y"], N, M * N, ws, ws.numel())
        return st["Y"]
    N, K, ws = st["N"], st["K"], st["workspace"]
    lda = _padded(K) if st["type"] == "int8" else K
    if op == "int8":
        sg.sgemm_run_int8(st["M"], N, K, 1.0, st["type"], st["A"], lda, st["scalesA"], st["B"],
                          _padded(K), st["scalesB"], 0.0, st["out"], st["C"], N, ws, ws.numel())
    else:
        sg.sgemm_run_int8_grouped(st["groups"], st["rows"], N, K, 1.0, st["type"], st["A"], lda,
                                  st["scalesA"], st["B"], _padded(K), st["scalesB"], 0.0,
                                  st["out"], st["C"], N, st["offsets"], ws, ws.numel())
    return st["C"]


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------ the definitions, 64 bits
def _ranked(c, n):
    """Indices of the n highest of each row, the lowest index first among equals: by counting how
    many come before each."""
    out = torch.full((c.shape[0], n), -1, dtype=torch.int64, device=c.device)
    index = torch.arange(c.shape[1], device=c.device)
    left = c.clone()
    for j in range(n):
        top = left.amax(1, keepdim=True)
        at = torch.where(left == top, index, torch.full_like(index, c.shape[1])).amin(1)
        out[:, j] = torch.where(top[:, 0] > -math.inf, at, torch.full_like(at, -1))
        left.scatter_(1, at.clamp(max=c.shape[1] - 1)[:, None], -math.inf)
    return out


def _exact_scores(kind, x):
    if kind == "sigmoid":
        return torch.special.expit(x)
    return torch.nan_to_num(torch.exp(x - torch.logsumexp(x, 1, keepdim=True)))


def _exact_route(st):
    x = st["logits"].double()
    s = _exact_scores(st["score"], x)
    c = s if st["b"] is None else s + st["b"].double()
    c = c.masked_fill(x == -math.inf, -math.inf)
    groups, size = st["groups"], st["experts"] // st["groups"]
    if groups > 1:
        sums = []
        for n in range(groups):
            part = c[:, n * size:(n + 1) * size]
            at = _ranked(part, min(st["top"], size))
            got = part.gather(1, at.clamp(min=0)).masked_fill(at < 0, 0.0).sum(1)
            sums.append(got.masked_fill(at[:, 0] < 0, -math.inf))
        chosen = _ranked(torch.stack(sums, 1), st["keep"])
        closed = torch.ones(c.shape[0], groups + 1, dtype=torch.bool, device=c.device)
        closed.scatter_(1, torch.where(chosen < 0, groups, chosen), False)
        for n in range(groups):
            c[:, n * size:(n + 1) * size].masked_fill_(closed[:, n:n + 1], -math.inf)
    picks = _ranked(c, st["topk"])
    w = s.gather(1, picks.clamp(min=0)).masked_fill(picks < 0, 0.0)
    if st["norm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return picks.to(torch.int32), w * st["scale"]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    if op == "route_back":
        # by the chain of derivatives: d weight_j / d logit_i, picked rows only
        x = st["logits"].double()
        s, picks = _exact_scores(st["score"], x), st["picks"].long()
        out = torch.zeros_like(x)
        valid = picks >= 0
        p = s.gather(1, picks.clamp(min=0)).masked_fill(~valid, 0.0)
        up = st["dweights"].double().masked_fill(~valid, 0.0) * case["scale"]
        if case["norm"]:
            total = p.sum(1, keepdim=True)
            share = torch.where(total > 0, p / total, torch.zeros_like(p))
            mean = (up * share).sum(1, keepdim=True)
            slope = share * (up - mean)  # d / d log s of the picked
        else:
            slope = up * p
        for j in range(case["topk"]):
            k = picks[:, j:j + 1].clamp(min=0)
            g = slope[:, j:j + 1]
            if case["score"] == "sigmoid":
                out.scatter_add_(1, k, g * (1 - s.gather(1, k)))
            else:
                out.scatter_add_(1, k, g)
                if not case["norm"]:
                    out -= g * s
        return out
    if op == "dispatch":
        e = st["picks"].reshape(-1).tolist()
        by_expert = [[] for _ in range(case["groups"])]
        for pair, k in enumerate(e):
            if 0 <= k - case["first"] < case["groups"]:
                by_expert[k - case["first"]].append(pair)
        rows = [pair for part in by_expert for pair in part]
        offsets = [0]
        for part in by_expert:
            offsets.append(offsets[-1] + len(part))
        places = [-1] * len(e)
        for row, pair in enumerate(rows):
            places[pair] = row
        sources = rows + [-1] * (len(e) - len(rows))
        y = torch.zeros(len(e), case["N"], dtype=F64, device="cuda")
        if rows:
            at = torch.tensor(rows, device="cuda") // case["topk"]
            y[:len(rows)] = st["X"][at].double()
        return (torch.tensor(offsets, device="cuda"),
                torch.tensor(sources, dtype=torch.int32, device="cuda"),
                torch.tensor(places, dtype=torch.int32, device="cuda").view(-1, case["topk"]), y)
    if op in ("combine", "combine_back"):
        places, w = st["places"].long(), st["weights"].double()
        here = places >= 0
        if op == "combine":
            y = torch.zeros(case["tokens"], case["N"], dtype=F64, device="cuda")
            for j in range(case["topk"]):
                t = here[:, j].nonzero()[:, 0]
                y[t] += w[t, j:j + 1] * st["X"][places[t, j]].double()
            return y
        dy = st["dY"].double()
        dx = torch.zeros(st["dX"].shape, dtype=F64, device="cuda")
        dw = torch.zeros(w.shape, dtype=F64, device="cuda")
        for j in range(case["topk"]):
            t = here[:, j].nonzero()[:, 0]
            dx[places[t, j]] = w[t, j:j + 1] * dy[t]
            dw[t, j] = torch.linalg.vecdot(st["X"][places[t, j]].double(), dy[t])
        return dx, dw
    if op == "orthogonalize":
        out = []
        a, b, c = STEP
        for x in st["X"].double():
            x = x / (torch.linalg.norm(x) + EPS)
            left = x.shape[0] <= x.shape[1]
            for _ in range(case["steps"]):
                s = x @ x.t() if left else x.t() @ x
                p = b * s + c * (s @ s)
                x = a * x + (p @ x if left else x @ p)
            out.append(x)
        return torch.stack(out)
    K, N = case["K"], case["N"]
    if case["type"] == "int8":
        a, scale = st["A"][:, :K].double(), st["scalesA"].double()
    else:
        x = st["A"].double()
        scale = (x.abs().amax(1) / 127).float().double()
        q = x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
        down = torch.floor(q)
        up = (q - down > 0.5) | ((q - down == 0.5) & (down % 2 == 1))
        a = down + up
    b, unit = st["B"][:, :K].double(), st["scalesB"].double()
    if op == "int8":
        return (a @ b.t()) * scale[:, None] * unit
    at = _offsets(case)
    return torch.cat([(a[i:j] @ b[n * N:(n + 1) * N].t()) * scale[i:j, None]
                      * unit[n * N:(n + 1) * N]
                      for n, (i, j) in enumerate(zip(at, at[1:]))])
