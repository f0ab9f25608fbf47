"""GPU parity of the feed-forward block with 4-bit weights against its formulas in 64 bits: the norms around a block, the
scored router, projections and the experts' products, alone and together.

Tolerances.  U = 2^-24 is half a step of an f32.  The norm rounds once (U) and carries 2^-44 up to there.  A product sums
its 32-value blocks' dots in f32: each dot is in error by at most a step of its size for each of its roundings, and an f32
activation enters as two f16 parts, which hold 2^-22 of its block's largest value.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ws(q8):
    w = q8.Workspace()
    yield w
    w.close()


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def quantize(torch, x, two):
    """The quantizer's rule in IEEE f32: words, low words and scales of every 32 values."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=x.device)
    t = torch.where(d > 0, b / d, torch.zeros_like(b))
    away = lambda v: (torch.sign(v) * torch.floor(v.abs() + 0.5)).clamp(-127, 127)  # noqa: E731
    hi = away(t)
    lo = away((t - hi) * 128).to(torch.int8).flatten(-2) if two else None
    return hi.to(torch.int8).flatten(-2), lo, d.squeeze(-1)


# ---- the norms around a block ----------------------------------------------------------------------------------------


def norm_inputs(torch, rows, d, gate, seed, post=True):
    g = gen(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gates = {None: None, "channel": (d,), "row": (rows, 1), "full": (rows, d)}[gate]
    return dict(a=3 * n(rows, d), b=n(rows, d) * 10 ** (2 * n(rows, 1)).clamp(-6, 6), w_post=1 + 0.1 * n(d) if post else None,
                w_pre=1 + 0.1 * n(d), gate=n(*gates) if gates else None)


def check_norm(torch, i, scale, eps, s, y=None, yq=None, ys=None, yl=None):
    d = i["a"].shape[-1]
    f = lambda t: t.double()  # noqa: E731
    p = f(i["b"])
    if i["w_post"] is not None:
        p = p / (p.pow(2).sum(-1, keepdim=True) / d + eps).sqrt() * f(i["w_post"])
    p = scale * p
    if i["gate"] is not None:
        p = p * f(i["gate"])
    want = f(i["a"]) + p
    assert ((f(s) - want).abs() <= U * want.abs() * 1.001 + 2.0 ** -40 * (f(i["a"]).abs() + p.abs())).all()
    want = f(s) / (f(s).pow(2).sum(-1, keepdim=True) / d + eps).sqrt() * f(i["w_pre"])
    if y is not None:
        assert ((f(y) - want).abs() <= U * want.abs() * 1.001 + 1e-44).all()
    if yq is not None:  # the words and scales of the rounded y
        words, low, scales = quantize(torch, want.float() if y is None else y, yl is not None)
        assert torch.equal(ys, scales)
        assert torch.equal(yq, words)
        if yl is not None:
            assert torch.equal(yl, low)


@pytest.mark.parametrize("gate", [None, "channel", "row", "full"])
@pytest.mark.parametrize("rows,d", [(1, 32), (1, 2048), (3, 96), (37, 5120), (5, 8192), (2, 16384), (700, 512), (401, 1056),
                                    (350, 4128), (310, 16384)])
def test_norm(q8, rows, d, gate):
    import torch
    i = norm_inputs(torch, rows, d, gate, rows + d)
    for two in (False, True):
        s, y = torch.empty_like(i["a"]), torch.empty_like(i["a"])
        yq, ys = torch.empty(rows, d, dtype=torch.int8, device="cuda"), torch.empty(rows, d // 32, device="cuda")
        yl = torch.empty_like(yq) if two else None
        q8.postnorm_add_rmsnorm_q8(**i, eps=1e-6, scale=0.22, sum_out=s, y_out=y, yq=yq, ys=ys, yl=yl)
        check_norm(torch, i, float(torch.tensor(0.22)), float(torch.tensor(1e-6)), s, y, yq, ys, yl)


@pytest.mark.parametrize("rows,d", [(1, 1), (2, 7), (9, 1001), (3, 4097), (400, 33), (1, 16383)])
def test_norm_odd_sizes(q8, rows, d):
    import torch
    for gate in (None, "full", "channel"):
        i = norm_inputs(torch, rows, d, gate, rows + d)
        s, y = torch.empty_like(i["a"]), torch.empty_like(i["a"])
        q8.postnorm_add_rmsnorm_q8(**i, eps=1e-6, sum_out=s, y_out=y)
        check_norm(torch, i, 1.0, float(torch.tensor(1e-6)), s, y)


def test_norm_outputs_one_at_a_time_in_place_and_off_alignment(q8):
    import torch
    rows, d = 5, 1024
    i = norm_inputs(torch, rows, d, "channel", 5)
    full = [torch.empty_like(i["a"]) for _ in range(2)]
    q8.postnorm_add_rmsnorm_q8(**i, eps=1e-5, scale=0.5, sum_out=full[0], y_out=full[1])
    one = torch.empty_like(i["a"])
    q8.postnorm_add_rmsnorm_q8(**i, eps=1e-5, scale=0.5, sum_out=one)
    assert torch.equal(one, full[0])
    q8.postnorm_add_rmsnorm_q8(**i, eps=1e-5, scale=0.5, y_out=one)
    assert torch.equal(one, full[1])
    off = {k: torch.empty(t.numel() + 1, device="cuda")[1:].view(t.shape).copy_(t) for k, t in i.items()}
    s, y = (torch.empty(rows * d + 1, device="cuda")[1:].view(rows, d) for _ in range(2))
    q8.postnorm_add_rmsnorm_q8(**off, eps=1e-5, scale=0.5, sum_out=s, y_out=y)
    check_norm(torch, i, 0.5, float(torch.tensor(1e-5)), s, y)
    wide = torch.zeros(rows, 2 * d, device="cuda")  # a gate whose values stand apart
    wide[:, ::2] = i["gate"]
    q8.postnorm_add_rmsnorm_q8(**{**i, "gate": wide[:, ::2]}, eps=1e-5, scale=0.5, sum_out=s, y_out=y)
    assert torch.equal(s, full[0]) and torch.equal(y, full[1])
    a, b = i["a"].clone(), i["b"].clone()  # the residual and the output in place
    q8.postnorm_add_rmsnorm_q8(**{**i, "a": a, "b": b}, eps=1e-5, scale=0.5, sum_out=a, y_out=b)
    assert torch.equal(a, full[0]) and torch.equal(b, full[1])
    i["w_post"] = None  # the output as it is
    q8.postnorm_add_rmsnorm_q8(**i, eps=1e-5, scale=0.5, sum_out=s, y_out=y)
    check_norm(torch, i, 0.5, float(torch.tensor(1e-5)), s, y)


def test_norm_zeros_infinities_and_their_neighbours(q8):
    import torch
    i = norm_inputs(torch, 4, 256, None, 9)
    i["b"][0] = 0
    i["a"][1], i["b"][1] = 0, 0
    i["a"][2, 17] = math.inf
    s, y = torch.empty_like(i["a"]), torch.empty_like(i["a"])
    yq, ys = torch.ones(4, 256, dtype=torch.int8, device="cuda"), torch.ones(4, 8, device="cuda")
    q8.postnorm_add_rmsnorm_q8(**i, eps=1e-6, sum_out=s, y_out=y, yq=yq, ys=ys)
    assert torch.equal(s[0], i["a"][0]) and s[2, 17] == math.inf and not torch.isfinite(y[2, 17])
    assert torch.isfinite(s[2, :17]).all()
    assert not y[1].any() and not yq[1].any() and not ys[1].any()
    at = torch.tensor([0, 1, 3], device="cuda")
    rest = {k: t[at] if k in "ab" else t for k, t in i.items()}
    check_norm(torch, rest, 1.0, float(torch.tensor(1e-6)), s[at], y[at], yq[at], ys[at])


# ---- the scored router -----------------------------------------------------------------------------------------------


def routed(torch, logits, k, score, bias, groups, keep, top, renorm, scale):
    """The rule in 64 bits, row by row: ids, gates and the gates' relative error by f32's roundings."""
    l = torch.nan_to_num(logits.double().cpu(), nan=-math.inf, posinf=3.402823466e38, neginf=-math.inf)
    ids, gates = [], []
    for row in l:
        off = row == -math.inf
        if score == 0:
            p = torch.zeros_like(row) if off.all() else torch.softmax(row, -1)
        else:
            p = torch.where(row < 0, row.exp() / (1 + row.exp()), 1 / (1 + (-row).exp()))
        c = p if bias is None else p + bias.double().cpu()
        off = off | torch.isnan(c) | (c == -math.inf)
        c = torch.where(off, torch.full_like(c, -math.inf), c)
        marks = []
        for j, part in enumerate(c.chunk(groups)):
            best = sorted(part[part > -math.inf].tolist(), reverse=True)[:top]
            marks.append((-sum(best) if best else math.inf, j))
        kept = {j for _, j in sorted(marks)[:keep]}
        size = len(row) // groups
        key = row if bias is None else c
        order = sorted((e for e in range(len(row)) if e // size in kept),
                       key=lambda e: (bool(off[e]), 0.0 if off[e] else -float(key[e]), e))[:k]
        g = [0.0 if off[e] else float(p[e]) for e in order]
        total = sum(g)
        if renorm:  # formed from the exponents, so that scores below f64's range keep their ratios
            best = max((float(row[e]) for e in order if not off[e]), default=0.0)
            if best < -30:
                g = [0.0 if off[e] else math.exp(float(row[e]) - best) for e in order]
                total = sum(g)
            g = [v / total if total > 0 else 0.0 for v in g]
        ids.append(order)
        gates.append([v * scale for v in g])
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(gates, dtype=torch.float64)


def grouped(ids, experts):
    flat = ids.flatten().tolist()
    counts = [flat.count(e) for e in range(experts)] if len(flat) < 5000 else None
    if counts is None:
        counts = [0] * experts
        for e in flat:
            counts[e] += 1
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    lists = sorted(range(len(flat)), key=lambda c: (flat[c], c))
    active = [e for e in range(experts) if counts[e]]
    return counts, offsets, lists, active


def route(q8, torch, ws, logits, k, plan=True, **rule):
    rows, E = logits.shape
    ids = torch.full((rows, k), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((rows, k), math.nan, device="cuda")
    arrays = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (E, E + 1, rows * k, E + 1)]
    q8.moe_route_scored(logits, ids, gates, plan=q8.plan_struct(*arrays) if plan else None, ws=ws if plan else None, **rule)
    return ids, gates, arrays


def check_route(torch, got, logits, k, plan=True, score=0, bias=None, groups=1, keep_groups=1, group_top=2, renorm=True,
                scale=1.0):
    ids, gates, arrays = got
    E = logits.shape[1]
    want, weights = routed(torch, logits, k, score, bias, groups, keep_groups, group_top, renorm, scale)
    assert torch.equal(ids.cpu(), want)
    # an exponential is 2 steps out beside its rounded argument (up to `span` U), a quotient and the scale's product one, the
    # sums of NL + 5 or of k values one for each term
    l = logits[torch.isfinite(logits)].double()
    span = float((l.max() - l.min()).clamp_max(110)) if l.numel() else 0.0
    tol = U * (8 + span + E / 32 + 5 + 5)
    assert ((gates.cpu().double() - weights).abs() <= tol * weights.abs() + 1e-44).all()
    if plan:
        counts, offsets, lists, active = grouped(want, E)
        assert arrays[0].tolist() == counts and arrays[1].tolist() == offsets and arrays[2].tolist() == lists
        assert arrays[3].tolist()[: 1 + len(active)] == [len(active)] + active


RULES = [dict(), dict(renorm=False, scale=2.5), dict(score=1), dict(score=1, renorm=False),
         dict(score=1, groups=4, keep_groups=2, scale=2.5), dict(groups=4, keep_groups=1, group_top=1, renorm=False)]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rows,E,k", [(1, 128, 8), (61, 256, 8), (5, 8, 2), (200, 60, 4), (33, 1000, 32), (3, 512, 10),
                                      (1100, 64, 6), (2, 1024, 1)])
def test_route(q8, ws, rows, E, k, biased, rule):
    import torch
    g = gen(rows * E + k)
    logits = 1.5 * torch.randn(rows, E, generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
    k = min(k, E // rule.get("groups", 1) * rule.get("keep_groups", 1))
    for plan in (False, True):
        check_route(torch, route(q8, torch, ws, logits, k, plan, bias=bias, **rule), logits, k, plan, bias=bias, **rule)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rule", RULES)
def test_route_ties_masks_and_extremes(q8, ws, rule, biased):
    import torch
    g = gen(3)
    E, k, rows = 96, 12, 40
    logits = torch.randn(rows, E, generator=g, device="cuda")
    logits[0] = 0.25  # all alike
    logits[1] = -math.inf  # nothing in service
    logits[2, 5:] = -math.inf  # fewer in service than choices
    logits[3] = -3.4028234663852886e38  # the type's lowest value everywhere
    logits[4, :50] = -3.4028234663852886e38
    logits[5, 7], logits[5, 60] = math.inf, math.inf
    logits[6, 3], logits[6, 4] = math.nan, -math.nan
    logits[7] = -120 + logits[7]  # scores below f32's range
    logits[8] = 60 + logits[8]  # sigmoids that round to 1
    logits[9:20] = (2 * logits[9:20]).round() / 2  # many equal ones
    logits[20:30] = 1 + 3e-8 * torch.arange(E, device="cuda") * torch.randn(10, E, generator=g, device="cuda").sign()
    logits[30:34, ::2] = -math.inf
    logits[34, :24] = -math.inf  # a whole group
    bias = None
    if biased:
        bias = 0.05 * torch.randn(E, generator=g, device="cuda")
        bias[::3] = bias[0]  # equal ones, so that equal scores tie
        bias[10], bias[11], bias[12] = -math.inf, math.nan, 2.0
    if rule.get("score") == 1 and biased or rule.get("groups", 1) > 1:
        logits[8] = logits[10]  # (sums of sigmoids of 60 are one 64-bit number for distinct logits: no order by the formula)
    got = route(q8, torch, ws, logits, k, True, bias=bias, **rule)
    check_route(torch, got, logits, k, True, bias=bias, **rule)


@pytest.mark.parametrize("rows", [127, 128, 129, 153, 2311, 15001])
def test_route_grouping_of_many_rows(q8, ws, rows):
    import torch
    g = gen(rows)
    logits = torch.randn(rows, 256, generator=g, device="cuda") + 2 * torch.randn(256, generator=g, device="cuda")
    logits[rows // 3 : rows // 2] = logits[0]  # long runs of one choice
    bias = 0.05 * torch.randn(256, generator=g, device="cuda")
    rule = dict(score=1, bias=bias, groups=8, keep_groups=4, scale=2.5)
    ids, gates, arrays = route(q8, torch, ws, logits, 8, True, **rule)
    p = torch.sigmoid(logits.double())
    c = p + bias.double()
    best = c.unflatten(1, (8, 32)).topk(2, -1).values.sum(-1)
    hidden = torch.ones(rows, 8, dtype=torch.bool, device="cuda").scatter_(1, best.topk(4, -1).indices, False)
    want = c.masked_fill(hidden.repeat_interleave(32, 1), -1).topk(8, -1).indices
    assert torch.equal(ids.long(), want)
    w = p.gather(1, want)
    w = 2.5 * w / w.sum(-1, keepdim=True)
    assert ((gates.double() - w).abs() <= U * 30 * w).all()
    flat = want.flatten()
    counts = torch.bincount(flat, minlength=256)
    assert torch.equal(arrays[0].long(), counts)
    assert torch.equal(arrays[1][1:].long(), counts.cumsum(0)) and arrays[1][0] == 0
    assert torch.equal(arrays[2].long(), torch.sort(flat, stable=True).indices)
    hit = counts.nonzero().flatten()
    assert arrays[3][0] == len(hit) and torch.equal(arrays[3][1 : 1 + len(hit)].long(), hit)


def test_route_rows_apart_and_one_row_without_dimensions(q8, ws):
    import torch
    wide = torch.randn(9, 100, generator=gen(1), device="cuda")
    got = route(q8, torch, ws, wide[:, 3:67], 4, True, score=1)
    check_route(torch, got, wide[:, 3:67], 4, True, score=1)
    ids, gates = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    q8.moe_route_scored(wide[2, 3:67], ids, gates, score=1)
    assert torch.equal(ids, got[0][2]) and torch.equal(gates, got[1][2])


# ---- products with 4-bit weights -------------------------------------------------------------------------------------


def matrix(torch, rows, cols, group, kind, zeros, g):
    """Words, scales and zero points, with scales of very different sizes and zero points over their whole range."""
    q = torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.randn(rows, cols // group, generator=g, device="cuda") * 0.02).to(torch.float16 if kind == "f16" else torch.bfloat16)
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    if zeros:
        z[:, -1] = 255
    return q, s, z


def values(torch, m):
    q, s, z = m
    w = torch.stack((q & 15, q >> 4), -1).flatten(-2).double()
    width = w.shape[1] // s.shape[1]
    z = z.double() if z is not None else torch.full(s.shape, 8.0, device="cuda", dtype=torch.float64)
    return (w - z.repeat_interleave(width, 1)) * s.double().repeat_interleave(width, 1)


def activation(torch, rows, cols, form, g, merged=False):
    """The call's arguments and the values they stand for."""
    x = torch.randn(rows, cols + 64 * merged, generator=g, device="cuda")[:, 64 * merged :]
    x *= 10 ** torch.randn(rows, 1, generator=g, device="cuda")
    x[:, 5 % cols] *= 100  # an outlier
    if form == "f32":
        return dict(x=x), x.double()
    q, lo, s = quantize(torch, x.contiguous(), form == "two")
    v = q.double() if lo is None else q.double() + lo.double() / 128
    return dict(xq=q, xs=s, xl=lo), v * s.double().repeat_interleave(32, 1)


def product_error(torch, W, x, form):
    """The bound on |y - W x|.  Words: each 32-value block's dot is exact, and enters by the product of two scales and one sum
    (2 U of it), and every partial sum is rounded once for each of the nb blocks: (nb + 8) U sum |block|, at most of the
    blocks' sums of absolute terms.  f32 values: beside that, 2^-22 of a block's largest |x| for every weight, and the
    block's own sum of 32 products in f32 by steps that may be cut off (32 * 2 U)."""
    nb = x.shape[1] // 32
    tol = (nb + 8) * U * (x.abs() @ W.abs().T)
    if form == "f32":
        most = x.abs().unflatten(1, (nb, 32)).amax(-1).repeat_interleave(32, 1)
        tol = tol + 2.0 ** -22 * (most @ W.abs().T) + 64 * U * (x.abs() @ W.abs().T)
    return tol


@pytest.mark.parametrize("form", ["f32", "one", "two"])
@pytest.mark.parametrize("group,kind,zeros", [(32, "f16", False), (64, "bf16", True), (128, "f16", True), (128, "bf16", False)])
@pytest.mark.parametrize("rows,n,cols", [(1, 5120, 2048), (1, 1, 128), (1, 17, 384), (2, 33, 256), (3, 100, 1152), (4, 64, 128),
                                         (5, 1000, 640), (8, 48, 4096), (17, 259, 512), (64, 130, 1024), (100, 31, 256)])
def test_projection(q8, ws, rows, n, cols, group, kind, zeros, form):
    import torch
    g = gen(rows * n + cols)
    m = matrix(torch, n, cols, group, kind, zeros, g)
    merged = rows % 2 == 0 and form == "f32"
    call, x = activation(torch, rows, cols, form, g, merged)
    wide = torch.full((rows + 1, n + 3), 7.0, device="cuda")
    y = wide[:rows, :n]
    q8.q4_gemv(q8.q4_mat(*m), y, **call, ws=ws)
    W = values(torch, m)
    assert ((y.double() - x @ W.T).abs() <= product_error(torch, W, x, form)).all()
    assert (wide[:, n:] == 7).all() and (wide[rows] == 7).all()


@pytest.mark.parametrize("cols,group", [(32, 32), (96, 32), (160, 32), (64, 64), (192, 64), (32768, 128)])
def test_projection_odd_columns(q8, ws, cols, group):
    import torch
    for rows in (1, 3, 9):
        for form in ("f32", "one", "two"):
            g = gen(cols + rows)
            m = matrix(torch, 37, cols, group, "f16", True, g)
            call, x = activation(torch, rows, cols, form, g)
            y = torch.empty(rows, 37, device="cuda")
            q8.q4_gemv(q8.q4_mat(*m), y, **call, ws=ws)
            W = values(torch, m)
            assert ((y.double() - x @ W.T).abs() <= product_error(torch, W, x, form)).all()


@pytest.mark.parametrize("rows", [1, 2, 6, 40])
def test_projection_of_values_that_are_not_finite_and_of_extremes(q8, ws, rows):
    import torch
    g = gen(rows)
    m = matrix(torch, 50, 256, 32, "f16", False, g)
    x = torch.randn(rows, 256, generator=g, device="cuda")
    plain = torch.empty(rows, 50, device="cuda")
    q8.q4_gemv(q8.q4_mat(*m), plain, x=x, ws=ws)
    bad = x.clone()
    bad[rows - 1, 40] = math.inf
    y = torch.empty(rows, 50, device="cuda")
    q8.q4_gemv(q8.q4_mat(*m), y, x=bad, ws=ws)
    assert not torch.isfinite(y[rows - 1]).any()
    assert torch.equal(y[: rows - 1], plain[: rows - 1])  # the other rows do not see it
    bad[rows - 1, 40] = math.nan
    q8.q4_gemv(q8.q4_mat(*m), y, x=bad, ws=ws)
    assert torch.isnan(y[rows - 1]).all() and torch.equal(y[: rows - 1], plain[: rows - 1])
    W = values(torch, m)
    for size in (1e30, 1e-30):  # far from 1, the result within f32's range
        big = x * size
        q8.q4_gemv(q8.q4_mat(*m), y, x=big, ws=ws)
        assert ((y.double() - big.double() @ W.T).abs() <= product_error(torch, W, big.double(), "f32")).all()
    q8.q4_gemv(q8.q4_mat(*m), y, x=torch.zeros_like(x), ws=ws)
    assert not y.any()


@pytest.mark.parametrize("rows", [1, 5, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_projection_with_scales_off_their_loads_alignment(q8, ws, rows, group):
    """Scales at 2 bytes and zero points at 1 past an aligned address: the same results as from aligned ones."""
    import torch
    g = gen(rows + group)
    q, s, z = matrix(torch, 200, 512, group, "bf16", True, g)
    off = [torch.cat((t.new_zeros(1), t.flatten()))[1:].view(t.shape) for t in (s, z)]
    assert off[0].data_ptr() % 4 == 2 and off[1].data_ptr() % 2 == 1
    x = torch.randn(rows, 512, generator=g, device="cuda")
    y, want = torch.empty(rows, 200, device="cuda"), torch.empty(rows, 200, device="cuda")
    q8.q4_gemv(q8.q4_mat(q, s, z), want, x=x, ws=ws)
    q8.q4_gemv(q8.q4_mat(q, *off), y, x=x, ws=ws)
    assert torch.equal(y, want)


def test_projection_into_columns_beside_its_rows(q8, ws):
    import torch
    g = gen(11)
    m = matrix(torch, 100, 128, 32, "f16", False, g)
    for rows in (3, 40):
        wide = torch.randn(rows, 300, generator=g, device="cuda")
        kept = wide.clone()
        q8.q4_gemv(q8.q4_mat(*m), wide[:, 160:260], x=wide[:, 16:144], ws=ws)
        x, W = kept[:, 16:144].double(), values(torch, m)
        assert ((wide[:, 160:260].double() - x @ W.T).abs() <= product_error(torch, W, x, "f32")).all()
        assert torch.equal(wide[:, :160], kept[:, :160]) and torch.equal(wide[:, 260:], kept[:, 260:])
        with pytest.raises(q8.Q8Error):
            q8.q4_gemv(q8.q4_mat(*m), wide[:, 140:240], x=wide[:, 16:144], ws=ws)


@pytest.mark.parametrize("form", ["f32", "one", "two"])
def test_projection_of_more_rows_than_the_workspace_holds(q8, form):
    """Rows taken so many at a time, and a workspace that holds none."""
    import torch
    rows, n, cols = 2113, 200, 512
    g = gen(7)
    m = matrix(torch, n, cols, 64, "f16", True, g)
    call, x = activation(torch, rows, cols, form, g)
    y = torch.full((rows, n), math.nan, device="cuda")
    small = q8.Workspace(8 << 20)
    q8.q4_gemv(q8.q4_mat(*m), y, **call, ws=small)
    W = values(torch, m)
    assert ((y.double() - x @ W.T).abs() <= product_error(torch, W, x, form)).all()
    small.check()
    small.close()
    tiny = q8.Workspace(4096)
    with pytest.raises(q8.Q8Error) as e:
        q8.q4_gemv(q8.q4_mat(*m), y, **call, ws=tiny)
    assert e.value.code == -5
    tiny.close()


def test_projection_on_a_workspace_of_which_a_wait_gave_up(q8):
    """Nothing is written until the workspace has been checked."""
    import torch
    ws = q8.Workspace()
    words = [torch.zeros(4, 2, 16, 64, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(4, 2, 16, device="cuda") for _ in range(2)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = q8.kv_pages(words[0], scales[0], words[1], scales[1])
    q = torch.zeros(1, 4, 64, device="cuda")
    q8.q8_paged_wait_selftest(pages, q8.kv_batch(i32(0, 1), i32(40), i32(0, 1, 2).view(1, 3)), q, torch.zeros_like(q), 16, ws)
    g = gen(3)
    m = matrix(torch, 300, 1024, 64, "f16", True, g)
    x = torch.randn(64, 1024, generator=g, device="cuda")
    y = torch.full((64, 300), 7.0, device="cuda")
    q8.q4_gemv(q8.q4_mat(*m), y, x=x, ws=ws)
    assert (y == 7).all()
    with pytest.raises(q8.Q8Error) as e:
        ws.check()
    assert e.value.code == -4
    q8.q4_gemv(q8.q4_mat(*m), y, x=x, ws=ws)
    W = values(torch, m)
    assert ((y.double() - x.double() @ W.T).abs() <= product_error(torch, W, x.double(), "f32")).all()
    ws.check()
    ws.close()


# ---- the experts' products -------------------------------------------------------------------------------------------


def plan_of(q8, torch, ids, experts):
    counts, offsets, lists, active = grouped(ids, experts)
    arrays = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in (counts, offsets, lists, [len(active)] + active)]
    arrays[3] = torch.cat((arrays[3], torch.full((experts - len(active),), -5, dtype=torch.int32, device="cuda")))
    return q8.plan_struct(*arrays), arrays


def choices(torch, rows, experts, k, g, skew):
    score = torch.rand(rows, experts, generator=g, device="cuda")
    if skew:  # most rows choose the same few experts
        score[:, : k + 1] += 0.9
    return score.topk(k, -1).indices.to(torch.int32)


def silu(x):
    return x / (1 + (-x).exp())


def check_hidden(torch, h, W, U_, x, ids, dff, form):
    """h against silu(Wg x) (Wu x): the products' errors through the formula (|silu'| <= 1.1), and 6 U for silu and the product."""
    for e in ids.unique().tolist():
        r, j = (ids == e).nonzero(as_tuple=True)
        Wg, Wu = W[e * dff : (e + 1) * dff], U_[e * dff : (e + 1) * dff]
        gate, up = x[r] @ Wg.T, x[r] @ Wu.T
        eg, eu = product_error(torch, Wg, x[r], form), product_error(torch, Wu, x[r], form)
        want = silu(gate) * up
        tol = 1.1 * eg * (up.abs() + eu) + silu(gate).abs() * eu + 6 * U * want.abs() + 1e-44
        assert ((h[r, j].double() - want).abs() <= tol).all()


def check_combined(torch, y, W, h, ids, gates, residual, d, form):
    """y against the gated sum of the products: their errors, k + 2 roundings of the sum's parts."""
    rows, k = ids.shape
    want = residual.double() if residual is not None else torch.zeros(rows, d, dtype=torch.float64, device="cuda")
    tol, size = torch.zeros_like(want), want.abs()
    for e in ids.unique().tolist():
        r, j = (ids == e).nonzero(as_tuple=True)
        We, g = W[e * d : (e + 1) * d], gates.double()[r, j, None]
        part = h[r, j] @ We.T
        want = want.index_add(0, r, g * part)
        size = size.index_add(0, r, (g * part).abs())
        tol = tol.index_add(0, r, g.abs() * product_error(torch, We, h[r, j], form))
    assert ((y.double() - want).abs() <= tol * 1.01 + (k + 2) * U * size + 1e-44).all()


@pytest.mark.parametrize("form", ["f32", "one", "two"])
@pytest.mark.parametrize("rows,E,k,d,dff,group,kind,zeros,skew", [
    (1, 16, 4, 256, 128, 32, "f16", False, False), (1, 128, 8, 2048, 768, 32, "f16", True, False),
    (1, 8, 8, 384, 640, 128, "bf16", True, False), (2, 16, 2, 256, 96, 32, "f16", False, False),
    (7, 20, 3, 512, 192, 64, "bf16", True, False), (24, 32, 8, 256, 256, 128, "f16", True, True),
    (70, 8, 2, 256, 160, 32, "bf16", False, True), (130, 6, 6, 128, 128, 64, "f16", True, False),
    (300, 4, 1, 256, 128, 128, "f16", False, True)])
def test_experts(q8, ws, rows, E, k, d, dff, group, kind, zeros, skew, form):
    import torch
    g = gen(rows * E + d)
    gate, up, down = (matrix(torch, n, c, group, kind, zeros, g) for n, c in ((E * dff, d), (E * dff, d), (E * d, dff)))
    ids = choices(torch, rows, E, k, g, skew)
    gates = torch.softmax(torch.randn(rows, k, generator=g, device="cuda"), -1)
    plan, kept = plan_of(q8, torch, ids, E) if rows > 1 else (None, None)
    call, x = activation(torch, rows, d, form, g)
    x = x / 16
    call = {n: (t / 16 if n in ("x", "xs") else t) for n, t in call.items()}
    h = torch.full((rows, k, dff), math.nan, device="cuda")
    q8.moe_gate_up_q4(q8.q4_mat(*gate), q8.q4_mat(*up), ids, h, **call, plan=plan, ws=ws)
    check_hidden(torch, h, values(torch, gate), values(torch, up), x, ids, dff, form)
    if form == "f32":
        hidden, hv = dict(h=h), h.double()
    else:
        q, lo, s = quantize(torch, h, form == "two")
        hidden = dict(hq=q, hs=s, hl=lo)
        hv = (q.double() if lo is None else q.double() + lo.double() / 128) * s.double().repeat_interleave(32, -1)
    residual = torch.randn(rows, d, generator=g, device="cuda")
    y = torch.full((rows, d), math.nan, device="cuda")
    W = values(torch, down)
    q8.moe_down_combine_q4(q8.q4_mat(*down), ids, gates, y, **hidden, plan=plan, residual=residual, ws=ws)
    check_combined(torch, y, W, hv, ids, gates, residual, d, form)
    q8.moe_down_combine_q4(q8.q4_mat(*down), ids, gates, y, **hidden, plan=plan, ws=ws)
    check_combined(torch, y, W, hv, ids, gates, None, d, form)
    q8.moe_down_combine_q4(q8.q4_mat(*down), ids, gates, residual, **hidden, plan=plan, residual=residual, ws=ws)  # in place
    del kept


@pytest.mark.parametrize("E,k,d,dff", [(3, 2, 32768, 32), (4, 3, 64, 32768), (9, 8, 128, 8192)])
def test_experts_of_a_row_longer_than_a_cta_holds(q8, ws, E, k, d, dff):
    """One row whose activations do not fit a CTA, with the same expert chosen twice and one out of range."""
    import torch
    g = gen(d + dff)
    gate, up, down = (matrix(torch, n, c, 32, "f16", True, g) for n, c in ((E * dff, d), (E * dff, d), (E * d, dff)))
    ids = choices(torch, 1, E, k, g, False)
    ids[0, 0] = ids[0, 1]
    gates = torch.rand(1, k, generator=g, device="cuda")
    x = torch.randn(1, d, generator=g, device="cuda") / 64
    h = torch.full((1, k, dff), math.nan, device="cuda")
    q8.moe_gate_up_q4(q8.q4_mat(*gate), q8.q4_mat(*up), ids, h, x=x, ws=ws)
    check_hidden(torch, h, values(torch, gate), values(torch, up), x.double(), ids, dff, "f32")
    y = torch.empty(1, d, device="cuda")
    q8.moe_down_combine_q4(q8.q4_mat(*down), ids, gates, y, h=h, ws=ws)
    check_combined(torch, y, values(torch, down), h.double(), ids, gates, None, d, "f32")


def test_experts_of_more_tiles_than_a_cta_looks_up(q8, ws):
    """Thousands of (expert, tile) items, the experts' rows from none to many."""
    import torch
    E, k, d, dff, rows = 300, 2, 128, 1280, 1500
    g = gen(5)
    gate, up, down = (matrix(torch, n, c, 32, "f16", False, g) for n, c in ((E * dff, d), (E * dff, d), (E * d, dff)))
    score = torch.rand(rows, E, generator=g, device="cuda") + 0.4 * (torch.arange(E, device="cuda") % 3 == 0)
    score[:, 7] = 2  # every row's
    ids = score.topk(k, -1).indices.to(torch.int32)
    gates = torch.rand(rows, k, generator=g, device="cuda")
    plan, kept = plan_of(q8, torch, ids, E)
    x = torch.randn(rows, d, generator=g, device="cuda") / 8
    h = torch.full((rows, k, dff), math.nan, device="cuda")
    q8.moe_gate_up_q4(q8.q4_mat(*gate), q8.q4_mat(*up), ids, h, x=x, plan=plan, ws=ws)
    check_hidden(torch, h, values(torch, gate), values(torch, up), x.double(), ids, dff, "f32")
    y = torch.full((rows, d), math.nan, device="cuda")
    q8.moe_down_combine_q4(q8.q4_mat(*down), ids, gates, y, h=h, plan=plan, ws=ws)
    check_combined(torch, y, values(torch, down), h.double(), ids, gates, None, d, "f32")
    del kept


def test_experts_out_of_range_and_the_same_expert_twice(q8, ws):
    import torch
    g = gen(1)
    E, k, d, dff = 8, 4, 256, 128
    gate, up, down = (matrix(torch, n, c, 32, "f16", False, g) for n, c in ((E * dff, d), (E * dff, d), (E * d, dff)))
    mats = [q8.q4_mat(*m) for m in (gate, up, down)]
    x = torch.randn(1, d, generator=g, device="cuda") / 8
    ids = torch.tensor([[3, -1, 3, E]], dtype=torch.int32, device="cuda")
    gates = torch.rand(1, k, generator=g, device="cuda")
    h = torch.full((1, k, dff), 5.0, device="cuda")
    q8.moe_gate_up_q4(mats[0], mats[1], ids, h, x=x, ws=ws)
    assert (h[0, 1] == 5).all() and (h[0, 3] == 5).all() and torch.equal(h[0, 0], h[0, 2])
    y = torch.empty(1, d, device="cuda")
    q8.moe_down_combine_q4(mats[2], ids, gates, y, h=h, ws=ws)
    one = torch.tensor([[3, 3]], dtype=torch.int32, device="cuda")
    check_combined(torch, y, values(torch, down), h[:, [0, 2]].double(), one, gates[:, [0, 2]], None, d, "f32")
    # several rows: a choice out of range is in no list
    rows = 3
    ids = torch.tensor([[3, -1, 3, E], [0, 1, 2, 3], [7, 7, 99, 7]], dtype=torch.int32, device="cuda")
    flat = [e for e in ids.flatten().tolist()]
    lists = sorted((c for c in range(12) if 0 <= flat[c] < E), key=lambda c: (flat[c], c))
    counts = [flat.count(e) for e in range(E)]
    offsets = [sum(counts[:e]) for e in range(E + 1)]
    active = [e for e in range(E) if counts[e]]
    arrays = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in (
        counts, offsets, lists + [-1] * (12 - len(lists)), [len(active)] + active + [0] * (E - len(active)))]
    plan = q8.plan_struct(*arrays)
    x = torch.randn(rows, d, generator=g, device="cuda") / 8
    h = torch.full((rows, k, dff), 5.0, device="cuda")
    q8.moe_gate_up_q4(mats[0], mats[1], ids, h, x=x, plan=plan, ws=ws)
    ok = (ids >= 0) & (ids < E)
    assert (h[~ok] == 5).all()
    h[~ok] = 0
    safe = torch.where(ok, ids, torch.zeros_like(ids))
    gates = torch.rand(rows, k, generator=g, device="cuda")
    y = torch.empty(rows, d, device="cuda")
    q8.moe_down_combine_q4(mats[2], ids, gates, y, h=h, plan=plan, ws=ws)
    check_combined(torch, y, values(torch, down), h.double(), safe, torch.where(ok, gates, torch.zeros_like(gates)), None, d, "f32")


# ---- together, as a layer calls them ---------------------------------------------------------------------------------


@pytest.mark.parametrize("rows", [1, 9, 150])
def test_layer_in_a_graph_and_on_another_stream(q8, rows):
    """The block's calls in a layer's order, each checked on what the one before it left; then captured and replayed on new
    inputs, with the results of plain launches bit for bit."""
    import torch
    g = gen(rows)
    E, k, d, dff, group = 32, 4, 512, 256, 64
    ws = q8.Workspace()
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gate, up, down = (matrix(torch, r, c, group, "f16", True, g) for r, c in ((E * dff, d), (E * dff, d), (E * d, dff)))
    router = matrix(torch, E, d, 32, "bf16", False, g)
    mats = [q8.q4_mat(*m) for m in (gate, up, down, router)]
    w_post, w_pre, bias = 1 + 0.1 * n(d), 1 + 0.1 * n(d), 0.05 * n(E)
    a, b = n(rows, d), n(rows, d)
    s, y, out = (torch.empty(rows, d, device="cuda") for _ in range(3))
    yq, ys = torch.empty(rows, d, dtype=torch.int8, device="cuda"), torch.empty(rows, d // 32, device="cuda")
    logits, h = torch.empty(rows, E, device="cuda"), torch.empty(rows, k, dff, device="cuda")
    ids, gates = torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, device="cuda")
    arrays = [torch.zeros(m, dtype=torch.int32, device="cuda") for m in (E, E + 1, rows * k, E + 1)]
    plan = q8.plan_struct(*arrays)
    rule = dict(score=q8.SCORE_SIGMOID, bias=bias, groups=4, keep_groups=2, scale=2.5)

    def layer():
        q8.postnorm_add_rmsnorm_q8(a, b, w_post, w_pre, 1e-6, scale=0.5, sum_out=s, y_out=y, yq=yq, ys=ys)
        q8.q4_gemv(mats[3], logits, x=y, ws=ws)
        q8.moe_route_scored(logits, ids, gates, **rule, plan=plan, ws=ws)
        q8.moe_gate_up_q4(mats[0], mats[1], ids, h, xq=yq, xs=ys, plan=plan, ws=ws)
        q8.moe_down_combine_q4(mats[2], ids, gates, out, h=h, plan=plan, residual=s, ws=ws)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (s, y, yq, ys, logits, ids, gates, h, out, *arrays)]

    layer()
    torch.cuda.synchronize()
    check_norm(torch, dict(a=a, b=b, w_post=w_post, w_pre=w_pre, gate=None), 0.5, float(torch.tensor(1e-6)), s, y, yq, ys)
    W = values(torch, router)
    assert ((logits.double() - y.double() @ W.T).abs() <= product_error(torch, W, y.double(), "f32")).all()
    check_route(torch, (ids, gates, arrays), logits, k, **rule)
    x = yq.double() * ys.double().repeat_interleave(32, 1)
    check_hidden(torch, h, values(torch, gate), values(torch, up), x, ids, dff, "one")
    check_combined(torch, out, values(torch, down), h.double(), ids, gates, s, d, "f32")
    first = results()
    layer()
    assert all(torch.equal(p, q) for p, q in zip(first, results()))  # a call repeats bit for bit
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer()
    a.copy_(n(rows, d))
    b.copy_(n(rows, d))
    graph.replay()
    replayed = results()
    assert not torch.equal(replayed[0], first[0])
    layer()
    assert all(torch.equal(p, q) for p, q in zip(replayed, results()))
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        layer()
    assert all(torch.equal(p, q) for p, q in zip(replayed, results()))
    ws.close()


def test_refusals_of_the_binding(q8, ws):
    """Wrong types, shapes and devices are named before anything is launched."""
    import torch
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    m = q8.q4_mat(z(64, 64, dtype=torch.uint8), z(64, 2, dtype=torch.float16))
    ids, gates = z(2, 4, dtype=torch.int32), z(2, 4)
    for word, call in [
        ("q, s", lambda: q8.q4_mat(z(64, 64), z(64, 2, dtype=torch.float16))),
        ("s: not", lambda: q8.q4_mat(z(64, 64, dtype=torch.uint8), z(64, 2))),
        ("s: ", lambda: q8.q4_mat(z(64, 64, dtype=torch.uint8), z(64, 3, dtype=torch.float16))),
        ("z: not", lambda: q8.q4_mat(z(64, 64, dtype=torch.uint8), z(64, 2, dtype=torch.float16), z(64, 2))),
        ("contiguous", lambda: q8.q4_mat(z(64, 128, dtype=torch.uint8)[:, ::2], z(64, 2, dtype=torch.float16))),
        ("current device", lambda: q8.q4_mat(torch.zeros(64, 64, dtype=torch.uint8), z(64, 2, dtype=torch.float16))),
        ("y: ", lambda: q8.q4_gemv(m, z(2, 63), x=z(2, 128), ws=ws)),
        ("x: rows differ", lambda: q8.q4_gemv(m, z(2, 64), x=z(3, 128), ws=ws)),
        ("x: not an f32", lambda: q8.q4_gemv(m, z(2, 64), x=z(2, 128).half(), ws=ws)),
        ("x: ", lambda: q8.q4_gemv(m, z(2, 64), x=z(2, 256)[:, ::2], ws=ws)),
        ("x: words without", lambda: q8.q4_gemv(m, z(2, 64), xq=z(2, 128, dtype=torch.int8), ws=ws)),
        ("x: given as", lambda: q8.q4_gemv(m, z(2, 64), x=z(2, 128), xq=z(2, 128, dtype=torch.int8), ws=ws)),
        ("ids", lambda: q8.moe_route_scored(z(2, 64), ids.long(), gates)),
        ("ids: rows", lambda: q8.moe_route_scored(z(3, 64), ids, gates)),
        ("gates", lambda: q8.moe_route_scored(z(2, 64), ids, z(2, 5))),
        ("bias", lambda: q8.moe_route_scored(z(2, 64), ids, gates, bias=z(63))),
        ("h: not", lambda: q8.moe_gate_up_q4(m, m, ids, z(2, 3, 16), x=z(2, 128), ws=ws)),
        ("plan", lambda: q8.moe_gate_up_q4(m, m, ids, z(2, 4, 16), x=z(2, 128), ws=ws)),
        ("x: not contiguous", lambda: q8.moe_gate_up_q4(m, m, ids, z(2, 4, 16), x=z(2, 256)[:, :128], ws=ws)),
        ("h: ", lambda: q8.moe_down_combine_q4(m, ids, gates, z(2, 16), h=z(2, 4, 64), ws=ws)),
        ("residual", lambda: q8.moe_down_combine_q4(m, ids, gates, z(2, 16), h=z(2, 4, 128), residual=z(2, 8), ws=ws)),
        ("b: not", lambda: q8.postnorm_add_rmsnorm_q8(z(2, 64), z(2, 32), None, z(64), 1e-6, y_out=z(2, 64))),
        ("gate: ", lambda: q8.postnorm_add_rmsnorm_q8(z(2, 64), z(2, 64), None, z(64), 1e-6, gate=z(3), y_out=z(2, 64))),
        ("yq: ", lambda: q8.postnorm_add_rmsnorm_q8(z(2, 64), z(2, 64), None, z(64), 1e-6, yq=z(2, 64, dtype=torch.int8))),
        ("a: not on", lambda: q8.postnorm_add_rmsnorm_q8(torch.zeros(2, 64), z(2, 64), None, z(64), 1e-6, y_out=z(2, 64))),
    ]:
        with pytest.raises(q8.Q8Error) as e:
            call()
        assert word in str(e.value), (word, str(e.value))
