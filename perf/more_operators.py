"""A sparse feed-forward block with 4-bit weights: the cases it is measured on, and its operators in plain torch operations.

Four operators, in the order a layer calls them (everything f32 unless said otherwise):

  norm     the block before ends in a norm and the next one begins with one: with the block's output b and the residual a
           s = a + scale * gate * norm(b) * w_post,  y = norm(s) * w_pre,  and y's int8 form (one or two words a value)
  route    expert scores from the router's logits: p = softmax(l) or sigmoid(l), chosen by p + bias among the experts of the
           best groups (a group's mark is its best, or the sum of its two best), weighed by p; and the choices grouped by
           expert.  A logit of -infinity takes its expert out of service
  project  y = W x with W = s (word - z): 4-bit words, a 16-bit scale s and a zero point z for every group of columns; x is
           f32, or int8 words with a scale for every 32 values (one or two words a value)
  experts  h = silu(Wg x) * (Wu x) of each row's chosen experts, y = residual + sum_j gate_j Wd h_j, the matrices as above

A 4-bit matrix [rows, cols] is words uint8 [rows, cols / 2] (value 2i in the low half of byte i, 2i + 1 in the high one),
scales float16 or bfloat16 [rows, cols / group] and zero points uint8 of the same shape, or none of these (8 everywhere).
"""
import math

import torch

own = False

_EPS = 1e-6


def _norm(name, rows, d, gate, words, scale=1.0):
    return dict(name=name, do="norm", rows=rows, d=d, gate=gate, words=words, scale=scale)


def _route(name, rows, experts, k, score, bias, groups, keep, renorm, scale, plan, masked=False, top=2):
    return dict(name=name, do="route", rows=rows, experts=experts, k=k, score=score, bias=bias, groups=groups, keep=keep,
                renorm=renorm, scale=scale, plan=plan, masked=masked, top=top)


def _project(name, rows, n, cols, group, kind, zeros, act, merged=False):
    return dict(name=name, do="project", rows=rows, n=n, cols=cols, group=group, kind=kind, zeros=zeros, act=act,
                merged=merged)


def _experts(name, rows, experts, k, d, dff, group, kind, zeros, act):
    return dict(name=name, do="experts", rows=rows, experts=experts, k=k, d=d, dff=dff, group=group, kind=kind, zeros=zeros,
                act=act)


def listed():
    return [
        # one decode step of one sequence
        _norm("norm_token", 1, 2048, "none", "one"),
        # one decode step of a serving batch, each row with a gate of its own
        _norm("norm_batch", 37, 5120, "row", "two", 0.5),
        # prompts of several requests, a gate a channel
        _norm("norm_prompts", 4096, 4096, "channel", "none"),
        # one decode step of one sequence, the framework's own routing rule
        _route("route_token", 1, 128, 8, "softmax", False, 1, 1, True, 1.0, False),
        # one decode step of a serving batch, balanced by a bias, grouped for the experts
        _route("route_batch", 61, 256, 8, "sigmoid", True, 8, 4, True, 2.5, True),
        # prompts of several requests
        _route("route_prompts", 15001, 256, 8, "sigmoid", True, 8, 4, True, 2.5, True),
        # one decode step: queries, keys and values of one sequence
        _project("project_token", 1, 5120, 2048, 32, "f16", False, "f32"),
        # one decode step: the head over the vocabulary, from a row the norm left quantized
        _project("project_head", 1, 151936, 2048, 128, "bf16", True, "one"),
        # a chunk of a prompt, its rows columns of a wider buffer
        _project("project_chunk", 61, 8192, 4096, 64, "f16", True, "f32", merged=True),
        # one decode step of one sequence
        _experts("experts_token", 1, 128, 8, 2048, 768, 32, "f16", False, "f32"),
        # one decode step of a serving batch, from rows the norm left quantized
        _experts("experts_batch", 24, 128, 8, 2048, 768, 128, "bf16", True, "one"),
        # a chunk of a prompt
        _experts("experts_chunk", 200, 64, 6, 2048, 1408, 64, "f16", False, "f32"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    do = rng.choice(("norm", "route", "project", "experts"))
    matrix = (rng.choice((32, 64, 128)), rng.choice(("f16", "bf16")), rng.choice((False, True)),
              rng.choice(("f32", "f32", "one", "two")))
    if do == "norm":
        d = 32 * _log(rng, 4, 256)
        rows = _log(rng, 1, min(8192, 4096 * 4096 // d))
        case = _norm("", rows, d, rng.choice(("none", "channel", "row", "full")), rng.choice(("none", "one", "two")),
                     rng.choice((1.0, 0.5, 0.22)))
    elif do == "route":
        groups, each = rng.choice((1, 1, 2, 4, 8)), rng.choice((8, 12, 16, 20, 32))
        if groups == 1:
            each = rng.choice((8, 60, 64, 96, 128, 160, 256, 512))
        keep = rng.randint(1, groups)
        experts = groups * each
        rows = _log(rng, 1, min(16384, 15001 * 256 // experts))
        case = _route("", rows, experts, rng.randint(1, min(10, keep * each)), rng.choice(("softmax", "sigmoid")),
                      rng.choice((False, True)), groups, keep, rng.choice((False, True)), rng.choice((1.0, 2.5)),
                      rng.choice((False, True)), rng.choice((False, False, True)), rng.choice((1, 2)))
    elif do == "project":
        cols = 128 * _log(rng, 2, 64)
        rows = _log(rng, 1, 64)
        n = _log(rng, 64, min(160000, 151936 * 2048 // cols, 61 * 8192 * 4096 // (rows * cols)))
        case = _project("", rows, n, cols, *matrix, merged=rng.choice((False, True)))
    else:
        experts, k, d, dff = rng.choice(((128, 8, 2048, 768), (64, 6, 2048, 1408), (16, 2, 2048, 4096), (32, 4, 1536, 1024),
                                         (60, 4, 1024, 640), (160, 6, 2560, 384)))
        rows = _log(rng, 1, min(256, 200 * 6 * 2048 * 1408 // (k * d * dff)))
        case = _experts("", rows, experts, k, d, dff, *matrix)
    del case["name"]
    return case


# ---- inputs ----------------------------------------------------------------------------------------------------------


def _words_of(x, two):
    """The int8 form of x: words, low words (or None) and the scale of every 32 values, as the framework's quantizer."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=x.device)  # a number would multiply by its inverse
    t = torch.where(d > 0, b / d, torch.zeros_like(b))
    hi = (torch.sign(t) * torch.floor(t.abs() + 0.5)).clamp(-127, 127)
    lo = None
    if two:
        r = (t - hi) * 128
        lo = (torch.sign(r) * torch.floor(r.abs() + 0.5)).clamp(-127, 127).to(torch.int8).flatten(-2)
    return hi.to(torch.int8).flatten(-2), lo, d.squeeze(-1)


def _matrix(case, rows, cols, g):
    groups = cols // case["group"]
    kind = torch.float16 if case["kind"] == "f16" else torch.bfloat16
    words = torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = (0.004 + 0.008 * torch.rand(rows, groups, generator=g, device="cuda")).to(kind)
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(5, 12, (rows, groups), generator=g, device="cuda", dtype=torch.uint8)
    return words, scale, zeros


def _grouping(ids, experts):
    """The choices of ids [rows, k] by expert: counts, offsets, lists, active (as the framework's plan holds them)."""
    flat = ids.flatten().long()
    counts = torch.zeros(experts, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((torch.zeros_like(counts[:1]), counts.cumsum(0)))
    lists = torch.sort(flat, stable=True).indices
    some = counts > 0
    place = torch.where(some, some.cumsum(0), torch.full_like(counts, experts + 1))
    active = torch.zeros(experts + 2, dtype=torch.int64, device="cuda")
    active.scatter_(0, place, torch.arange(experts, device="cuda"))
    active[0] = some.sum()
    return [t.to(torch.int32) for t in (counts, offsets, lists, active[: experts + 1])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    do, rows = case["do"], case["rows"]
    state = dict(case=case)
    if do == "norm":
        d = case["d"]
        state.update(a=4 * normal(rows, d), b=normal(rows, d) * (0.5 + normal(rows, 1).abs()), w_post=1 + 0.1 * normal(d),
                     w_pre=1 + 0.1 * normal(d), gate=None, sum=torch.empty(rows, d, device="cuda"))
        if case["gate"] != "none":
            state["gate"] = torch.sigmoid(normal(*{"channel": (d,), "row": (rows, 1), "full": (rows, d)}[case["gate"]]))
        if case["words"] == "none":
            state["y"] = torch.empty(rows, d, device="cuda")
        else:
            state["yq"] = torch.empty(rows, d, dtype=torch.int8, device="cuda")
            state["yl"] = torch.empty_like(state["yq"]) if case["words"] == "two" else None
            state["ys"] = torch.empty(rows, d // 32, device="cuda")
    elif do == "route":
        experts, k = case["experts"], case["k"]
        state["logits"] = 1.5 * normal(rows, experts)
        if case["masked"]:  # experts out of service, differing from row to row
            state["logits"][torch.rand(rows, experts, generator=g, device="cuda") < 0.1] = -math.inf
        state["bias"] = 0.05 * normal(experts) if case["bias"] else None
        state["ids"] = torch.empty(rows, k, dtype=torch.int32, device="cuda")
        state["gates"] = torch.empty(rows, k, device="cuda")
        state["plan"] = None
        if case["plan"]:
            state["plan"] = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (experts, experts + 1, rows * k,
                                                                                      experts + 1)]
    else:
        cols = case["cols"] if do == "project" else case["d"]
        wide = cols + 128 if case.get("merged") else cols
        x = normal(rows, wide)[:, wide - cols:]
        if case["act"] == "f32":
            state["x"] = x
        else:
            state["xq"], state["xl"], state["xs"] = _words_of(x, case["act"] == "two")
        if do == "project":
            state["W"] = _matrix(case, case["n"], cols, g)
            state["y"] = torch.empty(rows, case["n"], device="cuda")
        else:
            experts, k, d, dff = case["experts"], case["k"], case["d"], case["dff"]
            state["gate"], state["up"] = _matrix(case, experts * dff, d, g), _matrix(case, experts * dff, d, g)
            state["down"] = _matrix(case, experts * d, dff, g)
            chosen = torch.rand(rows, experts, generator=g, device="cuda").topk(k, -1).indices
            state["ids"] = chosen.to(torch.int32)
            state["gates"] = torch.softmax(normal(rows, k), -1)
            state["plan"] = _grouping(chosen, experts) if rows > 1 else None
            state["residual"] = normal(rows, d)
            state["h"] = torch.empty(rows, k, dff, device="cuda")
            state["y"] = torch.empty(rows, d, device="cuda")
    return state


# ---- the plain forms -------------------------------------------------------------------------------------------------


def _plain_norm(state):
    case = state["case"]
    a, b = state["a"].double(), state["b"].double()  # the words turn on values next to a border: 64 bits up to the roundings
    p = b * torch.rsqrt(b.square().mean(-1, keepdim=True) + _EPS) * state["w_post"]
    if state["gate"] is not None:
        p = p * state["gate"]
    s = (a + case["scale"] * p).float()
    state["sum"].copy_(s)
    s = s.double()
    y = (s * torch.rsqrt(s.square().mean(-1, keepdim=True) + _EPS) * state["w_pre"]).float()
    if case["words"] == "none":
        state["y"].copy_(y)
    else:
        hi, lo, d = _words_of(y, case["words"] == "two")
        state["yq"].copy_(hi)
        state["ys"].copy_(d)
        if lo is not None:
            state["yl"].copy_(lo)


def _plain_route(state):
    case = state["case"]
    rows, E, k, G = case["rows"], case["experts"], case["k"], case["groups"]
    l = state["logits"].double()  # choices turn on scores next to one another: 64 bits
    most = l.amax(-1, keepdim=True)
    off = l == -math.inf
    if case["score"] == "softmax":
        e = torch.where(off, torch.zeros_like(l), (l - most.clamp_min(-1e30)).exp())
        p = e / e.sum(-1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1 / (1 + (-l).exp())
    # without a bias the order of the scores is the logits'
    mark = p + state["bias"].double() if case["bias"] else (p if G > 1 else l)
    mark = mark.masked_fill(off, -math.inf)
    if G > 1:
        best = torch.sort(mark.unflatten(1, (G, -1)), dim=-1, descending=True, stable=True).values[..., : case["top"]]
        best = torch.where(best[..., 0] > -math.inf, best.masked_fill(best == -math.inf, 0).sum(-1), best[..., 0])
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, : case["keep"]]
        hidden = torch.ones(rows, G, dtype=torch.bool, device="cuda").scatter_(1, kept, False)
        hidden = hidden.repeat_interleave(E // G, 1)
        order = l if not case["bias"] else mark
        order = torch.where(off, torch.full_like(l, -1e300), order).masked_fill(hidden, -math.inf)
    else:
        order = mark
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :k]
    gate = p.gather(1, ids)
    if case["renorm"]:
        gate = gate / gate.sum(-1, keepdim=True).clamp_min(1e-300)
    state["ids"].copy_(ids)
    state["gates"].copy_(gate * case["scale"])
    if state["plan"] is not None:
        for to, made in zip(state["plan"], _grouping(ids, E)):
            to.copy_(made)


def _values(matrix, part=slice(None)):
    """A 4-bit matrix's values (of some of its rows) in f32."""
    words, scale, zeros = matrix
    words, scale = words[part], scale[part].float()
    w = torch.stack((words & 15, words >> 4), -1).flatten(-2).float().unflatten(-1, (scale.shape[-1], -1))
    z = zeros[part].float()[..., None] if zeros is not None else 8.0
    return ((w - z) * scale[..., None]).flatten(-2)


def _activation(state):
    if "x" in state:
        return state["x"]
    x = state["xq"].float()
    if state["xl"] is not None:
        x = x + state["xl"].float() / 128
    return (x.unflatten(-1, (-1, 32)) * state["xs"][..., None]).flatten(-2)


def _plain_project(state):
    state["y"].copy_(_activation(state) @ _values(state["W"]).T)


def _plain_experts(state):
    case = state["case"]
    rows, E, k, d, dff = (case[n] for n in ("rows", "experts", "k", "d", "dff"))
    x, ids = _activation(state), state["ids"].long()
    if rows * k <= E:  # the chosen experts' rows
        at = (ids.flatten()[:, None] * dff + torch.arange(dff, device="cuda")).flatten()
        xs = x.repeat_interleave(k, 0)[:, :, None]
        gate, up = (_values(state[n], at).unflatten(0, (rows * k, dff)) @ xs for n in ("gate", "up"))
        h = (gate / (1 + (-gate).exp()) * up).squeeze(-1)
        state["h"].copy_(h.unflatten(0, (rows, k)))
        at = (ids.flatten()[:, None] * d + torch.arange(d, device="cuda")).flatten()
        out = (_values(state["down"], at).unflatten(0, (rows * k, d)) @ h[:, :, None]).squeeze(-1)
        y = (out.unflatten(0, (rows, k)) * state["gates"][..., None]).sum(1)
    else:  # every expert over every row
        hs, y = torch.zeros(rows, k, dff, device="cuda"), torch.zeros(rows, d, device="cuda")
        for e in range(E):
            mine = (ids == e)[..., None]
            rows_of = slice(e * dff, (e + 1) * dff)
            gate, up = (x @ _values(state[n], rows_of).T for n in ("gate", "up"))
            h = gate / (1 + (-gate).exp()) * up
            hs += torch.where(mine, h[:, None], torch.zeros_like(hs))
            weight = torch.where(mine[..., 0], state["gates"], torch.zeros_like(state["gates"])).sum(-1, keepdim=True)
            y += weight * (h @ _values(state["down"], slice(e * d, (e + 1) * d)).T)
        state["h"].copy_(hs)
    state["y"].copy_(state["residual"] + y)


# ---- one pass --------------------------------------------------------------------------------------------------------

_workspace = None


def _own(state):
    import moe_add_rmsnorm_gb300 as q8

    global _workspace
    case, do = state["case"], state["case"]["do"]
    if do == "norm":
        q8.postnorm_add_rmsnorm_q8(state["a"], state["b"], state["w_post"], state["w_pre"], _EPS, gate=state["gate"],
                                   scale=case["scale"], sum_out=state["sum"], y_out=state.get("y"), yq=state.get("yq"),
                                   ys=state.get("ys"), yl=state.get("yl"))
        return
    if _workspace is None:
        _workspace = q8.Workspace()
    if "handles" not in state:  # a program builds its matrices' and plans' structs once
        state["handles"] = {n: q8.q4_mat(*state[n]) for n in ("W", "gate", "up", "down") if n in state}
        if state.get("plan") is not None:
            state["handles"]["plan"] = q8.plan_struct(*state["plan"])
    m = state["handles"]
    if do == "route":
        q8.moe_route_scored(state["logits"], state["ids"], state["gates"],
                            score=q8.SCORE_SOFTMAX if case["score"] == "softmax" else q8.SCORE_SIGMOID, bias=state["bias"],
                            groups=case["groups"], keep_groups=case["keep"], group_top=case["top"], renorm=case["renorm"],
                            scale=case["scale"], plan=m.get("plan"), ws=_workspace)
    elif do == "project":
        q8.q4_gemv(m["W"], state["y"], x=state.get("x"), xq=state.get("xq"), xs=state.get("xs"), xl=state.get("xl"),
                   ws=_workspace)
    else:
        q8.moe_gate_up_q4(m["gate"], m["up"], state["ids"], state["h"], x=state.get("x"), xq=state.get("xq"),
                          xs=state.get("xs"), xl=state.get("xl"), plan=m.get("plan"), ws=_workspace)
        q8.moe_down_combine_q4(m["down"], state["ids"], state["gates"], state["y"], h=state["h"], plan=m.get("plan"),
                               residual=state["residual"], ws=_workspace)


def run(state):
    do = state["case"]["do"]
    if own:
        _own(state)
    else:
        {"norm": _plain_norm, "route": _plain_route, "project": _plain_project, "experts": _plain_experts}[do](state)
    if do == "norm":
        return {n: state[n] for n in ("sum", "y", "yq", "yl", "ys") if state.get(n) is not None}
    if do == "route":
        return [state["ids"], state["gates"]] + (state["plan"] or [])
    return state["y"] if do == "project" else [state["h"], state["y"]]


def _matrix_bytes(case, rows, cols):
    return rows * (cols // 2 + cols // case["group"] * (3 if case["zeros"] else 2))


def _act_bytes(case, rows, cols):
    return {"f32": 4 * rows * cols, "one": rows * (cols + cols // 8), "two": rows * (2 * cols + cols // 8)}[case["act"]]


def work(case):
    do, rows = case["do"], case["rows"]
    if do == "norm":
        d = case["d"]
        gate = {"none": 0, "channel": d, "row": rows, "full": rows * d}[case["gate"]]
        out = {"none": 4 * d, "one": d + d // 8, "two": 2 * d + d // 8}[case["words"]]
        return {"bytes": rows * (12 * d + out) + 4 * (2 * d + gate), "flops": 11 * rows * d}
    if do == "route":
        E, k = case["experts"], case["k"]
        plan = 4 * (3 * E + rows * k) if case["plan"] else 0
        return {"bytes": 4 * rows * E + (4 * E if case["bias"] else 0) + 8 * rows * k + plan, "flops": 6 * rows * E}
    if do == "project":
        n, cols = case["n"], case["cols"]
        return {"bytes": _matrix_bytes(case, n, cols) + _act_bytes(case, rows, cols) + 4 * rows * n,
                "flops": 2 * rows * n * cols}
    E, k, d, dff = (case[n] for n in ("experts", "k", "d", "dff"))
    hit = E * (1 - (1 - k / E) ** rows)  # distinct experts, on average
    matrices = 2 * _matrix_bytes(case, dff, d) + _matrix_bytes(case, d, dff)
    return {"bytes": int(hit * matrices) + _act_bytes(case, rows, d) + rows * (8 * d + 4 * k * (dff + 2)),
            "flops": 6 * rows * k * d * dff}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------------


def _exact_matrix(matrix):
    words, scale, zeros = matrix
    cols = 2 * words.shape[1]
    w = torch.empty(words.shape[0], cols, dtype=torch.float64, device="cuda")
    w[:, 0::2] = (words % 16).double()
    w[:, 1::2] = torch.div(words, 16, rounding_mode="floor").double()
    width = cols // scale.shape[1]
    z = zeros.double() if zeros is not None else torch.full(scale.shape, 8.0, dtype=torch.float64, device="cuda")
    return (w - z.repeat_interleave(width, 1)) * scale.double().repeat_interleave(width, 1)


def _exact_activation(state):
    if "x" in state:
        return state["x"].double()
    x = state["xq"].double()
    if state["xl"] is not None:
        x = (128 * x + state["xl"].double()) / 128
    return x * state["xs"].double().repeat_interleave(32, 1)


def _exact_route(case, state):
    E, k, G = case["experts"], case["k"], case["groups"]
    l = state["logits"].cpu().double()
    p = torch.softmax(l, -1) if case["score"] == "softmax" else torch.sigmoid(l)
    mark = p + state["bias"].cpu().double() if case["bias"] else p
    mark[l == -math.inf] = -math.inf
    if G > 1:
        each = mark.reshape(-1, G, E // G)
        best = each.topk(case["top"], -1).values
        best = torch.where(best[..., 0] == -math.inf, best[..., 0], torch.nan_to_num(best, neginf=0.0).sum(-1))
        least = best.topk(case["keep"], -1).values[:, -1:]
        mark = each.masked_fill((best < least)[..., None], -math.inf).reshape(-1, E)
    ids = mark.topk(k, -1).indices
    gates = p.gather(1, ids)
    chosen = mark.gather(1, ids) > -math.inf
    if not bool(chosen.all()):  # fewer experts in service than choices
        return None
    if case["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    out = [ids.to(torch.int32).cuda(), (gates * case["scale"]).cuda()]
    if case["plan"]:
        flat = ids.flatten().numpy()
        counts = torch.bincount(ids.flatten(), minlength=E)
        lists = torch.from_numpy(flat.argsort(kind="stable"))
        active = torch.zeros(E + 1, dtype=torch.int64)
        hit = counts.nonzero().flatten()
        active[0] = len(hit)
        active[1 : 1 + len(hit)] = hit
        offsets = torch.tensor([0] + counts.cumsum(0).tolist())
        out += [t.to(torch.int32).cuda() for t in (counts, offsets, lists, active)]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    do = case["do"]
    if do == "norm":
        a, b = state["a"].double(), state["b"].double()
        d = case["d"]
        p = b / (b.pow(2).sum(-1, keepdim=True) / d + _EPS).sqrt() * state["w_post"].double() * case["scale"]
        s = a + (p * state["gate"].double() if state["gate"] is not None else p)
        y = s / (s.pow(2).sum(-1, keepdim=True) / d + _EPS).sqrt() * state["w_pre"].double()
        if case["words"] == "none":
            return {"sum": s, "y": y}
        scale = y.reshape(case["rows"], d // 32, 32).abs().amax(-1) / 127
        return {"sum": s, "yq": None, **({"yl": None} if case["words"] == "two" else {}), "ys": scale}
    if do == "route":
        return _exact_route(case, state)
    x = _exact_activation(state)
    if do == "project":
        return x @ _exact_matrix(state["W"]).T
    rows, k, d, dff = (case[n] for n in ("rows", "k", "d", "dff"))
    h = torch.zeros(rows, k, dff, dtype=torch.float64, device="cuda")
    y = state["residual"].double()
    ids = state["ids"].long()
    for e in ids.unique().tolist():
        r, j = (ids == e).nonzero(as_tuple=True)
        part = {n: _exact_matrix([t if t is None else t[e * m : (e + 1) * m] for t in state[n]])
                for n, m in (("gate", dff), ("up", dff), ("down", d))}
        g, u = x[r] @ part["gate"].T, x[r] @ part["up"].T
        h[r, j] = g * torch.sigmoid(g) * u
        y[r] = y[r] + state["gates"].double()[r, j, None] * (h[r, j] @ part["down"].T)
    return [h, y]
