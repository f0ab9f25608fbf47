"""The paged, quantized key/value cache: the cases it is measured on, and its operators in plain torch operations.

Three operators share one layout.  A page holds `page` positions of every key/value head; a cached row of `hd` values is
8-bit words and one f32 scale, d = max|x| / M with M = 127 (int8 words, rounded half away from zero) or 448 (e4m3 words).
A batch is `seqs` sequences; sequence b owns the rows row_start[b] .. row_start[b + 1] - 1 and has kv_len[b] cached
positions, its own rows the last of them; its position p is slot p % page of page table[b][p / page].

  write   RMS norm of every query and key head, rotation by position, then the keys and values quantized into the pages
  read    the values of the rows' cached keys and values
  attend  causal attention of the rows over their sequence's cached positions
"""
import math

import torch

own = False

_CONFIG = dict(heads=32, kv=4, hd=128)  # the framework's decode configuration
_EPS = 1e-6
_THETA = 1e6


def _case(name, do, seqs, new, length, rows="one", lengths="even", words="int8", page=16, **layout):
    case = dict(name=name, do=do, seqs=seqs, new=new, length=length, rows=rows, lengths=lengths, words=words, page=page)
    return {**case, **_CONFIG, **layout}


def listed():
    return [
        # one decode step of one sequence at the end of a 4096-position context
        _case("write_token", "write", 1, 1, 4096),
        # one decode step of a serving batch, every sequence somewhere else
        _case("write_batch", "write", 64, 1, 4096, lengths="ragged", words="e4m3"),
        # prompts of several requests written at once, q/k/v columns of one merged projection
        _case("write_prompts", "write", 5, 1021, 1500, rows="ragged", lengths="ragged", page=64, heads=24, kv=8),
        # a cached prefix read back, as when it moves to a dense cache
        _case("read_prefix", "read", 1, 4096, 4096, rows="even"),
        # long documents read back, ragged, narrow heads
        _case("read_long", "read", 3, 20011, 20011, rows="ragged", words="e4m3", page=32, heads=16, kv=8, hd=64),
        # one decode step, one sequence, a short chat
        _case("attend_token", "attend", 1, 1, 517),
        # one decode step, one sequence, a very long document
        _case("attend_long", "attend", 1, 1, 100003, page=64),
        # one decode step of a serving batch
        _case("attend_batch", "attend", 64, 1, 4096, lengths="ragged"),
        # a serving batch without shared heads, a few drafted tokens a sequence to verify
        _case("attend_drafts", "attend", 33, 3, 9001, rows="even", lengths="ragged", words="e4m3", page=32, heads=8, kv=8,
              hd=64),
        # a chunk of a long prompt over the part already cached
        _case("attend_chunk", "attend", 1, 2048, 32768, rows="even"),
        # whole prompts of several requests
        _case("attend_prompts", "attend", 4, 2048, 2048, rows="ragged", words="e4m3", page=64),
        # decoding sequences and prompt chunks in one batch
        _case("attend_mixed", "attend", 24, 300, 3000, rows="mixed", lengths="ragged", page=64, heads=24, kv=8),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    do = rng.choice(("write", "read", "attend", "attend"))
    heads, kv, hd = rng.choice(((32, 4, 128), (8, 2, 128), (24, 8, 128), (16, 8, 64), (14, 2, 64), (8, 8, 64)))
    words, page = rng.choice(("int8", "e4m3")), rng.choice((16, 32, 64, 128))
    rows, lengths = rng.choice(("one", "even", "ragged", "mixed")), rng.choice(("even", "ragged"))
    if do == "attend" and rows == "one":
        seqs = _log(rng, 1, 64)
        length = _log(rng, 1, 250000 // seqs)
        new = 1
    elif do == "attend":
        seqs = rng.randint(1, 8)
        new = _log(rng, 2, 512)
        length = new + _log(rng, 1, max(2, min(8192, 4000000 // (seqs * new))))
    else:
        seqs = _log(rng, 1, 64)
        new = 1 if rows == "one" else _log(rng, 2, max(2, 3000 // seqs))
        length = new + _log(rng, 1, max(2, 30000 // seqs))
    return dict(do=do, seqs=seqs, new=new, length=length, rows=rows, lengths=lengths, words=words, page=page, heads=heads,
                kv=kv, hd=hd)


def _sizes(case):
    """The rows and cached positions of each sequence, fixed by the case."""
    new, length = [], []
    for b in range(case["seqs"]):
        u, w = ((b + 1) * 2654435761 % 2**32) / 2**32, ((b + 1) * 2246822519 % 2**32) / 2**32
        most = case["new"]
        n = {"one": 1, "even": most, "ragged": max(1, round(u * most)), "mixed": most if b % 8 == 3 else 1}[case["rows"]]
        L = case["length"] if case["lengths"] == "even" else max(n, round((0.1 + 0.9 * w) * case["length"]))
        new.append(n)
        length.append(max(n, L))
    if case["rows"] == "ragged" and case["new"] == case["length"]:  # whole prompts: nothing cached before them
        length = list(new)
    return new, length


def _quantize(x, words):
    """The 8-bit words and the scale of every row of x (32 bits, both quotients rounded as IEEE divisions)."""
    most = torch.full((), 127.0 if words == "int8" else 448.0, device=x.device)  # a number would multiply by its inverse
    d = x.abs().amax(-1, keepdim=True) / most
    t = torch.where(d > 0, x / d, torch.zeros_like(x))
    if words == "int8":
        w = (torch.sign(t) * torch.floor(t.abs() + 0.5)).clamp(-127, 127).to(torch.int8)
    else:
        w = t.clamp(-448, 448).to(torch.float8_e4m3fn)
    return w, d.squeeze(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    H, KV, hd, page = case["heads"], case["kv"], case["hd"], case["page"]
    new, length = _sizes(case)
    rows, most = sum(new), max(length)
    held = [-(-L // page) for L in length]
    order = torch.randperm(sum(held) + 3, generator=g, device="cuda").to(torch.int32)  # pages in no order, three unused
    table = torch.zeros(case["seqs"], max(held), dtype=torch.int32)
    mine = torch.arange(table.shape[1])[None, :] < torch.tensor(held)[:, None]
    table[mine] = order[: sum(held)].cpu()
    state = dict(
        case=case, most_new=max(new), table=table.cuda(),
        row_start=torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda(),
        kv_len=torch.tensor(length, dtype=torch.int32).cuda(),
    )
    pages = sum(held) + 3
    for name in ("k", "v"):
        if case["do"] == "write":
            kind = torch.int8 if case["words"] == "int8" else torch.float8_e4m3fn
            state[name + "_words"] = torch.zeros(pages, KV, page, hd, device="cuda").to(kind)
            state[name + "_scale"] = torch.zeros(pages, KV, page, device="cuda")
        else:  # unit-sized heads, as the norm leaves them
            w, d = _quantize(normal(pages, KV, page, hd), case["words"])
            state[name + "_words"], state[name + "_scale"] = w, d
    if case["do"] == "write":
        merged = normal(rows, (H + 2 * KV) * hd)  # one projection's output: queries, keys, values
        state["q"] = merged[:, : H * hd].unflatten(1, (H, hd))
        state["k"] = merged[:, H * hd : (H + KV) * hd].unflatten(1, (KV, hd))
        state["v"] = merged[:, (H + KV) * hd :].unflatten(1, (KV, hd))
        state["q_norm"], state["k_norm"] = 1 + 0.1 * normal(hd), 1 + 0.1 * normal(hd)
        i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
        angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * _THETA ** (-2 * i / hd)
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
        state["q_out"] = torch.empty(rows, H, hd, device="cuda")
    elif case["do"] == "read":
        state["k_out"], state["v_out"] = (torch.empty(rows, KV, hd, device="cuda") for _ in range(2))
    else:
        state["q"] = 1.5 * normal(rows, H, hd)
        state["out"] = torch.empty(rows, H, hd, device="cuda")
    return state


def _places(state):
    """Each row's sequence, its place among the sequence's rows, its position, page and slot."""
    start, page = state["row_start"].long(), state["case"]["page"]
    rows = (state["q"] if "q" in state else state["k_out"]).shape[0]
    r = torch.arange(rows, device="cuda")
    b = torch.searchsorted(start[1:], r, right=True)
    position = state["kv_len"].long()[b] - start[b + 1] + r
    return b, r - start[b], position, state["table"][b, position // page].long(), position % page


def _turn(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _write(state):
    _, _, position, page, slot = _places(state)
    cos, sin = state["cos"][position][:, None], state["sin"][position][:, None]
    q, k = state["q"], state["k"].double()  # a key's words turn on values next to a border: 64 bits up to its rounding
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + _EPS) * state["q_norm"]
    k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + _EPS) * state["k_norm"]
    state["q_out"].copy_(_turn(q, cos, sin))
    for name, x in (("k", _turn(k, cos, sin).float()), ("v", state["v"])):
        words, scale = _quantize(x, state["case"]["words"])
        state[name + "_words"].view(torch.int8)[page, :, slot] = words.view(torch.int8)
        state[name + "_scale"][page, :, slot] = scale


def _read(state):
    _, _, _, page, slot = _places(state)
    for name in ("k", "v"):
        words = state[name + "_words"].view(torch.int8)[page, :, slot].view(state[name + "_words"].dtype)
        torch.mul(words.float(), state[name + "_scale"][page, :, slot][..., None], out=state[name + "_out"])


def _dense(state, name):
    """A sequence's cached rows in order, as values: [seqs, kv, positions, hd]."""
    at = state["table"].long()
    words = state[name + "_words"].view(torch.int8)[at].view(state[name + "_words"].dtype)
    x = words.float() * state[name + "_scale"][at][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(state):
    case = state["case"]
    KV, hd, group = case["kv"], case["hd"], case["heads"] // case["kv"]
    b, i, position, _, _ = _places(state)
    seqs, new = case["seqs"], state["most_new"]
    q = torch.zeros(seqs, new, KV, group, hd, device="cuda")
    q[b, i] = state["q"].unflatten(1, (KV, group))
    last = torch.full((seqs, new), -1, device="cuda")
    last[b, i] = position
    k, v = _dense(state, "k"), _dense(state, "v")
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = (q @ k.transpose(2, 3)).mul_(hd**-0.5).unflatten(2, (group, new))
    seen = torch.arange(k.shape[2], device="cuda") <= last[:, :, None]
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    total = s.sum(-1, keepdim=True)
    out = (s.flatten(2, 3) @ v).unflatten(2, (group, new)) / total
    state["out"].copy_(out.permute(0, 3, 1, 2, 4)[b, i].flatten(1, 2))


_workspace = None


def run(state):
    do = state["case"]["do"]
    if own:
        import moe_add_rmsnorm_gb300 as q8

        global _workspace
        if _workspace is None:
            _workspace = q8.Workspace()
        pages = q8.kv_pages(state["k_words"], state["k_scale"], state["v_words"], state["v_scale"])
        batch = q8.kv_batch(state["row_start"], state["kv_len"], state["table"])
        if do == "write":
            q8.q8_kv_append(pages, batch, state["q"], state["k"], state["v"], state["q_out"], q_norm=state["q_norm"],
                            k_norm=state["k_norm"], eps=_EPS, cos=state["cos"], sin=state["sin"])
        elif do == "read":
            q8.q8_kv_read(pages, batch, state["k_out"], state["v_out"])
        else:
            q8.q8_paged_attention(pages, batch, state["q"], state["out"], ws=_workspace)
    else:
        {"write": _write, "read": _read, "attend": _attend}[do](state)
    if do == "write":
        return {n: state[n] for n in ("q_out", "k_words", "k_scale", "v_words", "v_scale")}
    return [state["k_out"], state["v_out"]] if do == "read" else state["out"]


def work(case):
    H, KV, hd, page = case["heads"], case["kv"], case["hd"], case["page"]
    new, length = _sizes(case)
    rows, cached = sum(new), sum(length)
    row_bytes = 2 * KV * (hd + 4)  # a position's words and scales
    index = 8 * case["seqs"]
    if case["do"] == "write":
        table = 4 * sum(-(-L // page) - (L - n) // page for n, L in zip(new, length))
        tables = 4 * hd * rows  # a row's cosines and sines
        return {"bytes": 4 * rows * hd * (2 * H + 2 * KV) + rows * row_bytes + tables + table + index,
                "flops": rows * hd * (H + KV) * 8}
    if case["do"] == "read":
        return {"bytes": rows * (row_bytes + 8 * KV * hd) + 4 * sum(-(-L // page) for L in length) + index,
                "flops": 2 * rows * KV * hd}
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for n, L in zip(new, length))
    return {"bytes": 8 * rows * H * hd + cached * row_bytes + 4 * sum(-(-L // page) for L in length) + index,
            "flops": 4 * hd * H * pairs}


def _exact_rows(state, name, b):
    """Sequence b's cached rows in 64 bits: [kv, positions, hd]."""
    L, page = int(state["kv_len"][b]), state["case"]["page"]
    p = torch.arange(L, device="cuda")
    at, slot = state["table"][b].long()[p // page], p % page
    words = state[name + "_words"]
    words = words.view(torch.int8)[at, :, slot].view(words.dtype).float().double()
    return (words * state[name + "_scale"].double()[at, :, slot][..., None]).transpose(0, 1)


def exact(case, seed):
    state = prepare(case, seed)
    new, length = _sizes(case)
    H, KV, hd, page = case["heads"], case["kv"], case["hd"], case["page"]
    starts = [sum(new[:b]) for b in range(len(new))]
    if case["do"] == "attend":
        out = torch.empty(sum(new), H, hd, dtype=torch.float64, device="cuda")
        for b, (n, L, r) in enumerate(zip(new, length, starts)):
            k, v = _exact_rows(state, "k", b), _exact_rows(state, "v", b)
            for h in range(H):
                j = h // (H // KV)
                s = state["q"][r : r + n, h].double() @ k[j].T / math.sqrt(hd)
                hidden = torch.arange(L, device="cuda")[None, :] > torch.arange(L - n, L, device="cuda")[:, None]
                out[r : r + n, h] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[j]
        return out
    if case["do"] == "read":
        return [torch.cat([_exact_rows(state, name, b)[:, L - n :].transpose(0, 1)
                           for b, (n, L) in enumerate(zip(new, length))]) for name in ("k", "v")]

    place = torch.cat([torch.arange(L - n, L) for n, L in zip(new, length)]).cuda()

    def normed(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / hd + _EPS).sqrt() * w.double()
        z = torch.complex(x[..., : hd // 2], x[..., hd // 2 :])
        z = z * torch.complex(state["cos"].double()[place], state["sin"].double()[place])[:, None]
        return torch.cat((z.real, z.imag), -1)

    most = 127.0 if case["words"] == "int8" else 448.0
    found = {"q_out": normed(state["q"], state["q_norm"])}
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
    at, slot = state["table"][seq, place // page].long(), place % page
    for name, x in (("k", normed(state["k"], state["k_norm"])), ("v", state["v"].double())):
        scale = torch.zeros_like(state[name + "_scale"], dtype=torch.float64)
        scale[at, :, slot] = x.abs().amax(-1) / most
        found[name + "_scale"], found[name + "_words"] = scale, None
        if case["words"] == "e4m3":  # the quotient before its rounding to 4 bits
            found[name + "_words"] = torch.zeros(scale.shape + (hd,), dtype=torch.float64, device="cuda")
            found[name + "_words"][at, :, slot] = x / scale[at, :, slot][..., None]
    return found
