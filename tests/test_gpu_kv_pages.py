"""The paged, quantized key/value cache on the GPU: q8_kv_append, q8_kv_read and q8_paged_attention against their formulas in
64 bits, at the sizes, layouts and masks where they can go wrong, and together as a layer uses them.

Tolerances.  Words and scales follow the formula rounded to f32 once and are compared exactly.  Queries are normed and
rotated in f32: the sum of squares, root, quotient and three products of a value are at most 20 roundings of 2^-24, and
the rotation adds |a| + |b|.  Attention: a query is split into two 11-bit parts (2^-22 of each product) and a score's
products are added in f32 by at most 16 truncating steps of 2^-23, so a score is off by at most 2^-18 of its products'
magnitudes; the weighted values are added the same way, with one exponential (2^-22), 16 steps between folds and a fold
every 128 positions; both enter the output times the weights: (2 delta + 2^-17) * sum p |v|.  A weight times its value
row's scale is split into two f16 parts after a scaling that puts a tile's largest scale times weight 1 at 2^14 or above;
what lies under f16's smallest normal number, 2^-14, may be lost, so a position's share is off by at most the smaller of
its weight (relative to the row's largest, 1) and 2^-28, times the largest value there is.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

EPS = 1e-6


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def quantize(x, words):
    """The rule of q8_kv_pages for every row of an f32 tensor."""
    import torch
    most = torch.full((), 127.0 if words == "int8" else 448.0, device=x.device)  # (a number would multiply by its inverse)
    d = x.abs().amax(-1, keepdim=True) / most
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    t = torch.where((d > 0) & ~bad, x / d, torch.zeros_like(x))
    if words == "int8":
        w = (torch.sign(t) * torch.floor(t.abs() + 0.5)).clamp(-127, 127).to(torch.int8)
    else:
        w = t.clamp(-448, 448).to(torch.float8_e4m3fn)
    d = torch.where(bad, torch.full_like(d, math.nan), d)
    return w, d.squeeze(-1)


class Cache:
    """Pages in no order with some spare, and the batch over them."""

    def __init__(self, q8, new, length, kv, hd, page, words, seed, fill=True):
        import torch
        g = gen(seed)
        held = [-(-L // page) for L in length]
        self.q8, self.new, self.length, self.kv, self.hd, self.page, self.kind = q8, new, length, kv, hd, page, words
        pages = sum(held) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        width = max(1, max(held))
        self.table = torch.full((len(new), width + 2), 10 ** 9, dtype=torch.int32, device="cuda")
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order[at:at + h]
            at += h
        self.row_start = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        self.kv_len = torch.tensor(length, dtype=torch.int32).cuda()
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")
        kind = torch.int8 if words == "int8" else torch.float8_e4m3fn
        # slots past a sequence's end hold what an allocation may: every bit set, and scales that are not numbers
        self.kw, self.vw = (torch.full((pages, kv, page, hd), -1, dtype=torch.int8, device="cuda").view(kind)
                            for _ in range(2))
        self.ks, self.vs = (torch.full((pages, kv, page), math.nan, device="cuda") for _ in range(2))
        if fill:
            for b, L in enumerate(length):
                for w, s in ((self.kw, self.ks), (self.vw, self.vs)):
                    x = torch.randn(L, kv, hd, generator=g, device="cuda") * \
                        torch.exp(torch.randn(L, kv, 1, generator=g, device="cuda"))
                    qw, d = quantize(x, words)
                    a, o = self.where(b, torch.arange(L, device="cuda"))
                    w.view(torch.int8)[a, :, o] = qw.view(torch.int8)
                    s[a, :, o] = d

    def where(self, b, p):
        return self.table[b].long()[p // self.page], p % self.page

    def pages(self):
        return self.q8.kv_pages(self.kw, self.ks, self.vw, self.vs)

    def batch(self):
        t = self.table[:, :self.table.shape[1] - 2]  # strided: two columns of the tensor are not the table's
        return self.q8.kv_batch(self.row_start, self.kv_len, t, self.error)

    def values(self, name, b, dtype=None):
        """[L, kv, hd] of sequence b."""
        import torch
        w, s = (self.kw, self.ks) if name == "k" else (self.vw, self.vs)
        a, o = self.where(b, torch.arange(self.length[b], device="cuda"))
        w = w.view(torch.int8)[a, :, o].view(w.dtype).float()
        dtype = dtype or torch.float64
        return w.to(dtype) * s[a, :, o][..., None].to(dtype)


@pytest.fixture(scope="module")
def ws(q8):
    w = q8.Workspace()
    yield w
    w.close()


# ---- writing ---------------------------------------------------------------------------------------------------------

def rope(q8, positions, hd):
    import torch
    cos, sin = (torch.empty(positions, hd // 2, device="cuda") for _ in range(2))
    q8.q8_rope_table(1e6, cos, sin)
    return cos, sin


@pytest.mark.parametrize("hd,positions", [(64, 1), (128, 4096), (128, 200001)])
def test_rope_table(q8, hd, positions):
    import torch
    cos, sin = rope(q8, positions, hd)
    i = torch.arange(hd // 2, dtype=torch.float64)
    p = torch.tensor(sorted({0, positions // 3, positions - 1}), dtype=torch.float64)
    a = p[:, None] * 1e6 ** (-2 * i / hd)
    at = p.long()
    # half a step of f32 at 1, and the angle's own error (a few steps of f64 of an angle up to `positions`)
    tol = 2 ** -25 + 2 ** -50 * positions
    assert (cos.cpu()[at].double() - a.cos()).abs().max() <= tol
    assert (sin.cpu()[at].double() - a.sin()).abs().max() <= tol


def expected_append(c, x, w, cos, sin, positions):
    """Norm and rotation of [rows, heads, hd] in f64."""
    import torch
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
    if cos is None:
        return x
    h = c.hd // 2
    cs, sn = cos[positions].double()[:, None], sin[positions].double()[:, None]
    a, b = x[..., :h], x[..., h:]
    return torch.cat((a * cs - b * sn, a * sn + b * cs), -1)


APPEND = [
    # new rows, lengths, heads, kv, hd, page, words, norm, rope
    ([1], [1], 8, 2, 128, 16, "int8", True, True),
    ([1], [4096], 32, 4, 128, 16, "int8", True, True),
    ([1, 1, 1], [17, 16, 300], 32, 4, 128, 16, "e4m3", True, True),
    ([5, 0, 33, 1, 0], [5, 7, 64, 65, 0], 8, 2, 128, 32, "int8", True, True),
    ([100, 3], [100, 129], 14, 2, 64, 64, "e4m3", True, True),
    ([7, 90], [40, 90], 9, 3, 64, 1024, "int8", False, True),
    ([64], [70], 6, 6, 128, 16, "e4m3", True, False),
    ([19, 20], [19, 21], 5, 5, 64, 16, "int8", False, False),
    ([1] * 70, list(range(1, 71)), 4, 1, 128, 16, "int8", True, True),
    ([2] * 1100, [5] * 1100, 2, 1, 64, 16, "int8", True, True),
]


@pytest.mark.parametrize("new,length,heads,kv,hd,page,words,norm,turn", APPEND)
@pytest.mark.parametrize("merged", [False, True])
def test_append(q8, new, length, heads, kv, hd, page, words, norm, turn, merged):
    import torch
    c = Cache(q8, new, length, kv, hd, page, words, 3, fill=False)
    g, rows = gen(4), sum(new)
    tail = 2  # rows behind the last sequence
    wide = torch.randn(rows + tail, heads + 2 * kv, hd, generator=g, device="cuda") * 3
    q, k, v = wide[:, :heads], wide[:, heads:heads + kv], wide[:, heads + kv:]
    if not merged:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    k[0, 0] = 0  # a row of zeros has no scale
    v[0, 0] = 0
    qw, kw = ((1 + 0.1 * torch.randn(hd, generator=g, device="cuda") if norm else None) for _ in range(2))
    cos, sin = rope(q8, max(length), hd) if turn else (None, None)
    before = [t.clone() for t in (c.kw.view(torch.int8), c.vw.view(torch.int8), c.ks, c.vs)]
    q_out = torch.full((rows + tail, heads, hd), 7.5, device="cuda")
    q8.q8_kv_append(c.pages(), c.batch(), q, k, v, q_out, q_norm=qw, k_norm=kw, eps=EPS, cos=cos, sin=sin)
    assert c.error.item() == 0
    positions = torch.cat([torch.arange(L - n, L) for n, L in zip(new, length)]).cuda()
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
    page_of, slot = c.table[seq, positions // page].long(), positions % page
    z = expected_append(c, q[:rows], qw, cos, sin, positions)
    lim = z.abs() + z.roll(hd // 2, -1).abs()
    assert ((q_out[:rows].double() - z).abs() <= 20 * 2 ** -24 * lim + 1e-30).all()
    assert (q_out[rows:] == 7.5).all()
    zk = expected_append(c, k[:rows], kw, cos, sin, positions).float()
    for x, w, s, w0, s0 in ((zk, c.kw, c.ks, before[0], before[2]), (v[:rows], c.vw, c.vs, before[1], before[3])):
        qx, d = quantize(x, words)
        w0[page_of, :, slot] = qx.view(torch.int8)
        s0[page_of, :, slot] = d
        assert torch.equal(s.view(torch.int32), s0.view(torch.int32))  # every slot, those not written among them
        # (as values: -0 and 0 are the same word)
        assert torch.equal(w.float().nan_to_num(1e4), w0.view(w.dtype).float().nan_to_num(1e4))


def test_append_in_place_and_keys_only(q8):
    import torch
    c = Cache(q8, [3, 2], [20, 2], 2, 128, 16, "int8", 5, fill=False)
    g = gen(6)
    q, k, v = (torch.randn(5, h, 128, generator=g, device="cuda") for h in (8, 2, 2))
    cos, sin = rope(q8, 32, 128)
    w = 1 + 0.1 * torch.randn(128, generator=g, device="cuda")
    out = torch.empty_like(q)
    q8.q8_kv_append(c.pages(), c.batch(), q, k, v, out, q_norm=w, k_norm=w, cos=cos, sin=sin)
    kw, vs = c.kw.clone(), c.vs.clone()
    c.kw.fill_(-1)
    q8.q8_kv_append(c.pages(), c.batch(), q, k, v, q, q_norm=w, k_norm=w, cos=cos, sin=sin)
    assert torch.equal(q, out) and torch.equal(c.kw, kw)
    c.kw.fill_(-1)
    q8.q8_kv_append(c.pages(), c.batch(), None, k, v, None, k_norm=w, cos=cos, sin=sin)
    assert torch.equal(c.kw, kw) and torch.equal(c.vs.nan_to_num(), vs.nan_to_num())


@pytest.mark.parametrize("words", ["int8", "e4m3"])
def test_append_extreme_rows(q8, words):
    """Rows with an infinity or a NaN read back as NaN; tiny, huge and zero rows follow the rule."""
    import torch
    c = Cache(q8, [8], [8], 1, 64, 16, words, 7, fill=False)
    g = gen(8)
    k = torch.randn(8, 1, 64, generator=g, device="cuda")
    k[0, 0, 5], k[1, 0, 63], k[2, 0, 0] = math.inf, -math.inf, math.nan
    k[3] *= 1e-38
    k[4] *= 1e-42  # subnormal: its scale is subnormal or zero
    k[5] *= 1e37
    k[6] = 0
    v = k.flip(2).contiguous()
    q8.q8_kv_append(c.pages(), c.batch(), None, k, v, None)
    for x, w, s in ((k, c.kw, c.ks), (v, c.vw, c.vs)):
        qx, d = quantize(x, words)
        a, o = c.where(0, torch.arange(8, device="cuda"))
        assert torch.equal(s[a, :, o].nan_to_num(-1), d.nan_to_num(-1))
        assert torch.equal(w.view(torch.int8)[a, :, o].view(w.dtype).float(), qx.float())
    back = torch.empty(8, 1, 64, device="cuda")
    q8.q8_kv_read(c.pages(), c.batch(), k_out=back)
    assert back[:3].isnan().all() and back[3:].isfinite().all()


# ---- reading ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("new,length,kv,hd,page,words", [
    ([1], [1], 1, 64, 16, "int8"), ([4096], [4096], 4, 128, 16, "int8"), ([3, 0, 50, 1], [9, 40, 50, 17], 2, 128, 32, "e4m3"),
    ([200, 7], [700, 1025], 8, 64, 64, "e4m3"), ([33], [40], 3, 64, 1024, "int8"), ([1] * 40, [5] * 40, 5, 128, 16, "int8")])
def test_read(q8, new, length, kv, hd, page, words):
    import torch
    c = Cache(q8, new, length, kv, hd, page, words, 9)
    rows = sum(new)
    ref = {n: torch.cat([c.values(n, b, torch.float32)[L - m:] for b, (m, L) in enumerate(zip(new, length))]) for n in "kv"}
    k, v = (torch.full((rows + 2, kv, hd), 7.5, device="cuda") for _ in range(2))
    q8.q8_kv_read(c.pages(), c.batch(), k, v)
    assert torch.equal(k[:rows], ref["k"]) and torch.equal(v[:rows], ref["v"])
    assert (k[rows:] == 7.5).all() and (v[rows:] == 7.5).all() and c.error.item() == 0
    dense = torch.full((kv, rows + 5, hd), 7.5, device="cuda")  # a dense cache's layout, values alone
    q8.q8_kv_read(c.pages(), c.batch(), None, dense.transpose(0, 1)[:rows])
    assert torch.equal(dense[:, :rows].transpose(0, 1), ref["v"]) and (dense[:, rows:] == 7.5).all()


# ---- attention -------------------------------------------------------------------------------------------------------

def attention64(c, q, scale, hidden=None):
    """Output, lse and the bound on the output's error, in f64; hidden(b, positions): positions left out of sequence b."""
    import torch
    rows, heads, hd = q.shape
    out, lse, lim = (torch.zeros(rows, heads, n, dtype=torch.float64, device="cuda") for n in (hd, 1, hd))
    lse.fill_(-math.inf)
    r = 0
    for b, (n, L) in enumerate(zip(c.new, c.length)):
        if n == 0:
            continue
        k, v = c.values("k", b), c.values("v", b)
        x = q[r:r + n].double().unflatten(1, (c.kv, heads // c.kv))
        p = torch.arange(L, device="cuda")
        seen = p[None, :] <= torch.arange(L - n, L, device="cuda")[:, None]
        if hidden is not None:
            seen = seen & ~hidden(b, p)[None, :]
        gone = ~seen.any(0)
        k[gone], v[gone] = 0, 0
        s = torch.einsum("nkgd,tkd->nkgt", x, k) * scale
        size = torch.einsum("nkgd,tkd->nkgt", x.abs(), k.abs()) * scale
        s = s.masked_fill(~seen[:, None, None], -math.inf)
        some = seen.any(1)
        m = s.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        e = (s - m).exp()
        total = e.sum(-1, keepdim=True)
        w = torch.where(total > 0, e / total, torch.zeros_like(e))
        delta = size.masked_fill(~seen[:, None, None], 0).amax(-1, keepdim=True) * 2 ** -18
        o = torch.einsum("nkgt,tkd->nkgd", w, v)
        near = torch.einsum("nkgt,tkd->nkgd", w, v.abs()) * (2 * delta + 2 ** -17)
        small = e.clamp_max(2 ** -28).sum(-1, keepdim=True) / total.clamp_min(1)
        near = near + small * v.abs().amax(0).amax(-1)[None, :, None, None]
        out[r:r + n], lim[r:r + n] = o.flatten(1, 2), near.flatten(1, 2)
        lse[r:r + n] = torch.where(some[:, None, None, None], m + total.log(), torch.full_like(m, -math.inf)).flatten(1, 2)
        r += n
    return out, lse.squeeze(-1), lim


def close(out, lse, ref):
    o, l, lim = ref
    rows = o.shape[0]
    assert ((out[:rows].double() - o).abs() <= lim).all(), \
        f"off by {(out[:rows].double() - o).abs().max():.3e}, allowed up to {lim.max():.3e}"
    if lse is not None:
        fine = l.isfinite()
        got = lse[:rows].double()
        assert bool((got[~fine] == -math.inf).all())
        assert ((got - l)[fine].abs() <= 2 ** -17 + 2 ** -18 * 64 * l[fine].abs().clamp_min(1)).all()


ATTEND = [
    # new rows, lengths, heads, kv, hd, page, words
    ([1], [1], 8, 2, 128, 16, "int8"),
    ([1], [2], 1, 1, 64, 16, "e4m3"),
    ([1], [127], 32, 4, 128, 16, "int8"),
    ([1], [128], 32, 4, 128, 32, "e4m3"),
    ([1], [129], 32, 4, 128, 64, "int8"),
    ([1], [5000], 32, 4, 128, 16, "int8"),
    ([1], [40001], 8, 1, 128, 64, "int8"),
    ([1], [3001], 14, 2, 64, 16, "e4m3"),
    ([1] * 9, [1, 15, 16, 17, 255, 256, 257, 1000, 31], 32, 4, 128, 16, "int8"),
    ([1] * 33, [37 * (i + 1) for i in range(33)], 8, 8, 64, 32, "int8"),
    ([1] * 200, [(i * 97) % 700 + 1 for i in range(200)], 16, 4, 128, 16, "e4m3"),
    ([1] * 1500, [(i * 89) % 90 + 1 for i in range(1500)], 4, 2, 64, 16, "int8"),
    ([1, 0, 1, 0], [300, 5, 7, 0], 24, 8, 128, 16, "int8"),
    ([2], [2], 8, 8, 128, 16, "int8"),
    ([3, 3, 3], [500, 3, 77], 32, 4, 128, 16, "e4m3"),
    ([16], [16], 8, 1, 64, 16, "int8"),
    ([17], [18], 32, 4, 128, 16, "int8"),
    ([128], [128], 8, 8, 128, 128, "int8"),
    ([129], [400], 8, 2, 128, 16, "int8"),
    ([200], [1000], 14, 2, 64, 64, "e4m3"),
    ([513], [513], 32, 4, 128, 64, "int8"),
    ([300], [5000], 9, 3, 128, 16, "e4m3"),
    ([40, 0, 1, 260, 5], [40, 9, 1000, 300, 129], 10, 2, 128, 32, "int8"),
    ([64, 1, 1, 1, 30], [64, 2000, 3, 129, 4000], 32, 4, 64, 16, "int8"),
    ([20], [20], 64, 1, 128, 16, "int8"),
    ([33], [333], 48, 1, 64, 1024, "e4m3"),
    ([1], [700], 64, 1, 128, 16, "int8"),
    ([2], [100], 23, 1, 128, 16, "int8"),
    ([1], [3000], 16, 1, 128, 16, "int8"),
    ([1, 1, 1], [33, 2500, 700], 24, 2, 64, 32, "e4m3"),
    ([1] * 30, [100 + 61 * i for i in range(30)], 22, 2, 128, 16, "e4m3"),
    ([1, 300, 1], [900, 400, 77], 12, 1, 128, 16, "int8"),
    ([2, 2, 1, 40], [700, 2, 1300, 40], 8, 1, 128, 64, "int8"),
    ([1], [3000], 32, 1, 128, 16, "int8"),
    ([1, 1], [2000, 9], 30, 1, 64, 1024, "e4m3"),
    ([2, 3, 4, 5, 1], [900, 500, 64, 3000, 7], 8, 1, 128, 16, "int8"),
    ([20] + [0] * 19, [900] + [0] * 19, 32, 4, 128, 16, "e4m3"),
    ([1, 0, 33, 4] * 200, [(i * 53) % 200 + 40 for i in range(800)], 8, 2, 128, 16, "int8"),
    ([16, 1, 700, 17, 2], [16, 1, 700, 2500, 1100], 8, 1, 64, 16, "e4m3"),
]


@pytest.mark.parametrize("new,length,heads,kv,hd,page,words", ATTEND)
def test_attention(q8, ws, new, length, heads, kv, hd, page, words):
    import torch
    c = Cache(q8, new, length, kv, hd, page, words, 11)
    rows = sum(new)
    wide = torch.randn(rows + 2, heads + 1, hd, generator=gen(12), device="cuda")
    q = wide[:, :heads]  # strided rows
    out = torch.full((rows + 2, heads + 2, hd), 7.5, device="cuda")
    lse = torch.full((rows + 2, heads), 7.5, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, out[:, :heads], lse=lse, ws=ws)
    assert c.error.item() == 0
    close(out[:, :heads], lse, attention64(c, q[:rows], hd ** -0.5))
    assert (out[rows:] == 7.5).all() and (out[:, heads:] == 7.5).all() and (lse[rows:] == 7.5).all()
    again = torch.empty(rows + 2, heads, hd, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, again, ws=ws)  # the same bits, and no lse
    assert torch.equal(again[:rows], out[:rows, :heads])


@pytest.mark.parametrize("new,length,heads,kv,hd,words", [([1] * 40, [300 + 41 * i for i in range(40)], 32, 4, 128, "int8"),
                                                          ([700, 1, 90], [700, 3000, 1500], 24, 8, 128, "int8"),
                                                          ([400, 300], [400, 900], 14, 2, 64, "e4m3"),
                                                          ([3], [20000], 32, 2, 128, "e4m3"),
                                                          ([5, 40, 17, 1] * 9, [60 + 31 * i for i in range(36)], 16, 2, 64, "int8")])
def test_attention_back_to_back(q8, ws, new, length, heads, kv, hd, words):
    """Many launches in a row, on two batches in turn: every one gives the first one's bits (the order in which CTAs meet
    decides nothing, and no launch leaves anything behind for the next)."""
    import torch
    caches = [Cache(q8, new, length, kv, hd, 16, words, seed) for seed in (31, 32)]
    q = torch.randn(sum(new), heads, hd, generator=gen(33), device="cuda")
    first = []
    for c in caches:
        first.append(torch.empty_like(q))
        q8.q8_paged_attention(c.pages(), c.batch(), q, first[-1], ws=ws)
    outs = [torch.empty_like(q) for _ in range(60)]
    for i, o in enumerate(outs):
        q8.q8_paged_attention(caches[i % 2].pages(), caches[i % 2].batch(), q, o, ws=ws)
    assert all(torch.equal(o, first[i % 2]) for i, o in enumerate(outs))
    assert caches[0].error.item() == 0 and caches[1].error.item() == 0


@pytest.mark.parametrize("new,length,words", [([1, 1], [400, 70], "int8"), ([150, 1], [600, 200], "e4m3")])
@pytest.mark.parametrize("factor", [0.01, 30.0])
def test_attention_flat_and_sharp(q8, ws, new, length, words, factor):
    """Nearly equal weights, and weights of one position alone (scores in the thousands)."""
    import torch
    c = Cache(q8, new, length, 2, 128, 16, words, 13)
    q = torch.randn(sum(new), 8, 128, generator=gen(14), device="cuda") * factor
    out = torch.empty_like(q)
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, scale=0.25, ws=ws)
    close(out, None, attention64(c, q, 0.25))


@pytest.mark.parametrize("new,length", [([1], [300]), ([140], [300])])
def test_attention_not_finite(q8, ws, new, length):
    """A key or value row that is not a number reaches the rows that see it and no others; so does a query."""
    import torch
    c = Cache(q8, new, length, 2, 128, 16, "int8", 15)
    n, L = new[0], length[0]
    q = torch.randn(n, 8, 128, generator=gen(16), device="cuda")
    ref = attention64(c, q, 128 ** -0.5)
    out = torch.empty_like(q)
    if n > 1:
        at = L - n + 70  # rows 70 .. see it
        a, o = c.where(0, torch.tensor([at], device="cuda"))
        c.ks[a, 0, o] = math.nan
        c.vs[a, 1, o] = math.inf
        q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=ws)
        assert not out[70:].isfinite().any()
        close(out[:70], None, tuple(t[:70] for t in ref))
        c = Cache(q8, new, length, 2, 128, 16, "int8", 15)
    q[n - 1, 3, 7] = math.inf
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=ws)
    assert not out[n - 1, 3].isfinite().any()
    out[n - 1, 3] = ref[0][n - 1, 3].float()
    close(out, None, ref)


@pytest.mark.parametrize("new,length", [([1, 1, 1], [300, 40, 600]), ([100, 30, 1], [300, 40, 600])])
def test_attention_value_scales_far_apart(q8, ws, new, length):
    """Key and value rows of very different magnitude in one tile, the values tiny."""
    import torch
    c = Cache(q8, new, length, 2, 128, 16, "int8", 17)
    g = gen(18)
    for s in (c.ks, c.vs):
        s.mul_(torch.exp2(torch.randint(-6, 7, s.shape, generator=g, device="cuda").float()))
    c.vs.mul_(1e-20)
    q = torch.randn(sum(new), 8, 128, generator=g, device="cuda") * 0.1
    out = torch.empty_like(q)
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=ws)
    close(out, None, attention64(c, q, 128 ** -0.5))


@pytest.mark.parametrize("new,length", [([1, 1], [200, 40]), ([60, 50], [200, 50])])
def test_bad_pages_and_lengths_are_left_out(q8, ws, new, length):
    """Page ids and lengths out of range: flagged, never followed."""
    import torch
    c = Cache(q8, new, length, 2, 128, 16, "int8", 19)
    rows = sum(new)
    q = torch.randn(rows, 8, 128, generator=gen(20), device="cuda")
    table = c.table.clone()
    c.table[0, 2], c.table[0, 5] = -1, c.kw.shape[0]
    hidden = lambda b, p: ((p // 16 == 2) | (p // 16 == 5)) if b == 0 else torch.zeros_like(p, dtype=torch.bool)  # noqa: E731
    good = Cache(q8, new, length, 2, 128, 16, "int8", 19)
    ref = attention64(good, q, 128 ** -0.5, hidden)
    out, lse = torch.empty_like(q), torch.empty(rows, 8, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
    close(out, lse, ref)
    assert c.error.item() == q8.KV_ERR_PAGE
    c.table[0].fill_(-7)  # no page of the first sequence
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
    assert (out[:new[0]] == 0).all() and (lse[:new[0]] == -math.inf).all()
    close(out, lse, attention64(good, q, 128 ** -0.5, lambda b, p: torch.full_like(p, b == 0, dtype=torch.bool)))
    back = torch.full((rows, 2, 128), 7.5, device="cuda")
    q8.q8_kv_read(c.pages(), c.batch(), back)
    assert (back[:new[0]] == 7.5).all() and (back[new[0]:] != 7.5).any()
    words = c.kw.clone()
    k = torch.randn(rows, 2, 128, generator=gen(21), device="cuda")
    q_out = torch.zeros_like(q)
    q8.q8_kv_append(c.pages(), c.batch(), q, k, k, q_out)
    assert torch.equal(q_out, q)  # the queries are written all the same
    page = c.table[1, (length[1] - new[1]) // 16: -(-length[1] // 16)].long()
    other = torch.ones(c.kw.shape[0], dtype=torch.bool, device="cuda")
    other[page] = False
    assert torch.equal(c.kw[other], words[other])
    c.table.copy_(table)
    for bad in (new[0] - 1, 10 ** 6, -5):
        c.error.zero_()
        c.kv_len[0] = bad
        out.fill_(7.5)
        q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
        assert (out[:new[0]] == 0).all() and (lse[:new[0]] == -math.inf).all() and (out[new[0]:] != 7.5).all()
        back.fill_(7.5)
        q8.q8_kv_read(c.pages(), c.batch(), back)
        assert (back[:new[0]] == 7.5).all() and c.error.item() == q8.KV_ERR_LENGTH
    c.kv_len[0] = length[0]
    c.error.zero_()
    c.row_start[0] = -3  # the first sequence's rows are not the call's
    out.fill_(7.5)
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=ws)
    assert (out[:new[0]] == 7.5).all() and (out[new[0]:] != 7.5).all() and c.error.item() == q8.KV_ERR_LENGTH
    c.row_start[0] = 0
    c.error.zero_()
    cos, sin = rope(q8, length[0] - 1, 128)  # the first sequence's last row lies past the tables
    q_out.fill_(7.5)
    q8.q8_kv_append(c.pages(), c.batch(), q, k, k, q_out, cos=cos, sin=sin)
    assert (q_out[new[0] - 1] == 7.5).all() and (q_out[new[0]:] != 7.5).any() and c.error.item() == q8.KV_ERR_ROPE


@pytest.mark.parametrize("starts", [[7, 0, 1, 9], [0, 9, 3, 9], [5, 5, 0, 9], [-4, 0, -9, 2 ** 31 - 1]])
def test_decreasing_row_starts(q8, ws, starts):
    """Rows that no sequence owns are left as they were, whatever a search among the starts lands on; nothing is read or
    written past a table's row or outside the sequences' pages."""
    import torch
    rows, page = 9, 16
    c = Cache(q8, [3, 3, 3], [48, 48, 48], 2, 128, page, "int8", 31)
    c.row_start.copy_(torch.tensor(starts, dtype=torch.int64).to(torch.int32))
    table = c.table[:, :3].contiguous()  # (positions 48 on are past its row: another sequence's pages, or the end)
    owned = torch.zeros(rows, dtype=torch.bool)
    slots = torch.zeros(c.kw.shape[0], page, dtype=torch.bool, device="cuda")
    for b in range(3):
        first, n = starts[b], starts[b + 1] - starts[b]
        if first >= 0 and 0 <= n <= 48 and first + n <= rows:
            owned[first:first + n] = True
            for p in range(48 - n, 48):
                slots[table[b, p // page].long(), p % page] = True
    batch = q8.kv_batch(c.row_start, c.kv_len, table, c.error)
    back = torch.full((rows, 2, 128), 7.5, device="cuda")
    q8.q8_kv_read(c.pages(), batch, back)
    assert (back[~owned.cuda()] == 7.5).all() and c.error.item() == q8.KV_ERR_LENGTH
    before = c.kw.clone()
    x = torch.randn(rows, 2, 128, generator=gen(32), device="cuda")
    q_out = torch.full_like(x, 7.5)
    q8.q8_kv_append(c.pages(), batch, x, x, x, q_out)
    assert (q_out[~owned.cuda()] == 7.5).all()
    assert torch.equal(c.kw.transpose(1, 2)[~slots], before.transpose(1, 2)[~slots])
    out = torch.full((rows, 4, 128), 7.5, device="cuda")
    q8.q8_paged_attention(c.pages(), batch, torch.randn(rows, 4, 128, generator=gen(33), device="cuda"), out, ws=ws)
    assert (out[~owned.cuda()] == 7.5).all()


def test_pages_and_batches_of_another_device_are_refused(q8, ws):
    import torch
    c = Cache(q8, [1], [5], 1, 64, 16, "int8", 34)
    x = torch.ones(1, 1, 64, device="cuda")
    for which in range(2):
        both = [c.pages(), c.batch()]
        both[which].device += 1
        for call in (lambda: q8.q8_kv_append(*both, x, x, x, x), lambda: q8.q8_kv_read(*both, x),
                     lambda: q8.q8_paged_attention(*both, x, torch.empty_like(x), ws=ws)):
            with pytest.raises(q8.Q8Error, match="current device"):
                call()


def test_addresses_past_32_bits(q8, ws):
    """Words behind 2^32 bytes and scales behind 2^27 values."""
    import torch
    pages, kv, page, hd = 1 << 17, 5, 64, 128  # 5.4 GB of words each, 168 MB of scales
    c = Cache(q8, [70, 1], [300, 1000], kv, hd, page, "int8", 23)
    big = [torch.zeros(pages, kv, page, hd, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.zeros(pages, kv, page, device="cuda") for _ in range(2)]
    shift = pages - c.kw.shape[0]
    for t, s in zip(big + scale, (c.kw, c.vw, c.ks, c.vs)):
        t[shift:] = s
    table = torch.where(c.table < 10 ** 8, c.table + shift, c.table)
    q = torch.randn(71, 10, hd, generator=gen(24), device="cuda")
    ref, out = torch.empty_like(q), torch.empty_like(q)
    q8.q8_paged_attention(c.pages(), c.batch(), q, ref, ws=ws)
    far = q8.kv_pages(big[0], scale[0], big[1], scale[1])
    batch = q8.kv_batch(c.row_start, c.kv_len, table[:, :16], c.error)
    q8.q8_paged_attention(far, batch, q, out, ws=ws)
    assert torch.equal(out, ref)
    k, v, k2, v2 = (torch.empty(71, kv, hd, device="cuda") for _ in range(4))
    q8.q8_kv_read(c.pages(), c.batch(), k, v)
    q8.q8_kv_read(far, batch, k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    q8.q8_kv_append(c.pages(), c.batch(), None, v, k, None)
    q8.q8_kv_append(far, batch, None, v, k, None)
    assert torch.equal(big[0][shift:], c.kw) and torch.equal(scale[1][shift:].nan_to_num(), c.vs.nan_to_num())
    assert not big[0][:shift].any() and c.error.item() == 0


# ---- together --------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("new", [[1, 1, 1], [1, 40, 3]])
def test_captured_step_follows_the_device_arrays(q8, new):
    """Append and attention captured once on a side stream and replayed as the sequences grow: each replay does what the
    plain calls do.  Two graphs share one workspace, replayed in turn on one stream."""
    import torch
    kv, hd, heads, page = 2, 128, 8, 16
    base = [200, 40, 7]
    steps, rows = 5, sum(new)
    full = [L + steps * n for L, n in zip(base, new)]
    c = Cache(q8, new, full, kv, hd, page, "int8", 25)
    ref = Cache(q8, new, full, kv, hd, page, "int8", 25)
    w = q8.Workspace()
    cos, sin = rope(q8, 512, hd)
    g = gen(26)
    q, k, v, out, out2 = (torch.empty(rows, h, hd, device="cuda") for h in (heads, kv, kv, heads, heads))
    turned = torch.empty_like(q)

    def step(cache, o, work):
        q8.q8_kv_append(cache.pages(), cache.batch(), q, k, v, turned, cos=cos, sin=sin)
        q8.q8_paged_attention(cache.pages(), cache.batch(), turned, o, ws=work)

    side = torch.cuda.Stream()
    graphs = []
    for scale in (None, 0.5):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            if scale is None:
                step(c, out, w)
            else:
                q8.q8_paged_attention(c.pages(), c.batch(), turned, out2, scale=scale, ws=w)
        graphs.append(gr)
    for i in range(steps):
        lens = torch.tensor([L + (i + 1) * n for L, n in zip(base, new)], dtype=torch.int32)
        for t in (c, ref):
            t.kv_len.copy_(lens)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graphs[0].replay()
        graphs[1].replay()
        got, got2 = out.clone(), out2.clone()
        step(ref, out, w)
        q8.q8_paged_attention(ref.pages(), ref.batch(), turned, out2, scale=0.5, ws=w)
        assert torch.equal(got, out) and torch.equal(got2, out2) and torch.equal(c.kw, ref.kw)
    assert c.error.item() == 0
    w.close()


@pytest.mark.parametrize("nbytes,new", [(1 << 20, [1, 1]), (1 << 20, [90]), (8 << 20, [1, 90])])
def test_a_small_workspace_is_refused(q8, ws, nbytes, new):
    """Nothing of the call is launched, not the half that would have had room either; the next call is as ever."""
    import torch
    c = Cache(q8, new, [200] * len(new), 2, 128, 16, "int8", 35)
    q = torch.randn(sum(new), 8, 128, generator=gen(36), device="cuda")
    out, want = torch.full_like(q, 7.5), torch.empty_like(q)
    small = q8.Workspace(nbytes)
    with pytest.raises(q8.Q8Error, match="workspace too small"):
        q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=small)
    torch.cuda.synchronize()
    assert (out == 7.5).all()
    q8.q8_paged_attention(c.pages(), c.batch(), q, want, ws=ws)
    close(want, None, attention64(c, q, 128 ** -0.5))
    small.close()


def test_two_streams_with_their_own_workspaces(q8):
    import torch
    c = Cache(q8, [1] * 20 + [60], [500] * 21, 4, 128, 16, "int8", 27)
    q = torch.randn(80, 32, 128, generator=gen(28), device="cuda")
    spaces = [q8.Workspace() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = torch.empty_like(q)
    q8.q8_paged_attention(c.pages(), c.batch(), q, want, ws=spaces[0])
    outs = [[torch.empty_like(q) for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for s, w, o in zip(streams, spaces, outs):
            q8.q8_paged_attention(c.pages(), c.batch(), q, o[i], ws=w, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for each in outs for o in each)
    for w in spaces:
        w.close()


def test_a_layer_over_pages_and_back_into_the_dense_cache(q8, ws):
    """What a serving program does: a layer's attention side over pages (norm, projections, append, attention, output
    projection) against the same layer in f64 over the values the cache holds; then the cache is read back into a dense
    model's caches and the model takes its next step from there."""
    import numpy as np
    import torch

    import oracle
    from synth import recipes
    cfg = dict(layers=1, d=256, heads=8, kv_heads=2, hd=128, experts=16, k=4, dff=64, vocab=512, ctx=64, eps=1e-6,
               rope_theta=1e6)
    arr = recipes.decode_model(cfg, seed=1)

    def dv(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    t = {k: ([tuple(map(dv, e)) if isinstance(e, tuple) else dv(e) for e in v] if isinstance(v, list)
             else tuple(map(dv, v)) if isinstance(v, tuple) else dv(v)) for k, v in arr.items()}
    n = 21
    tokens = [(37 * i + 5) % cfg["vocab"] for i in range(n)]
    h = t["embed"][torch.tensor(tokens, device="cuda")]
    c = Cache(q8, [n], [n], 2, 128, 16, "int8", 29, fill=False)
    cos, sin = rope(q8, cfg["ctx"], 128)
    x, q, k, v = (torch.empty(n, w, device="cuda") for w in (256, 1024, 256, 256))
    q8.add_rmsnorm_q8(h, None, t["attn_norm"][0], cfg["eps"], y_out=x)
    for name, y in (("wq", q), ("wk", k), ("wv", v)):
        q8.q8_gemv(*t[name][0], q8.F32ACT_F64SUM, y, x=x, rows=n, ws=ws)
    qr, att = torch.empty(n, 8, 128, device="cuda"), torch.empty(n, 8, 128, device="cuda")
    q8.q8_kv_append(c.pages(), c.batch(), q.view(n, 8, 128), k.view(n, 2, 128), v.view(n, 2, 128), qr,
                    q_norm=t["q_norm"][0], k_norm=t["k_norm"][0], eps=cfg["eps"], cos=cos, sin=sin)
    q8.q8_paged_attention(c.pages(), c.batch(), qr, att, ws=ws)
    o = torch.empty(n, 256, device="cuda")
    q8.q8_gemv(*t["wo"][0], q8.F32ACT_F64SUM, o, x=att.view(n, 1024), rows=n, ws=ws)

    # the same in f64, over the values the cache holds
    hd64 = h.double()
    x64 = hd64 * torch.rsqrt(hd64.square().mean(-1, keepdim=True) + cfg["eps"]) * t["attn_norm"][0].double()
    dense = lambda m: m[0].double() * m[1].double().repeat_interleave(32, 1)  # noqa: E731
    positions = torch.arange(n, device="cuda")
    q64 = expected_append(c, (x64 @ dense(t["wq"][0]).T).view(n, 8, 128), t["q_norm"][0], cos, sin, positions)
    k64 = expected_append(c, (x64 @ dense(t["wk"][0]).T).view(n, 2, 128), t["k_norm"][0], cos, sin, positions)
    ck = c.values("k", 0)
    # one step of a word is at most 1/127 of its row's largest value; half of it is the rounding
    assert ((ck - k64).abs() <= k64.abs().amax(-1, keepdim=True) * (0.5 / 127) * 1.01).all()
    out64, _, _ = attention64(c, q64, 128 ** -0.5)
    want = out64.reshape(n, 1024) @ dense(t["wo"][0]).T
    assert (o.double() - want).abs().max() <= 1e-4 * want.abs().max()  # the f32-activation mode's tolerance

    # into a dense model's caches, and one token further
    for name, out in (("k", t["k_cache"][0]), ("v", t["v_cache"][0])):
        q8.q8_kv_read(c.pages(), c.batch(), **{name + "_out": out.transpose(0, 1)[:n]})
    host = dict(recipes.decode_model(cfg, seed=1))
    host["k_cache"] = [t["k_cache"][0].cpu().numpy()]
    host["v_cache"] = [t["v_cache"][0].cpu().numpy()]
    om = oracle.ModelArrays(cfg, **host)
    tok, pos = (torch.full((1,), z, dtype=torch.int32, device="cuda") for z in (7, n))
    logits = torch.empty(cfg["vocab"], device="cuda")
    model = q8.Model(cfg, t, q8.F32ACT_F64SUM, tok, pos, logits)
    model.step()
    model.check()
    _, ref = oracle.decode_step(q8.F32ACT_F64SUM, om, 7, n)
    got = logits.cpu().numpy().astype(np.float64)
    assert np.max(np.abs(got - ref)) <= 1e-4 * np.max(np.abs(ref))
    model.close()
