"""The paged key/value cache on the GPU where one row's numbers meet another's.

Tolerances.  As in test_gpu_kv_pages.py, but every row's bound is formed from the positions which that row sees: a score is
off by at most delta = 2^-18 of its products' magnitudes; the output by (2 delta + 2^-17) sum p |v|, and by what a split
weight may lose, the smaller of the weight and 2^-28 times the largest value the row sees.  lse is off by delta, by the sum's
rounding (an exponential of 2^-22 and, at the lengths here, fewer than 2^5 additions of 2^-24: 2^-18 in all), and by the
scores' own rounding to f32 and that of the logarithm's result (2^-20 of the largest of them).
"""
import math

import pytest

from test_gpu_kv_pages import Cache, gen, quantize, rope, ws  # noqa: F401  (ws: a fixture)

pytestmark = pytest.mark.gpu


def attention_seen(c, q, scale):
    """Output, lse and both bounds in f64, each row's from the positions that it sees alone."""
    import torch
    rows, heads, hd = q.shape
    group = heads // c.kv
    out, lim = (torch.zeros(rows, heads, hd, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, off = (torch.zeros(rows, heads, dtype=torch.float64, device="cuda") for _ in range(2))
    r = 0
    for b, (n, L) in enumerate(zip(c.new, c.length)):
        for i in range(n if n else 0):
            k, v = (c.values(name, b)[:L - n + i + 1].transpose(0, 1) for name in "kv")  # [kv, seen, hd]
            x = q[r].double().unflatten(0, (c.kv, group))
            s = torch.einsum("kgd,ktd->kgt", x, k) * scale
            delta = torch.einsum("kgd,ktd->kgt", x.abs(), k.abs()).amax(-1, keepdim=True) * scale * 2 ** -18
            m = s.amax(-1, keepdim=True)
            e = (s - m).exp()
            total = e.sum(-1, keepdim=True)
            o = torch.einsum("kgt,ktd->kgd", e / total, v)
            near = torch.einsum("kgt,ktd->kgd", e / total, v.abs()) * (2 * delta + 2 ** -17)
            near = near + (e.clamp_max(2 ** -28).sum(-1, keepdim=True) / total) * v.abs().amax((1, 2))[:, None, None]
            out[r], lim[r] = o.flatten(0, 1), near.flatten(0, 1)
            lse[r] = (m + total.log()).flatten()
            off[r] = (delta + 2 ** -18 + 2 ** -20 * (s.abs().amax(-1, keepdim=True) + total.log().abs())).flatten()
            r += 1
    return out, lim, lse, off


def near(out, lse, ref, rows, heads):
    """Rows `rows` (an index) and heads `heads` of out and lse against the reference; the others are another check's."""
    o, lim, l, off = (t[rows][:, heads] for t in ref)
    d = (out[rows][:, heads].double() - o).abs()
    assert (d <= lim).all(), f"off by {d.nan_to_num(math.inf).max():.3e}, allowed up to {lim.max():.3e}"
    assert ((lse[rows][:, heads].double() - l).abs() <= off).all()


# A sequence of a few rows and one of many (the two kernels), and one of many beside places that hold none (which the first
# kernel takes): the bad position is one that the last rows see.
MASKED = [([3], [300], 299), ([4], [290], 288), ([140], [300], 270), ([257], [257], 130),
          ([40] + [0] * 39, [300] + [0] * 39, 281)]


@pytest.mark.parametrize("new,length,at", MASKED)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("size", [8.0, 1000.0, 2.0 ** -40])
@pytest.mark.parametrize("words", ["int8", "e4m3"])
def test_a_value_row_that_is_not_finite_stays_behind_the_mask(q8, ws, new, length, at, bad, size, words):  # noqa: F811
    """Rows before it are as if it were not there, whatever the size of the values that they see."""
    import torch
    c = Cache(q8, new, length, 2, 128, 16, words, 41)
    n, L = new[0], length[0]
    c.vs.copy_(c.vs * 0 + size * (1 + torch.rand(c.vs.shape, generator=gen(42), device="cuda")))
    q = torch.randn(n, 8, 128, generator=gen(43), device="cuda")
    ref = attention_seen(c, q, 128 ** -0.5)
    a, o = c.where(0, torch.tensor([at], device="cuda"))
    c.vs[a, 0, o] = bad
    out, lse = torch.empty_like(q), torch.empty(n, 8, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
    first = at - (L - n)  # the first row that sees it
    assert c.error.item() == 0
    near(out, lse, ref, slice(0, first), slice(0, 8))
    near(out, lse, ref, slice(first, n), slice(4, 8))  # (the other key/value head)
    assert not out[first:, :4].isfinite().any()


@pytest.mark.parametrize("new,length,at", MASKED)
@pytest.mark.parametrize("power", [20, 45, 90])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -20])
def test_a_large_value_row_costs_the_rows_before_it_no_bits(q8, ws, new, length, at, power, size):  # noqa: F811
    import torch
    c = Cache(q8, new, length, 2, 128, 16, "int8", 44)
    n, L = new[0], length[0]
    c.vs.mul_(size)
    a, o = c.where(0, torch.arange(at, L, device="cuda"))
    c.vs[a, :, o] = c.vs[a, :, o] * 2.0 ** power
    q = torch.randn(n, 8, 128, generator=gen(45), device="cuda")
    ref = attention_seen(c, q, 128 ** -0.5)
    out, lse = torch.empty_like(q), torch.empty(n, 8, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
    near(out, lse, ref, slice(0, n), slice(0, 8))


@pytest.mark.parametrize("new,length,keys", [
    ([1], [1], [0]), ([1], [17], [16]), ([1], [300], range(32, 48)), ([1], [4097], range(1024, 1040)),
    ([1], [4097], range(4097)), ([1] * 3, [900, 1, 33], range(900)), ([2], [130], [128]), ([140], [300], [160, 299]),
    ([140], [300], range(300))])
def test_lse_beside_keys_that_are_not_numbers(q8, ws, new, length, keys):  # noqa: F811
    """A row that sees such a key has no lse, whichever positions are looked at together; others keep theirs."""
    import torch
    c = Cache(q8, new, length, 2, 128, 16, "int8", 48)
    rows = sum(new)
    q = torch.randn(rows, 8, 128, generator=gen(49), device="cuda")
    ref = attention_seen(c, q, 128 ** -0.5)
    a, o = c.where(0, torch.tensor(list(keys), device="cuda"))
    c.ks[a, 1, o] = math.nan
    out, lse = torch.empty_like(q), torch.empty(rows, 8, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
    first = max(0, min(keys) - (length[0] - new[0]))
    assert out[first:new[0], 4:].isnan().all() and lse[first:new[0], 4:].isnan().all()
    near(out, lse, ref, slice(0, rows), slice(0, 4))
    near(out, lse, ref, slice(0, first), slice(4, 8))
    near(out, lse, ref, slice(new[0], rows), slice(4, 8))


@pytest.mark.parametrize("new,length", [([1], [1]), ([1], [5000]), ([3], [700]), ([140], [300])])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_lse_of_a_query_that_is_not_finite(q8, ws, new, length, bad):  # noqa: F811
    import torch
    c = Cache(q8, new, length, 2, 128, 16, "int8", 50)
    n = new[0]
    q = torch.randn(n, 8, 128, generator=gen(51), device="cuda")
    ref = attention_seen(c, q, 128 ** -0.5)
    q[n - 1, 3, 7] = bad
    out, lse = torch.empty_like(q), torch.empty(n, 8, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
    assert out[n - 1, 3].isnan().all() and lse[n - 1, 3].isnan()
    out[n - 1, 3], lse[n - 1, 3] = ref[0][n - 1, 3].float(), ref[2][n - 1, 3].float()
    near(out, lse, ref, slice(0, n), slice(0, 8))


def test_a_batch_without_rows_or_sequences(q8, ws):  # noqa: F811
    """Empty tensors, whose address is none, are a batch with nothing to do."""
    import torch
    c = Cache(q8, [1, 1], [5, 9], 2, 128, 16, "int8", 52)
    words = c.kw.clone()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    for rows, batch in ((0, c.batch()), (0, q8.kv_batch(none, none[:0], c.table[:0, :1], c.error)),
                        (2, q8.kv_batch(none, none[:0], c.table[:0, :0], c.error))):
        q, k = torch.ones(rows, 8, 128, device="cuda"), torch.ones(rows, 2, 128, device="cuda")
        out = torch.full_like(q, 7.5)
        q8.q8_kv_append(c.pages(), batch, q, k, k, out)
        q8.q8_kv_append(c.pages(), batch, None, k, k, None)
        q8.q8_kv_read(c.pages(), batch, k, torch.empty_like(k))
        q8.q8_kv_read(c.pages(), batch, None, k)
        q8.q8_paged_attention(c.pages(), batch, q, out, lse=torch.empty(rows, 8, device="cuda"), ws=ws)
        assert (out == 7.5).all() and (k == 1).all()
    assert torch.equal(c.kw, words) and c.error.item() == 0


def test_the_largest_scales(q8, ws):  # noqa: F811
    """Value scales up to the largest that the pages can hold."""
    import torch
    for new, length in (([2], [40]), ([60], [200])):
        c = Cache(q8, new, length, 2, 128, 16, "int8", 46)
        c.vs.copy_(c.vs * 0 + 2.6e36)  # words of up to 127: values up to 3.3e38
        q = torch.randn(new[0], 8, 128, generator=gen(47), device="cuda")
        ref = attention_seen(c, q, 128 ** -0.5)
        out, lse = torch.empty_like(q), torch.empty(new[0], 8, device="cuda")
        q8.q8_paged_attention(c.pages(), c.batch(), q, out, lse=lse, ws=ws)
        near(out, lse, ref, slice(0, new[0]), slice(0, 8))


@pytest.mark.parametrize("new,length,heads,kv,hd,words", [
    ([1], [1], 8, 2, 128, "int8"), ([1], [5000], 32, 1, 64, "e4m3"), ([1] * 40, [300 + 41 * i for i in range(40)], 32, 4, 128, "int8"),
    ([1, 1], [900, 70], 12, 1, 128, "e4m3"), ([140], [300], 8, 2, 64, "int8"), ([2000], [4000], 32, 4, 128, "e4m3"),
    ([1, 90, 3, 1], [400, 900, 77, 3000], 8, 2, 128, "int8")])
@pytest.mark.parametrize("polls", [1, 64])
def test_waits_that_give_up(q8, new, length, heads, kv, hd, words, polls):
    """Copies that never complete, as far as their barriers know: the launches end, write nothing and say so; the workspace
    takes no further call until it has been checked, and works as before then."""
    import torch
    c = Cache(q8, new, length, kv, hd, 16, words, 59)
    w, q = q8.Workspace(), torch.randn(sum(new), heads, hd, generator=gen(60), device="cuda")
    want, out = torch.empty_like(q), torch.full_like(q, 7.5)
    q8.q8_paged_attention(c.pages(), c.batch(), q, want, ws=w)
    w.check()
    q8.q8_paged_wait_selftest(c.pages(), c.batch(), q, out, polls, w)
    torch.cuda.synchronize()
    assert (out == 7.5).all() and c.error.item() == q8.KV_ERR_WAIT
    c.error.zero_()
    q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=w)
    assert (out == 7.5).all() and c.error.item() == q8.KV_ERR_WAIT
    q8.q8_paged_attention(c.pages(), q8.kv_batch(c.row_start, c.kv_len, c.table), q, out, ws=w)  # (no error word)
    assert (out == 7.5).all()
    with pytest.raises(q8.Q8Error, match="Q8_ETIMEOUT"):
        w.check()
    w.check()  # cleared
    c.error.zero_()
    for _ in range(3):
        q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=w)
        assert torch.equal(out, want) and c.error.item() == 0
    w.check()
    w.close()


@pytest.mark.parametrize("starts,lens", [([0, 9, 20], [9, 30]), ([0, 9, 9, 30], [9, 0, 30]), ([0, 9, 12], [9, 30]),
                                         ([-3, 0, 9], [9, 30]), ([0, 9] + [9] * 300 + [20], [9] + [5] * 300 + [30])])
def test_a_sequence_with_no_row_of_the_call_is_recorded(q8, ws, starts, lens):  # noqa: F811
    """Its rows are skipped by every call, and the error word says so, although no row of the call leads to it."""
    import torch
    rows, seqs = 9, len(lens)
    c = Cache(q8, [0] * seqs, lens, 2, 128, 16, "int8", 53)
    c.row_start.copy_(torch.tensor(starts, dtype=torch.int32))
    k = torch.randn(rows, 2, 128, generator=gen(54), device="cuda")
    q = torch.randn(rows, 8, 128, generator=gen(55), device="cuda")
    back, out = torch.empty_like(k), torch.empty_like(q)
    for call in (lambda: q8.q8_kv_append(c.pages(), c.batch(), q, k, k, out), lambda: q8.q8_kv_read(c.pages(), c.batch(), back),
                 lambda: q8.q8_paged_attention(c.pages(), c.batch(), q, out, ws=ws)):
        c.error.zero_()
        call()
        assert c.error.item() == q8.KV_ERR_LENGTH


def test_pages_and_batches_keep_their_tensors(q8):
    """The structs hold addresses: the tensors behind them live as long as they do."""
    import gc
    import weakref
    c = Cache(q8, [1], [5], 1, 64, 16, "int8", 56)
    made = [t.clone() for t in (c.kw, c.ks, c.vw, c.vs, c.row_start, c.kv_len, c.table, c.error)]
    refs = [weakref.ref(t) for t in made]
    pages, batch = q8.kv_pages(*made[:4]), q8.kv_batch(*made[4:])
    del made
    gc.collect()
    assert all(r() is not None for r in refs)
    del pages, batch
    gc.collect()
    assert all(r() is None for r in refs)


def test_append_into_columns_of_one_buffer(q8):
    """The queries' places among what is read: q itself, and columns beside q, k and v in one buffer."""
    import torch
    c = Cache(q8, [3, 2], [20, 2], 2, 128, 16, "int8", 61, fill=False)
    cos, sin = rope(q8, 32, 128)
    wide = torch.randn(5, 12 + 8, 128, generator=gen(62), device="cuda")
    want = torch.empty(5, 8, 128, device="cuda")
    q, k, v, beside = wide[:, :8], wide[:, 8:10], wide[:, 10:12], wide[:, 12:]
    q8.q8_kv_append(c.pages(), c.batch(), q, k, v, want, cos=cos, sin=sin)
    q8.q8_kv_append(c.pages(), c.batch(), q, k, v, beside, cos=cos, sin=sin)
    assert torch.equal(beside, want)
    q8.q8_kv_append(c.pages(), c.batch(), q, k, v, q, cos=cos, sin=sin)
    assert torch.equal(q, want)
    for bad in (wide[:, 4:12], wide[:, 9:17], wide[:, 3:11]):
        with pytest.raises(q8.Q8Error, match="q_out: overlaps"):
            q8.q8_kv_append(c.pages(), c.batch(), q, k, v, bad, cos=cos, sin=sin)


@pytest.mark.parametrize("kv,hd", [(1, 64), (3, 64), (2, 128)])
def test_read_into_layouts_of_one_buffer(q8, kv, hd):
    """Keys and values side by side in one buffer, in several orders, and layouts that overlap."""
    import torch
    n = 21
    c = Cache(q8, [n], [40], kv, hd, 16, "int8", 63)
    k, v = (torch.empty(n, kv, hd, device="cuda") for _ in range(2))
    q8.q8_kv_read(c.pages(), c.batch(), k, v)
    for shape, at in (((n, 2, kv, hd), lambda t, i: t[:, i]), ((2, n, kv, hd), lambda t, i: t[i]),
                      ((kv, 2, n + 3, hd), lambda t, i: t[:, i, :n].transpose(0, 1)),
                      ((kv, n, 2, hd), lambda t, i: t[:, :, i].transpose(0, 1)),
                      ((n, kv, 2 * hd + 8), lambda t, i: t[:, :, i * hd:(i + 1) * hd]),
                      ((2, kv, n + 5, hd + 8), lambda t, i: t[i, :, 5:, 8:].transpose(0, 1))):
        t = torch.full(shape, 7.5, device="cuda")
        kept = torch.ones(shape, dtype=torch.bool, device="cuda")
        at(kept, 0)[:] = False
        at(kept, 1)[:] = False
        q8.q8_kv_read(c.pages(), c.batch(), at(t, 0), at(t, 1))
        assert torch.equal(at(t, 0), k) and torch.equal(at(t, 1), v) and (t[kept] == 7.5).all()
    t = torch.zeros(4 * n * kv * hd, device="cuda")
    with pytest.raises(q8.Q8Error, match="overlap"):
        q8.q8_kv_read(c.pages(), c.batch(), k, k)
    with pytest.raises(q8.Q8Error, match="overlap"):
        q8.q8_kv_read(c.pages(), c.batch(), t[:n * kv * hd].view(n, kv, hd), t[hd - 8:n * kv * hd + hd - 8].view(n, kv, hd))
    if kv > 1:
        with pytest.raises(q8.Q8Error, match="overlap"):  # heads within one another's rows
            q8.q8_kv_read(c.pages(), c.batch(), t.as_strided((n, kv, hd), (hd, hd, 1)))


def test_a_workspace_of_another_device_is_refused(q8):
    import torch
    c = Cache(q8, [1], [5], 1, 64, 16, "int8", 64)
    q = torch.ones(1, 1, 64, device="cuda")
    w = q8.Workspace()
    assert w.device == torch.cuda.current_device()
    w.device += 1
    for call in (lambda: q8.q8_paged_attention(c.pages(), c.batch(), q, torch.empty_like(q), ws=w),
                 lambda: q8.q8_paged_wait_selftest(c.pages(), c.batch(), q, torch.empty_like(q), 64, w)):
        with pytest.raises(q8.Q8Error, match="ws: not on the current device"):
            call()
    w.close()
    with pytest.raises(q8.Q8Error, match="ws: null"):
        q8.q8_paged_attention(c.pages(), c.batch(), q, torch.empty_like(q))
    with pytest.raises(q8.Q8Error, match="ws: null"):  # closed
        w.device -= 1
        q8.q8_paged_attention(c.pages(), c.batch(), q, torch.empty_like(q), ws=w)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("words", ["int8", "e4m3"])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_rows_at_the_ends_of_the_norms_range(q8, hd, words, eps):
    """Rows whose squares add up to little less than f32's largest number, and, without eps, to 2^-72."""
    import torch
    n = 4
    c = Cache(q8, [n], [n], 2, hd, 16, words, 57, fill=False)
    g = gen(58)
    size = torch.tensor([1.0, 1e12, 1e18, 1e-3 if eps else 1e-12], device="cuda")[:, None, None]
    q, k = (torch.randn(n, h, hd, generator=g, device="cuda") * size for h in (4, 2))
    w = 1 + 0.1 * torch.randn(hd, generator=g, device="cuda")
    cos, sin = rope(q8, n, hd)
    out = torch.empty_like(q)
    q8.q8_kv_append(c.pages(), c.batch(), q, k, torch.ones_like(k), out, q_norm=w, k_norm=w, eps=eps, cos=cos, sin=sin)

    eps32 = torch.tensor(eps, dtype=torch.float32).item()  # (what the call takes: 2.5e-9 from 1e-6, which turns last bits of f32)

    def turned(x):
        x = x.double()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps32) * w.double()
        a, b = x.chunk(2, -1)
        cs, sn = cos.double()[:, None], sin.double()[:, None]
        return torch.cat((a * cs - b * sn, a * sn + b * cs), -1)

    z = turned(q)
    lim = z.abs() + z.roll(hd // 2, -1).abs()
    assert ((out.double() - z).abs() <= 20 * 2 ** -24 * lim).all()
    qx, d = quantize(turned(k).float(), words)
    a, o = c.where(0, torch.arange(n, device="cuda"))
    assert torch.equal(c.ks[a, :, o], d)
    assert torch.equal(c.kw.view(torch.int8)[a, :, o].view(c.kw.dtype).float(), qx.float())


def test_binding_refuses_tensors_of_other_dimensions(q8, ws):  # noqa: F811
    """With a Q8Error that names the tensor, whatever its number of dimensions."""
    import torch
    c = Cache(q8, [2], [5], 2, 64, 16, "int8", 65)
    p, b, x = c.pages(), c.batch(), torch.ones(2, 2, 64, device="cuda")
    o, t = torch.empty_like(x), torch.ones(8, 32, device="cuda")
    for bad in (x.view(-1), x.view(2, 128), x[0, 0, 0], x.view(1, 2, 2, 64), x.view(2, 4, 32), x[:, :, ::2], x.double(),
                x.cpu(), x[:1].expand(2, 2, 64)):
        for call, name in ((lambda: q8.q8_kv_append(p, b, bad, x, x, o), "q"), (lambda: q8.q8_kv_append(p, b, x, bad, x, o), "k"),
                           (lambda: q8.q8_kv_append(p, b, x, x, bad, o), "v"), (lambda: q8.q8_kv_append(p, b, x, x, x, bad), "q_out"),
                           (lambda: q8.q8_paged_attention(p, b, bad, o, ws=ws), "q"),
                           (lambda: q8.q8_paged_attention(p, b, x, bad, ws=ws), "out"),
                           (lambda: q8.q8_paged_wait_selftest(p, b, x, bad, 64, ws), "out"),
                           (lambda: q8.q8_kv_read(p, b, bad), "k_out")):
            with pytest.raises(q8.Q8Error, match=rf"\b{name}\b"):
                call()
    for bad in (t.view(-1), t[0, 0], t.view(8, 1, 32), t[:, :16]):
        with pytest.raises(q8.Q8Error):
            q8.q8_kv_append(p, b, x, x, x, o, cos=bad, sin=t)
        with pytest.raises(q8.Q8Error):
            q8.q8_rope_table(1e6, bad, t)
    with pytest.raises(q8.Q8Error):
        q8.q8_kv_append(p, b, x, x, x, o, cos=t, sin=None)
    for rows in (1, 3):
        with pytest.raises(q8.Q8Error, match="rows differ"):
            q8.q8_paged_wait_selftest(p, b, x, torch.empty(rows, 2, 64, device="cuda"), 64, ws)
    assert c.error.item() == 0


@pytest.mark.parametrize("new,length", [([1, 1], [400, 70]), ([60, 1], [200, 33])])
def test_attention_into_columns_beside_the_queries(q8, ws, new, length):  # noqa: F811
    import torch
    c = Cache(q8, new, length, 2, 128, 16, "int8", 66)
    wide = torch.randn(sum(new), 20, 128, generator=gen(67), device="cuda")
    q, want = wide[:, 4:12], torch.empty(sum(new), 8, 128, device="cuda")
    q8.q8_paged_attention(c.pages(), c.batch(), q, want, ws=ws)
    kept = wide.clone()
    q8.q8_paged_attention(c.pages(), c.batch(), q, wide[:, 12:], ws=ws)
    assert torch.equal(wide[:, 12:], want) and torch.equal(wide[:, :12], kept[:, :12])
    for bad in (wide[:, 5:13], wide[:, 11:19], q):
        with pytest.raises(q8.Q8Error, match="out"):
            q8.q8_paged_attention(c.pages(), c.batch(), q, bad, ws=ws)
