"""Host-side refusals of the paged key/value cache's calls: every bad argument is named before anything is launched (no
GPU: the addresses are never used)."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def q8():
    import __graft_entry__
    __graft_entry__.build()
    import moe_add_rmsnorm_gb300 as m
    return m


def pages(q8, **other):
    f = dict(k=4096, v=4096, ks=4096, vs=4096, pages=10, page_size=16, kv_heads=2, head_dim=128, words=0)
    return q8.q8_kv_pages(**{**f, **other})


def batch(q8, **other):
    f = dict(row_start=4096, kv_len=4096, table=4096, seqs=3, table_pages=4, table_stride=4, error=None)
    return q8.q8_kv_batch(**{**f, **other})


A = 8192  # an aligned address


def append(q8, pg=None, bt=None, rows=3, heads=4, q=A, qs=512, k=A, ks=256, v=A, vs=256, qn=None, kn=None, eps=1e-6, cos=None,
           sin=None, n=0, out=A, os=512):
    return q8.lib.q8_kv_append(ctypes.byref(pg or pages(q8)), ctypes.byref(bt or batch(q8)), rows, heads, P(q), qs, P(k), ks,
                               P(v), vs, P(qn), P(kn), eps, P(cos), P(sin), n, P(out), os, None)


def read(q8, pg=None, bt=None, rows=3, k=A, v=A, rs=256, hs=128):
    return q8.lib.q8_kv_read(ctypes.byref(pg or pages(q8)), ctypes.byref(bt or batch(q8)), rows, P(k), P(v), rs, hs, None)


def attend(q8, pg=None, bt=None, rows=3, heads=4, q=A, qs=512, scale=0.1, out=2 * A, os=512, lse=None, ws=A):
    return q8.lib.q8_paged_attention(ctypes.byref(pg or pages(q8)), ctypes.byref(bt or batch(q8)), rows, heads, P(q), qs,
                                     scale, P(out), os, P(lse), P(ws), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(k=None), -1, "null words"), (dict(vs=None), -1, "null words"), (dict(words=2), -1, "words 2"),
    (dict(pages=0), -1, "0 pages"), (dict(kv_heads=0), -1, "0 heads"), (dict(kv_heads=1025), -2, "1025 heads"),
    (dict(head_dim=96), -2, "head_dim 96"), (dict(head_dim=256), -2, "head_dim 256"), (dict(page_size=8), -2, "page_size 8"),
    (dict(page_size=48), -2, "page_size 48"), (dict(page_size=2048), -2, "page_size 2048"),
    (dict(v=4096 + 16), -1, "32-byte"), (dict(ks=4096 + 4), -1, "16-byte")])
def test_pages(q8, change, code, word):
    for call in (append, read, attend):
        assert call(q8, pg=pages(q8, **change)) == code
        assert word in q8.last_error()


@pytest.mark.parametrize("change,code,word", [
    (dict(row_start=None), -1, "null row_start"), (dict(table=None), -1, "table"), (dict(seqs=-1), -1, "negative"),
    (dict(seqs=65537), -2, "65537"), (dict(table_pages=0), -1, "0 pages"), (dict(table_stride=3), -1, "3 apart"),
    (dict(table_pages=1 << 27, table_stride=1 << 27), -2, "2^30"), (dict(kv_len=4098), -1, "4-byte"),
    (dict(error=4097), -1, "4-byte")])
def test_batch(q8, change, code, word):
    for call in (append, read, attend):
        assert call(q8, bt=batch(q8, **change)) == code
        assert word in q8.last_error()


@pytest.mark.parametrize("change,code,word", [
    (dict(rows=-1), -1, "negative"), (dict(rows=(1 << 24) + 1), -2, "rows"), (dict(q=None), -1, "q: null"),
    (dict(out=None), -1, "q_out: null"), (dict(k=None), -1, "k: null"), (dict(v=A + 4), -1, "v: address"),
    (dict(ks=254), -1, "k: address or stride"), (dict(ks=252), -1, "252 apart"), (dict(qs=508), -1, "508 apart"),
    (dict(os=510), -1, "q_out"), (dict(eps=-1.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"),
    (dict(cos=A, n=9), -1, "one without"), (dict(cos=A, sin=A), -1, "rope_positions 0"),
    (dict(cos=A + 4, sin=A, n=9), -1, "16-byte"), (dict(heads=0), -1, "without heads"), (dict(heads=-1), -1, "heads"),
    (dict(qn=4097), -1, "q_norm")])
def test_append(q8, change, code, word):
    assert append(q8, **change) == code
    assert word in q8.last_error()


@pytest.mark.parametrize("change,code,word", [
    (dict(k=None, v=None), -1, "both null"), (dict(k=A + 16), -1, "32-byte"), (dict(rs=260), -1, "32-byte"),
    (dict(rs=64), -1, "rows 64"), (dict(hs=64), -1, "heads 64"), (dict(hs=1 << 37), -2, "2^36")])
def test_read(q8, change, code, word):
    assert read(q8, **change) == code
    assert word in q8.last_error()


@pytest.mark.parametrize("change,code,word", [
    (dict(heads=0), -1, "heads 0"), (dict(heads=5), -1, "heads 5"), (dict(heads=130), -2, "heads 130"),
    (dict(q=None), -1, "q: null"), (dict(out=None), -1, "out: null"), (dict(out=A), -1, "q itself"),
    (dict(qs=510), -1, "q: address or stride"), (dict(os=256), -1, "256 apart"), (dict(scale=0.0), -1, "scale"),
    (dict(scale=float("nan")), -1, "scale"), (dict(scale=float("inf")), -1, "scale"), (dict(lse=4098), -1, "lse"),
    (dict(ws=None), -1, "ws: null")])
def test_attention(q8, change, code, word):
    assert attend(q8, **change) == code
    assert word in q8.last_error()


def test_rope_table(q8):
    f = q8.lib.q8_rope_table
    assert f(1e6, 4, 128, None, P(A), None) == -1 and "cos" in q8.last_error()
    assert f(0.0, 4, 128, P(A), P(A), None) == -1 and "theta" in q8.last_error()
    assert f(1e6, 4, 127, P(A), P(A), None) == -1 and "head_dim 127" in q8.last_error()
    assert f(1e6, 1 << 31, 128, P(A), P(A), None) == -2
    assert f(1e6, 0, 128, P(A), P(A), None) == 0


def test_nothing_to_do_is_no_error(q8):
    for call in (append, read, attend):
        assert call(q8, rows=0) == 0
        assert call(q8, bt=batch(q8, seqs=0)) == 0


def test_binding_refuses_wrong_tensors(q8):
    import torch
    w, s = torch.zeros(4, 2, 16, 128, dtype=torch.int8), torch.zeros(4, 2, 16)
    for bad in ((w.float(), s, w, s), (w, s, w[:2], s), (w, s.double(), w, s), (w, s, w, s)):  # the last: not on a GPU
        with pytest.raises(q8.Q8Error):
            q8.kv_pages(*bad)
    i = torch.zeros(3, dtype=torch.int32)
    for bad in ((i, i, i[:, None]), (torch.zeros(4, dtype=torch.int64), i, i[:, None]),
                (torch.zeros(4, dtype=torch.int32), i, i[:, None])):
        with pytest.raises(q8.Q8Error):
            q8.kv_batch(*bad)
