"""Host-side refusals of overlapping buffers in the paged key/value cache's calls (no GPU: the addresses are never used, for
every call is refused or has no sequences; layouts that are taken run on real tensors in test_gpu_kv_edges.py)."""
import pytest

from test_kv_empty import NONE
from test_kv_refusals import A, append, attend, batch, pages, q8, read  # noqa: F401  (q8: a fixture)

B = 1 << 20  # far from A


def ok(call, q8, **change):  # noqa: F811
    return call(q8, bt=batch(q8, **NONE), **change) == 0


@pytest.mark.parametrize("change", [
    dict(out=A + 16), dict(out=A + 512 * 4 - 16), dict(out=A + 512 * 4), dict(q=2 * A + 64, out=2 * A), dict(qs=1024, os=1024, out=A + 511 * 4 + 4 - 16),
    dict(qs=1024, os=1024, out=A + 516 * 4), dict(qs=1024, os=1024, out=A + 1024 * 4), dict(qs=1024, os=512, out=A + 2048),
    dict(qs=1024, os=1024, rows=2, out=A + 1023 * 4 + 4 - 16), dict(rows=1, out=A + 511 * 4 + 4 - 16)])
def test_attention_out_over_q(q8, change):  # noqa: F811
    assert attend(q8, bt=batch(q8, **NONE), **change) == -1
    assert "out: overlaps q" in q8.last_error()


@pytest.mark.parametrize("change", [
    dict(out=A + 3 * 512 * 4), dict(q=A + 3 * 512 * 4, out=A), dict(qs=1024, os=1024, out=A + 512 * 4),
    dict(qs=1024, os=1024, q=A + 512 * 4, out=A), dict(qs=1040, os=1040, out=A + 520 * 4), dict(rows=1, out=A + 512 * 4),
    dict(rows=1, qs=0, os=4, out=A + 512 * 4), dict(qs=2048, os=1024, out=B)])
def test_attention_out_beside_q(q8, change):  # noqa: F811
    assert ok(attend, q8, **change)


# one merged projection of rows 1024 values apart: 4 query heads, 2 key and 2 value heads of 128
MERGED = dict(qs=1024, ks=1024, vs=1024, q=A, k=A + 512 * 4, v=A + 768 * 4)


@pytest.mark.parametrize("change,name", [
    (dict(out=A, os=1024), "q"), (dict(out=A + 16), "q"), (dict(qs=520, out=A), "q"), (dict(k=B, out=B), "k"),
    (dict(v=B, out=B + 1024), "v"), (dict(MERGED, out=A + 256 * 4, os=1024), "q"), (dict(MERGED, out=A + 512 * 4, os=1024), "k"),
    (dict(MERGED, k=B, out=A + 512 * 4, os=1024), "v"), (dict(MERGED, out=A, os=512), "q"), (dict(rows=1, out=A + 16), "q")])
def test_append_q_out_over_its_inputs(q8, change, name):  # noqa: F811
    change = dict(dict(q=A, k=4 * B, v=5 * B, out=6 * B), **change)
    assert append(q8, **change) == -1
    assert f"q_out: overlaps {name}" in q8.last_error()


def meet(at, rows, rs, heads, hs, hd):
    """Whether two of the vectors of hd values at r rs + h hs, and (with `at` given) those `at` values on, share a value."""
    a = sorted(r * rs + h * hs for r in range(rows) for h in range(heads))
    if at is None:
        return any(y - x < hd for x, y in zip(a, a[1:]))
    return any(abs(x - y - at) < hd for x in a for y in a)


@pytest.mark.parametrize("hd,kv", [(64, 1), (64, 3), (128, 2), (128, 5)])
def test_read_outputs(q8, hd, kv):  # noqa: F811
    """A layout of rows and heads whose vectors share a value is refused, and no other; so is a v_out over k_out."""
    pg = pages(q8, head_dim=hd, kv_heads=kv)
    for rows in (1, 2, 5):
        for rs in {hd, hd + 8, 2 * hd, 3 * hd, kv * hd, kv * hd + 8, 2 * kv * hd}:
            for hs in {hd, hd + 8, 2 * hd, 3 * hd + 16, rows * hd, rows * hd + 8, rows * rs, 2 * rows * hd}:
                bad = meet(None, rows, rs, kv, hs, hd)
                assert read(q8, pg=pg, bt=batch(q8, **NONE), rows=rows, k=B, v=None, rs=rs, hs=hs) == (-1 if bad else 0)
                if bad:
                    assert "overlap" in q8.last_error()
                    continue
                for at in {0, 8, hd - 8, hd, hd + 8, 2 * hd, kv * hd, rows * hd, rows * rs, rows * rs + kv * hs}:
                    for sign in (1, -1):  # (the other layouts go on to a launch: taken on real tensors, on a GPU)
                        if meet(sign * at, rows, rs, kv, hs, hd):
                            assert read(q8, pg=pg, rows=rows, k=B, v=B + 4 * sign * at, rs=rs, hs=hs) == -1
                            assert "overlap" in q8.last_error()
