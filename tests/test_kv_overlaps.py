"""Host-side refusals of overlapping buffers in the paged key/value cache's calls (no GPU: the addresses are never used; a
call that would go on to a launch has no sequences)."""
import pytest

from test_kv_empty import NONE
from test_kv_refusals import A, append, attend, batch, q8, read  # noqa: F401  (q8: a fixture)

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
