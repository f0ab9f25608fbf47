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
