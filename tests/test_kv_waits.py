"""Host-side refusals of the calls about bounded waits (no GPU: the addresses are never used)."""
import ctypes

from test_kv_refusals import A, P, batch, pages, q8  # noqa: F401  (q8: a fixture)


def test_workspace_check_needs_a_workspace(q8):  # noqa: F811
    assert q8.lib.q8_workspace_check(None, None) == -1 and "ws: null" in q8.last_error()


def test_wait_selftest(q8):  # noqa: F811
    def call(polls, heads=4, ws=A, rows=3, out=2 * A):
        return q8.lib.q8_paged_wait_selftest(ctypes.byref(pages(q8)), ctypes.byref(batch(q8)), rows, heads, P(A), 512, 0.1,
                                             P(out), 512, P(ws), polls, None)
    for polls in (0, 4097, 2 ** 32 - 1):
        assert call(polls) == -1 and "polls" in q8.last_error()
    assert call(64, heads=5) == -1 and "heads 5" in q8.last_error()
    assert call(64, ws=None) == -1 and "ws: null" in q8.last_error()
    assert call(64, out=A) == -1 and "q itself" in q8.last_error()
    assert call(64, rows=0) == 0
