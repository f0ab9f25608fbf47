"""Calls of the paged key/value cache with nothing to do (no GPU: nothing is launched).  An empty tensor's address is null, so
null is no mistake where there are no values; everything else is checked as ever."""
import pytest

from test_kv_refusals import append, attend, batch, pages, q8, read  # noqa: F401  (q8: a fixture)

NONE = dict(row_start=None, kv_len=None, table=None, seqs=0)


def test_no_rows(q8):  # noqa: F811
    assert append(q8, rows=0, q=None, k=None, v=None, out=None) == 0
    assert append(q8, rows=0, heads=0, q=None, k=None, v=None, out=None) == 0
    assert read(q8, rows=0, k=None, v=None) == 0 and read(q8, rows=0, k=None) == 0
    assert attend(q8, rows=0, q=None, out=None) == 0


@pytest.mark.parametrize("table", [dict(), dict(table_pages=0, table_stride=0)])
def test_no_sequences(q8, table):  # noqa: F811
    for rows in (0, 3):
        assert append(q8, bt=batch(q8, **NONE, **table), rows=rows) == 0
        assert read(q8, bt=batch(q8, **NONE, **table), rows=rows) == 0
        assert attend(q8, bt=batch(q8, **NONE, **table), rows=rows) == 0


def test_the_other_arguments_are_still_checked(q8):  # noqa: F811
    for call in (append, read, attend):
        assert call(q8, rows=0, bt=batch(q8, kv_len=None)) == -1 and "kv_len" in q8.last_error()
        assert call(q8, rows=0, bt=batch(q8, table_pages=0, table_stride=0)) == -1 and "0 pages" in q8.last_error()
        assert call(q8, rows=0, pg=pages(q8, k=None)) == -1 and "null words" in q8.last_error()
        assert call(q8, bt=batch(q8, **{**NONE, "seqs": -1})) == -1
    assert append(q8, bt=batch(q8, **NONE), k=None) == -1 and "k: null" in q8.last_error()
    assert read(q8, bt=batch(q8, **NONE), k=None, v=None) == -1 and "both null" in q8.last_error()
    assert attend(q8, bt=batch(q8, **NONE), out=None) == -1 and "out: null" in q8.last_error()
