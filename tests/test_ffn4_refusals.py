"""Host-side refusals of the feed-forward block with 4-bit weights: every bad argument is named before anything is launched
(no GPU: the addresses are never used), and calls without rows do nothing."""
import ctypes

import pytest

P = ctypes.c_void_p
A = 1 << 20  # an aligned address; others lie at multiples of it, further apart than any call reaches


@pytest.fixture(scope="module")
def q8():
    import __graft_entry__
    __graft_entry__.build()
    import moe_add_rmsnorm_gb300 as m
    return m


def norm(q8, a=A, b=2 * A, wpost=3 * A, wpre=4 * A, gate=None, gr=0, gc=0, scale=1.0, rows=2, d=64, eps=1e-6, sum=5 * A,
         y=6 * A, q=7 * A, s=8 * A, lo=None, yq=True):
    act = ctypes.byref(q8.q8_act(q, s, lo)) if yq else None
    return q8.lib.postnorm_add_rmsnorm_q8(P(a), P(b), P(wpost), P(wpre), P(gate), gr, gc, scale, rows, d, eps, P(sum), P(y),
                                          act, None)


@pytest.mark.parametrize("change,code,word", [
    (dict(rows=-1), -1, "rows -1"), (dict(d=0), -1, "d 0"), (dict(d=16385), -2, "16384"), (dict(d=48), -2, "32-value"),
    (dict(eps=-1.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"), (dict(a=None), -1, "a: null"),
    (dict(b=None), -1, "b: null"), (dict(wpre=None), -1, "w_pre: null"), (dict(sum=None, y=None, yq=False), -1, "no output"),
    (dict(gr=-1), -1, "negative stride"), (dict(a=A + 2), -1, "a: not 4-byte"), (dict(q=7 * A + 16), -1, "32-byte"),
    (dict(lo=7 * A + 16), -1, "32-byte"), (dict(s=None), -1, "null words or scales"), (dict(s=8 * A + 1), -1, "4-byte"),
    (dict(sum=A + 4), -1, "sum_out: overlaps a"), (dict(y=2 * A + 64), -1, "y_out: overlaps b"),
    (dict(y=3 * A), -1, "y_out: overlaps w_post"), (dict(sum=4 * A), -1, "sum_out: overlaps w_pre"),
    (dict(y=5 * A), -1, "y_out: overlaps sum_out"), (dict(q=A), -1, "yq: overlaps a"),
    (dict(s=7 * A + 64), -1, "scales: overlaps yq"), (dict(lo=7 * A + 96), -1, "low words: overlaps yq"),
    (dict(gate=5 * A + 128, gc=1), -1, "sum_out: overlaps gate"), (dict(rows=1 << 31), -2, "rows")])
def test_norm(q8, change, code, word):
    assert norm(q8, **change) == code
    assert word in q8.last_error()


PLAN = (9 * A, 10 * A, 11 * A, 12 * A)


def route(q8, logits=A, stride=64, rows=3, experts=64, rule=True, k=4, ids=2 * A, gates=3 * A, plan=None, ws=A, **other):
    f = dict(score=0, bias=None, groups=4, keep_groups=2, group_top=2, renorm=1, scale=1.0)
    r = ctypes.byref(q8.q8_route_rule(**{**f, **other})) if rule else None
    pl = ctypes.byref(q8.q8_moe_plan(*plan)) if plan else None
    return q8.lib.moe_route_scored(P(logits), stride, rows, experts, r, k, P(ids), P(gates), pl, P(ws), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(rows=-1), -1, "rows -1"), (dict(experts=0), -1, "experts 0"), (dict(experts=1028), -2, "at most 1024"),
    (dict(rule=False), -1, "rule: null"), (dict(score=2), -1, "score 2"), (dict(groups=0), -2, "0 groups"),
    (dict(groups=33), -2, "33 groups"), (dict(groups=5), -1, "64 experts in 5 groups"), (dict(keep_groups=0), -1, "keep_groups 0"),
    (dict(keep_groups=5), -1, "keep_groups 5"), (dict(group_top=3), -1, "group_top 3"), (dict(renorm=2), -1, "renorm 2"),
    (dict(scale=float("inf")), -1, "scale"), (dict(k=0), -2, "k 0"), (dict(k=33), -2, "k 33"),
    (dict(keep_groups=1, k=17), -1, "k 17 above the 16"), (dict(rows=1 << 23), -2, "2^24"), (dict(logits=None), -1, "null"),
    (dict(ids=None), -1, "null"), (dict(gates=3 * A + 2), -1, "4-byte"), (dict(bias=A + 1), -1, "4-byte"),
    (dict(stride=63), -1, "63 apart"), (dict(plan=(A, A, A, None)), -1, "plan: null"),
    (dict(plan=(A, A, A, A + 2)), -1, "plan: not 4-byte"), (dict(plan=PLAN, ws=None), -1, "ws: null"),
    (dict(ids=A + 128), -1, "ids or gates: overlaps"), (dict(gates=2 * A + 16), -1, "ids or gates: overlaps"),
    (dict(bias=3 * A + 8), -1, "ids or gates: overlaps"), (dict(plan=(A, *PLAN[1:])), -1, "plan: overlaps"),
    (dict(plan=(*PLAN[:3], 9 * A + 4)), -1, "plan: overlaps"), (dict(plan=(*PLAN[:2], 2 * A, PLAN[3])), -1, "plan: overlaps")])
def test_route(q8, change, code, word):
    assert route(q8, **change) == code
    assert word in q8.last_error()


def mat(q8, **other):
    f = dict(q=16 * A, s=32 * A, z=None, rows=64, cols=128, group=64, scale_type=0)
    return ctypes.byref(q8.q4_matrix(**{**f, **other}))


def act(q8, q, s, lo=None):
    return ctypes.byref(q8.q8_act(q, s, lo))


def gemv(q8, W=None, x=A, xs=128, xq=None, rows=3, y=2 * A, ys=64, ws=A):
    return q8.lib.q4_gemv(W or mat(q8), P(x), xs, xq, rows, P(y), ys, P(ws), None)


def gate_up(q8, W=None, U=None, dff=16, x=A, xq=None, rows=3, k=2, ids=3 * A, plan=(A, A, A, A), h=4 * A, ws=A):
    pl = ctypes.byref(q8.q8_moe_plan(*plan)) if plan else None
    return q8.lib.moe_gate_up_q4(W or mat(q8), U or mat(q8), dff, P(x), xq, rows, k, P(ids), pl, P(h), P(ws), None)


def down(q8, W=None, d=16, h=A, hq=None, rows=3, k=2, ids=3 * A, gates=4 * A, plan=(A, A, A, A), residual=5 * A, y=6 * A, ws=A):
    pl = ctypes.byref(q8.q8_moe_plan(*plan)) if plan else None
    return q8.lib.moe_down_combine_q4(W or mat(q8), d, P(h), hq, rows, k, P(ids), P(gates), pl, P(residual), P(y), P(ws), None)


@pytest.mark.parametrize("change,code,word", [
    (dict(q=None), -1, "null words"), (dict(s=None), -1, "null words"), (dict(rows=0), -1, "0 x 128"),
    (dict(cols=0), -1, "64 x 0"), (dict(group=48), -2, "group 48"), (dict(cols=96), -2, "whole groups of 64"),
    (dict(cols=32768 + 64), -2, "32768"), (dict(rows=(1 << 30) + 64), -2, "2^30"), (dict(scale_type=2), -1, "scale type 2"),
    (dict(q=16 * A + 8), -1, "16-byte"), (dict(s=32 * A + 1), -1, "2-byte")])
def test_matrix(q8, change, code, word):
    for call in (gemv, gate_up, down):
        assert call(q8, W=mat(q8, **change)) == code
        assert word in q8.last_error()


@pytest.mark.parametrize("change,code,word", [
    (dict(rows=-1), -1, "negative"), (dict(rows=65537), -2, "65536"), (dict(x=None), -1, "x: null"),
    (dict(x=A + 4), -1, "16 bytes"), (dict(xs=130), -1, "16 bytes"), (dict(xs=124), -1, "124 apart"), (dict(y=None), -1, "y: null"),
    (dict(y=2 * A + 2), -1, "y: null or not"), (dict(ys=63), -1, "63 apart"), (dict(ws=None), -1, "ws: null"),
    (dict(y=A + 1024), -1, "y: overlaps"), (dict(y=16 * A), -1, "y: overlaps"), (dict(y=32 * A + 64), -1, "y: overlaps")])
def test_gemv(q8, change, code, word):
    assert gemv(q8, **change) == code
    assert word in q8.last_error()


def test_activation(q8):
    for call, name, words in ((gemv, "x", "xq"), (gate_up, "x", "xq"), (down, "h", "hq")):
        for q, code, word in ((act(q8, A, A), -1, "as values and as words"),):
            assert call(q8, **{words: q}) == code
            assert word in q8.last_error()
        for q, word in ((act(q8, None, A), "null words"), (act(q8, A, None), "null words"), (act(q8, A + 16, A), "32-byte"),
                        (act(q8, A, A + 2), "4-byte"), (act(q8, A, A, A + 16), "32-byte")):
            assert call(q8, **{name: None, words: q}) == -1
            assert word in q8.last_error()


@pytest.mark.parametrize("change,code,word", [
    (dict(rows=-1), -1, "negative"), (dict(k=0), -2, "k 0"), (dict(k=33), -2, "k 33"), (dict(rows=1 << 24), -2, "2^24"),
    (dict(ids=None), -1, "ids or ws"), (dict(ws=None), -1, "ids or ws"), (dict(ids=3 * A + 2), -1, "4-byte"),
    (dict(plan=None), -1, "plan: null"), (dict(plan=(A, None, A, A)), -1, "plan: null")])
def test_experts(q8, change, code, word):
    for call in (gate_up, down):
        assert call(q8, **change) == code
        assert word in q8.last_error()


def test_gate_up(q8):
    for change, word in ((dict(dff=0), "dff 0"), (dict(dff=24), "dff 24"), (dict(h=None), "h: null"), (dict(h=A), "h: overlaps"),
                         (dict(h=3 * A), "h: overlaps"), (dict(h=32 * A), "h: overlaps"),
                         (dict(U=mat(q8, rows=32)), "differ"), (dict(U=mat(q8, z=A)), "differ"),
                         (dict(U=mat(q8, scale_type=1)), "differ"), (dict(U=mat(q8, group=32)), "differ")):
        assert gate_up(q8, **change) == -1
        assert word in q8.last_error()


def test_down(q8):
    for change, word in ((dict(d=0), "d 0"), (dict(d=24), "d 24"), (dict(gates=None), "gates: null"), (dict(y=None), "y: null"),
                         (dict(residual=5 * A + 2), "residual not 4-byte"), (dict(y=A), "y: overlaps"), (dict(y=4 * A), "y: overlaps"),
                         (dict(y=5 * A + 64), "y: overlaps")):
        assert down(q8, **change) == -1
        assert word in q8.last_error()


@pytest.mark.parametrize("array", [1, 2, 3])
def test_outputs_over_the_plan(q8, array):
    plan = [A, A, A, A]
    plan[array] = 40 * A
    assert gate_up(q8, plan=tuple(plan), h=40 * A + 4) == -1 and "h: overlaps" in q8.lib.q8_last_error().decode()
    assert down(q8, plan=tuple(plan), y=40 * A + 4) == -1 and "y: overlaps" in q8.lib.q8_last_error().decode()


def test_no_rows(q8):
    assert norm(q8, rows=0, a=None, b=None, sum=A) == 0
    assert route(q8, rows=0, logits=None, ids=None, gates=None, ws=None) == 0
    assert gemv(q8, rows=0, x=None, y=None, ws=None) == 0
    assert gate_up(q8, rows=0, x=None, h=None, ids=None, plan=None, ws=None) == 0
    assert down(q8, rows=0, h=None, y=None, ids=None, gates=None, plan=None, ws=None) == 0
