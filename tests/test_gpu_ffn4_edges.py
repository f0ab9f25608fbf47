"""GPU tests of the 4-bit feed-forward block at its edges.  Bounds and helpers as in test_gpu_ffn4.py."""
import math

import pytest

from test_gpu_ffn4 import (activation, check_combined, check_hidden, check_route, choices, gen, matrix, plan_of,
                           product_error, quantize, route, values)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws(q8):
    w = q8.Workspace()
    yield w
    w.close()


def give_up(q8, torch, ws):
    """Marks the workspace: an attention on it whose waits run out."""
    words = [torch.zeros(4, 2, 16, 64, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(4, 2, 16, device="cuda") for _ in range(2)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = q8.kv_pages(words[0], scales[0], words[1], scales[1])
    q = torch.zeros(1, 4, 64, device="cuda")
    q8.q8_paged_wait_selftest(pages, q8.kv_batch(i32(0, 1), i32(40), i32(0, 1, 2).view(1, 3)), q, torch.zeros_like(q), 16, ws)


def experts(torch, rows, E, k, d, dff, form, seed):
    """Matrices, choices, gates, an activation and hidden rows of a call."""
    g = gen(seed)
    mats = [matrix(torch, n, c, 32, "f16", True, g) for n, c in ((E * dff, d), (E * dff, d), (E * d, dff))]
    ids = choices(torch, rows, E, k, g, False)
    gates = torch.rand(rows, k, generator=g, device="cuda") + 0.1
    call, x = activation(torch, rows, d, form, g)
    h = torch.randn(rows, k, dff, generator=g, device="cuda")
    if form == "f32":
        hidden, hv = dict(h=h), h.double()
    else:
        q, lo, s = quantize(torch, h, form == "two")
        hidden = dict(hq=q, hs=s, hl=lo)
        hv = (q.double() if lo is None else q.double() + lo.double() / 128) * s.double().repeat_interleave(32, -1)
    residual = torch.randn(rows, d, generator=g, device="cuda")
    return mats, ids, gates, call, x, hidden, hv, residual


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("form", ["f32", "one"])
def test_experts_on_a_workspace_of_which_a_wait_gave_up(q8, form, in_place):
    """Products on the tensor cores, and the sum over their choices, write nothing until the workspace has been checked."""
    import torch
    rows, E, k, d, dff = 130, 6, 6, 128, 128
    mats, ids, gates, call, x, hidden, hv, residual = experts(torch, rows, E, k, d, dff, form, 21)
    m = [q8.q4_mat(*t) for t in mats]
    plan, kept = plan_of(q8, torch, ids, E)
    ws = q8.Workspace()
    give_up(q8, torch, ws)
    h = torch.full((rows, k, dff), 7.0, device="cuda")
    y = residual.clone() if in_place else torch.full((rows, d), 7.0, device="cuda")
    was = y.clone()
    q8.moe_gate_up_q4(m[0], m[1], ids, h, **call, plan=plan, ws=ws)
    q8.moe_down_combine_q4(m[2], ids, gates, y, **hidden, plan=plan, residual=y if in_place else residual, ws=ws)
    assert (h == 7).all()
    assert torch.equal(y, was)
    with pytest.raises(q8.Q8Error) as e:
        ws.check()
    assert e.value.code == -4
    q8.moe_gate_up_q4(m[0], m[1], ids, h, **call, plan=plan, ws=ws)
    q8.moe_down_combine_q4(m[2], ids, gates, y, **hidden, plan=plan, residual=y if in_place else residual, ws=ws)
    check_hidden(torch, h, values(torch, mats[0]), values(torch, mats[1]), x, ids, dff, form)
    check_combined(torch, y, values(torch, mats[2]), hv, ids, gates, residual, d, form)
    ws.check()
    ws.close()
    del kept


@pytest.mark.parametrize("rows", [1, 5, 61, 2311])
def test_route_on_a_workspace_of_which_a_wait_gave_up(q8, rows):
    """With a plan nothing is written until the workspace has been checked; without one no workspace is looked at."""
    import torch
    E, k, rule = 64, 6, dict(score=1, groups=4, keep_groups=2)
    logits = torch.randn(rows, E, generator=gen(rows), device="cuda")
    ids, gates = torch.full((rows, k), 3, dtype=torch.int32, device="cuda"), torch.full((rows, k), 7.0, device="cuda")
    arrays = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (E, E + 1, rows * k, E + 1)]
    ws = q8.Workspace()
    give_up(q8, torch, ws)
    for _ in range(2):
        q8.moe_route_scored(logits, ids, gates, plan=q8.plan_struct(*arrays), ws=ws, **rule)
    assert (ids == 3).all() and (gates == 7).all() and all((a == -9).all() for a in arrays)
    check_route(torch, route(q8, torch, ws, logits, k, False, **rule), logits, k, False, **rule)
    with pytest.raises(q8.Q8Error) as e:
        ws.check()
    assert e.value.code == -4
    for _ in range(2):
        check_route(torch, route(q8, torch, ws, logits, k, True, **rule), logits, k, True, **rule)
    ws.check()
    ws.close()


@pytest.mark.parametrize("xe,se", [(-106, -23), (110, -60), (-100, 60), (120, -6), (-60, -60)])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_projection_of_magnitudes_far_from_1(q8, ws, rows, xe, se):
    """Values of 2^xe by scales of 2^se, whose products' sums are normal numbers: the usual bound, and half a step of the
    smallest numbers for every sum."""
    import torch
    g = gen(rows + 7)
    q = torch.randint(0, 256, (50, 128), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.randn(50, 8, generator=g, device="cuda", dtype=torch.float64) * 2.0 ** se).to(torch.bfloat16)
    x = (torch.randn(rows, 256, generator=g, device="cuda", dtype=torch.float64) * 2.0 ** xe).float()
    y = torch.empty(rows, 50, device="cuda")
    q8.q4_gemv(q8.q4_mat(q, s), y, x=x, ws=ws)
    W = values(torch, (q, s, None))
    tol = product_error(torch, W, x.double(), "f32") + (8 + 8) * 2.0 ** -149
    assert ((y.double() - x.double() @ W.T).abs() <= tol).all()


@pytest.mark.parametrize("zero", [None, 0, 15])
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_two_word_dots_are_exact(q8, ws, rows, zero):
    """A block's two-word dot is an integer of 128ths: with zero points up to 15 it is below 32 * 15 * 16383 < 2^23, which f32
    holds exactly, as are all its parts' sums."""
    import torch
    g = gen(rows)
    q = torch.randint(0, 256, (64, 16), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.ones(64, 1, dtype=torch.float16, device="cuda")
    z = None if zero is None else torch.full((64, 1), zero, dtype=torch.uint8, device="cuda")
    hi, lo = (torch.randint(-127, 128, (rows, 32), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    hi[0], lo[0] = 127, 127
    q[0], q[1] = 0, 255
    y = torch.empty(rows, 64, device="cuda")
    q8.q4_gemv(q8.q4_mat(q, s, z), y, xq=hi, xs=torch.ones(rows, 1, device="cuda"), xl=lo, ws=ws)
    x = hi.double() + lo.double() / 128
    assert torch.equal(y.double(), x @ values(torch, (q, s, z)).T)


@pytest.mark.parametrize("form", ["f32", "one", "two"])
@pytest.mark.parametrize("rows", [1, 7, 130])
def test_combine_in_place(q8, ws, rows, form):
    """The residual's own place as the result's: bit for bit what another place gets."""
    import torch
    E, k, d, dff = 9, 4, 256, 128
    mats, ids, gates, call, x, hidden, hv, residual = experts(torch, rows, E, k, d, dff, form, rows)
    m = q8.q4_mat(*mats[2])
    plan, kept = plan_of(q8, torch, ids, E) if rows > 1 else (None, None)
    y = torch.full((rows, d), math.nan, device="cuda")
    q8.moe_down_combine_q4(m, ids, gates, y, **hidden, plan=plan, residual=residual, ws=ws)
    check_combined(torch, y, values(torch, mats[2]), hv, ids, gates, residual, d, form)
    q8.moe_down_combine_q4(m, ids, gates, residual, **hidden, plan=plan, residual=residual, ws=ws)
    assert torch.equal(residual, y)
    del kept


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("rows", [1, 7, 130])
def test_experts_of_values_that_are_not_finite(q8, ws, rows, bad):
    """A row with such a value has hidden rows and a result that are not finite; the others do not see it."""
    import torch
    E, k, d, dff, r = 9, 4, 256, 128, rows // 2
    mats, ids, gates, call, x, hidden, hv, residual = experts(torch, rows, E, k, d, dff, "f32", rows + 5)
    m = [q8.q4_mat(*t) for t in mats]
    plan, kept = plan_of(q8, torch, ids, E) if rows > 1 else (None, None)
    clean, h = (torch.full((rows, k, dff), 5.0, device="cuda") for _ in range(2))
    q8.moe_gate_up_q4(m[0], m[1], ids, clean, **call, plan=plan, ws=ws)
    values_ = call["x"].clone()
    values_[r, 33] = bad
    q8.moe_gate_up_q4(m[0], m[1], ids, h, x=values_, plan=plan, ws=ws)
    rest = [i for i in range(rows) if i != r]
    assert not torch.isfinite(h[r]).any() and torch.equal(h[rest], clean[rest])
    y, want = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, device="cuda")
    q8.moe_down_combine_q4(m[2], ids, gates, want, **hidden, plan=plan, ws=ws)
    hidden["h"][r, 1, 33] = bad
    q8.moe_down_combine_q4(m[2], ids, gates, y, **hidden, plan=plan, ws=ws)
    assert not torch.isfinite(y[r]).any() and torch.equal(y[rest], want[rest])
    del kept


@pytest.mark.parametrize("rows", [9, 150])
def test_products_by_a_plan_of_the_softmax_router(q8, ws, rows):
    """moe_route_topk's plan groups the rows for the 4-bit products."""
    import torch
    E, k, d, dff = 32, 4, 256, 128
    mats, _, _, call, x, hidden, hv, residual = experts(torch, rows, E, k, d, dff, "f32", rows + 2)
    g = gen(rows)
    rq = torch.randint(-127, 128, (E, d), generator=g, device="cuda", dtype=torch.int8)
    rs = torch.full((E, d // 32), 1e-3, device="cuda")
    ids, gates = torch.empty(rows, k, dtype=torch.int32, device="cuda"), torch.empty(rows, k, device="cuda")
    arrays = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E, E + 1, rows * k, E + 1)]
    plan = q8.plan_struct(*arrays)
    q8.moe_route_topk(rq, rs, 0, k, ids, gates, x=call["x"], rows=rows, plan=plan, ws=ws)
    h, y = torch.full((rows, k, dff), math.nan, device="cuda"), torch.full((rows, d), math.nan, device="cuda")
    q8.moe_gate_up_q4(q8.q4_mat(*mats[0]), q8.q4_mat(*mats[1]), ids, h, **call, plan=plan, ws=ws)
    q8.moe_down_combine_q4(q8.q4_mat(*mats[2]), ids, gates, y, **hidden, plan=plan, residual=residual, ws=ws)
    check_hidden(torch, h, values(torch, mats[0]), values(torch, mats[1]), x, ids, dff, "f32")
    check_combined(torch, y, values(torch, mats[2]), hv, ids, gates, residual, d, "f32")


def need(rows, k, E, cols, d=0):
    """The workspace that a call of several rows needs at most: of every choice, and up to eight more an expert, 544 bytes for
    each 128 columns started and 4; for down also its outputs."""
    n = rows * k + 8 * min(E, rows * k) + 16
    return n * ((cols + 127) // 128 * 544 + 4) + 4 * rows * k * d + 1024


@pytest.mark.parametrize("form", ["f32", "one", "two"])
@pytest.mark.parametrize("rows,E,k,d,dff", [(7, 40, 3, 416, 96), (24, 32, 8, 256, 256), (130, 6, 6, 128, 160), (300, 4, 1, 256, 128)])
def test_experts_in_a_workspace_that_just_holds_them(q8, ws, rows, E, k, d, dff, form):
    import torch
    mats, ids, gates, call, x, hidden, hv, residual = experts(torch, rows, E, k, d, dff, form, rows + E)
    m = [q8.q4_mat(*t) for t in mats]
    plan, kept = plan_of(q8, torch, ids, E)
    small, tiny = [q8.Workspace(need(rows, k, E, d)), q8.Workspace(need(rows, k, E, dff, d))], q8.Workspace(4096)
    h, y = torch.full((rows, k, dff), 7.0, device="cuda"), torch.full((rows, d), 7.0, device="cuda")
    for call_ in (lambda w: q8.moe_gate_up_q4(m[0], m[1], ids, h, **call, plan=plan, ws=w),
                  lambda w: q8.moe_down_combine_q4(m[2], ids, gates, y, **hidden, plan=plan, residual=residual, ws=w)):
        with pytest.raises(q8.Q8Error) as e:
            call_(tiny)
        assert e.value.code == -5
    assert (h == 7).all() and (y == 7).all()
    want = torch.empty_like(h), torch.empty_like(y)
    q8.moe_gate_up_q4(m[0], m[1], ids, want[0], **call, plan=plan, ws=ws)
    q8.moe_down_combine_q4(m[2], ids, gates, want[1], **hidden, plan=plan, residual=residual, ws=ws)
    q8.moe_gate_up_q4(m[0], m[1], ids, h, **call, plan=plan, ws=small[0])
    q8.moe_down_combine_q4(m[2], ids, gates, y, **hidden, plan=plan, residual=residual, ws=small[1])
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    for w in (*small, tiny):
        w.close()
    del kept
