"""What the binding of the 4-bit feed-forward block passes on and refuses, without a GPU: tensors that give a device, and calls of
the library that are recorded in place of being made."""
import pytest


@pytest.fixture()
def made(monkeypatch):
    """The binding with device 0 as the current one, and the calls that reach the library."""
    import __graft_entry__
    __graft_entry__.build()
    import moe_add_rmsnorm_gb300 as q8

    calls = []
    q8._lazy_torch()
    monkeypatch.setattr(q8, "_current_device", lambda: 0)
    for name in ("q4_gemv", "moe_gate_up_q4", "moe_down_combine_q4", "moe_route_scored", "postnorm_add_rmsnorm_q8"):
        monkeypatch.setattr(q8.lib, name, lambda *a, name=name: calls.append((name, a)) or 0)
    return q8, calls


class Workspace:
    device, handle = 0, 1


def on(*shape, dtype=None, device=0):
    """A tensor that says it is on the device."""
    import torch

    class On(torch.Tensor):
        def get_device(self):
            return device

    return torch.zeros(*shape, dtype=dtype or torch.float32).as_subclass(On)


def matrix(q8, rows, cols, group=32):
    import torch
    return q8.q4_mat(on(rows, cols // 2, dtype=torch.uint8), on(rows, cols // group, dtype=torch.float16))


def refused(q8, calls, word, call):
    with pytest.raises(q8.Q8Error) as e:
        call()
    assert word in str(e.value), (word, str(e.value))
    assert not calls


def test_gate_up_takes_dense_rows(made):
    """Rows that stand apart, or all at one place (a row expanded to a batch), are refused: the call reads rows * d values."""
    import torch
    q8, calls = made
    gate, up = matrix(q8, 64, 128), matrix(q8, 64, 128)
    ids, h = on(3, 2, dtype=torch.int32), on(3, 2, 16)
    plan = q8.plan_struct(*(on(n, dtype=torch.int32) for n in (4, 5, 6, 5)))
    call = lambda x: q8.moe_gate_up_q4(gate, up, ids, h, x=x, plan=plan, ws=Workspace, stream=1)  # noqa: E731
    refused(q8, calls, "x: not contiguous", lambda: call(on(128).expand(3, 128)))
    refused(q8, calls, "x: not contiguous", lambda: call(on(1, 128).expand(3, 128)))
    refused(q8, calls, "x: not contiguous", lambda: call(on(3, 256)[:, :128]))
    call(on(3, 128))
    q8.moe_gate_up_q4(gate, up, ids, h, xq=on(3, 128, dtype=torch.int8), xs=on(3, 4), plan=plan, ws=Workspace, stream=1)
    assert [n for n, _ in calls] == ["moe_gate_up_q4"] * 2


def test_other_rows_at_one_place(made):
    """The other calls' rows: dense, or passed on with their stride, which the library checks."""
    import torch
    q8, calls = made
    down, ids, gates = matrix(q8, 64, 128), on(3, 2, dtype=torch.int32), on(3, 2)
    plan = q8.plan_struct(*(on(n, dtype=torch.int32) for n in (4, 5, 6, 5)))
    refused(q8, calls, "h: not contiguous", lambda: q8.moe_down_combine_q4(
        down, ids, gates, on(3, 16), h=on(1, 1, 128).expand(3, 2, 128), plan=plan, ws=Workspace, stream=1))
    refused(q8, calls, "residual: not a contiguous", lambda: q8.moe_down_combine_q4(
        down, ids, gates, on(3, 16), h=on(3, 2, 128), plan=plan, residual=on(16).expand(3, 16), ws=Workspace, stream=1))
    q8.q4_gemv(down, on(3, 64), x=on(128).expand(3, 128), ws=Workspace, stream=1)
    assert calls.pop()[1][2] == 0  # its stride: "x: rows 0 apart"
    q8.moe_route_scored(on(8).expand(3, 8), ids, gates, stream=1)
    assert calls.pop()[1][1] == 0


@pytest.mark.parametrize("change,word", [
    (dict(counts=3), "plan: for 3 experts and 6 choices, not 4 and 6"), (dict(offsets=4), "plan: for 3 experts"),
    (dict(lists=5), "plan: for 4 experts and 5 choices"), (dict(active=4), "plan: for 3 experts"),
    (dict(dtype="int64"), "plan: not contiguous int32"), (dict(device=1), "plan: not contiguous int32"),
    (dict(device=-1), "plan: not contiguous int32"), (dict(apart=True), "plan: not contiguous int32")])
def test_plans_that_do_not_hold_the_call(made, change, word):
    """A plan of fewer experts or rows, of another type or device: the calls would write, or read, past it."""
    import torch
    q8, calls = made
    gate, up, down = matrix(q8, 64, 128), matrix(q8, 64, 128), matrix(q8, 512, 32)
    ids, gates = on(3, 2, dtype=torch.int32), on(3, 2)

    def plan(counts=4, offsets=5, lists=6, active=5, dtype="int32", device=0, apart=False):
        sizes = (counts, offsets, lists, active)
        if apart:
            return q8.plan_struct(*(on(2 * n, dtype=torch.int32)[::2] for n in sizes))
        return q8.plan_struct(*(on(n, dtype=getattr(torch, dtype), device=device) for n in sizes))

    def each(p):
        yield lambda: q8.moe_route_scored(on(3, 4), ids, gates, plan=p, ws=Workspace, stream=1)
        yield lambda: q8.moe_gate_up_q4(gate, up, ids, on(3, 2, 16), x=on(3, 128), plan=p, ws=Workspace, stream=1)
        yield lambda: q8.moe_down_combine_q4(down, ids, gates, on(3, 128), h=on(3, 2, 32), plan=p, ws=Workspace, stream=1)

    for call in each(plan(**change)):
        refused(q8, calls, word, call)
    for call in each(plan(counts=9, offsets=12, lists=100, active=10)):  # larger ones hold it
        call()
    assert len(calls) == 3


def test_one_row_needs_no_plan(made):
    """A row's choices are not grouped: whatever plan comes along is not looked at."""
    import torch
    q8, calls = made
    gate, up, ids = matrix(q8, 64, 128), matrix(q8, 64, 128), on(1, 2, dtype=torch.int32)
    plan = q8.plan_struct(*(on(1, dtype=torch.int32) for _ in range(4)))
    q8.moe_gate_up_q4(gate, up, ids, on(1, 2, 16), x=on(1, 128), plan=plan, ws=Workspace, stream=1)
    assert len(calls) == 1 and calls[0][1][8] is None


def test_a_plan_keeps_its_tensors(made):
    import gc
    import weakref

    import torch
    q8, calls = made
    arrays = [on(n, dtype=torch.int32) for n in (4, 5, 6, 5)]
    held = [weakref.ref(a) for a in arrays]
    plan = q8.plan_struct(*arrays)
    del arrays
    gc.collect()
    assert all(r() is not None for r in held) and plan.lists == held[2]().data_ptr()


def test_low_words_alone_are_refused(made):
    """Low words without words would be left unwritten."""
    import torch
    q8, calls = made
    a, b, w = on(2, 64), on(2, 64), on(64)
    low = on(2, 64, dtype=torch.int8)
    refused(q8, calls, "yq: words without scales", lambda: q8.postnorm_add_rmsnorm_q8(a, b, None, w, 1e-6, y_out=on(2, 64), yl=low,
                                                                                      stream=1))
    q8.postnorm_add_rmsnorm_q8(a, b, None, w, 1e-6, yq=on(2, 64, dtype=torch.int8), ys=on(2, 2), yl=low, stream=1)
    assert len(calls) == 1
