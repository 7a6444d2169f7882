"""More of the adapters' calls against 64 bits, with the tolerances derived in test_gpu_adapter.py: offsets that fall, in both forms."""

import numpy as np
import pytest
import torch

from gpu_util import dev, note
from oracle import adapter as oracle
from test_gpu_adapter import U, check_forward, make, ops, plan_of, val, within

pytestmark = pytest.mark.gpu


def with_offsets(c, off):
    """The case under other offsets: of rows that their running maximum within [0, n] gives to an expert."""
    c["off"] = np.array(off, dtype=np.int64).astype(np.int32)
    eff = np.maximum.accumulate(np.clip(np.array(off, dtype=np.int64), 0, c["n"]))
    c["e"], c["l"] = oracle.row_groups(c["ids"], eff, c["token"], c["n"], c["L"])
    c["s"] = np.where(c["l"] >= 0, c["scale"].astype(np.float64)[c["l"]], 0.0)[:, None]
    return eff


@pytest.mark.parametrize("sort", [False, True], ids=["few", "sorted"])
@pytest.mark.parametrize("bad", [[0, 250, 40, 2 ** 31 - 1, 300], [-5, 7, 309, 3, 100], [0, 300, 0, 300, 0], [0, 100, 50, 200, 300],
                                 [-2 ** 31, -1, 150, 150, 301]], ids=str)
def test_offsets_that_fall_are_their_running_maximum_in_both_forms(bad, sort):
    note(f"adapter falling offsets {bad} sorted={sort}")
    c = make(30, 300, 1, 4, 2, 64, 64, 8)
    with_offsets(c, bad)
    assert c["e"].min() >= 0
    check_forward(c, plan_of(c, sort))


def test_many_experts_with_falling_offsets():
    """The running maximum over all four groups of 64 experts."""
    note("adapter falling offsets of 256 experts")
    for sort in (False, True):
        c = make(31, 400, 1, 256, 1, 64, 64, 8, "one")
        g = np.random.default_rng(4)
        off = np.concatenate([[0], np.sort(g.integers(0, 401, 255)), [400]])
        fall = g.random(257) < 0.5
        off[fall] -= g.integers(0, 300, 257)[fall]
        off[0], off[256] = -3, 500
        with_offsets(c, off)
        assert c["e"].min() >= 0 and len(np.unique(c["e"])) > 64
        check_forward(c, plan_of(c, sort))


@pytest.mark.parametrize("sort", [False, True], ids=["few", "sorted"])
def test_rows_outside_falling_offsets_are_left_as_they_were(sort):
    """The C call on a prefilled output: rows before the first and from the largest offset on keep every byte."""
    from expert_ffn_layer_top_amd._lib import call, lib
    note(f"adapter rows outside falling offsets sorted={sort}")
    c = make(32, 60, 1, 4, 2, 64, 64, 8)
    eff = with_offsets(c, [5, 30, 9, 41, 20])
    plan = plan_of(c, sort)
    v, y = (torch.full((60, cols), 7.25, dtype=torch.bfloat16, device=dev()) for cols in (8, 64))
    nbytes = lib.moe_adapter_workspace_bytes(60, 4, 2, 64, 64, 8, sort, False)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev())
    p = lambda name: c["t_" + name].data_ptr()                                                    # noqa: E731
    call("moe_adapter_down", p("a"), *plan._args(), 64, 64, 8, p("a_down"), p("b_down"), p("scale"), None, 0.0, 0, p("y"),
         v.data_ptr(), y.data_ptr(), ws.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream)
    out = c["e"] < 0
    assert np.array_equal(out, (np.arange(60) < 5) | (np.arange(60) >= 41)) and eff[-1] == 41
    for t in (v, y):
        assert bool((t[torch.from_numpy(out)] == 7.25).all())
    ref, mag = oracle.shrink(c["a"], c["a_down"], c["e"], c["l"])
    within(val(v)[~out], ref[~out], (U * np.abs(ref) + 64 * 2.0 ** -23 * mag)[~out], "v")


def test_a_plan_used_on_another_stream_and_dropped():
    """Its buffer is not handed out again while the other stream's calls that read it are still to run."""
    note("adapter plan on another stream")
    n, d, f, r = 300000, 64, 64, 8
    g = torch.Generator(device=dev()).manual_seed(1)
    bf = lambda *s: torch.randn(s, generator=g, device=dev()).to(torch.bfloat16)          # noqa: E731
    a, y, A, B = bf(n, f), bf(n, d), bf(2, 3, r, f), bf(2, 3, r, d)
    scale = torch.ones(2, dtype=torch.float32, device=dev())
    ids = torch.randint(-1, 2, (n,), generator=g, device=dev()).int()
    off = torch.tensor([0, n // 3, n // 2, n], dtype=torch.int32, device=dev())
    want = ops().adapter_down(a, y, ops().adapter_plan(ids, off, 2), A, B, scale)[0]
    work = torch.randn(8192, 8192, generator=g, device=dev())
    busy = work @ work
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    plan = ops().adapter_plan(ids, off, 2)
    at, size = plan.buf.data_ptr(), plan.buf.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(8):
            torch.mm(work, work, out=busy)          # a millisecond or more each
        got = ops().adapter_down(a, y, plan, A, B, scale)[0]
    del plan
    again = torch.empty(size, dtype=torch.uint8, device=dev())
    assert not other.query()                        # (the other stream was still at work when the memory was asked for)
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, want)
