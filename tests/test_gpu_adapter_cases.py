"""More of the adapters' calls against 64 bits, with the tolerances derived in test_gpu_adapter.py (whose bound of v's error, that of two
bf16 values, is wider than what fp32 needs): wide matrices of few rows, whose sums are cut into slices and columns into groups,
dropout at every rank in every form, many rows in pieces of every length, offsets that fall, a plan on two streams.
"""

import numpy as np
import pytest
import torch

from gpu_util import dev, note
from oracle import adapter as oracle
from test_gpu_adapter import U, check_backward, check_forward, make, ops, plan_of, val, within

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


def test_a_plan_made_before_a_capture():
    """Calls captured with a plan of eager work, replayed with eager work in between; the plan is dropped after the last replay."""
    note("adapter plan before a capture")
    c = make(38, 700, 2, 4, 3, 192, 128, 16)
    plan = plan_of(c, True)
    up, down = [c["t_" + w] for w in ("a_gu", "b_gate", "b_up", "scale")], [c["t_" + w] for w in ("a_down", "b_down", "scale")]

    def step():
        g, u, a, v1 = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, *up, want_v=True)
        y, v2 = ops().adapter_down(a, c["t_y"], plan, *down, want_v=True)
        return (g, u, a, v1, y, v2, *ops().adapter_down_bwd(c["t_y"], a, v2, g, u, c["t_dg"], c["t_du"], plan, *down))
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(got, want)), i
        assert all(torch.equal(s, t) for s, t in zip(step(), want)), i
    del plan, graph, got
    torch.cuda.synchronize()
    check_forward(c, plan_of(c, True))


# (T, k, E, L, d, f, r): eight slices of 2112 and six of 1344, column groups of unequal width, ranks in two workgroups; many experts
WIDE = [(40, 2, 3, 2, 2112, 1344, 16), (40, 2, 3, 2, 2112, 1344, 64), (40, 2, 3, 2, 1344, 2112, 40), (128, 2, 64, 1, 2048, 640, 8),
        (9, 1, 1, 1, 4096, 576, 24)]


@pytest.mark.parametrize("p", [0.0, 0.25], ids=["plain", "dropout"])
@pytest.mark.parametrize("sort", [False, True], ids=["few", "sorted"])
@pytest.mark.parametrize("T,k,E,L,d,f,r", WIDE)
def test_forward_of_wide_matrices(T, k, E, L, d, f, r, sort, p):
    note(f"adapter wide forward {T} {k} {E} {L} {d} {f} {r} sorted={sort} p={p}")
    c = make(33, T, k, E, L, d, f, r)
    check_forward(c, plan_of(c, sort), p=p)


@pytest.mark.parametrize("p", [0.0, 0.1], ids=["plain", "dropout"])
@pytest.mark.parametrize("T,k,E,L,d,f,r", WIDE)
def test_backward_of_wide_matrices(T, k, E, L, d, f, r, p):
    note(f"adapter wide backward {T} {k} {E} {L} {d} {f} {r} p={p}")
    c = make(34, T, k, E, L, d, f, r)
    check_backward(c, plan_of(c, True), p=p)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64])
def test_dropout_at_every_rank_of_few_rows_and_of_the_backward(r):
    note(f"adapter dropout few, backward r={r}")
    c = make(35, 150, 2, 3, 2, 192, 128, r)
    check_forward(c, plan_of(c, False), p=0.25)
    check_backward(c, plan_of(c, True), p=0.1)


# (T, E, L): pieces of 256, 640 and 2048 rows of a contraction, several to a group, next to groups of one
@pytest.mark.parametrize("T,E,L,p", [(7000, 2, 3, 0.0), (20002, 1, 2, 0.1), (70001, 1, 1, 0.0)])
def test_backward_of_many_rows(T, E, L, p):
    note(f"adapter backward many rows {T} {E} {L} p={p}")
    c = make(36, T, 1, E, L, 64, 64, 8)
    check_backward(c, plan_of(c, True), p=p)


def test_backward_of_many_rows_and_wide_matrices():
    """Pieces, column groups and ranks in two workgroups together, and both products of gate/up."""
    note("adapter backward many rows, wide")
    c = make(37, 1500, 1, 2, 2, 1344, 640, 40)
    check_backward(c, plan_of(c, True), p=0.1)
