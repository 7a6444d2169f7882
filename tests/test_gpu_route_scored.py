"""The scored router on the GPU against the float64 oracle: chosen experts and row metadata exactly, gates
and gradients to fp32 accuracy.

Tolerances.  Gates are computed in 64 bits and rounded to fp32 once: at most 2^-24 of the value (2^-23
allows the 64-bit steps), or, below 2^-126, where fp32 values are the multiples of 2^-149, half of that step.  Only the softmax's sum over all experts, by which its gates are divided when they
are not renormalised, is made of fp32 exponentials: one of x = l - max is off by (|x| + 1) 2^-23 of itself
(its argument is rounded twice, the exponential by a unit), on average over the sum at most (ln E + 1) 2^-23
since the softmax's mean of |x| is at most its entropy; adding 4 per lane over 6 levels, or 16 as
a tree over 4, rounds at most 9 times by 2^-24; with ln 256 = 5.6 that is less than 12 * 2^-23.  A gradient is g (ds - sum g ds) or s (1 - s) ds in fp32: exponentials are off by
a few units plus the rounding of their argument (2^-24 of |l - max|, at most 2^-24 * 32 for the logits
here), sums run over at most 256 terms in a tree of 10 levels, so every term is off by less than 64 * 2^-24
of the sum of magnitudes that enters it.  The oracle multiplies by a whole Jacobian in 64 bits, whose at
most 256 terms leave up to 256 * 2^-52 of that sum where the exact gradient is zero.
"""

import numpy as np
import pytest
import torch

from gpu_util import dev, f32_to_dev, host, i32_to_dev, note
from oracle import moe, scored

pytestmark = pytest.mark.gpu

CASES = [
    # T, E, k, n_group, topk_group, group_top, score, renormalize, bias
    (1, 256, 8, 8, 4, 2, "sigmoid", True, True),
    (1, 1, 1, 1, 1, 1, "softmax", True, False),
    (3, 64, 16, 1, 1, 1, "softmax", False, True),
    (65, 160, 6, 8, 3, 1, "softmax", False, False),
    (130, 256, 8, 8, 4, 2, "sigmoid", True, True),
    (64, 96, 4, 96, 7, 2, "sigmoid", False, True),
    (200, 7, 7, 1, 1, 1, "sigmoid", True, False),
    (77, 192, 5, 64, 3, 2, "softmax", True, True),
    (129, 256, 16, 256, 16, 1, "sigmoid", True, False),
    (500, 24, 3, 4, 2, 2, "sigmoid", False, False),
]


def _inputs(T, E, seed, bias):
    rng = np.random.default_rng([seed, T, E])
    logits = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    return rng, logits, (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None


def _check_forward(logits, k, bias, out, pad=128, **kw):
    T, E = logits.shape
    idx, gate, s = scored.route(logits, k, bias=bias, **kw)
    assert np.array_equal(host(out["topk_idx"]), idx)
    got = host(out["topk_gate"]).astype(np.float64)
    units = 13 if kw.get("score") == "softmax" and not kw.get("renormalize", True) else 1
    assert np.all(np.abs(got - gate) <= units * 2.0 ** -23 * np.abs(gate) + 2.0 ** -149)
    meta = moe.route_metadata(idx, E, pad=pad)
    for name, want in zip(("counts", "offsets", "dest", "row_token", "offsets_pad"), meta):
        assert np.array_equal(host(out[name]), want), name
    if out["scores"] is not None:
        assert np.all(np.abs(host(out["scores"]).astype(np.float64) - s) <= 2.0 ** -23 * s + 2.0 ** -149)


@pytest.mark.parametrize("T,E,k,n_group,topk_group,group_top,score,renormalize,bias", CASES)
def test_forward(T, E, k, n_group, topk_group, group_top, score, renormalize, bias):
    from expert_ffn_layer_top_amd import ops
    _, logits, b = _inputs(T, E, 1, bias)
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top, renormalize=renormalize, scale=2.5)
    note(f"route_scored T={T} E={E} k={k} {kw}")
    out = ops.route_scored(f32_to_dev(logits), k, bias=None if b is None else f32_to_dev(b), pad=128,
                           want_scores=True, **kw)
    _check_forward(logits, k, b, out, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_absent_experts_ties_and_infinities(score):
    from expert_ffn_layer_top_amd import ops
    inf, nan = np.inf, np.nan
    logits = np.zeros((8, 8), np.float32)
    logits[0] = [1, -inf, nan, 0.5, -inf, -inf, 3, -inf]
    logits[1] = -inf
    logits[2] = nan
    logits[3] = [inf, 0, inf, -1, -inf, 0, 0, 0]
    logits[4] = [-0.0, 0.0, -0.0, 0.0, 0.0, -0.0, 0.0, 0.0]
    logits[5] = -np.finfo(np.float32).max
    logits[6] = [-200, -201, -202, -203, -200, -201, -202, -203]
    logits[7] = [1e-40, -1e-40, 0, 5, 5, 5, 5, 5]
    bias = np.array([0.0, 1.0, 0.5, -inf, nan, 0.0, 0.0, 1e30], np.float32)
    for b in (None, bias):
        for n_group, topk_group, group_top in ((1, 1, 1), (4, 2, 2), (2, 1, 1)):
            kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
            note(f"route_scored edges {kw} bias={b is not None}")
            out = ops.route_scored(f32_to_dev(logits), 4, bias=None if b is None else f32_to_dev(b), pad=128, **kw)
            _check_forward(logits, 4, b, out, **kw)


# shapes of every form of the choice from fp32 scores (no score output, more than 64 tokens): 4, 8 or 16 experts
# per lane with whole lanes per group, experts that fill no last lane or no vector load, groups of odd sizes
FAST = [
    # E, k, n_group, topk_group, group_top, score, bias
    (256, 8, 8, 4, 2, "sigmoid", True), (256, 16, 16, 16, 1, "softmax", True), (256, 1, 16, 3, 2, "softmax", False),
    (200, 11, 1, 1, 1, "sigmoid", True), (130, 16, 1, 1, 1, "softmax", False), (128, 8, 16, 5, 2, "sigmoid", False),
    (72, 9, 9, 2, 2, "softmax", True), (65, 7, 1, 1, 1, "sigmoid", True), (64, 6, 2, 1, 2, "sigmoid", True),
    (48, 4, 12, 3, 1, "softmax", True), (33, 16, 1, 1, 1, "softmax", True), (16, 16, 4, 4, 2, "sigmoid", True),
    (5, 5, 1, 1, 1, "sigmoid", False), (1, 1, 1, 1, 1, "softmax", True),
    (160, 6, 8, 3, 2, "sigmoid", True), (96, 4, 96, 7, 1, "sigmoid", True), (255, 10, 5, 2, 2, "softmax", True),
]


@pytest.mark.parametrize("E,k,n_group,topk_group,group_top,score,bias", FAST)
def test_choice_of_many_tokens(E, k, n_group, topk_group, group_top, score, bias):
    from expert_ffn_layer_top_amd import ops
    _, logits, b = _inputs(333, E, 7, bias)
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    note(f"route_scored many E={E} k={k} {kw} bias={bias}")
    out = ops.route_scored(f32_to_dev(logits), k, bias=None if b is None else f32_to_dev(b), pad=128, **kw)
    assert out["scores"] is None
    _check_forward(logits, k, b, out, **kw)


@pytest.mark.parametrize("E,k,n_group,topk_group,group_top,score,bias", FAST)
def test_choice_of_many_tokens_with_absent_experts_ties_and_infinities(E, k, n_group, topk_group, group_top, score, bias):
    from expert_ffn_layer_top_amd import ops
    rng = np.random.default_rng([13, E])
    inf, nan, top = np.inf, np.nan, np.finfo(np.float32).max
    kinds = [np.array(v, np.float32) for v in
             ([0.0], [-0.0, 0.0], [-inf], [nan], [inf], [-top], [top, -inf], [0.0, -inf, nan], [1.0, 2.0], [1e-40, -1e-40, 0.0],
              [-200.0, -201.0], [inf, 0.0, -inf], [90.0, -90.0], [nan, 0.5, 0.5, 0.25])]
    logits = np.stack([rng.choice(kinds[t % len(kinds)], E) for t in range(7 * len(kinds))])
    logits[::5, E // 2] = -inf
    some = np.array([0.0, 0.0, 0.0, 1.0, 0.5, -inf, nan, 1e30, inf], np.float32)
    b = rng.choice(some, E) if bias else None
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    note(f"route_scored many edges E={E} k={k} {kw} bias={bias}")
    out = ops.route_scored(f32_to_dev(logits), k, bias=None if b is None else f32_to_dev(b), pad=128, **kw)
    _check_forward(logits, k, b, out, **kw)


def test_choice_next_to_ties_is_made_in_64_bits():
    """Scores that differ by less than one fp32 rounding: biases cancel the sigmoids' fp32 values."""
    from expert_ffn_layer_top_amd import ops
    rng = np.random.default_rng(11)
    T, E = 300, 64
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:] = logits[:1]                                   # one row, its last bits varied
    logits += (rng.integers(-2, 3, (T, E)) * 2.0 ** -23).astype(np.float32) * np.abs(logits)
    bias = (1.0 - 1.0 / (1.0 + np.exp(-logits[0].astype(np.float64)))).astype(np.float32)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2)
    out = ops.route_scored(f32_to_dev(logits), 6, bias=f32_to_dev(bias), pad=128, **kw)
    _check_forward(logits, 6, bias, out, **kw)


@pytest.mark.parametrize("T,E,k,score,renormalize", [
    (1, 256, 8, "sigmoid", True), (5, 256, 8, "softmax", True), (130, 128, 8, "softmax", False),
    (67, 33, 3, "sigmoid", False), (3, 1, 1, "softmax", True), (257, 200, 16, "softmax", False)])
def test_backward(T, E, k, score, renormalize):
    from expert_ffn_layer_top_amd import ops
    rng, logits, _ = _inputs(T, E, 2, False)
    if E > 8:
        logits[0, :3] = [-np.inf, np.nan, -120.0]
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if E > 8:
        idx[0, :min(k, 3)] = np.arange(min(k, 3))
    dg = rng.standard_normal((T, k)).astype(np.float32)
    note(f"route_scored_bwd T={T} E={E} k={k} {score} {renormalize}")
    got = host(ops.route_scored_bwd(f32_to_dev(logits), i32_to_dev(idx), f32_to_dev(dg), score=score,
                                    renormalize=renormalize, scale=2.5)).astype(np.float64)
    want = scored.route_bwd(logits.astype(np.float64), idx, dg.astype(np.float64), score=score, renormalize=renormalize,
                            scale=2.5)
    for t in range(T):
        _, s = scored.scores(logits[t], score)
        w = s[idx[t]]
        g = w / w.sum() if renormalize and w.sum() > 0 else w
        most = 2.5 * (np.abs(dg[t]).max() + (g * np.abs(dg[t])).sum())
        at = np.zeros(E)
        np.maximum.at(at, idx[t], g)
        if score == "softmax" and not renormalize:
            at = np.maximum(at, s)
        assert np.all(np.abs(got[t] - want[t]) <= 64 * 2.0 ** -24 * at * most + 2.0 ** -44 * most), t


def test_backward_repeated_and_foreign_indices():
    """An index that repeats adds up, one outside the experts takes no part."""
    from expert_ffn_layer_top_amd import ops
    logits = np.array([[0.5, -1.0, 2.0, 0.0]], np.float32)
    dg = np.array([[1.0, 2.0, 4.0]], np.float32)
    s = 1 / (1 + np.exp(-logits[0].astype(np.float64)))
    got = host(ops.route_scored_bwd(f32_to_dev(logits), i32_to_dev([[2, 2, 7]]), f32_to_dev(dg), renormalize=False))
    assert np.allclose(got[0], [0, 0, 3 * s[2] * (1 - s[2]), 0], rtol=1e-6)
    got = host(ops.route_scored_bwd(f32_to_dev(logits), i32_to_dev([[1, -1, 4]]), f32_to_dev(dg), renormalize=False))
    assert np.allclose(got[0], [0, s[1] * (1 - s[1]), 0, 0], rtol=1e-6)


def test_repeats_strided_streams_and_graphs():
    """Two calls give the same bits; a call on another stream and a replayed graph too."""
    from expert_ffn_layer_top_amd import ops
    _, logits, b = _inputs(1000, 256, 5, True)
    x, bias = f32_to_dev(logits), f32_to_dev(b)
    kw = dict(score="sigmoid", bias=bias, n_group=8, topk_group=4, group_top=2, pad=128)
    first = ops.route_scored(x, 8, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = ops.route_scored(x, 8, **kw)
        grad = ops.route_scored_bwd(x, first["topk_idx"], first["topk_gate"])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        third = ops.route_scored(x, 8, **kw)
        third_grad = ops.route_scored_bwd(x, third["topk_idx"], third["topk_gate"])
    want = ops.route_scored(x, 8, **kw)
    for replay in range(3):
        for t in third.values():
            if t is not None:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name, t in want.items():
            if t is not None:
                assert torch.equal(t, third[name]), (replay, name)
        assert torch.equal(third_grad, grad)
    for name, t in want.items():
        if t is not None:
            assert torch.equal(t, first[name]) and torch.equal(t, second[name])
    with pytest.raises(ValueError, match="contiguous"):
        ops.route_scored(x[:, ::2], 8)
