"""The scored router's oracle against other statements of it: torch's sort-free formulas on the CPU,
brute force over groups, central differences of the gates."""

import itertools

import numpy as np
import pytest
import torch

from oracle import moe, scored


def test_plain_softmax_is_the_other_router():
    rng = np.random.default_rng(1)
    logits = rng.standard_normal((40, 12)).astype(np.float32)
    idx, gate, _ = scored.route(logits, 3, score="softmax")
    want = moe.route_topk(logits, 3)
    assert np.array_equal(idx, want[0])
    assert np.allclose(gate, want[1], rtol=1e-12, atol=0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_against_brute_force(score, group_top):
    rng = np.random.default_rng(2)
    logits = rng.standard_normal((30, 12)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(12)).astype(np.float32)
    idx, gate, s = scored.route(logits, 2, score=score, bias=bias, n_group=4, topk_group=2, group_top=group_top)
    t = torch.from_numpy(logits).double()
    p = (torch.sigmoid(t) if score == "sigmoid" else torch.softmax(t, dim=1)).numpy()
    assert np.allclose(s, p, rtol=1e-13, atol=0)
    c = p + bias.astype(np.float64)
    for r in range(30):
        value = [np.sort(c[r, 3 * g:3 * g + 3])[::-1][:group_top].sum() for g in range(4)]
        kept = max(itertools.combinations(range(4), 2), key=lambda gs: sum(value[g] for g in gs))
        allowed = [e for e in range(12) if e // 3 in kept]
        best = max(itertools.permutations(allowed, 2), key=lambda es: (c[r, es[0]], c[r, es[1]]))
        assert tuple(idx[r]) == best
        assert np.allclose(gate[r], p[r, list(best)] / p[r, list(best)].sum(), rtol=1e-13)


def test_absent_experts():
    inf = np.inf
    logits = np.array([[1.0, -inf, np.nan, 0.5], [-inf] * 4, [inf, 0.0, inf, -1.0]], np.float32)
    idx, gate, _ = scored.route(logits, 3, score="sigmoid")
    assert idx.tolist() == [[0, 3, 1], [0, 1, 2], [0, 2, 1]]
    assert gate[0, 2] == 0 and gate[0].sum() == pytest.approx(1) and not gate[1].any()
    idx, gate, _ = scored.route(logits, 3, score="softmax")
    assert gate[2].tolist() == [0.5, 0.5, 0.0]
    # a group whose experts are all absent is kept last, whatever its bias
    idx, _, _ = scored.route(np.array([[-inf, -inf, -5.0, -inf]], np.float32), 1,
                             bias=np.array([9, 9, 0, 0], np.float32), n_group=2, topk_group=1, group_top=2)
    assert idx.tolist() == [[2]]


def test_ties_go_to_the_lower_index():
    idx, _, _ = scored.route(np.zeros((1, 8), np.float32), 3, bias=np.zeros(8, np.float32), n_group=4, topk_group=2)
    assert idx.tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((4, 6))
    d_gate = rng.standard_normal((4, 2))
    idx = np.stack([rng.permutation(6)[:2] for _ in range(4)])
    got = scored.route_bwd(logits, idx, d_gate, score=score, renormalize=renormalize, scale=1.7)

    def loss(l):
        total = 0.0
        for t in range(4):
            w = scored.scores(l[t], score)[1][idx[t]]
            total += 1.7 * ((w / w.sum() if renormalize else w) * d_gate[t]).sum()
        return total

    h = 1e-5
    for t in range(4):
        for e in range(6):
            up, down = logits.copy(), logits.copy()
            up[t, e] += h
            down[t, e] -= h
            assert got[t, e] == pytest.approx((loss(up) - loss(down)) / (2 * h), abs=1e-8)
