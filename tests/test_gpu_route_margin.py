"""Choices of the scored router that fp32 scores get wrong: the margin within which they count as undecided has
to cover every rounding on the way.  Gates are not compared here; the chosen experts are, exactly."""

import numpy as np
import pytest

from gpu_util import f32_to_dev, host, note
from oracle import scored

pytestmark = pytest.mark.gpu


def _cancelling(T, E, n_group, B, gap, score, seed):
    """Logits and a bias: the best two of the first group carry biases B and -B (its others -4 |B|), those of the second
    none, and in 64 bits the two groups' values differ by `gap` (of either sign); every other expert's score is far below.  Adding
    B rounds a score to a multiple of B 2^-24 or so, which neither the value nor a margin relative to it shows."""
    rng = np.random.default_rng([seed, T, E, n_group])
    per = E // n_group
    logits = rng.uniform(-9.0, -8.0, (T, E))
    a, b, c = (rng.uniform(0.8, 1.2, T) for _ in range(3))           # exponentials of the softmax, odds of the sigmoid
    sign = rng.choice([-1.0, 1.0], T)
    if score == "softmax":
        rest = a + b + c + np.exp(np.delete(logits, [0, 1, per, per + 1], axis=1)).sum(axis=1)
        d = (a + b - c - sign * gap * rest) / (1.0 + sign * gap)
    else:
        p = a / (1 + a) + b / (1 + b) - c / (1 + c) - sign * gap
        d = p / (1 - p)
    logits[:, 0], logits[:, 1], logits[:, per], logits[:, per + 1] = (np.log(v) for v in (a, b, c, d))
    bias = np.zeros(E, np.float32)
    bias[:per] = -4 * abs(B)
    bias[0], bias[1] = B, -B
    return logits.astype(np.float32), bias


def _fp32_first_group_wins(logits, bias, per, score):
    s = np.stack([scored.scores(l, score)[1] for l in logits]).astype(np.float32)
    c = s + bias                                       # rounded to fp32
    return c[:, 0] + c[:, 1] > c[:, per] + c[:, per + 1]


# whole lanes of 16 experts, 4 and 8 per lane in groups of two lanes; groups of 20, 5 and 12 experts; more groups
# than fill a wave's lanes with whole lanes each
FORMS = [(256, 16), (64, 8), (128, 8), (160, 8), (40, 8), (96, 8), (256, 32)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("B,gap", [(64.0, 3.5e-6), (1000.0, 1e-5), (-5000.0, 2e-4)])
@pytest.mark.parametrize("E,n_group", FORMS)
@pytest.mark.parametrize("T", [64, 700])
def test_groups_whose_best_two_cancel(T, E, n_group, B, gap, score):
    from expert_ffn_layer_top_amd import ops
    logits, bias = _cancelling(T, E, n_group, B, gap, score, 1)
    kw = dict(score=score, n_group=n_group, topk_group=1, group_top=2)
    idx, _, _ = scored.route(logits, 3, bias=bias, **kw)
    first = idx.min(axis=1) < E // n_group
    wrong = first != _fp32_first_group_wins(logits, bias, E // n_group, score)
    assert wrong.any()                                 # fp32 values alone would choose otherwise
    note(f"route_scored cancelling groups T={T} E={E} n_group={n_group} B={B} {score}")
    out = ops.route_scored(f32_to_dev(logits), 3, bias=f32_to_dev(bias), **kw)
    bad = (host(out["topk_idx"]) != idx).any(axis=1)
    assert not bad.any(), f"{bad.sum()} of {T} tokens, {wrong.sum()} of them undecided in fp32"


@pytest.mark.parametrize("E,n_group", FORMS)
def test_group_values_past_the_largest_float(E, n_group):
    """Sums of two biases that overflow fp32 in either direction, beside absent groups."""
    from expert_ffn_layer_top_amd import ops
    rng = np.random.default_rng(E)
    T, per = 100, E // n_group
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[::7, 3 * per:4 * per] = -np.inf
    big = np.array([-3.4e38, -3.3e38, -1.7e38, 1.7e38, 3.3e38, 3.4e38, 0.0], np.float32)
    bias = rng.choice(big, E)
    bias[:per], bias[per:2 * per] = -3.3e38, -3.2e38
    for group_top in (1, 2):
        kw = dict(n_group=n_group, topk_group=2, group_top=group_top)
        idx, _, _ = scored.route(logits, 4, bias=bias, **kw)
        note(f"route_scored huge biases E={E} n_group={n_group} group_top={group_top}")
        out = ops.route_scored(f32_to_dev(logits), 4, bias=f32_to_dev(bias), **kw)
        assert np.array_equal(host(out["topk_idx"]), idx)


@pytest.mark.parametrize("beta", [0.9, 0.5, 0.05])
@pytest.mark.parametrize("E", [256, 100, 64, 5])
@pytest.mark.parametrize("T", [64, 900])
def test_softmax_scores_next_to_a_biased_one(T, E, beta):
    """One expert's softmax score and a small one with a bias of `beta`, some 2^-20 apart in 64 bits: as close as
    the errors of their fp32 values, which share the error of one sum."""
    from expert_ffn_layer_top_amd import ops
    rng = np.random.default_rng([T, E])
    logits = rng.uniform(-4.0, 0.0, (T, E))
    rest = np.exp(logits[:, 2:]).sum(axis=1)
    small = 10.0 ** rng.uniform(-5, -2, T)
    gap = rng.choice([-1.0, 1.0], T) * rng.uniform(0.5e-6, 2.5e-6, T)
    a, b = beta + small + gap, small
    total = rest / (1 - a - b)
    logits[:, 0], logits[:, 1] = np.log(a * total), np.log(b * total)
    logits = logits.astype(np.float32)
    bias = np.full(E, -4.0, np.float32)
    bias[0], bias[1] = 0.0, beta
    idx, _, _ = scored.route(logits, 2, score="softmax", bias=bias)
    assert (idx[:, 0] == 0).any() and (idx[:, 0] == 1).any() and idx.max() == 1
    note(f"route_scored softmax pairs T={T} E={E} beta={beta}")
    out = ops.route_scored(f32_to_dev(logits), 2, score="softmax", bias=f32_to_dev(bias))
    assert np.array_equal(host(out["topk_idx"]), idx)
