"""Pins of the adapters' and the dropout's oracle: published vectors of the generator, dense products for one adapter,
gradients against differences."""

import numpy as np
import pytest

from oracle import adapter, dropout


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_against_its_published_vectors(counter, key, want):
    """Ten rounds; the rounds themselves are the same for any number."""
    got = dropout.philox([np.array([c], dtype=np.uint64) for c in counter], key, 10)
    assert tuple(int(w[0]) for w in got) == want


def test_factors_share_mean_and_independence():
    """The share of zeros is p within 5 standard deviations, their mean factor 1 likewise; other sites, offsets and
    seeds agree no more often than chance."""
    n, p = 512 * 512, 0.3
    f = dropout.factors(5, 7, 0, 512, 512, p)
    dev = np.sqrt(p * (1 - p) / n)
    assert abs(np.mean(f == 0) - p) < 5 * dev + 2.0 ** -16
    assert abs(f.mean() - 1.0) < 5 * dev / (1 - p) + 1e-12
    for other in ((5, 7, 1), (5, 8, 0), (6, 7, 0), (5, 7 + (1 << 32), 0), (5 + (1 << 32), 7, 0)):
        h = dropout.factors(*other, 512, 512, p)
        both = np.mean((f == 0) & (h == 0))
        assert abs(both - p * p) < 5 * np.sqrt(p * p * (1 - p * p) / n) + 2.0 ** -15
    # rows and columns: neighbours agree no more often than chance either
    for a, b in ((f[1:], f[:-1]), (f[:, 1:], f[:, :-1])):
        assert abs(np.mean((a == 0) & (b == 0)) - p * p) < 6 * np.sqrt(p * p * (1 - p * p) / n) + 2.0 ** -15


def test_factors_of_no_dropout_and_of_the_largest():
    assert np.all(dropout.factors(1, 2, 0, 4, 24, 0.0) == 1.0)
    f = dropout.factors(1, 2, 0, 64, 1024, 1 - 2.0 ** -16)
    assert set(np.unique(f)) <= {0.0, 65536.0}


def case(seed=0, T=6, E=3, L=2, d=8, f=6, r=2):
    g = np.random.default_rng(seed)
    n = 2 * T
    tok = np.concatenate([np.sort(g.permutation(T)[:k]) for k in (5, 0, 7 - 2)] + [g.integers(0, T, 2)])[:n]
    n = len(tok)
    off = np.array([0, 5, 5, n])
    ids = np.array([0, 1, -1, 0, 5, 1])[:T]
    e, l = adapter.row_groups(ids, off, tok, n, L)
    z = lambda *s: g.standard_normal(s)                                          # noqa: E731
    w = dict(a_gu=z(L, E, 2 * r, d), b_gate=z(L, E, r, f), b_up=z(L, E, r, f), a_down=z(L, E, r, f), b_down=z(L, E, r, d))
    return dict(n=n, e=e, l=l, x=z(n, d), g=z(n, f), u=z(n, f), y=z(n, d), w=w, scale=g.random(L) + 0.5,
                m1=(g.random((n, d)) > 0.3) / 0.7, m2=(g.random((n, f)) > 0.3) / 0.7, dy=z(n, d))


def test_rows_without_an_adapter_and_numbers_out_of_range():
    c = case()
    out = adapter.forward(c["x"], c["g"], c["u"], *c["w"].values(), c["y"], c["scale"], c["e"], c["l"])
    none = c["l"] < 0
    assert none.any() and (~none).any()
    for name in ("g", "u", "y"):
        assert np.array_equal(out[name][none], c[name][none])
    assert np.all(out["v1"][none] == 0) and np.all(out["v2"][none] == 0)


def test_one_adapter_of_one_expert_is_the_dense_product():
    g = np.random.default_rng(1)
    x, w = g.standard_normal((5, 8)), g.standard_normal((1, 1, 3, 8))
    zero = np.zeros(5, dtype=int)
    v, _ = adapter.shrink(x, w, zero, zero)
    assert np.allclose(v, x @ w[0, 0].T, rtol=1e-13)
    assert np.allclose(adapter.expand(v, w, zero, zero, [2.0])[0], 2 * v @ w[0, 0], rtol=1e-13)
    assert np.allclose(adapter.wgrad(v, x, zero, zero, w.shape)[0][0, 0], v.T @ x, rtol=1e-12)


@pytest.mark.parametrize("dropped", [False, True])
def test_gradients_against_differences(dropped):
    """d (sum of y dy) by each matrix and each input, central differences with a step of 1e-6: off by about 1e-12 / 1e-6 of
    rounding and 1e-12 of the third derivative; 1e-6 of the largest is asked."""
    c = case(2)
    m1, m2 = (c["m1"], c["m2"]) if dropped else (1.0, 1.0)

    def value(x, g, u, y, w):
        return np.sum(adapter.forward(x, g, u, *w.values(), y, c["scale"], c["e"], c["l"], m1, m2)["y"] * c["dy"])

    out = adapter.forward(c["x"], c["g"], c["u"], *c["w"].values(), c["y"], c["scale"], c["e"], c["l"], m1, m2)
    w, has = c["w"], c["l"] >= 0
    da, d_a, d_b = adapter.down_backward(c["dy"], out["a"], out["v2"], w["a_down"], w["b_down"], c["scale"], c["e"], c["l"], m2)
    s = adapter.sigmoid(out["g"])
    dg, du = da * out["u"] * s * (1 + out["g"] * (1 - s)), da * out["g"] * s
    dx, d_agu, d_bg, d_bu = adapter.gate_up_backward(dg, du, c["x"], out["v1"], w["a_gu"], w["b_gate"], w["b_up"], c["scale"],
                                                     c["e"], c["l"], m1)
    got = dict(x=dx, g=dg, u=du, y=c["dy"], a_gu=d_agu, b_gate=d_bg, b_up=d_bu, a_down=d_a, b_down=d_b)
    args = dict(x=c["x"], g=c["g"], u=c["u"], y=c["y"])
    for name, grad in got.items():
        src = args[name] if name in args else w[name]
        num = np.zeros_like(src)
        for i in np.ndindex(src.shape):
            old = src[i]
            src[i] = old + 1e-6
            hi = value(**args, w=w)
            src[i] = old - 1e-6
            lo = value(**args, w=w)
            src[i] = old
            num[i] = (hi - lo) / 2e-6
        if name in ("g", "u"):
            num, grad = num[has], grad[has]      # without an adapter nothing else of the value depends on them
        assert np.max(np.abs(num - grad)) <= 1e-6 * max(1.0, np.max(np.abs(grad))), name
