"""The adapters' products on inputs whose sums are exact in fp32: every result has to be the rounded 64-bit one, bit for bit.

v = x A^T is a whole number of up to 22 bits and a half: x holds -1, 0 and 1 times a power of two (large in few columns, 1 in most),
A whole numbers up to 2.  The ranks come in pairs whose v differ in the low bits alone and whose rows of B are each other's negative,
so what reaches the second result is only what v's last bits hold: a v of fewer bits than fp32 between the two products gives other numbers.
The sums of magnitudes are asserted to stay below 2^24 wherever an order of summation could meet them.
"""

import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, bits, dev, f32_to_dev, i32_to_dev, note
from oracle import adapter as oracle
from oracle import codecs, dropout

pytestmark = pytest.mark.gpu

SEED, OFFSET = 5, 9


def ops():
    from expert_ffn_layer_top_amd import ops
    return ops


def digits(g, n, K):
    """[n, K]: rows in pairs that differ in the columns of weight 1 alone."""
    c = np.arange(K)
    weight = np.where(c % 32 == 5, 2.0 ** np.floor(np.log2(2 ** 22 / (2 * (K // 32)))), np.where(c % 32 == 11, 64.0, 1.0))
    x = g.integers(-1, 2, (n, K)) * weight
    x[1::2] = np.where(weight > 1, x[:n - n % 2:2][:n // 2], x[1::2])
    return x


def paired(g, L, E, R, K, signs):
    """signs: rows 2i and 2i + 1 are each other's negative; else they differ in the columns of weight 1 alone."""
    if signs:
        w = g.choice([-1.0, 1.0], (L, E, R, K))
        w[:, :, 1::2] = -w[:, :, ::2]
        return w
    w = g.integers(-2, 3, (L, E, R, K)).astype(np.float64)
    c = np.arange(K) % 32
    w[:, :, 1::2] = np.where((c == 5) | (c == 11), w[:, :, ::2], w[:, :, 1::2])
    return w


def make(n, E, L, d, f, r):
    """Row r is token r; neighbours (2i, 2i + 1) have the same expert and adapter."""
    g = np.random.default_rng([n, E, L, d, f, r])
    c = dict(n=n, E=E, L=L, d=d, f=f, r=r)
    cut = 2 * np.sort(g.integers(0, n // 2 + 1, E - 1))
    c["off"] = np.concatenate([[0], cut, [n]]).astype(np.int32)
    c["ids"] = np.repeat(g.integers(-1 if L > 1 else 0, L, n // 2), 2).astype(np.int32)
    c["e"], c["l"] = oracle.row_groups(c["ids"], c["off"], None, n, L)
    # +-1 in two neighbouring rows of every 32 of a group, other ones in other columns
    rank = np.zeros(n, dtype=np.int64)
    key = c["e"] * (L + 1) + c["l"]
    for q in np.unique(key):
        rank[key == q] = np.arange((key == q).sum())
    pick = lambda cols: np.where((rank[:, None] // 2 % 16 == np.arange(cols) % 16), 1.0 - 2.0 * (rank[:, None] % 2), 0.0)   # noqa: E731
    small = lambda *shape: g.integers(-8, 9, shape).astype(np.float64)                                                     # noqa: E731
    values = dict(x=digits(g, n, d), xa=digits(g, n, f), dy=digits(g, n, d), hg=digits(g, n, f), hu=digits(g, n, f),
                  pd=pick(d), pf=pick(f), nd=small(n, d), nf=small(n, f), nf2=small(n, f), v1=small(n, 2 * r), v2=small(n, r),
                  g=np.full((n, f), 64.0), u=g.choice([1.0, 2.0], (n, f)))
    for name, R, C in (("a_gu", 2 * r, d), ("b_gate", r, f), ("b_up", r, f), ("a_down", r, f), ("b_down", r, d)):
        values["up_" + name], values["pm_" + name] = paired(g, L, E, R, C, False), paired(g, L, E, R, C, True)
    for name, v in values.items():
        b = codecs.f64_to_bf16(v)
        assert np.array_equal(codecs.bf16_to_f64(b), v), name
        c[name], c["t_" + name] = v, bf16_to_dev(b)
    c["scale"] = g.choice([0.5, 1.0], L).astype(np.float32)
    c["t_scale"] = f32_to_dev(c["scale"])
    c["s"] = np.where(c["l"] >= 0, c["scale"].astype(np.float64)[c["l"]], 0.0)[:, None]
    return c


def drop_of(p, site):
    return ops().Dropout(p, torch.tensor([SEED, OFFSET], device=dev()), site) if p else None


def mask(c, p, site, cols):
    return dropout.factors(SEED, OFFSET, site, c["n"], cols, p) if p else 1.0


def is_rounded(out, want, what):
    got, want = codecs.bf16_to_f64(bits(out)), codecs.bf16_to_f64(codecs.f64_to_bf16(want))
    bad = got != want
    assert not bad.any(), (what, int(bad.sum()), bad.size, got[bad][:4].tolist(), want[bad][:4].tolist())


def shrink(c, x, w, m=1.0):
    v, mag = oracle.shrink(x, w, c["e"], c["l"], m)
    assert mag.max(initial=0) < 2 ** 24 and np.array_equal(v, np.rint(v))
    return v


def expand(c, v, w, scale=None):
    return oracle.expand(v, w, c["e"], c["l"], scale)[0]


# (n, E, L, d, f, r): both products in one kernel by 16, 32 and 64 rows, few rows, two kernels, K in one slice and in several; what the
# 16 bits of two bf16 values lack is there in each (asserted)
SIZES = [(2, 1, 1, 64, 64, 8), (96, 2, 1, 2112, 1344, 64), (96, 2, 2, 1344, 2112, 16), (130, 3, 2, 192, 320, 40), (700, 4, 3, 64, 192, 24),
         (5000, 4, 3, 64, 64, 16), (9000, 2, 3, 64, 64, 32), (600, 16, 16, 64, 64, 8), (17000, 1, 1, 64, 64, 32)]


def lacks(v):
    """Whether two bf16 values are not enough for all of v."""
    hi = codecs.bf16_to_f64(codecs.f64_to_bf16(v))
    return not np.array_equal(hi + codecs.bf16_to_f64(codecs.f64_to_bf16(v - hi)), v)


@pytest.mark.parametrize("p", [0.0, 0.5], ids=["plain", "dropout"])
@pytest.mark.parametrize("n,E,L,d,f,r,sort", [(*size, sort) for size in SIZES for sort in (False, True) if sort or size[0] <= 512])
def test_forward(n, E, L, d, f, r, sort, p):
    note(f"adapter exact forward {n} {E} {L} {d} {f} {r} sorted={sort} p={p}")
    c = make(n, E, L, d, f, r)
    plan = ops().adapter_plan(i32_to_dev(c["ids"]), i32_to_dev(c["off"]), L, backward=sort)
    v = shrink(c, c["x"], c["up_a_gu"], mask(c, p, 1, d))
    assert n < 8 or lacks(v)
    g, u, _, v1 = ops().adapter_gate_up(c["t_x"], c["t_nf"], c["t_nf2"], c["t_nf"], plan, c["t_up_a_gu"], c["t_pm_b_gate"],
                                        c["t_pm_b_up"], c["t_scale"], drop=drop_of(p, 1), want_v=True)
    is_rounded(v1, v, "v1")
    is_rounded(g, c["nf"] + expand(c, v[:, :r], c["pm_b_gate"], c["scale"]), "g")
    is_rounded(u, c["nf2"] + expand(c, v[:, r:], c["pm_b_up"], c["scale"]), "u")
    v = shrink(c, c["xa"], c["up_a_down"], mask(c, p, 2, f))
    y, v2 = ops().adapter_down(c["t_xa"], c["t_nd"], plan, c["t_up_a_down"], c["t_pm_b_down"], c["t_scale"], drop=drop_of(p, 2),
                               want_v=True)
    is_rounded(v2, v, "v2")
    is_rounded(y, c["nd"] + expand(c, v, c["pm_b_down"], c["scale"]), "y")
    y2, _ = ops().adapter_down(c["t_xa"], c["t_nd"], plan, c["t_up_a_down"], c["t_pm_b_down"], c["t_scale"], drop=drop_of(p, 2))
    assert torch.equal(y, y2)


def wgrad(c, dv, y, shape):
    """Within 32 rows one pair of rows counts in a column: the sums that can be met stay below 2^24."""
    out, _ = oracle.wgrad(dv, y, c["e"], c["l"], shape)
    assert np.abs(dv).max() < 2 ** 23 and np.abs(out).max() < 2 ** 22
    return out


@pytest.mark.parametrize("p", [0.0, 0.5], ids=["plain", "dropout"])
@pytest.mark.parametrize("n,E,L,d,f,r", SIZES)
def test_backward(n, E, L, d, f, r, p):
    """Where g is 64 its logistic function is 1, so dg' = dg + da u and du' = du + 64 da.  With dropout the rows of a pair no longer
    cancel in A's gradients, which are left to the plain case."""
    note(f"adapter exact backward {n} {E} {L} {d} {f} {r} p={p}")
    c = make(n, E, L, d, f, r)
    plan = ops().adapter_plan(i32_to_dev(c["ids"]), i32_to_dev(c["off"]), L, backward=True)
    dv = c["s"] * shrink(c, c["dy"], c["up_b_down"])
    assert n < 8 or lacks(dv)
    dg, du, d_a, _ = ops().adapter_down_bwd(c["t_dy"], c["t_pf"], c["t_v2"], c["t_g"], c["t_u"], c["t_nf"], c["t_nf2"], plan,
                                            c["t_pm_a_down"], c["t_up_b_down"], c["t_scale"], drop=drop_of(p, 2))
    da = mask(c, p, 2, f) * expand(c, dv, c["pm_a_down"])
    is_rounded(dg, c["nf"] + da * c["u"], "dg")
    is_rounded(du, c["nf2"] + da * 64, "du")
    if p == 0:
        is_rounded(d_a, wgrad(c, dv, c["pf"], c["pm_a_down"].shape), "d_a_down")
    dv = c["s"] * np.concatenate([shrink(c, c["hg"], c["up_b_gate"]), shrink(c, c["hu"], c["up_b_up"])], axis=1)
    dxp, d_a, _, _ = ops().adapter_gate_up_bwd(c["t_hg"], c["t_hu"], c["t_pd"], c["t_v1"], c["t_nd"], plan, c["t_pm_a_gu"],
                                               c["t_up_b_gate"], c["t_up_b_up"], c["t_scale"], drop=drop_of(p, 1))
    is_rounded(dxp, c["nd"] + mask(c, p, 1, d) * expand(c, dv, c["pm_a_gu"]), "dxp")
    if p == 0:
        is_rounded(d_a, wgrad(c, dv, c["pd"], c["pm_a_gu"].shape), "d_a_gu")
