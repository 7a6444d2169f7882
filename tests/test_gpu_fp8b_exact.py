"""Exact block sums of the products of few rows whose results are quantised again (G, U, dG, dU).

The operands are codes made by hand: in every aligned group of 8 along the contraction +448 * 448 and -448 * 448
cancel beside one small product.  The exact sum is that of the small ones; the fp8 matrix core, which cuts every
product of a group to a multiple of 2^4 beside 448 * 448, loses a 7 and makes 8 of a 15.  All sums are small whole
numbers and the scales powers of two, so the expected values are exact up to the one rounding to bf16.
"""

import numpy as np
import pytest
import torch

from gpu_util import bits, dev, f32_to_dev, i32_to_dev, note
from oracle import codecs

pytestmark = pytest.mark.gpu

BIG, ONE = 448.0, 1.0


def _codes(values):
    return torch.from_numpy(codecs.e4m3_encode_rne_sat(values)).to(dev())


def _operands(rng, n, counts, K, cols, small):
    """(x codes, x scales, w codes, w scales, the exact product [n, cols]) of rows dealt to len(counts) experts."""
    E = len(counts)
    x, w = np.zeros((n, K)), np.zeros((E, cols, K))
    place = np.argsort(rng.random((K // 8, 8)), axis=1)[:, :3] + 8 * np.arange(K // 8)[:, None]
    x[:, place[:, :2]] = BIG
    x[:, place[:, 2]] = small * rng.choice([-1.0, 1.0], (n, K // 8))
    sign = rng.choice([-1.0, 1.0], (E, cols, K // 8))
    w[:, :, place[:, 0]], w[:, :, place[:, 1]] = BIG * sign, -BIG * sign
    w[:, :, place[:, 2]] = ONE
    blocks = -(-K // 128)
    xs = np.exp2(rng.integers(-3, 4, (1, n))) * np.ones((blocks, 1))
    ws = np.exp2(rng.integers(-3, 4, (E, 1, 1))) * np.ones((1, -(-cols // 128), blocks))
    expert = np.repeat(np.arange(E), counts)
    exact = x[:, place[:, 2]].sum(axis=1)[:, None] * xs[0][:, None] * ws[expert, 0, 0][:, None] * np.ones((1, cols))
    return _codes(x), f32_to_dev(xs), _codes(w), f32_to_dev(ws), exact


CASES = [([5], 128, 64), ([1, 0, 2], 192, 320), ([40], 128, 192), ([70, 0, 3], 320, 64), ([130], 1024, 128)]


@pytest.mark.parametrize("form", ["", "few", "mid", "half", "big"])
@pytest.mark.parametrize("small", [7.0, 15.0])
@pytest.mark.parametrize("counts,d,f", CASES, ids=[f"{sum(c)}-{d}-{f}" for c, d, f in CASES])
def test_cancelling_products(counts, d, f, small, form, monkeypatch):
    """The library's choice and the two kernels that have exact sums give them; the two that have none, on the same
    operands, do not: a control, without which the operands might not tell the difference."""
    from expert_ffn_layer_top_amd import ops
    if form:
        monkeypatch.setenv("MOE_FP8B_FORM", form)
    rng = np.random.default_rng([d, f, int(small)])
    n, E = sum(counts), len(counts)
    off = i32_to_dev(np.concatenate([[0], np.cumsum(counts)]))
    xq, xs, wq, ws, exact = _operands(rng, n, counts, d, f, small)
    wu, wus = wq.flip(1).contiguous(), ws * 2.0
    note(f"fp8b cancelling products {form} n={n} E={E} d={d} f={f}")
    g, u, _ = ops.grouped_gemm_gate_up_fp8b(xq, xs, off, wq, ws, wu, wus)
    # silu(64) is 64 and its derivative 1 in fp32
    gb = torch.full((n, f), 64.0, device=dev()).bfloat16()
    dg, du = ops.grouped_gemm_dgrad_down_fp8b(xq, xs, off, wq, ws, gb, torch.ones_like(gb))
    for what, got, want in (("g", g, exact), ("u", u, 2 * exact), ("dg", dg, exact), ("du", du, 64 * exact)):
        same = bits(got) == codecs.f64_to_bf16(want)
        zero = (want == 0) & (bits(got) & 0x7fff == 0)
        assert (same | zero).all() if form not in ("half", "big") else not (same | zero).all(), what


def test_an_unknown_form_is_refused(monkeypatch):
    from expert_ffn_layer_top_amd import _lib, ops
    monkeypatch.setenv("MOE_FP8B_FORM", "small")
    z = torch.zeros(4, 64, dtype=torch.uint8, device=dev())
    s = f32_to_dev(np.ones((1, 4)))
    w, ws = torch.zeros(1, 64, 64, dtype=torch.uint8, device=dev()), f32_to_dev(np.ones((1, 1, 1)))
    with pytest.raises(_lib.MoeError, match="MOE_FP8B_FORM"):
        ops.grouped_gemm_down_fp8b(z, s, i32_to_dev([0, 4]), w, ws)


@pytest.mark.parametrize("form", ["mid", "half", "big"])
@pytest.mark.parametrize("counts,d,f", [([700, 3, 0, 321], 192, 320), ([2050], 320, 64)], ids=["1024", "2050"])
def test_products_of_many_blocks_in_every_form(counts, d, f, form, monkeypatch):
    """... of 2048 result blocks and more, where the 64-row tiles run on the fp8 core too."""
    from expert_ffn_layer_top_amd import ops
    from oracle import fp8b, moe
    from test_gpu_fp8b import Case, assert_bf16, silu_slack, sum_tol
    monkeypatch.setenv("MOE_FP8B_FORM", form)
    c = Case(counts, d, f, seed=8)
    x, xv = c.rows(d)
    (wg, wgv), (wu, wuv) = c.weight(f, d), c.weight(f, d)
    note(f"fp8b many blocks {form} n={c.n} d={d} f={f}")
    g, u, a = ops.grouped_gemm_gate_up_fp8b(*x, c.offsets, *wg, *wu)
    gr, gs, lgs = fp8b.grouped_nt(xv, wgv, c.off)
    ur, us, lus = fp8b.grouped_nt(xv, wuv, c.off)
    eg, eu = sum_tol(gs, lgs, d), sum_tol(us, lus, d)
    assert_bf16(g, gr, eg, "g")
    assert_bf16(u, ur, eu, "u")
    assert_bf16(a, moe.silu(gr) * ur, silu_slack(gr, ur, eg, eu), "a")
    gb, gv = c.bf16(f)
    ub, uv = c.bf16(f)
    dg, du = ops.grouped_gemm_dgrad_down_fp8b(*x, c.offsets, *wg, gb, ub)
    s = 1 / (1 + np.exp(-gv))
    kg, ku = uv * s * (1 + gv * (1 - s)), gv * s
    assert_bf16(dg, gr * kg, eg * np.abs(kg) + 16 * 2.0 ** -24 * np.abs(gr * uv) * (1 + np.abs(gv)), "dg")
    assert_bf16(du, gr * ku, eg * np.abs(ku) + 16 * 2.0 ** -24 * np.abs(gr * gv), "du")
