"""Dropout without a stored mask against 64 bits: rows, the combined output with the residual, its gradient.

Tolerances, element by element: an fp32 sum of k products and the factor is off by at most (k + 3) 2^-24 of the sum of
magnitudes (each product, addition and the factor's own rounding), the result is rounded once more: bf16 by 2^-8 of it.
"""

import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, bits, dev, f32_to_dev, host, i32_to_dev, note
from oracle import codecs, dropout as oracle

pytestmark = pytest.mark.gpu

SEEDS = [(0, 0), (-1, 1 << 40), (1234567890123456789, -5)]


def ops():
    from expert_ffn_layer_top_amd import ops
    return ops


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device=dev())


def bf16(g, *shape):
    b = codecs.f64_to_bf16(g.standard_normal(shape))
    return b, codecs.bf16_to_f64(b)


def within(out, ref, tol, what):
    bad = np.abs(out - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), np.max(np.abs(out - ref) - tol))


def routing(g, T, k, E):
    idx = np.stack([g.permutation(E)[:k] for _ in range(T)]).reshape(-1)
    order = np.argsort(idx, kind="stable")
    dest = np.empty(T * k, dtype=np.int32)
    dest[order] = np.arange(T * k)
    return dest.reshape(T, k), g.random((T, k), dtype=np.float32)


@pytest.mark.parametrize("T,d,p,site,res", [(1, 64, 0.5, 0, False), (1, 64, 0.1, 15, True), (7, 192, 0.3, 1, True),
                                            (130, 640, 0.05, 0, False), (33, 2112, 1 - 2.0 ** -16, 2, True),
                                            (65, 128, 0.0, 0, True), (5, 8256, 2.0 ** -16, 3, False)])
def test_rows(T, d, p, site, res):
    note(f"dropout rows T={T} d={d} p={p}")
    for seed, offset in SEEDS:
        g = np.random.default_rng([T, d])
        xb, x = bf16(g, T, d)
        rb, r = bf16(g, T, d)
        y = ops().dropout(bf16_to_dev(xb), ops().Dropout(p, rng_of(seed, offset), site),
                          residual=bf16_to_dev(rb) if res else None)
        got = codecs.bf16_to_f64(bits(y))
        m = oracle.factors(seed, offset, site, T, d, p)
        ref = x * m + (r if res else 0.0)
        within(got, ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * (np.abs(x * m) + np.abs(r)), "y")
        if not res:
            assert np.array_equal(got == 0, (m == 0) | (x == 0))


@pytest.mark.parametrize("T,k,E,d,p,res", [(1, 1, 1, 64, 0.5, True), (5, 3, 7, 192, 0.1, False), (67, 4, 8, 640, 0.2, True),
                                           (31, 8, 16, 2112, 0.1, True), (9, 16, 16, 128, 0.4, False),
                                           (40, 2, 8, 320, 0.0, True)])
def test_combine_and_its_gradient(T, k, E, d, p, res):
    note(f"dropout combine T={T} k={k} d={d} p={p}")
    g = np.random.default_rng([T, k, d])
    dest, gate = routing(g, T, k, E)
    (yb, y), (rb, r), (db, dy) = bf16(g, T * k, d), bf16(g, T, d), bf16(g, T, d)
    seed, offset = SEEDS[2]
    drop = ops().Dropout(p, rng_of(seed, offset), 4)
    m = oracle.factors(seed, offset, 4, T, d, p)
    args = (bf16_to_dev(yb), f32_to_dev(gate), i32_to_dev(dest))
    out = ops().unpermute_combine_dropout(*args, drop, residual=bf16_to_dev(rb) if res else None)
    g64 = gate.astype(np.float64)[:, :, None]
    ref = m * (g64 * y[dest]).sum(1) + (r if res else 0.0)
    mag = m * np.abs(g64 * y[dest]).sum(1) + np.abs(r)
    within(codecs.bf16_to_f64(bits(out)), ref, 2.0 ** -8 * np.abs(ref) + (k + 3) * 2.0 ** -23 * mag, "y")
    dyexp, d_gate = ops().unpermute_combine_dropout_bwd(bf16_to_dev(db), *args, drop)
    want = np.empty_like(y)
    want[dest.reshape(-1)] = (g64 * (m * dy)[:, None]).reshape(T * k, d)
    within(codecs.bf16_to_f64(bits(dyexp)), want, (2.0 ** -8 + 2.0 ** -22) * np.abs(want), "dyexp")
    dots, mags = (m * dy)[:, None] * y[dest], np.abs((m * dy)[:, None] * y[dest])
    within(host(d_gate).astype(np.float64), dots.sum(2), (d + 3) * 2.0 ** -24 * mags.sum(2), "d_gate")
    if p == 0.0 and not res:
        return
    if p == 0.0:          # without dropout and residual: the calls that were there, bit for bit
        plain = ops().unpermute_combine_dropout(*args, drop)
        assert torch.equal(plain, ops().unpermute_combine(*args))
        for a, b in zip((dyexp, d_gate), ops().unpermute_combine_bwd(bf16_to_dev(db), *args)):
            assert torch.equal(a, b)


def test_no_dropout_reads_no_generator():
    """drop = None hands the library a null rng: the sums alone, with and without the residual."""
    note("dropout without a generator")
    g = np.random.default_rng(3)
    T, k, d = 21, 3, 320
    dest, gate = routing(g, T, k, 4)
    y, dy, res = (bf16_to_dev(bf16(g, n, d)[0]) for n in (T * k, T, T))
    args = (y, f32_to_dev(gate), i32_to_dev(dest))
    assert torch.equal(ops().unpermute_combine_dropout(*args, None), ops().unpermute_combine(*args))
    for a, b in zip(ops().unpermute_combine_dropout_bwd(dy, *args, None), ops().unpermute_combine_bwd(dy, *args)):
        assert torch.equal(a, b)
    assert torch.equal(ops().dropout(dy, None), dy)
    assert torch.equal(ops().dropout(dy, None, residual=res), (dy.float() + res.float()).to(torch.bfloat16))


def test_what_is_dropped_is_zero_whatever_it_was():
    note("dropout of infinities and NaN")
    T, d, p = 16, 256, 0.5
    x = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device=dev())
    x[:, ::2] = float("inf")
    y = ops().dropout(x, ops().Dropout(p, rng_of(3, 4), 0)).float().cpu().numpy()
    kept = oracle.factors(3, 4, 0, T, d, p) != 0
    assert np.all(y[~kept] == 0)
    assert np.all(np.isinf(y[:, ::2][kept[:, ::2]])) and np.all(np.isnan(y[:, 1::2][kept[:, 1::2]]))


def test_rows_whose_offsets_pass_32_bits():
    """T d 2 bytes > 2^32: the last rows are those of their own numbers."""
    note("dropout of more than 4 GiB")
    T, d, p = 263000, 8256, 0.25
    x = torch.ones((T, d), dtype=torch.bfloat16, device=dev())
    y = ops().dropout(x, ops().Dropout(p, rng_of(11, 12), 0))
    last = y[-3:].float().cpu().numpy()
    w = oracle.philox([np.repeat([np.arange(d // 8, dtype=np.uint64)], 3, 0),
                       np.repeat(np.arange(T - 3, T, dtype=np.uint64)[:, None], d // 8, 1),
                       np.full((3, d // 8), 12, dtype=np.uint64), np.zeros((3, d // 8), dtype=np.uint64)], (11, 0), 7)
    u = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], axis=2).reshape(3, d)
    assert np.array_equal(last != 0, u >= 16384)


def test_replayed_graph_draws_anew_where_the_program_advances_the_offset():
    note("dropout captured and replayed")
    g = np.random.default_rng(0)
    xb, x = bf16(g, 40, 320)
    t, rng = bf16_to_dev(xb), rng_of(9, 100)
    drop = ops().Dropout(0.3, rng, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops().dropout(t, drop)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops().dropout(t, drop)
    seen = []
    for i in range(3):
        rng[1] = 100 + i
        graph.replay()
        torch.cuda.synchronize()
        m = oracle.factors(9, 100 + i, 0, 40, 320, 0.3)
        got = codecs.bf16_to_f64(bits(y))
        within(got, x * m, (2.0 ** -8 + 2.0 ** -22) * np.abs(x * m), i)
        assert torch.equal(y, ops().dropout(t, drop))
        seen.append(got)
    assert not np.array_equal(seen[0], seen[1]) and not np.array_equal(seen[1], seen[2])
