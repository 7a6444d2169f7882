"""The adapters' products against 64 bits, each step on the GPU's own inputs to it.

Tolerances, element by element.  A sum of N products of bf16 values in fp32 is off by at most N 2^-23 of the sum of
magnitudes, in any order (each of up to N additions by 2^-24, and as much again for the way the matrix core aligns
its terms); a result in bf16 by 2^-8 of it (half a step).  v and dv are held as two bf16 values between their two products,
off by at most 2^-16 (what the first lacks is at most 2^-8 of it, and is rounded by 2^-8 of that), and their error counts
with the magnitudes that it meets in the second product.  The logistic function in fp32 is
good to 2^-18 (exp of up to |x| < 32: |x| 2^-24 from its argument, and about 2 ulp each for exp and the reciprocal).
"""

import numpy as np
import pytest
import torch

from gpu_util import bf16_to_dev, bits, dev, f32_to_dev, i32_to_dev, note
from oracle import adapter as oracle
from oracle import codecs, dropout

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
V = 2.0 ** -16
SEED, OFFSET = 77, 1 << 33


def ops():
    from expert_ffn_layer_top_amd import ops
    return ops


def val(t):
    return codecs.bf16_to_f64(bits(t))


def within(out, ref, tol, what):
    assert out.shape == ref.shape, (what, out.shape, ref.shape)
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), np.max(np.abs(out - ref) - tol))


def make(seed, T, k, E, L, d, f, r, ids="mixed", spread=True):
    """Inputs of a random routing; bf16 tensors as (device tensor, values)."""
    g = np.random.default_rng([seed, T, k, E, L, d, f, r])
    n = T * k
    weight = g.random(E) ** 3 if spread else np.ones(E)
    idx = np.stack([np.argsort(-weight * g.random(E), kind="stable")[:k] for _ in range(T)]).reshape(-1)
    order = np.argsort(idx, kind="stable")
    c = dict(T=T, k=k, n=n, E=E, L=L, d=d, f=f, r=r)
    c["token"] = (order // k).astype(np.int32)
    c["off"] = np.concatenate([[0], np.cumsum(np.bincount(idx, minlength=E))]).astype(np.int32)
    c["ids"] = {"mixed": g.integers(-1, L, T), "none": np.full(T, -1), "one": np.full(T, L - 1),
                "outside": g.choice([-7, 0, L - 1, L, L + 3, 2 ** 31 - 1, -2 ** 31], T)}[ids].astype(np.int32)

    def t(*shape, std=1.0):
        b = codecs.f64_to_bf16(g.standard_normal(shape) * std)
        return bf16_to_dev(b), codecs.bf16_to_f64(b)

    for name, shape, std in (("x", (T, d), 1), ("g", (n, f), 1), ("u", (n, f), 1), ("a", (n, f), 1), ("y", (n, d), 1),
                             ("dg", (n, f), 1), ("du", (n, f), 1), ("dxp", (n, d), 1),
                             ("a_gu", (L, E, 2 * r, d), d ** -0.5), ("b_gate", (L, E, r, f), r ** -0.5),
                             ("b_up", (L, E, r, f), r ** -0.5), ("a_down", (L, E, r, f), f ** -0.5),
                             ("b_down", (L, E, r, d), r ** -0.5), ("v1", (n, 2 * r), 1), ("v2", (n, r), 1)):
        c["t_" + name], c[name] = t(*shape, std=std)
    c["scale"] = (g.random(L) + 0.5).astype(np.float32)
    c["t_scale"] = f32_to_dev(c["scale"])
    c["e"], c["l"] = oracle.row_groups(c["ids"], c["off"], c["token"], n, L)
    c["s"] = np.where(c["l"] >= 0, c["scale"].astype(np.float64)[c["l"]], 0.0)[:, None]
    return c


def plan_of(c, backward):
    return ops().adapter_plan(i32_to_dev(c["ids"]), i32_to_dev(c["off"]), c["L"], row_token=i32_to_dev(c["token"]),
                              backward=backward)


def drop_of(p, site):
    return ops().Dropout(p, torch.tensor([SEED, OFFSET], device=dev()), site) if p else None


def mask(c, p, site, cols):
    return dropout.factors(SEED, OFFSET, site, c["n"], cols, p) if p else np.ones((c["n"], cols))


def check_forward(c, plan, p=0.0):
    up, down = [c["t_" + w] for w in ("a_gu", "b_gate", "b_up", "scale")], [c["t_" + w] for w in ("a_down", "b_down", "scale")]
    r, none = c["r"], c["l"] < 0
    g, u, a, v1 = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, *up, drop=drop_of(p, 1), want_v=True)
    ref, mag = oracle.shrink(c["x"][c["token"]], c["a_gu"], c["e"], c["l"], mask(c, p, 1, c["d"]))
    within(val(v1), ref, U * np.abs(ref) + c["d"] * 2.0 ** -23 * mag, "v1")
    v1_off = V * np.abs(ref) + c["d"] * 2.0 ** -23 * mag
    tol, pre = {}, {}
    for name, base, out, at in (("g", c["g"], g, slice(0, r)), ("u", c["u"], u, slice(r, None))):
        w = c["b_gate" if name == "g" else "b_up"]
        add, mag = oracle.expand(ref[:, at], w, c["e"], c["l"], c["scale"])
        _, off = oracle.expand(v1_off[:, at], w, c["e"], c["l"], c["scale"])
        pre[name], tol[name] = base + add, off + (2 * r + 4) * 2.0 ** -23 * (np.abs(base) + mag)
        within(val(out), pre[name], U * np.abs(pre[name]) + tol[name], name)
    s = oracle.sigmoid(pre["g"])
    ref = np.where(none[:, None], c["a"], pre["g"] * s * pre["u"])
    # silu has a slope of at most 1.1
    within(val(a), ref, U * np.abs(ref) + 2.0 ** -18 * np.abs(ref) + 1.2 * np.abs(pre["u"]) * tol["g"]
           + np.abs(pre["g"] * s) * tol["u"] + 1.2 * tol["g"] * tol["u"] + 1e-30, "a")
    for out, base in ((g, c["t_g"]), (u, c["t_u"]), (a, c["t_a"])):
        assert torch.equal(out[torch.from_numpy(none)], base[torch.from_numpy(none)])
    y, v2 = ops().adapter_down(a, c["t_y"], plan, *down, drop=drop_of(p, 2), want_v=True)
    ref, mag = oracle.shrink(val(a), c["a_down"], c["e"], c["l"], mask(c, p, 2, c["f"]))
    within(val(v2), ref, U * np.abs(ref) + c["f"] * 2.0 ** -23 * mag, "v2")
    v2_off = V * np.abs(ref) + c["f"] * 2.0 ** -23 * mag
    add, mag = oracle.expand(ref, c["b_down"], c["e"], c["l"], c["scale"])
    _, off = oracle.expand(v2_off, c["b_down"], c["e"], c["l"], c["scale"])
    within(val(y), c["y"] + add, (U * np.abs(c["y"] + add) + 1.01 * off + (2 * r + 4) * 2.0 ** -23 * (np.abs(c["y"]) + mag)), "y")
    assert torch.equal(y[torch.from_numpy(none)], c["t_y"][torch.from_numpy(none)])
    # a serving pass: the same a and y, bit for bit
    g2, u2, a2, w1 = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, *up, drop=drop_of(p, 1), want_gu=False)
    y2, w2 = ops().adapter_down(a2, c["t_y"], plan, *down, drop=drop_of(p, 2))
    assert g2 is u2 is w1 is w2 is None and torch.equal(a, a2) and torch.equal(y, y2)


def check_wgrad(out, v, y, c, shape, scale, what):
    ref, mag = oracle.wgrad(v, y, c["e"], c["l"], shape, scale)
    rows = max(1, int(np.max(np.bincount(c["e"][c["l"] >= 0], minlength=1), initial=1)))
    within(val(out), ref, U * np.abs(ref) + (1 + U) * (rows + 4) * 2.0 ** -23 * mag, what)


def check_backward(c, plan, p=0.0):
    up, down = [c["t_" + w] for w in ("a_gu", "b_gate", "b_up", "scale")], [c["t_" + w] for w in ("a_down", "b_down", "scale")]
    e, l, r, d, f = c["e"], c["l"], c["r"], c["d"], c["f"]
    none = torch.from_numpy(l < 0)
    m1, m2 = mask(c, p, 1, d), mask(c, p, 2, f)
    dg, du, d_a, d_b = ops().adapter_down_bwd(c["t_y"], c["t_a"], c["t_v2"], c["t_g"], c["t_u"], c["t_dg"], c["t_du"], plan,
                                              *down, drop=drop_of(p, 2))
    dv, mag = oracle.shrink(c["y"], c["b_down"], e, l)
    dv, mag = c["s"] * dv, c["s"] * mag
    check_wgrad(d_b, c["v2"], c["y"], c, d_b.shape, c["scale"], "d_b_down")
    dv_off = V * np.abs(dv) + (d + 2) * 2.0 ** -23 * mag
    ref, wmag = oracle.wgrad(dv, c["a"] * m2, e, l, d_a.shape)
    _, off = oracle.wgrad(dv_off, np.abs(c["a"] * m2), e, l, d_a.shape)
    rows = c["n"]
    within(val(d_a), ref, U * np.abs(ref) + (1 + U) * off + (rows + 4) * 2.0 ** -23 * 2 * wmag, "d_a_down")
    da, damag = oracle.expand(dv, c["a_down"], e, l)
    _, daoff = oracle.expand(dv_off, np.abs(c["a_down"]), e, l)
    da, daoff = m2 * da, m2 * (daoff + (2 * r + 4) * 2.0 ** -23 * damag)
    s = oracle.sigmoid(c["g"])
    for name, out, base, k in (("dg", dg, c["dg"], c["u"] * s * (1 + c["g"] * (1 - s))), ("du", du, c["du"], c["g"] * s)):
        ref = base + da * k
        slack = np.abs(c["u"]) * (1 + np.abs(c["g"])) if name == "dg" else np.abs(c["g"])
        within(val(out), ref, U * np.abs(ref) + (1 + U) * daoff * np.abs(k) + 2.0 ** -18 * (np.abs(da) * slack + np.abs(base)), name)
        assert torch.equal(out[none], c["t_" + name][none])
    hg, hu = val(dg), val(du)
    dxp, d_agu, d_bg, d_bu = ops().adapter_gate_up_bwd(dg, du, c["t_x"], c["t_v1"], c["t_dxp"], plan, *up, drop=drop_of(p, 1))
    check_wgrad(d_bg, c["v1"][:, :r], hg, c, d_bg.shape, c["scale"], "d_b_gate")
    check_wgrad(d_bu, c["v1"][:, r:], hu, c, d_bu.shape, c["scale"], "d_b_up")
    parts = [oracle.shrink(h, c[w], e, l) for h, w in ((hg, "b_gate"), (hu, "b_up"))]
    dv, mag = (c["s"] * np.concatenate([q[i] for q in parts], axis=1) for i in (0, 1))
    dv_off = V * np.abs(dv) + (f + 2) * 2.0 ** -23 * mag
    x = c["x"][c["token"]] * m1
    ref, wmag = oracle.wgrad(dv, x, e, l, d_agu.shape)
    _, off = oracle.wgrad(dv_off, np.abs(x), e, l, d_agu.shape)
    within(val(d_agu), ref, U * np.abs(ref) + (1 + U) * off + (rows + 4) * 2.0 ** -23 * 2 * wmag, "d_a_gu")
    add, mag = oracle.expand(dv, c["a_gu"], e, l)
    _, off = oracle.expand(dv_off, np.abs(c["a_gu"]), e, l)
    ref = c["dxp"] + m1 * add
    within(val(dxp), ref, U * np.abs(ref) + (1 + U) * m1 * (off + (4 * r + 4) * 2.0 ** -23 * mag) + 2.0 ** -22 * np.abs(c["dxp"]), "dxp")
    assert torch.equal(dxp[none], c["t_dxp"][none])
    # groups without rows: zeros
    empty = np.ones((c["L"], c["E"]), dtype=bool)
    empty[l[l >= 0], e[l >= 0]] = False
    for t in (d_a, d_b, d_agu, d_bg, d_bu):
        assert torch.count_nonzero(t[torch.from_numpy(empty)]) == 0


# (T, k, E, L, d, f, r, ids): one token; half a stripe of columns; odd numbers of rows, a tile and one more; every
# size of the rank's tiles; experts without rows; absent and impossible adapters; many adapters
SIZES = [(1, 1, 1, 1, 64, 64, 8, "one"), (1, 8, 16, 3, 192, 128, 16, "one"), (3, 2, 4, 2, 128, 320, 24, "mixed"),
         (65, 1, 1, 1, 64, 192, 40, "one"), (37, 3, 5, 4, 320, 64, 32, "mixed"), (64, 4, 8, 2, 192, 192, 64, "mixed"),
         (50, 2, 64, 3, 64, 128, 8, "mixed"), (33, 2, 3, 2, 128, 64, 56, "outside"), (20, 2, 3, 2, 64, 64, 16, "none"),
         (300, 1, 2, 256, 64, 64, 8, "mixed"), (129, 2, 256, 1, 64, 64, 16, "one")]


@pytest.mark.parametrize("T,k,E,L,d,f,r,ids", SIZES)
@pytest.mark.parametrize("sort", [False, True], ids=["few", "sorted"])
def test_forward(T, k, E, L, d, f, r, ids, sort):
    note(f"adapter forward {T} {k} {E} {L} {d} {f} {r} {ids} sorted={sort}")
    c = make(0, T, k, E, L, d, f, r, ids)
    check_forward(c, plan_of(c, sort))


@pytest.mark.parametrize("T,k,E,L,d,f,r,ids", SIZES)
def test_backward(T, k, E, L, d, f, r, ids):
    note(f"adapter backward {T} {k} {E} {L} {d} {f} {r} {ids}")
    c = make(1, T, k, E, L, d, f, r, ids)
    check_backward(c, plan_of(c, True))


# (T, E, L, d, f): both products in one kernel by 16, 32 and 64 rows (full tiles, tiles of few rows), with more stripes of
# columns than it has waves, and in two kernels
FORMS = [(700, 4, 3, 64, 192), (150, 1, 2, 1088, 64), (90, 2, 1, 64, 1216), (5000, 4, 3, 64, 64), (9000, 2, 3, 64, 64),
         (600, 16, 16, 64, 64), (3000, 30, 20, 64, 64), (17000, 1, 1, 64, 64)]


@pytest.mark.parametrize("r", [8, 16, 24, 32, 64])
@pytest.mark.parametrize("T,E,L,d,f", FORMS)
def test_every_form_of_the_sorted_forward(T, E, L, d, f, r):
    note(f"adapter forms {T} {E} {L} {d} {f} {r}")
    c = make(12, T, 1, E, L, d, f, r)
    check_forward(c, plan_of(c, True))


@pytest.mark.parametrize("r", [8, 16, 24, 32, 64])
def test_dropout_at_every_rank(r):
    note(f"adapter dropout r={r}")
    c = make(13, 150, 2, 3, 2, 192, 128, r)
    check_forward(c, plan_of(c, True), p=0.25)


@pytest.mark.parametrize("sort", [False, True], ids=["few", "sorted"])
def test_dropout_of_the_inputs(sort):
    note(f"adapter dropout sorted={sort}")
    c = make(2, 45, 2, 3, 2, 192, 128, 16)
    check_forward(c, plan_of(c, sort), p=0.25)
    if sort:
        check_backward(c, plan_of(c, True), p=0.25)


def test_more_rows_than_one_piece_of_a_contraction():
    """More than 512 rows of one expert and adapter: chunks of the sort, several pieces of the weight gradients, next to groups of one piece."""
    note("adapter rows in several pieces")
    c = make(3, 2100, 2, 3, 2, 64, 64, 16, "mixed")
    has = c["l"] >= 0
    assert max(np.bincount(c["e"][has] * 2 + c["l"][has])) > 512
    check_forward(c, plan_of(c, True), p=0.1)
    check_backward(c, plan_of(c, True), p=0.1)


@pytest.mark.parametrize("T,k,E,L,ids", [(70001, 1, 1, 3, "mixed"), (40000, 2, 3, 2, "outside"), (5000, 8, 64, 9, "mixed"),
                                         (66000, 1, 2, 256, "mixed")])
def test_many_rows(T, k, E, L, ids):
    """Chunks of several blocks of the sort, experts of very different size; against the definition in 64 bits on the GPU, written with
    every row's matrices gathered."""
    note(f"adapter many rows {T} {k} {E} {L} {ids}")
    d, f, r = 64, 64, 8
    c = make(10, T, k, E, L, d, f, r, ids)
    plan = plan_of(c, True)
    e, l = (torch.from_numpy(c[name]).to(dev()) for name in "el")
    has, l0 = (l >= 0)[:, None], l.clamp(min=0)
    A, B, s = c["t_a_down"].double()[l0, e], c["t_b_down"].double()[l0, e], c["t_scale"].double()[l0][:, None]
    y, v = ops().adapter_down(c["t_a"], c["t_y"], plan, c["t_a_down"], c["t_b_down"], c["t_scale"], want_v=True)
    a64 = c["t_a"].double()
    v64 = torch.where(has, (A * a64[:, None]).sum(2), 0.0)
    vmag = (A * a64[:, None]).abs().sum(2)
    assert bool(((v.double() - v64).abs() <= U * v64.abs() + f * 2.0 ** -23 * vmag).all())
    y64 = c["t_y"].double() + torch.where(has, s * (B * v64[:, :, None]).sum(1), 0.0)
    off = s * (B.abs() * (V * v64.abs() + f * 2.0 ** -23 * vmag)[:, :, None]).sum(1)
    mag = c["t_y"].double().abs() + s * (B * v64[:, :, None]).abs().sum(1)
    assert bool(((y.double() - y64).abs() <= U * y64.abs() + 1.01 * off + (2 * r + 4) * 2.0 ** -23 * mag).all())
    out = ops().adapter_down_bwd(c["t_y"], c["t_a"], c["t_v2"], c["t_g"], c["t_u"], c["t_dg"], c["t_du"], plan, c["t_a_down"],
                                 c["t_b_down"], c["t_scale"])
    key = (l0 * E + e)[has[:, 0]]
    part = (s * c["t_v2"].double())[has[:, 0]][:, :, None] * c["t_y"].double()[has[:, 0]][:, None]
    want = torch.zeros((L * E, r, d), dtype=torch.float64, device=dev()).index_add_(0, key, part).view(L, E, r, d)
    size = torch.zeros((L * E, r, d), dtype=torch.float64, device=dev()).index_add_(0, key, part.abs()).view(L, E, r, d)
    rows = int(torch.bincount(key).max())
    assert bool(((out[3].double() - want).abs() <= U * want.abs() + (1 + U) * (rows + 4) * 2.0 ** -23 * size).all())
    assert torch.equal(out[0][~has[:, 0]], c["t_dg"][~has[:, 0]])


def test_rows_are_tokens_without_row_token():
    note("adapter without row_token")
    c = make(4, 70, 1, 4, 2, 128, 128, 16)
    c["x"], c["token"] = c["x"][c["token"]], np.arange(c["n"], dtype=np.int32)
    c["t_x"] = bf16_to_dev(codecs.f64_to_bf16(c["x"]))
    c["e"], c["l"] = oracle.row_groups(c["ids"], c["off"], None, c["n"], c["L"])
    c["s"] = np.where(c["l"] >= 0, c["scale"].astype(np.float64)[c["l"]], 0.0)[:, None]
    for sort in (False, True):
        plan = ops().adapter_plan(i32_to_dev(c["ids"]), i32_to_dev(c["off"]), c["L"], backward=sort)
        check_forward(c, plan)
    check_backward(c, plan)


@pytest.mark.parametrize("sort", [False, True], ids=["few", "sorted"])
def test_rows_behind_the_last_expert_are_left_as_they_were(sort):
    """The C calls on prefilled outputs: rows from offsets[E] on keep every byte."""
    from expert_ffn_layer_top_amd._lib import call, lib
    note(f"adapter rows behind the last, sorted={sort}")
    c = make(5, 30, 2, 4, 2, 128, 64, 16)
    end = 41
    off = np.minimum(c["off"], end)
    ids, offs, token = i32_to_dev(c["ids"]), i32_to_dev(off), i32_to_dev(c["token"])
    plan = ops().adapter_plan(ids, offs, c["L"], row_token=token, backward=sort)
    fill = lambda cols: torch.full((c["n"], cols), 7.25, dtype=torch.bfloat16, device=dev())      # noqa: E731
    outs = dict(v=fill(32), g=fill(64), u=fill(64), a=fill(64))
    nbytes = lib.moe_adapter_workspace_bytes(c["n"], 4, 2, 128, 64, 16, sort, False)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev())
    p = lambda name: c["t_" + name].data_ptr()                                                    # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    call("moe_adapter_gate_up", p("x"), *plan._args(), 128, 64, 16, p("a_gu"), p("b_gate"), p("b_up"), p("scale"), None, 0.0, 0,
         p("g"), p("u"), p("a"), *(t.data_ptr() for t in outs.values()), ws.data_ptr(), nbytes, stream)
    v2, y = fill(16), fill(128)
    call("moe_adapter_down", outs["a"].data_ptr(), *plan._args(), 128, 64, 16, p("a_down"), p("b_down"), p("scale"), None, 0.0, 0,
         p("y"), v2.data_ptr(), y.data_ptr(), ws.data_ptr(), nbytes, stream)
    e, l = oracle.row_groups(c["ids"], off, c["token"], c["n"], c["L"])
    assert np.all(l[end:] == -1)
    for t in (*outs.values(), v2, y):
        assert bool((t[end:] == 7.25).all())
    ref, mag = oracle.shrink(c["x"][c["token"]], c["a_gu"], e, l)
    within(val(outs["v"])[:end], ref[:end], (U * np.abs(ref) + 128 * 2.0 ** -23 * mag)[:end], "v")
    whole = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, c["t_a_gu"], c["t_b_gate"], c["t_b_up"], c["t_scale"])
    assert torch.equal(whole[2][:end], outs["a"][:end])


@pytest.mark.parametrize("n", [300, 6000])
def test_offsets_that_fall_or_lie_outside_are_never_followed(n):
    """Offsets are the router's; others only the device can see.  Read as their running maximum within [0, n], they still
    give every row one place."""
    note(f"adapter bad offsets n={n}")
    c = make(11, n, 1, 4, 2, 64, 64, 8)
    for bad in ([0, 250, 40, 2 ** 31 - 1, n], [-5, 7, n + 9, 3, 100], [5, 5, 5, 5, 5], [0, n, 0, n, 0]):
        eff = np.maximum.accumulate(np.clip(np.array(bad, dtype=np.int64), 0, n))
        off, tok, ids = i32_to_dev(np.array(bad, dtype=np.int64).astype(np.int32)), i32_to_dev(c["token"]), i32_to_dev(c["ids"])
        plan = ops().adapter_plan(ids, off, 2, row_token=tok, backward=True)
        e, l = (torch.from_numpy(v).to(dev()) for v in oracle.row_groups(c["ids"], eff, c["token"], n, 2))
        y, v = ops().adapter_down(c["t_a"], c["t_y"], plan, c["t_a_down"], c["t_b_down"], c["t_scale"], want_v=True)
        has = l >= 0
        v64 = (c["t_a_down"].double()[l.clamp(min=0), e.clamp(min=0)] * c["t_a"].double()[:, None]).sum(2)
        vmag = (c["t_a_down"].double()[l.clamp(min=0), e.clamp(min=0)] * c["t_a"].double()[:, None]).abs().sum(2)
        assert bool(((v.double() - v64).abs() <= U * v64.abs() + 64 * 2.0 ** -23 * vmag)[has].all())
        assert torch.equal(y[~has & (e >= 0)], c["t_y"][~has & (e >= 0)])
        few = ops().adapter_down(c["t_a"], c["t_y"], ops().adapter_plan(ids, off, 2, row_token=tok), c["t_a_down"], c["t_b_down"], c["t_scale"])
        torch.cuda.synchronize()
        assert few[0].shape == y.shape


def test_a_bad_row_stays_a_bad_row():
    """NaN and infinities in one row's inputs, and in an adapter that no row has, reach no other row."""
    note("adapter NaN rows")
    c = make(6, 40, 2, 2, 3, 64, 64, 16)
    c["ids"][:] = np.where(c["ids"] == 2, 0, c["ids"])
    for sort in (False, True):
        plan = plan_of(c, sort)
        up = [c["t_" + w].clone() for w in ("a_gu", "b_gate", "b_up", "scale")]
        clean = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, *up)
        for w in up:
            w[2] = float("nan")
        x = c["t_x"].clone()
        x[11], x[12] = float("nan"), float("inf")
        out = ops().adapter_gate_up(x, c["t_g"], c["t_u"], c["t_a"], plan, *up)
        other = torch.from_numpy(~np.isin(c["token"], (11, 12)))
        for s, t in zip(clean[:3], out[:3]):
            assert torch.equal(s[other], t[other])


def test_ranks_padded_with_zeros_add_nothing():
    note("adapter padded ranks")
    c = make(7, 60, 2, 4, 2, 128, 128, 24)
    c["t_a_gu"][:, :, 8:24] = 0
    c["t_a_gu"][:, :, 32:] = 0
    c["t_b_gate"][:, :, 8:] = float(3)
    small = [torch.cat([c["t_a_gu"][:, :, 0:8], c["t_a_gu"][:, :, 24:32]], 2).contiguous(),
             c["t_b_gate"][:, :, :8].contiguous(), c["t_b_up"][:, :, :8].contiguous(), c["t_scale"]]
    for sort in (False, True):
        plan = plan_of(c, sort)
        a = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, c["t_a_gu"], c["t_b_gate"], c["t_b_up"], c["t_scale"])
        b = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, *small)
        for s, t in zip(a[:3], b[:3]):
            assert torch.equal(s, t)


def test_rows_whose_offsets_pass_32_bits():
    """yexp and dyexp of more than 4 GiB: the last rows, and a gradient that only they reach."""
    note("adapter rows past 4 GiB")
    n, d, f, r = 270000, 8192, 64, 8
    g = torch.Generator(device=dev()).manual_seed(5)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device=dev()) * std).to(torch.bfloat16)          # noqa: E731
    a, y = bf(n, f), torch.zeros((n, d), dtype=torch.bfloat16, device=dev())
    y[-70:] = bf(70, d)
    A, B, s = bf(2, 1, r, f, std=f ** -0.5), bf(2, 1, r, d, std=r ** -0.5), torch.ones(2, dtype=torch.float32, device=dev())
    ids = torch.zeros(n, dtype=torch.int32, device=dev())
    ids[-70:] = 1
    off = torch.tensor([0, n], dtype=torch.int32, device=dev())
    plan = ops().adapter_plan(ids, off, 2, backward=True)
    out, v = ops().adapter_down(a, y, plan, A, B, s, want_v=True)
    v64 = a[-70:].double() @ A[1, 0].double().t()
    vmag = a[-70:].double().abs() @ A[1, 0].double().abs().t()
    want = y[-70:].double() + v64 @ B[1, 0].double()
    off_v = V * v64.abs() + f * 2.0 ** -23 * vmag
    tol = U * want.abs() + 1.01 * off_v @ B[1, 0].double().abs() + (2 * r + 4) * 2.0 ** -23 * (y[-70:].double().abs() + v64.abs() @ B[1, 0].double().abs())
    assert bool(((out[-70:].double() - want).abs() <= tol).all())
    zero = torch.zeros((n, f), dtype=torch.bfloat16, device=dev())
    _, _, d_a, d_b = ops().adapter_down_bwd(y, a, v, zero, zero, zero, zero, plan, A, B, s)
    assert torch.count_nonzero(d_a[0]) == 0 and torch.count_nonzero(d_b[0]) == 0        # y is 0 in all other rows
    want = v[-70:].double().t() @ y[-70:].double()
    mag = v[-70:].double().abs().t() @ y[-70:].double().abs()
    assert bool(((d_b[1, 0].double() - want).abs() <= U * want.abs() + 80 * 2.0 ** -23 * mag).all())


def test_matrices_whose_offsets_pass_32_bits():
    """Adapters of more than 4 GiB: the last one, by both forms."""
    note("adapters past 4 GiB")
    L, E, r, d, f = 64, 64, 64, 4352, 64
    a_gu = torch.zeros((L, E, 2 * r, d), dtype=torch.bfloat16, device=dev())
    g = torch.Generator(device=dev()).manual_seed(6)
    bf = lambda *s, std=1.0: (torch.randn(s, generator=g, device=dev()) * std).to(torch.bfloat16)          # noqa: E731
    a_gu[-1, -1] = bf(2 * r, d, std=d ** -0.5)
    b_gate, b_up = torch.zeros((2, L, E, r, f), dtype=torch.bfloat16, device=dev())
    b_gate, b_up = b_gate.contiguous(), b_up.contiguous()
    x, gb = bf(3, d), bf(3, f)
    ids = torch.full((3,), L - 1, dtype=torch.int32, device=dev())
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev())
    off[-1] = 3
    v64 = x.double() @ a_gu[-1, -1].double().t()
    vmag = x.double().abs() @ a_gu[-1, -1].double().abs().t()
    for sort in (False, True):
        plan = ops().adapter_plan(ids, off, L, backward=sort)
        _, _, _, v = ops().adapter_gate_up(x, gb, gb, gb, plan, a_gu, b_gate, b_up, torch.ones(L, dtype=torch.float32, device=dev()), want_v=True)
        assert bool(((v.double() - v64).abs() <= U * v64.abs() + d * 2.0 ** -23 * vmag).all())


def test_two_streams_at_once():
    """The same calls on two streams, each with plans and workspaces of its own, against one after the other."""
    note("adapter on two streams")
    cases = [make(20 + i, 700, 2, 4, 3, 192, 128, 16) for i in range(2)]
    def step(c):
        plan = plan_of(c, True)
        up, down = [c["t_" + w] for w in ("a_gu", "b_gate", "b_up", "scale")], [c["t_" + w] for w in ("a_down", "b_down", "scale")]
        g, u, a, v1 = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, *up, want_v=True)
        y, v2 = ops().adapter_down(a, c["t_y"], plan, *down, want_v=True)
        one = ops().adapter_down_bwd(y, a, v2, g, u, c["t_dg"], c["t_du"], plan, *down)
        return (g, u, a, v1, y, v2, *one, *ops().adapter_gate_up_bwd(one[0], one[1], c["t_x"], v1, c["t_dxp"], plan, *up))
    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append([step(c) for _ in range(3)])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(s, t) for s, t in zip(w, run))


def test_repeated_calls_give_the_same_bits():
    note("adapter repeated")
    c = make(8, 700, 2, 2, 3, 64, 128, 16)
    plan = plan_of(c, True)
    first = None
    for _ in range(3):
        plan = plan_of(c, True)
        out = ops().adapter_down_bwd(c["t_y"], c["t_a"], c["t_v2"], c["t_g"], c["t_u"], c["t_dg"], c["t_du"], plan, c["t_a_down"],
                                     c["t_b_down"], c["t_scale"])
        if first is None:
            first = out
        assert all(torch.equal(s, t) for s, t in zip(first, out))


def test_captured_and_replayed_on_a_stream_of_its_own():
    """Plan and both passes in one graph; ids, routing and dropout change between the replays, eager work runs there too."""
    note("adapter captured")
    c = make(9, 48, 2, 4, 3, 128, 64, 16)
    ids, off, token = i32_to_dev(c["ids"]), i32_to_dev(c["off"]), i32_to_dev(c["token"])
    rng = torch.tensor([1, 2], device=dev())
    up, down = [c["t_" + w] for w in ("a_gu", "b_gate", "b_up", "scale")], [c["t_" + w] for w in ("a_down", "b_down", "scale")]

    def step():
        plan = ops().adapter_plan(ids, off, 3, row_token=token, backward=True)
        g, u, a, v1 = ops().adapter_gate_up(c["t_x"], c["t_g"], c["t_u"], c["t_a"], plan, *up, drop=ops().Dropout(0.2, rng, 1), want_v=True)
        y, v2 = ops().adapter_down(a, c["t_y"], plan, *down, drop=ops().Dropout(0.2, rng, 2), want_v=True)
        one = ops().adapter_down_bwd(y, a, v2, g, u, c["t_dg"], c["t_du"], plan, *down, drop=ops().Dropout(0.2, rng, 2))
        return (g, u, a, v1, y, v2, *one, *ops().adapter_gate_up_bwd(one[0], one[1], c["t_x"], v1, c["t_dxp"], plan, *up,
                                                                     drop=ops().Dropout(0.2, rng, 1)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    gen = np.random.default_rng(0)
    for i in range(4):
        ids.copy_(torch.from_numpy(gen.integers(-1, 3, 48).astype(np.int32)))
        rng[1] = i
        cut = np.sort(gen.integers(0, 97, 3))
        off.copy_(torch.from_numpy(np.concatenate([[0], cut, [96]]).astype(np.int32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        for j, (s, t) in enumerate(zip(out, eager)):
            assert torch.equal(s, t), (i, j)
