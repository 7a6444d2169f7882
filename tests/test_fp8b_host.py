"""Refusals of the scored router's and the block-128 E4M3 calls, on the host: the torch wrappers (CPU
tensors; a consistent call stops at the device check) and the C entry points (every call fails its
argument checks, so nothing is launched)."""

import ctypes

import pytest
import torch

from expert_ffn_layer_top_amd import _lib, ops

bf, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
T, d, E, k, f = 8, 192, 4, 2, 128
n = T * k
P = (n + 128 * E + 127) // 128 * 128


def z(*shape, dt=bf):
    return torch.zeros(shape, dtype=dt)


def q(*shape):
    return torch.zeros(shape, dtype=u8)


def s(*shape):
    return torch.zeros(shape, dtype=f32)


def consistent(fn, *args, **kw):
    with pytest.raises(ValueError, match="GPU"):
        fn(*args, **kw)


def refused(match, fn, *args, exc=ValueError, **kw):
    with pytest.raises(exc, match=match):
        fn(*args, **kw)


def test_route_scored():
    l = s(T, 32)
    consistent(ops.route_scored, l, 4, bias=s(32), n_group=8, topk_group=2, group_top=2, pad=128)
    refused("n_group", ops.route_scored, l, 4, n_group=5)
    refused("n_group", ops.route_scored, l, 4, n_group=0)
    refused("topk_group", ops.route_scored, l, 4, n_group=4, topk_group=5)
    refused("topk_group", ops.route_scored, l, 4, n_group=4, topk_group=0)
    refused("group_top", ops.route_scored, l, 4, group_top=3)
    refused("k = 9", ops.route_scored, l, 9, n_group=8, topk_group=2)
    refused("k = 17", ops.route_scored, l, 17)
    refused("k = 0", ops.route_scored, l, 0)
    refused("score", ops.route_scored, l, 4, score="relu")
    refused("bias", ops.route_scored, l, 4, bias=s(31))
    refused("bias", ops.route_scored, l, 4, bias=torch.zeros(32, dtype=torch.float64), exc=TypeError)
    refused("pad", ops.route_scored, l, 4, pad=0)
    refused("E <= 256", ops.route_scored, s(T, 257), 4)
    refused("T >= 1", ops.route_scored, s(0, 32), 4)
    refused("logits", ops.route_scored, z(T, 32), 4, exc=TypeError)
    consistent(ops.route_scored_bwd, l, z(T, k, dt=i32), s(T, k))
    refused("d_gate", ops.route_scored_bwd, l, z(T, k, dt=i32), s(T, k + 1))
    refused("topk_idx", ops.route_scored_bwd, l, z(T + 1, k, dt=i32), s(T, k))


def test_quantisers():
    off = z(E + 1, dt=i32)
    consistent(ops.fp8b_quantize_rows, z(T, d))
    consistent(ops.fp8b_quantize_rows, z(T, d), dest=z(T, k, dt=i32))
    refused("multiple of 64", ops.fp8b_quantize_rows, z(T, d + 32))
    refused("T >= 1", ops.fp8b_quantize_rows, z(0, d))
    refused("dest", ops.fp8b_quantize_rows, z(T, d), dest=z(T + 1, k, dt=i32))
    refused("k = 17", ops.fp8b_quantize_rows, z(T, d), dest=z(T, 17, dt=i32))
    refused("contiguous", ops.fp8b_quantize_rows, z(d, T).t())
    consistent(ops.fp8b_quantize_rows_grouped, z(n, d), off, off)
    consistent(ops.fp8b_quantize_rows_grouped, z(T, d), off, off, row_token=z(n, dt=i32), row_gate=s(n))
    refused("offsets_pad", ops.fp8b_quantize_rows_grouped, z(n, d), off, z(E, dt=i32))
    refused("row_gate", ops.fp8b_quantize_rows_grouped, z(T, d), off, off, row_token=z(n, dt=i32), row_gate=s(T))
    refused("E <= 256", ops.fp8b_quantize_rows_grouped, z(n, d), z(258, dt=i32), z(258, dt=i32))
    consistent(ops.fp8b_quantize_weights, z(E, f, d))
    consistent(ops.fp8b_quantize_weights, z(f, d))
    refused("multiples of 64", ops.fp8b_quantize_weights, z(E, f, d + 16))


def test_products():
    off = z(E + 1, dt=i32)
    w = (q(E, f, d), s(E, 1, 2))
    x = (q(n, d), s(2, n))
    consistent(ops.grouped_gemm_gate_up_fp8b, *x, off, *w, *w)
    refused("w_up", ops.grouped_gemm_gate_up_fp8b, *x, off, *w, q(E, f + 64, d), s(E, 2, 2))
    refused("w_gate_s", ops.grouped_gemm_gate_up_fp8b, *x, off, q(E, f, d), s(E, 2, 1), *w)
    refused("xq", ops.grouped_gemm_gate_up_fp8b, q(n, f), s(1, n), off, *w, *w)
    refused("xq_s", ops.grouped_gemm_gate_up_fp8b, q(n, d), s(n, 2), off, *w, *w)
    refused("offsets", ops.grouped_gemm_gate_up_fp8b, *x, z(E, dt=i32), *w, *w)
    refused("n >= 1", ops.grouped_gemm_gate_up_fp8b, q(0, d), s(2, 0), off, *w, *w)
    refused("multiples of 64", ops.grouped_gemm_down_fp8b, q(n, 96), s(1, n), off, q(E, d, 96), s(E, 2, 1))
    consistent(ops.grouped_gemm_down_fp8b, q(n, f), s(1, n), off, q(E, d, f), s(E, 2, 1))
    refused("aq", ops.grouped_gemm_down_fp8b, q(n, d), s(2, n), off, q(E, d, f), s(E, 2, 1))
    consistent(ops.grouped_gemm_dgrad_down_fp8b, *x, off, *w, z(n, f), z(n, f))
    refused("u:", ops.grouped_gemm_dgrad_down_fp8b, *x, off, *w, z(n, f), z(n, d))
    h, wt = (q(n, f), s(1, n)), (q(E, d, f), s(E, 2, 1))
    consistent(ops.grouped_gemm_dgrad_gate_up_fp8b, *h, *h, off, *wt, *wt)
    refused("duq", ops.grouped_gemm_dgrad_gate_up_fp8b, *h, q(n + 1, f), s(1, n + 1), off, *wt, *wt)
    dT, fT = (q(d, P), s(P // 128, d)), (q(f, P), s(P // 128, f))
    consistent(ops.grouped_gemm_wgrad_down_fp8b, *dT, *fT, off, off, n)
    refused("aT", ops.grouped_gemm_wgrad_down_fp8b, *dT, q(f, P - 128), s(P // 128, f), off, off, n)
    refused("dyT_s", ops.grouped_gemm_wgrad_down_fp8b, q(d, P), s(P // 32, d), *fT, off, off, n)
    consistent(ops.grouped_gemm_wgrad_gate_up_fp8b, *fT, *fT, *dT, off, off, n)
    refused("duT", ops.grouped_gemm_wgrad_gate_up_fp8b, *fT, *dT, *dT, off, off, n)
    refused("offsets_pad", ops.grouped_gemm_wgrad_gate_up_fp8b, *fT, *fT, *dT, off, z(E, dt=i32), n)


def test_c_entry_points_refuse_before_any_launch():
    L = _lib.lib
    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
    p, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)

    def route(logits=p, bias=p, T=16, E=32, k=4, score=0, G=4, tg=2, top=2, scale=1.0, pad=128, ws=p, nbytes=1 << 20):
        return L.moe_route_scored(logits, bias, T, E, k, score, G, tg, top, 1, scale, p, p, None, p, p, p, pad, p, p, ws,
                                  nbytes, None)

    assert route(T=0) == UNSUPPORTED and route(E=300) == UNSUPPORTED and route(k=17) == UNSUPPORTED
    assert route(G=5) == UNSUPPORTED and route(G=0) == UNSUPPORTED and route(tg=5) == UNSUPPORTED
    assert route(tg=0) == UNSUPPORTED and route(top=3) == UNSUPPORTED and route(k=9, tg=1) == UNSUPPORTED
    assert route(score=2) == INVALID and route(logits=None) == INVALID and route(bias=odd) == INVALID
    assert route(scale=float("nan")) == INVALID and route(pad=0) == INVALID
    size = L.moe_route_scored_workspace_bytes
    assert size(64, 256, 8) == 0 and size(65, 256, 8) == 2 * 256 * 4 + 16 + 65 * 8 and size(1000, 3, 2) == 16 * 3 * 4 + 16 + 8000
    assert route(T=65, ws=None) == WORKSPACE and route(T=65, nbytes=16) == WORKSPACE
    assert L.moe_route_scored_bwd(p, p, p, 4, 8, 2, 7, 1, 1.0, p, None) == INVALID
    assert L.moe_route_scored_bwd(p, None, p, 4, 8, 2, 0, 1, 1.0, p, None) == INVALID
    assert L.moe_route_scored_bwd(p, p, p, 4, 8, 9, 0, 1, 1.0, p, None) == UNSUPPORTED
    rows = L.moe_fp8b_quantize_rows
    assert rows(p, None, 4, 96, 1, p, p, None) == UNSUPPORTED and rows(p, None, 0, 64, 1, p, p, None) == UNSUPPORTED
    assert rows(p, None, 4, 64, 2, p, p, None) == UNSUPPORTED and rows(p, p, 4, 64, 17, p, p, None) == UNSUPPORTED
    assert rows(odd, None, 4, 64, 1, p, p, None) == INVALID and rows(p, p, 1 << 28, 64, 16, p, p, None) == UNSUPPORTED
    grp = L.moe_fp8b_quantize_rows_grouped
    assert grp(p, None, None, p, p, 4, 8, 64, p, None, p, p, None) == INVALID
    assert grp(p, None, None, p, p, 257, 8, 64, p, p, p, p, None) == UNSUPPORTED
    assert grp(p, None, None, p, p, 4, (1 << 31) - 1, 64, p, p, p, p, None) == UNSUPPORTED
    assert L.moe_fp8b_quantize_weights(p, 1, 64, 96, p, p, None, None, None) == UNSUPPORTED
    assert L.moe_fp8b_quantize_weights(p, 1, 64, 64, p, p, p, None, None) == INVALID
    gu = L.moe_grouped_gemm_gate_up_fp8b
    assert gu(4, 8, 96, 64, *[p] * 11) == UNSUPPORTED and gu(0, 8, 64, 64, *[p] * 11) == UNSUPPORTED
    assert gu(4, 0, 64, 64, *[p] * 11) == UNSUPPORTED and gu(4, 8, 64, 64, None, *[p] * 10) == INVALID
    assert gu(4, 8, 64, 64, *[p] * 7, p, None, p, None) == INVALID                  # g without u
    assert L.moe_grouped_gemm_down_fp8b(4, 8, 64, 64, p, odd, p, p, p, p, None) == INVALID
    assert L.moe_grouped_gemm_dgrad_down_fp8b(4, 8, 64, 64, p, p, p, p, p, p, None, p, p, None) == INVALID
    assert L.moe_grouped_gemm_dgrad_gate_up_fp8b(4, 8, 64, 72, *[p] * 11) == UNSUPPORTED
    assert L.moe_grouped_gemm_wgrad_down_fp8b(4, 8, 64, 64, p, None, p, p, p, p, p, None) == INVALID
    assert L.moe_grouped_gemm_wgrad_gate_up_fp8b(4, 1 << 30, 64, 64, *[p] * 10, None) == UNSUPPORTED   # P * 256 past 2^31
