"""Block-128 products at the limits of one of their kernels, where another one has to take over."""

import pytest
import torch

from gpu_util import dev, i32_to_dev, note

pytestmark = pytest.mark.gpu


def test_weight_gradients_of_a_token_axis_past_the_256_row_kernels_offsets(monkeypatch):
    """2^23 tokens: 256 rows of codes no longer fit 32-bit offsets, 128 do.  The tokens are zero but for a few
    blocks at both ends and past 2^31 codes, so the result has the bits of those blocks alone."""
    from expert_ffn_layer_top_amd import ops
    n, d, f = 1 << 23, 4096, 2176                      # more than two rounds of 128-row tiles: the estimate prefers 256
    P = n + 128
    at = [0, 1, 2, 40000, 65534, 65535]                # blocks of 128 tokens that are not zero
    gen = torch.Generator(device=dev()).manual_seed(3)

    def axis(*v):
        return torch.tensor(v, dtype=torch.int32, device=dev())

    m = 128 * len(at)
    small = axis(0, m), axis(0, m)
    long = axis(0, n), axis(0, n)
    note(f"fp8b weight gradients of {n} tokens, d={d} f={f}")

    def operand(C):
        x = torch.randn(m, C, device=dev(), generator=gen).bfloat16()
        _, _, q, s = ops.fp8b_quantize_rows_grouped(x, *small)
        codes = torch.zeros(C, P, dtype=torch.uint8, device=dev())
        scales = torch.ones(P // 128, C, dtype=torch.float32, device=dev())
        for i, b in enumerate(at):
            codes[:, 128 * b:128 * (b + 1)] = q[:, 128 * i:128 * (i + 1)]
            scales[b] = s[i]
        return (q, s), (codes, scales)

    (dy, dy_long), (a, a_long) = operand(d), operand(f)
    got = ops.grouped_gemm_wgrad_down_fp8b(*dy_long, *a_long, *long, n)
    monkeypatch.setenv("MOE_FP8B_FORM", "half")
    want = ops.grouped_gemm_wgrad_down_fp8b(*dy, *a, *small, m)
    assert torch.equal(got, want) and want.abs().max() > 0


@pytest.mark.parametrize("form", ["", "few", "mid", "half", "big"])
def test_offsets_past_the_rows_of_a_call(form, monkeypatch):
    """Offsets that name more rows than the call's n are a caller's mistake: whatever the rows below n hold then,
    nothing is written behind them, in any form."""
    from expert_ffn_layer_top_amd._lib import call
    from test_gpu_fp8b import Case
    if form:
        monkeypatch.setenv("MOE_FP8B_FORM", form)
    held, n, d, f = 200, 20, 192, 320
    c = Case([held], d, f, seed=12)
    (xq, xs), _ = c.rows(d)
    c.E = 3
    wg, wu = c.weight(f, d)[0], c.weight(f, d)[0]
    g, u = c.bf16(f)[0], c.bf16(f)[0]
    xs = xs[:, :n].contiguous()
    stream = torch.cuda.current_stream().cuda_stream

    note(f"fp8b offsets past n {form}")
    for offsets in ([0, 3, 90, 200], [0, 20, 21, 140]):
        off = i32_to_dev(offsets)
        out = [torch.full((held, f), 7.0, device=dev()).bfloat16() for _ in range(5)]
        call("moe_grouped_gemm_gate_up_fp8b", 3, n, d, f, *(t.data_ptr() for t in (off, xq, xs, *wg, *wu, *out[:3])), stream)
        call("moe_grouped_gemm_dgrad_down_fp8b", 3, n, d, f,
             *(t.data_ptr() for t in (off, xq, xs, *wg, g, u, *out[3:])), stream)
        for t in out:
            assert (t[n:] == 7.0).all()
