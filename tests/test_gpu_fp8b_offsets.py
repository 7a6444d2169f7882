"""Padded offsets that the block-128 token axis has no room for, or that split its blocks.  They live on the device,
so no call can refuse them: nothing may be read through them, and what they would make wrong is NaN."""

import numpy as np
import pytest
import torch

from gpu_util import dev, i32_to_dev, note

pytestmark = pytest.mark.gpu

P_OF = lambda n, E: (n + 128 * E + 127) // 128 * 128   # noqa: E731


def _offsets(counts, pad):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return i32_to_dev(off), i32_to_dev(np.concatenate([[0], np.cumsum([-(-c // pad) * pad for c in counts])]))


def _rows(n, C, seed):
    return torch.randn(n, C, device=dev(), generator=torch.Generator(device=dev()).manual_seed(seed)).bfloat16()


@pytest.fixture(params=["", "half", "big"])
def form(request, monkeypatch):
    if request.param:
        monkeypatch.setenv("MOE_FP8B_FORM", request.param)
    return request.param


# the last experts start past P (the first case), end past it, or start inside a block
BAD = [([1] * 8, 256), ([1] * 8, 1 << 20), ([300, 1, 1, 1], 512), ([5, 200, 64], 64), ([1] * 256, 256), ([3, 140], 96)]


@pytest.mark.parametrize("counts,pad", BAD, ids=[f"{len(c)}-{p}" for c, p in BAD])
def test_other_pads_give_nan(counts, pad, form):
    from expert_ffn_layer_top_amd import ops
    n, E, d, f = sum(counts), len(counts), 192, 320
    off, good = _offsets(counts, 128)
    _, bad = _offsets(counts, pad)
    x, h = _rows(n, d, 1), _rows(n, f, 2)
    note(f"fp8b offsets of pad {pad}, {E} experts {form}")
    for rows in (True, False):
        q, s, qT, sT = ops.fp8b_quantize_rows_grouped(x, off, bad, want_rows=rows)
        assert torch.isnan(sT).all() and (s is None or torch.isnan(s).all())
    xT, hT = ops.fp8b_quantize_rows_grouped(x, off, good)[2:], ops.fp8b_quantize_rows_grouped(h, off, good)[2:]
    start, P = bad.cpu().numpy(), P_OF(n, E)
    lost = [e for e in range(E) if start[e] % 128 or start[e + 1] % 128 or start[e + 1] > P]
    assert lost
    dwd = ops.grouped_gemm_wgrad_down_fp8b(*xT, *hT, off, bad, n)
    dwg, dwu = ops.grouped_gemm_wgrad_gate_up_fp8b(*hT, *hT, *xT, off, bad, n)
    for dw in (dwd, dwg, dwu):
        nan = torch.isnan(dw).flatten(1)
        assert nan[lost].all() and not nan[[e for e in range(E) if e not in lost]].any()


def test_a_larger_pad_that_fits_is_no_different(form):
    from expert_ffn_layer_top_amd import ops
    counts, d, f = [200, 0, 250], 128, 192
    n = sum(counts)
    x, h = _rows(n, d, 3), _rows(n, f, 4)
    note(f"fp8b offsets of pad 256 that fit {form}")
    got = []
    for pad in (128, 256):
        off, offp = _offsets(counts, pad)
        q, s, *xT = ops.fp8b_quantize_rows_grouped(x, off, offp)
        hT = ops.fp8b_quantize_rows_grouped(h, off, offp)[2:]
        got.append((q, s, ops.grouped_gemm_wgrad_down_fp8b(*xT, *hT, off, offp, n),
                    *ops.grouped_gemm_wgrad_gate_up_fp8b(*hT, *hT, *xT, off, offp, n)))
    for a, b in zip(*got):
        assert torch.equal(a, b) and not torch.isnan(a.float()).any()
