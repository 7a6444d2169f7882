"""The block-128 E4M3 oracle against torch's own float8 cast, closed forms and plain matrix products."""

import numpy as np
import pytest
import torch

from oracle import codecs, fp8b


def bf16(a):
    return codecs.bf16_to_f64(codecs.f64_to_bf16(a))


@pytest.mark.parametrize("C", [64, 128, 320])
def test_rows_against_torch(C):
    x = bf16(np.random.default_rng(C).standard_normal((7, C)))
    q, s = fp8b.quantize_rows(x)
    t = torch.from_numpy(x).float()
    for b in range(fp8b.blocks(C)):
        part = t[:, 128 * b:128 * (b + 1)]
        amax = part.abs().amax(dim=1, keepdim=True)
        want = (part * (torch.full_like(amax, 448.0) / amax)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(q[:, 128 * b:128 * (b + 1)], want)
        assert np.array_equal(s[b], (amax[:, 0] * torch.tensor(1.0 / 448.0)).numpy())


def test_values_are_within_half_a_step():
    x = bf16(np.random.default_rng(5).standard_normal((16, 256)))
    back = fp8b.row_values(*fp8b.quantize_rows(x))
    amax = np.abs(x.reshape(16, 2, 128)).max(axis=2).repeat(128, axis=1)
    # half a step of a normal code is 2^-4 of it; below the normals (2^-6 of 448) steps are 2^-9
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * amax / 448) * (1 + 1e-6))


def test_zero_and_tiny_blocks():
    x = np.zeros((2, 128))
    x[1, 3] = 2.0 ** -130
    q, s = fp8b.quantize_rows(x)
    assert not q.any() and np.all(s == np.float32(2.0 ** -100) * np.float32(1 / 448)) and np.all(s > 0)


def test_weights_and_tokens_agree_with_rows():
    rng = np.random.default_rng(6)
    w = bf16(rng.standard_normal((2, 192, 320)))
    q, s = fp8b.quantize_weights(w)
    inv, scale = fp8b.factors(np.abs(w[1, 128:, 256:]).max())
    assert s.shape == (2, 2, 3) and s[1, 1, 2] == scale
    assert np.array_equal(q[1, 128:, 256:], fp8b._codes(w[1, 128:, 256:], inv))
    # blocks of tokens of one expert are row blocks of its transposed rows
    x = bf16(rng.standard_normal((150, 64)))
    qT, sT = fp8b.quantize_tokens(x, [0, 20, 150], [0, 128, 384], 512)
    qr, sr = fp8b.quantize_rows(np.ascontiguousarray(x[20:].T))
    assert np.array_equal(qT[:, 128:258], qr) and np.array_equal(sT[1:3], sr)
    assert not qT[:, 20:128].any() and not qT[:, 258:].any()
    back = fp8b.token_values(qT, sT, [0, 20, 150], [0, 128, 384])
    assert np.allclose(back, x, atol=0.07 * np.abs(x).max())


def test_grouped_products_are_plain_products():
    rng = np.random.default_rng(7)
    x, w, y = rng.standard_normal((9, 64)), rng.standard_normal((3, 32, 64)), rng.standard_normal((9, 16))
    off = [0, 4, 4, 9]
    out, size, largest = fp8b.grouped_nt(x, w, off)
    dw, _, _ = fp8b.grouped_tn(x, y, off)
    for r in range(9):
        assert np.allclose(out[r], w[0 if r < 4 else 2] @ x[r])
    assert np.allclose(dw[2], sum(np.outer(x[r], y[r]) for r in range(4, 9))) and not dw[1].any()
    assert np.all(size >= np.abs(out) - 1e-12)
    terms = np.abs(x[5] * w[2, 7]).reshape(8, 8)
    assert largest[5, 7] == pytest.approx(terms.max(axis=1).sum())
