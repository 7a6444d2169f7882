"""Oracle of the block-128 E4M3 format: quantisation in its three layouts, the values that codes stand
for, and the grouped products of the expert FFN on those values in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A block's amax counts as at least 2^-100; inv = 448 / amax rounded to float32; a code is E4M3 of the
float32 product v * inv, round to nearest even; scale = amax * float32(1/448) rounded to float32.
Scales of rows are block-major [ceil(K/128), rows]; weights have one scale per 128 x 128 block.
"""

import numpy as np

from . import codecs, moe

BLOCK = 128
TINY = np.float32(2.0 ** -100)


def blocks(n):
    return -(-n // BLOCK)


def factors(amax):
    """(inv, scale) float32 of float32 amax."""
    a = np.maximum(np.asarray(amax, dtype=np.float32), TINY)
    return np.float32(448.0) / a, a * np.float32(1.0 / 448.0)


def _codes(v, inv):
    w = (v.astype(np.float32) * inv).astype(np.float32).astype(np.float64)
    return codecs.e4m3_encode_rne_sat(np.clip(w, -448.0, 448.0))


def quantize_rows(x):
    """x [n, C] (exact bf16 values) -> codes [n, C], scales [ceil(C/128), n]."""
    n, C = x.shape
    q = np.empty((n, C), np.uint8)
    s = np.empty((blocks(C), n), np.float32)
    for b in range(blocks(C)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        inv, s[b] = factors(np.abs(part).max(axis=1))
        q[:, b * BLOCK:(b + 1) * BLOCK] = _codes(part, inv[:, None])
    return q, s


def quantize_weights(w):
    """w [E, R, C] -> codes [E, R, C], scales [E, ceil(R/128), ceil(C/128)]."""
    E, R, C = w.shape
    q = np.empty((E, R, C), np.uint8)
    s = np.empty((E, blocks(R), blocks(C)), np.float32)
    for e in range(E):
        for i in range(blocks(R)):
            for j in range(blocks(C)):
                at = (e, slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
                inv, s[e, i, j] = factors(np.abs(w[at]).max())
                q[at] = _codes(w[at], inv)
    return q, s


def quantize_tokens(x, offsets, offsets_pad, P):
    """x [n, C] grouped rows -> codes [C, P], scales [P/128, C], every other position zero."""
    C = x.shape[1]
    q = np.zeros((C, P), np.uint8)
    s = np.empty((P // BLOCK, C), np.float32)
    s[:] = factors(0.0)[1]
    for e in range(len(offsets) - 1):
        for i, r in enumerate(range(offsets[e], offsets[e + 1], BLOCK)):
            part = x[r:min(r + BLOCK, offsets[e + 1])]
            p = offsets_pad[e] + i * BLOCK
            inv, s[p // BLOCK] = factors(np.abs(part).max(axis=0))
            q[:, p:p + part.shape[0]] = _codes(part, inv[None, :]).T
    return q, s


def row_values(q, s):
    return codecs.e4m3_to_f64(q) * np.repeat(s.astype(np.float64), BLOCK, axis=0)[:q.shape[1]].T


def weight_values(q, s):
    s = np.repeat(np.repeat(s.astype(np.float64), BLOCK, axis=1), BLOCK, axis=2)
    return codecs.e4m3_to_f64(q) * s[:, :q.shape[1], :q.shape[2]]


def token_values(q, s, offsets, offsets_pad):
    """The grouped rows [n, C] that transposed codes [C, P] stand for."""
    v = (codecs.e4m3_to_f64(q) * np.repeat(s.astype(np.float64), BLOCK, axis=0).T).T
    rows = [v[offsets_pad[e]:offsets_pad[e] + offsets[e + 1] - offsets[e]] for e in range(len(offsets) - 1)]
    return np.concatenate(rows, axis=0)


def _largest_by_eight(a, b):
    """Sum over aligned groups of 8 along K of the largest |a[i, k]| |b[j, k]| in the group: [I, J]."""
    a, b = np.abs(a), np.abs(b)
    out = np.zeros((a.shape[0], b.shape[0]))
    for k0 in range(0, a.shape[1], 8):
        most = np.zeros_like(out)
        for k in range(k0, min(k0 + 8, a.shape[1])):
            np.maximum(most, np.outer(a[:, k], b[:, k]), out=most)
        out += most
    return out


def grouped_nt(x, w, offsets):
    """(out, size, largest): x rows times their expert's w [E, N, K] transposed, the sum of |x||w|, and the
    sum over aligned groups of 8 of the largest |x||w|."""
    out = np.zeros((x.shape[0], w.shape[1]))
    size, largest = np.zeros_like(out), np.zeros_like(out)
    for e in range(w.shape[0]):
        r = slice(offsets[e], offsets[e + 1])
        out[r] = x[r] @ w[e].T
        size[r] = np.abs(x[r]) @ np.abs(w[e]).T
        largest[r] = _largest_by_eight(x[r], w[e])
    return out, size, largest


def grouped_tn(left, right, offsets):
    """(dW, size, largest) [E, R, C]: left^T right over each expert's rows, as grouped_nt."""
    E = len(offsets) - 1
    out = np.zeros((E, left.shape[1], right.shape[1]))
    size, largest = np.zeros_like(out), np.zeros_like(out)
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        out[e] = left[r].T @ right[r]
        size[e] = np.abs(left[r]).T @ np.abs(right[r])
        largest[e] = _largest_by_eight(left[r].T, right[r].T)
    return out, size, largest
