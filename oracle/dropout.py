"""Factors of the counter-based dropout, in whole numbers and 64 bits.

Philox4x32 (Salmon, Moraes, Dror, Shaw, SC 2011) with any number of rounds, pinned by the vectors its authors
publish for 10; the library takes 7.
"""

import numpy as np

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85
LOW = np.uint64(0xFFFFFFFF)


def philox(counter, key, rounds):
    """counter: four uint64 arrays of 32-bit words, key: two ints -> four arrays of words."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        p0, p1 = np.uint64(M0) * c[0], np.uint64(M1) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & LOW, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & LOW]
        k0, k1 = (k0 + W0) & 0xFFFFFFFF, (k1 + W1) & 0xFFFFFFFF
    return c


def pieces(seed, offset, site, rows, cols):
    """u(r, c) [rows, cols]: 16 bits each."""
    seed, offset = int(seed) % (1 << 64), int(offset) % (1 << 64)
    chunks = -(-cols // 8)
    c0 = np.broadcast_to(np.arange(chunks, dtype=np.uint64)[None] | np.uint64(site << 28), (rows, chunks))
    c1 = np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, chunks))
    full = lambda v: np.full((rows, chunks), v, dtype=np.uint64)                # noqa: E731
    w = philox((c0, c1, full(offset & 0xFFFFFFFF), full(offset >> 32)), (seed & 0xFFFFFFFF, seed >> 32), 7)
    out = np.empty((rows, chunks, 8), dtype=np.uint64)
    for i in range(4):
        out[:, :, 2 * i], out[:, :, 2 * i + 1] = w[i] & np.uint64(0xFFFF), w[i] >> np.uint64(16)
    return out.reshape(rows, -1)[:, :cols].astype(np.int64)


def factors(seed, offset, site, rows, cols, p):
    cut = int(np.rint(np.float32(p) * np.float32(65536)))
    return np.where(pieces(seed, offset, site, rows, cols) >= cut, 65536.0 / (65536 - cut), 0.0)
