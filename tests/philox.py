"""Philox4x32-10 in numpy, for the dropout tests (Salmon et al., "Parallel
random numbers: as easy as 1, 2, 3", 2011)."""
import numpy as np


def philox(counter, seed):
    """Words [4, ...] of a counter array [4, ...] under a 64-bit seed."""
    c = [np.asarray(x, np.uint64) for x in counter]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k0), b & low, (a >> half) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(np.broadcast_arrays(*c))


def keep_mask(ne0, ne1, p, seed, offset, rows=None):
    """[len(rows), ne0] truth values of the elements the dropout keeps."""
    rows = np.arange(ne1) if rows is None else np.asarray(rows)
    groups = -(-ne0 // 4)
    w = philox([np.arange(groups)[None, :], rows[:, None], offset & 0xFFFFFFFF, offset >> 32], seed)
    w = np.moveaxis(w, 0, -1).reshape(len(rows), groups * 4)[:, :ne0]
    return w >= np.uint64(int(float(np.float32(p)) * 4294967296.0))


def scale_of(p):
    return np.float32(0) if p == 1 else np.float32(1) / (np.float32(1) - np.float32(p))
