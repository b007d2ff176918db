"""Dropout mask of an adapter's input, as the C ABI defines it (qlr_dropout): Philox4x32-10 (Salmon, Moraes, Dror,
Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) of an element group's number and the mask's counter."""
import numpy as np

MASK64 = (1 << 64) - 1


def philox4x32(ctr, key, rounds=10):
    """ctr: four uint32 arrays (or numbers), key: two numbers; the four result words as uint32 arrays."""
    x = [np.asarray(c, dtype=np.uint64) for c in ctr]
    lo = np.uint64(0xFFFFFFFF)
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), b & lo, (a >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [v.astype(np.uint32) for v in x]


def dropout_threshold(p):
    """Numbers below it drop their element: p 65536 to the nearest integer, ties to even, at most 65535."""
    return min(round(65536 * p), 65535)


def dropout_factors(M, K, p, seed, counter):
    """(M, K) float64: 0 where the element is dropped, 65536 / (65536 - t) where it is kept."""
    t = dropout_threshold(p)
    if t == 0:
        return np.ones((M, K))
    g = np.arange(M * K // 8, dtype=np.uint64)
    c, seed = counter & MASK64, seed & MASK64
    words = philox4x32((g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), c & 0xFFFFFFFF, c >> 32), (seed & 0xFFFFFFFF, seed >> 32))
    n = np.stack([h for w in np.broadcast_arrays(*words) for h in (w & 0xFFFF, w >> 16)], 1)
    return np.where(n >= t, 65536.0 / (65536 - t), 0.0).reshape(M, K)
