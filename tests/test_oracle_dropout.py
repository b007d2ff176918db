"""Pins of the dropout mask: the generator's published known answers, the share of dropped elements, its layout."""
import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("ctr,key,want", [
    # the known answers published with the generator, ten rounds
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(ctr, key, want):
    assert tuple(int(v) for v in oracle.philox4x32(ctr, key)) == want


def test_rounds_against_whole_numbers():
    rng = np.random.default_rng(0)
    for _ in range(20):
        ctr, key = [int(v) for v in rng.integers(0, 1 << 32, 4)], [int(v) for v in rng.integers(0, 1 << 32, 2)]
        x, k = list(ctr), list(key)
        for _ in range(10):
            a, b = 0xD2511F53 * x[0], 0xCD9E8D57 * x[2]
            x = [(b >> 32) ^ x[1] ^ k[0], b % 2 ** 32, (a >> 32) ^ x[3] ^ k[1], a % 2 ** 32]
            k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
        assert [int(v) for v in oracle.philox4x32(ctr, key)] == x


def test_threshold():
    assert oracle.dropout_threshold(0.0) == 0 and oracle.dropout_threshold(0.5) == 32768
    assert oracle.dropout_threshold(0.5 / 65536) == 0 and oracle.dropout_threshold(1.5 / 65536) == 2  # ties to even
    assert oracle.dropout_threshold(0.9999999) == 65535


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_share_and_mean(p):
    M, K = 512, 1024
    f = oracle.dropout_factors(M, K, p, 12345, 6)
    n, t = M * K, oracle.dropout_threshold(p) / 65536
    sd = (t * (1 - t) / n) ** 0.5
    assert abs((f == 0).mean() - t) < 6 * sd          # six standard deviations of the share
    assert abs(f.mean() - 1) < 6 * sd / (1 - t)
    assert set(np.unique(f)) == {0.0, 1 / (1 - t)}
    # rows, columns and neighbouring masks are as independent as their size allows
    drop = (f == 0).astype(float) - t
    for other in (np.roll(drop, 1, 0), np.roll(drop, 1, 1), np.roll(drop, 8, 1),
                  (oracle.dropout_factors(M, K, p, 12345, 7) == 0) - t, (oracle.dropout_factors(M, K, p, 12346, 6) == 0) - t):
        assert abs((drop * other).mean()) < 6 * t * (1 - t) / n ** 0.5


def test_layout():
    """Element (m, k) takes half-word k % 8 of group (m K + k) / 8, whatever the matrix's height."""
    M, K, p, seed, c = 5, 64, 0.3, (7 << 32) | 9, (3 << 32) | 4
    f, t = oracle.dropout_factors(M, K, p, seed, c), oracle.dropout_threshold(p)
    for m, k in ((0, 0), (0, 7), (2, 33), (4, 63)):
        w = oracle.philox4x32(((m * K + k) // 8, 0, 4, 3), (9, 7))[(k % 8) // 2]
        assert (f[m, k] != 0) == (((int(w) >> (16 * (k % 2))) & 0xFFFF) >= t)
    assert np.array_equal(oracle.dropout_factors(3, K, p, seed, c), f[:3])
    assert np.array_equal(oracle.dropout_factors(M, K, 0.0, seed, c), np.ones((M, K)))
