"""The oracle's generator against its authors' published known answers, with no GPU."""
import random

import numpy as np
import pytest

from block_util import numbers


def philox(counter, key):
    """Philox4x32-10 of one counter, by whole numbers."""
    x, k, low = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        p, q = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [q >> 32 ^ x[1] ^ k[0], q & low, p >> 32 ^ x[3] ^ k[1], p & low]
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    return x


ONES = 0xFFFFFFFF


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((ONES, ONES, ONES, ONES), (ONES, ONES), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_known_answers(counter, key, want):
    assert tuple(philox(counter, key)) == want


def test_numbers_of_a_matrix():
    r = random.Random(0)
    for _ in range(20):
        seed, offset, site = r.getrandbits(64), r.getrandbits(64), r.randrange(32768)
        T, W = r.randrange(1, 9), r.randrange(1, 70)
        u = numbers(seed, offset, site, T, W)
        for _ in range(5):
            t, c = r.randrange(T), r.randrange(W)
            words = philox((c // 8 + (site << 17), t, offset & ONES, offset >> 32), (seed & ONES, seed >> 32))
            assert int(u[t, c]) == int(np.array(words, np.uint32).view(np.uint16)[c % 8])
