"""The tests' generator against the published known answers of Philox4x32-10, and its masks' shares."""
import numpy as np
import pytest

from philox import border_of, keep_mask, philox


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, words):
    assert tuple(philox(np.array([counter], dtype=np.uint64), key)[0]) == words


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_share(p):
    n = 512 * 1000
    kept = int(keep_mask(512, 1000, p, 7, 3).sum())
    q = 1 - border_of(p) / 65536
    assert abs(kept - n * q) < 6 * (n * q * (1 - q)) ** 0.5  # six standard deviations of a binomial


def test_masks_differ():
    a, b, c = keep_mask(64, 256, 0.5, 1, 0), keep_mask(64, 256, 0.5, 2, 0), keep_mask(64, 256, 0.5, 1, 1)
    for x, y in ((a, b), (a, c), (b, c)):
        assert 0.45 < float((x == y).mean()) < 0.55  # 16384 fair coins: 0.5 within 0.004 a standard deviation
