"""Philox4x32-10 in numpy, and the masks that dropout makes of it: the tests' own, from the published rounds."""
import numpy as np

MASK = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """The four result words of each counter [..., 4] (uint32 values) under the key (two words)."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & MASK, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & MASK]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=-1).astype(np.uint32)


def border_of(p):
    return int(np.rint(p * 65536))


def keep_mask(n, width, p, seed, step=0):
    """bool [n, width]: which elements stay."""
    seed, step = seed % 2 ** 64, step % 2 ** 64
    groups = -(-width // 8)
    at = np.arange(n * groups, dtype=np.uint64)
    counter = np.stack([at & MASK, at >> np.uint64(32), np.full_like(at, step & 0xFFFFFFFF), np.full_like(at, step >> 32)],
                       axis=-1)
    words = philox(counter, (seed & 0xFFFFFFFF, seed >> 32)).astype("<u4")
    return words.view("<u2").reshape(n, groups * 8)[:, :width] >= border_of(p)
