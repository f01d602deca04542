"""Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) in numpy's unsigned
64-bit arithmetic, for the dropout tests."""
import numpy as np

M32 = np.uint64(0xFFFFFFFF)
S32 = np.uint64(32)


def words(group, key, offset):
    """[n, 4] words (uint64 below 2^32) at the counters (group, offset)."""
    group = group.astype(np.uint64)
    c = [group & M32, group >> S32, np.full_like(group, offset & 0xFFFFFFFF), np.full_like(group, offset >> 32)]
    for r in range(10):
        k0 = np.uint64((key + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64(((key >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> S32) ^ c[1] ^ k0, b & M32, (a >> S32) ^ c[3] ^ k1, a & M32]
    return np.stack(c, axis=1)


def kept(N, d, rate, seed, offset, row0):
    """The mask of moe_dropout_forward for these parameters, [N, d] of truth values."""
    first = row0 * d // 4
    w = words(np.arange(N * d // 4, dtype=np.uint64) + np.uint64(first), seed % 2 ** 64, offset % 2 ** 64)
    return (w >= np.uint64(round(rate * 2 ** 32))).reshape(N, d)
