"""Plain forms of MXFP4 and of the counter-based dropout for the tests: numpy, 64
bits, written from the definitions."""
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def encode(x):
    """(codes 0 .. 15, exponent bytes) of x [M, K] in blocks of 32 columns."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    nb = -(-K // 32)
    v = np.zeros((M, nb * 32))
    v[:, :K] = x
    v = v.reshape(M, nb, 32)
    top = np.abs(v).max(axis=2)
    bad = ~np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(bad, 1.0, top)))
    e = np.where(top > 0, e, -200)
    # (log2 rounds next to a power of two)
    e += np.where(np.exp2(e + 1) <= np.where(bad, 0, top), 1, 0)
    e -= np.where((np.exp2(e) > top) & (top > 0) & ~bad, 1, 0)
    e = np.maximum(e - 2, -127)
    with np.errstate(invalid="ignore"):
        a = np.abs(v / np.exp2(e)[..., None])
    a = np.where(bad[..., None], 0.0, a)
    d = np.abs(a[..., None] - LEVELS)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])  # even codes first: they win ties
    c = order[np.argmin(d[..., order], axis=-1)]
    c = np.where(a >= 6, 7, c) + 8 * (np.signbit(v) & ~bad[..., None])
    return c.reshape(M, nb * 32), np.where(bad, 255, e + 127).astype(np.uint8)


def decode(c, E, K):
    v = np.where(c & 8, -1.0, 1.0) * LEVELS[c & 7]
    s = np.where(E == 255, np.nan, np.exp2(E.astype(np.float64) - 127))
    return (v * np.repeat(s, 32, axis=1))[:, :K]


def rounded(x):
    c, E = encode(x)
    return decode(c, E, np.shape(x)[1])


def layout(c, E):
    """The stored bytes: codes [M, 128 J] and scales [ceil(M / 32), J, 256]."""
    M, nb = E.shape
    J, R = -(-nb // 8), -(-M // 32)
    codes = np.zeros((M, 128 * J), np.uint8)
    codes[:, :16 * nb] = c[:, 0::2] | (c[:, 1::2] << 4)
    scales = np.full((R, J, 256), 127, np.uint8)
    for m in range(M):
        for b in range(nb):
            n, q = m % 32, b % 8
            scales[m // 32, b // 8, 4 * (16 * (q % 4) + n % 16) + 2 * (n // 16) + q // 4] = E[m, b]
    return codes, scales


def philox(counter, key):
    """Philox 4x32 with ten rounds; counter: four arrays or numbers, key: two numbers."""
    low = (1 << 32) - 1
    c = [np.asarray(v, dtype=object) for v in counter]
    k = list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def keep(n, p, seed, offset=0, first=0):
    """Which of the elements 8 first .. 8 first + n - 1 dropout keeps, and the factor of the kept ones."""
    low = (1 << 32) - 1
    b = np.array([first + i for i in range(-(-n // 8))], dtype=object)
    offset &= (1 << 64) - 1
    w = philox((b & low, b >> 32, offset & low, offset >> 32), (seed & low, seed >> 32))
    w = np.stack([np.broadcast_to(v, b.shape) for v in w], axis=1).astype(np.int64)
    half = np.stack([w & 0xffff, w >> 16], axis=2).reshape(-1)[:n]
    t = min(int(np.rint(np.float64(np.float32(p)) * 65536)), 65535)
    return half >= t, 65536.0 / (65536 - t)
