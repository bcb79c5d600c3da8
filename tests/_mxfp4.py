"""Plain MXFP4 arithmetic for the tests, from the definition in include/gq.h
(numpy, binary64), sharing nothing with csrc/ or gq.py."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
CODE_VALUES = np.concatenate([GRID, -GRID])
EPS2 = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}  # half a subnormal step


def to_bf16_bits(x):
    """binary32 -> bfloat16 bit patterns, nearest even (finite x)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def from_bf16_bits(b):
    return (np.asarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32)


def quantize(x):
    """x [N][K] binary64 -> (codes [N][K/2], scales [N][K/32]) uint8, one block at
    a time by search over the grid."""
    N, K = x.shape
    b = x.reshape(N, K // 32, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 0.0, amax)
    _, ex = np.frexp(amax)  # amax = m * 2^ex, m in [0.5, 1)
    e = np.where(amax > 0, np.clip(ex - 1 - 2, -127, 127), -127)
    v = np.where(bad[..., None], 0.0, np.where(np.isfinite(b), b, 0.0)) * np.exp2(-e.astype(np.float64))[..., None]
    a = np.minimum(np.abs(v), 6.0)
    d = np.abs(a[..., None] - GRID)  # distance to every grid value
    best = d.min(-1)
    code = np.full(a.shape, -1, np.int64)
    for c in (7, 5, 3, 1, 6, 4, 2, 0):  # of two equally near the even code is written last
        code = np.where(d[..., c] == best, c, code)
    code = code | np.where(np.signbit(v), 8, 0)
    code = np.where(bad[..., None], 0, code).reshape(N, K)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), s


def values(q, s):
    """Codes [.., K/2], scales [.., K/32] -> binary64 values [.., K]."""
    c = np.stack([q & 15, q >> 4], -1).reshape(q.shape[:-1] + (-1,))
    e = np.where(s == 255, 0, s.astype(np.int64) - 127)
    sc = np.where(s == 255, np.nan, np.exp2(e.astype(np.float64)))
    return CODE_VALUES[c] * np.repeat(sc, 32, -1)


def weights(seed, rows, K, lo=112, hi=124):
    """Random codes and scales in [lo, hi)."""
    g = np.random.default_rng([seed, rows, K])
    return (g.integers(0, 256, (rows, K // 2), np.uint8),
            g.integers(lo, hi, (rows, K // 32)).astype(np.uint8))


def products(W, X):
    """(Y, S) binary64: Y = X W^T and S = |X| |W|^T."""
    return X @ W.T, np.abs(X) @ np.abs(W).T
