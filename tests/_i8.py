"""Plain arithmetic of the int8 operators for the tests, from the definition in include/gq.h
(numpy, binary64 and whole numbers), sharing nothing with csrc/ or gq.py."""
import numpy as np

from tests._mxfp4 import EPS2, TINY, from_bf16_bits, to_bf16_bits

F = np.float32


def quantize(x):
    """x [N][K] binary64 (values of a binary32 number or shorter) -> (codes int64, scales
    binary32).  127 x is exact in binary64 and the quotient of two such numbers that is no half
    itself lies 2^-33 or more from one, so binary64 rounds it to the right side."""
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[:, None], 0.0, x)
    top = np.abs(x).max(-1)
    q = np.rint(127.0 * x / np.where(top > 0, top, 1.0)[:, None]).astype(np.int64)
    s = top.astype(F) / F(127.0)
    return q, np.where(bad, F(np.nan), s).astype(F)


def round_to(v, t):
    """binary32 values rounded to a type, as binary64."""
    v = np.asarray(v, F)
    if t == "f32":
        return v.astype(np.float64)
    if t == "f16":
        with np.errstate(over="ignore"):
            return v.astype(np.float16).astype(np.float64)
    nan = np.isnan(v)
    r = from_bf16_bits(to_bf16_bits(np.where(nan, F(0), v))).astype(np.float64)
    return np.where(nan, np.nan, r)


def sums(wq, xq):
    """Whole-number products [N][M]; below 2^31, so binary64 holds every partial sum."""
    return xq.astype(np.float64) @ wq.astype(np.float64).T


def product(wq, ws, xq, xs):
    """The product as binary32, three roundings as documented."""
    with np.errstate(all="ignore"):
        return sums(wq, xq).astype(F) * ws[None, :] * xs[:, None]


def weights16(wq, ws, t):
    """Weights rounded to the 16-bit type, as binary64."""
    with np.errstate(all="ignore"):
        return round_to(wq.astype(F) * ws[:, None], t)


def split_scales(s):
    """s = f 2^e with 1/2 <= f < 1: (f, 2^e) in binary64."""
    f, e = np.frexp(s.astype(np.float64))
    return f, np.exp2(e)


def act(z, kind):
    """(act(z), act'(z), p(z)) in binary64."""
    z = np.asarray(z, np.float64)
    if kind == "silu":
        p, dp = z, np.ones_like(z)
    else:
        c = np.sqrt(2 / np.pi)
        p, dp = 2 * c * (z + 0.044715 * z ** 3), 2 * c * (1 + 3 * 0.044715 * z ** 2)
    sig = np.where(p >= 0, 1 / (1 + np.exp(-np.abs(p))), np.exp(-np.abs(p)) / (1 + np.exp(-np.abs(p))))
    return z * sig, sig + z * dp * sig * (1 - sig), p


# Relative error of the kernels' sigmoid(p) in binary32: p itself is off by up to 5 half steps
# (GELU: two products, two fused steps and the constant), which e^-p turns into |p| 5 2^-24;
# the exponent's product with log2(e) and the instruction add |p| 2^-24 + 2 2^-23, the sum and
# the quotient 2 2^-24 more: (6 |p| + 6) 2^-24, taken as (4 |p| + 8) 2^-23.
def act_rel(p):
    return (4 * np.abs(p) + 8) * 2.0 ** -23


def half_step(v, t):
    """What rounding v to a type moves it by at most."""
    return EPS2[t] * np.abs(v) + TINY[t]


def rows(seed, n, K, lo=-127, hi=127):
    """Codes [n][K] and scales [n]."""
    g = np.random.default_rng([seed, n, K])
    return (g.integers(lo, hi + 1, (n, K)).astype(np.int8),
            (2.0 ** g.uniform(-12, -8, n)).astype(F))
