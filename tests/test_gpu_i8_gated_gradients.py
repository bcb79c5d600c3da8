"""The gated half's backward pass where its 16-bit operands could leave their type or lose bits:
gradients of g and u beyond binary16 and below it, sums that cancel, rows of zeros, infinities and
NaN.  Against the formula in binary64."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _i8 as i8
from tests._gpu import dev, torch_cuda
from tests.test_gpu_i8 import floats, gated_reference, grad_tolerance, matrix, near, ttype, values

pytestmark = pytest.mark.gpu


def scaled(seed, n, K, s, spread=1.0):
    """Codes [n][K] and scales near s."""
    g = np.random.default_rng([seed, n, K])
    return g.integers(-127, 128, (n, K)).astype(np.int8), (s * 2.0 ** g.uniform(0, spread, n)).astype(np.float32)


def want_and_tolerance(gate, up, xq, xs, d64, kind, t):
    """dX in binary64 and what may be lost: each operand dg ws and du us is rounded to binary16
    after a scaling by a power of two of its row, under which 1.13 max|dh ws us| |xs| 128 sum|xq| is
    at most 2^15 and, the five factors taken by their exponents and 1.13 as 2, at least 2^15 / 2^6:
    half a step of 11 bits, or 2^-25 scaled back, 2^-25 2^-15 2^6 of that bound."""
    g, u, (a, da, p) = gated_reference(gate, up, xq, xs, kind)
    sg, su = gate[1].astype(np.float64), up[1].astype(np.float64)
    raw = d64 * u * da
    dg, du = raw * sg, d64 * a * su
    sig = np.where(g != 0, a / np.where(g != 0, g, 1), 0.5)
    terms = np.abs(sig) + np.abs(da - sig) * 2
    eg = np.abs(d64 * u * sg) * terms * (2 * i8.act_rel(p) + 8 * 2.0 ** -24)
    eu = np.abs(du) * i8.act_rel(p)
    top = np.abs(d64 * sg * su).max(-1)
    least = 2.0 ** -34 * 1.13 * top * np.abs(xs.astype(np.float64)) * 128 * np.abs(xq.astype(np.float64)).sum(-1)
    eg, eu = (e + 2.0 ** -11 * (np.abs(v) + e) + least[:, None] for e, v in ((eg, dg), (eu, du)))
    qg, qu = gate[0].astype(np.float64), up[0].astype(np.float64)
    want = dg @ qg + du @ qu
    size = (np.abs(dg) + eg) @ np.abs(qg) + (np.abs(du) + eu) @ np.abs(qu)
    return want, eg @ np.abs(qg) + eu @ np.abs(qu) + grad_tolerance(size, 2 * dg.shape[1], want, t), raw


def check(gate, up, xq, xs, dh, d64, kind, t):
    want, tol, dg = want_and_tolerance(gate, up, xq, xs, d64, kind, t)
    assert np.abs(want).max() < 30000  # (the result itself fits its type)
    got, _ = gq.gated_i8_backward(matrix(*gate), matrix(*up), *matrix(xq, xs), dh, act=kind)
    near(got, want, tol, "dX")
    return dg


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("N", [1, 30, 130])
def test_gradients_of_g_beyond_binary16(N, kind):
    """Loss scaling: dh near the largest binary16 value, dg above it, dX far below."""
    I, H = 40, 64
    gate, up = scaled(1, I, H, 2.0 ** -17), scaled(2, I, H, 2.0 ** -7)
    xq, xs = scaled(3, N, H, 2.0 ** -6)
    dh, d64 = floats(4, N, I, "f16", 2.0 ** 14)
    assert np.isfinite(d64).all()
    dg = check(gate, up, xq, xs, dh, d64, kind, "f16")
    assert np.abs(dg).max() > 1.5 * 65504


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("N", [1, 30, 130])
def test_gradients_of_g_below_binary16(N, kind):
    """dh and dg of a few of binary16's smallest steps, large weights, dX of ordinary size."""
    torch = torch_cuda()
    I, H = 50, 70
    gate, up = scaled(5, I, H, 1.0), scaled(6, I, H, 1.0)
    xq, xs = scaled(7, N, H, 2.0 ** -17)
    steps = np.random.default_rng(8).integers(-15, 16, (N, I)).astype(np.float32)
    d64 = steps.astype(np.float64) * 2.0 ** -24
    dh = dev((steps * np.float32(2.0 ** -24))).to(torch.float16)
    assert (values(dh) == d64).all()
    dg = check(gate, up, xq, xs, dh, d64, kind, "f16")
    assert 0 < np.median(np.abs(dg)) < 2.0 ** -20


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("I", [1, 4, 9])
def test_sums_that_cancel(I, t, kind):
    """Few terms: what an operand loses shows where the result is small."""
    H, N = 300, 70
    gate, up = scaled(9, I, H, 2.0 ** -8), scaled(10, I, H, 2.0 ** -8)
    xq, xs = scaled(11, N, H, 2.0 ** -8)
    dh, d64 = floats(12, N, I, t)
    check(gate, up, xq, xs, dh, d64, kind, t)


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_scales_of_many_sizes(t):
    """Weight rows and tokens between 2^-30 and 2^12 side by side."""
    I, H, N = 90, 65, 40
    g = np.random.default_rng(13)
    gate = (scaled(14, I, H, 1)[0], (2.0 ** g.uniform(-30, 0, I)).astype(np.float32))
    up = (scaled(15, I, H, 1)[0], (2.0 ** g.uniform(-30, 0, I)).astype(np.float32))
    xq, xs = scaled(16, N, H, 1)[0], (2.0 ** g.uniform(-20, -12, N)).astype(np.float32)
    dh, d64 = floats(17, N, I, t)
    check(gate, up, xq, xs, dh, d64, "silu", t)


def test_bfloat16_range():
    """Gradients, scales and results near both ends of bfloat16's exponents."""
    I, H, N = 30, 40, 20
    for ed, es in ((100, -40), (-100, 20), (-60, -20), (60, 5)):
        gate, up = scaled(18, I, H, 2.0 ** es), scaled(19, I, H, 2.0 ** es)
        xq, xs = scaled(20, N, H, 2.0 ** (-es - 12))
        dh, d64 = floats(21, N, I, "bf16", 2.0 ** ed)
        want, tol, _ = want_and_tolerance(gate, up, xq, xs, d64, "silu", "bf16")
        assert np.isfinite(want).all()
        got, _ = gq.gated_i8_backward(matrix(*gate), matrix(*up), *matrix(xq, xs), dh)
        near(got, want, tol, "2^%d, 2^%d" % (ed, es))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("I,H,N", [(77, 130, 40), (64, 128, 3), (520, 96, 200)])
def test_zeros_infinities_and_nan_stay_in_their_rows(I, H, N, t):
    torch = torch_cuda()
    gate, up = scaled(22, I, H, 2.0 ** -10), scaled(23, I, H, 2.0 ** -10)
    for m in (gate, up):
        m[0][m[0] == 0] = 1
    xq, xs = scaled(24, N, H, 2.0 ** -8)
    dh, _ = floats(25, N, I, t)
    G, U = matrix(*gate), matrix(*up)
    ref = values(gq.gated_i8_backward(G, U, *matrix(xq, xs), dh)[0])
    assert np.isfinite(ref).all()
    dh[0] = 0
    dh[1, I - 1], dh[2, 0] = float("inf"), float("nan")
    rows = [0, 1, 2]
    if N > 3:
        xs[5], xq[6], xs[7] = np.nan, 0, 0
        rows += [5, 6, 7]
    got = values(gq.gated_i8_backward(G, U, *matrix(xq, xs), dh)[0])
    rest = np.setdiff1d(np.arange(N), rows)
    assert (got[rest] == ref[rest]).all()
    assert (got[0] == 0).all() and not np.isfinite(got[1]).any() and np.isnan(got[2]).all()
    if N > 3:
        assert np.isnan(got[5]).all() and (got[6] == 0).all() and (got[7] == 0).all()
    # a weight row of scale zero gives nothing, one of scale NaN reaches every token
    zero = (gate[0], np.where(np.arange(I) == I // 2, 0, gate[1]).astype(np.float32))
    w, _, _ = want_and_tolerance(zero, up, *scaled(24, N, H, 2.0 ** -8), values(floats(25, N, I, t)[0]), "silu", t)
    x2 = matrix(*scaled(24, N, H, 2.0 ** -8))
    got = values(gq.gated_i8_backward(matrix(*zero), U, *x2, floats(25, N, I, t)[0])[0])
    assert np.isfinite(got).all() and np.abs(got - w).max() <= 0.02 * np.abs(w).max()
    nan = (gate[0], np.where(np.arange(I) == I // 2, np.nan, gate[1]).astype(np.float32))
    got = values(gq.gated_i8_backward(matrix(*nan), U, *x2, floats(25, N, I, t)[0])[0])
    assert np.isnan(got).all()
    torch.cuda.synchronize()


def test_a_workspace_and_its_neighbour():
    """The documented workspace is enough, and calls of two sizes may take turns in one."""
    torch = torch_cuda()
    sets = []
    for i, (I, H, N) in enumerate([(64, 96, 200), (130, 2000, 3), (700, 300, 70)]):
        gate, up = scaled(30 + i, I, H, 2.0 ** -9), scaled(40 + i, I, H, 2.0 ** -9)
        dh, _ = floats(50 + i, N, I, "bf16")
        sets.append((matrix(*gate), matrix(*up), *matrix(*scaled(60 + i, N, H, 2.0 ** -8)), dh))
    need = [gq.gq_gated_i8_backward_workspace_bytes(s[4].shape[0], s[0][0].shape[1], s[0][0].shape[0]) for s in sets]
    buf = torch.full((max(need) + 64,), 9, dtype=torch.uint8, device="cuda")
    alone = [values(gq.gated_i8_backward(*s)[0]) for s in sets]
    for i in (0, 1, 2, 1, 0):
        got, _ = gq.gated_i8_backward(*sets[i], ws=buf[:need[i]])
        assert (values(got) == alone[i]).all()
    assert (buf[max(need):] == 9).all()
