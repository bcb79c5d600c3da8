"""The int8 operators on the GPU, against plain arithmetic in whole numbers and binary64
(tests/_i8.py).  Products of codes are whole numbers and their scaling is three documented
binary32 roundings, so quantiser, gemv and gemm are compared bit for bit."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _i8 as i8
from tests._gpu import dev, host, torch_cuda
from tests._mxfp4 import EPS2

pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]


def ttype(t):
    torch = torch_cuda()
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[t]


def values(t):
    """A device tensor as binary64."""
    return host(t.float()).astype(np.float64)


def floats(seed, n, K, t, scale=1.0):
    """(device tensor [n][K] of the type, its values in binary64)."""
    g = np.random.default_rng([seed, n, K])
    x = dev((g.standard_normal((n, K)) * scale).astype(np.float32)).to(ttype(t))
    return x, values(x)


def matrix(q, s, extra=0, fill=0x55):
    """Codes and scales on the device; rows a multiple of 16 bytes apart, what lies between
    them filled with codes that count if they are read as such."""
    n, K = q.shape
    ld = (K + 15) // 16 * 16 + 16 * extra
    buf = np.full((n, ld), fill, np.int8)
    buf[:, :K] = q
    return dev(buf)[:, :K], dev(s)


def same(got, want, what):
    g = values(got) if not isinstance(got, np.ndarray) else got
    bad = ~((g == want) | (np.isnan(g) & np.isnan(want)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d differ; first at %s: %r, expected %r"
                             % (what, bad.sum(), bad.size, i, g[i], want[i]))


def near(got, want, tol, what):
    g = values(got)
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        e = np.where(bad, np.nan_to_num(np.abs(g - want) / tol, nan=np.inf), 0)
        i = np.unravel_index(np.argmax(e), e.shape)
        raise AssertionError("%s: %d of %d out of tolerance; worst at %s: %r, expected %r within %r"
                             % (what, bad.sum(), bad.size, i, g[i], want[i], tol[i]))


# -- quantiser -----------------------------------------------------------------

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N,K", [(1, 1), (1, 7), (3, 8), (5, 15), (2, 64), (7, 100), (1, 4096),
                                 (3, 2049), (65, 257), (2, 14336), (2, 20011), (1, 70001)])
def test_quantize_exact(N, K, t):
    x, x64 = floats(1, N, K, t, 3.0)
    q, s = gq.quantize_i8(x)
    rq, rs = i8.quantize(x64)
    same(host(q).astype(np.float64), rq.astype(np.float64), "codes")
    same(s, rs.astype(np.float64), "scales")
    assert q.stride(0) % 16 == 0
    for td in TYPES:
        same(gq.dequant_i8(q, s, ttype(td)), i8.round_to(rq.astype(np.float32) * rs[:, None], td),
             "values")


@pytest.mark.parametrize("t", TYPES)
def test_quantize_borders(t):
    """Halves of codes and their neighbours, at the tie 63.5 of every row and where 127 divides
    the largest magnitude; magnitudes from subnormals to the largest."""
    rows = []
    half = {"f32": np.float32, "f16": np.float16, "bf16": np.float32}[t]
    for top in (127.0, 254.0, 4.0, 3.0, 1.9921875, 100.0):
        r = [top] + [top * (k + 0.5) / 127 for k in range(127)] + [top / 2, -top / 2, 0.0, -top]
        rows.append(r)
    x = np.array(rows, np.float32)
    torch = torch_cuda()
    base = dev(x).to(ttype(t))
    near_ = [base]
    if t == "f32":
        near_ += [dev(np.nextafter(x, np.float32(np.inf))), dev(np.nextafter(x, np.float32(-np.inf)))]
        for e in (-140, -126, -100, -61, -60, 60, 120):
            near_.append(dev(np.ldexp(x, e).astype(np.float32)))
    if t == "bf16":
        near_ += [(base.float() * 2.0 ** e).to(base.dtype) for e in (-126, -61, 100)]
    if t == "f16":
        near_ += [(base.float() * 2.0 ** e).half() for e in (-20, -14, 7)]
    xs = torch.cat(near_).contiguous()
    q, s = gq.quantize_i8(xs)
    rq, rs = i8.quantize(values(xs))
    same(host(q).astype(np.float64), rq.astype(np.float64), "codes")
    same(s, rs.astype(np.float64), "scales")


@pytest.mark.parametrize("t", TYPES)
def test_quantize_nonfinite_and_zero_rows(t):
    x, x64 = floats(2, 9, 333, t)
    x[1, 5], x[3, 332], x[5, 0] = float("inf"), float("nan"), float("-inf")
    x[7] = 0
    q, s = gq.quantize_i8(x)
    rq, rs = i8.quantize(values(x))
    assert np.isnan(rs[[1, 3, 5]]).all() and rs[7] == 0
    same(host(q).astype(np.float64), rq.astype(np.float64), "codes")
    same(s, rs.astype(np.float64), "scales")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("K", [100, 128])
def test_quantize_strided_and_bounds(K, t):
    """Rows of a wider matrix in, into columns of a wider one out; nothing else is written."""
    torch = torch_cuda()
    wide, _ = floats(3, 6, 301, t)
    x = wide[:, 3:3 + K] if t != "f32" else wide[:, 4:4 + K]
    # a base pointer is 16-byte aligned: start the view where it is
    off = 8 if t != "f32" else 4
    x = wide[:, off:off + K]
    buf = torch.full((6, 192), 77, dtype=torch.int8, device="cuda")
    s = torch.full((9,), -1.0, device="cuda")
    gq.quantize_i8(x, out=(buf[:, 32:32 + K], s[:6]))
    rq, rs = i8.quantize(values(x))
    b = host(buf).astype(np.float64)
    same(b[:, 32:32 + K], rq.astype(np.float64), "codes")
    assert (b[:, :32] == 77).all() and (b[:, 32 + K:] == 77).all()
    same(s, np.concatenate([rs, [-1, -1, -1]]).astype(np.float64), "scales")


# -- products ------------------------------------------------------------------

PRODUCTS = [  # M, K, N
    (1, 1, 1), (5, 15, 2), (16, 16, 3), (17, 17, 4), (31, 63, 5), (64, 64, 16), (33, 65, 17),
    (100, 127, 31), (128, 128, 32), (130, 129, 33), (65, 255, 64), (257, 256, 65), (96, 300, 77),
    (520, 1000, 130), (1003, 2083, 77), (300, 4096, 8), (129, 511, 257), (256, 384, 256),
    (700, 640, 300), (2050, 1030, 1), (64, 5000, 16), (1, 4099, 200), (4099, 96, 1), (1, 2, 600),
    (512, 512, 513),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K,N", PRODUCTS)
def test_gemm(M, K, N, t):
    wq, ws = i8.rows(10, M, K, -128, 127)
    xq, xs = i8.rows(11, N, K, -128, 127)
    W, X = matrix(wq, ws, extra=M % 3), matrix(xq, xs, extra=N % 2, fill=-0x56)
    same(gq.gemm_i8(*W, *X, dtype=ttype(t)), i8.round_to(i8.product(wq, ws, xq, xs), t), "gemm")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (15, 16), (16, 17), (100, 64), (33, 127), (260, 1000),
                                 (70, 4096), (4100, 130), (40, 14336), (37, 9999), (20, 70001),
                                 (50, 4097), (33, 8192), (9010, 8193), (17, 16384), (16, 16385)])
@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 8, 16])
def test_gemv(M, K, B, t):
    wq, ws = i8.rows(12, M, K, -128, 127)
    x, x64 = floats(13, B, K, t, 2.0)
    xq, xs = i8.quantize(x64)
    W = matrix(wq, ws, extra=M % 2)
    y = gq.gemv_i8(*W, x)
    same(y, i8.round_to(i8.product(wq, ws, xq, xs), t), "gemv")


def test_sums_at_the_ends_of_32_bits():
    """K = 131071 of the largest products of both signs."""
    K = 131071
    wq = np.full((18, K), -128, np.int8)
    xq = np.full((130, K), -128, np.int8)
    xq[1], xq[2, ::2] = 127, 127
    wq[3] = 127
    one = np.ones(130, np.float32)
    W = matrix(wq, one[:18])
    for N in (1, 5, 17, 130):
        ref = i8.product(wq, one[:18], xq[:N], one[:N])
        assert ref.max() == np.float32(131071 * 16384)
        same(gq.gemm_i8(*W, *matrix(xq[:N], one[:N])), ref.astype(np.float64), "gemm %d" % N)


@pytest.mark.parametrize("N", [1, 4, 16, 40, 70, 300])
def test_scales_reach_their_rows_only(N):
    """Infinite, NaN, zero and extreme scales of weights and tokens; a token holding an
    infinity."""
    M, K = 150, 200
    wq, ws = i8.rows(14, M, K)
    x, _ = floats(15, N, K, "f32")
    ws[3], ws[77], ws[100], ws[101], ws[149] = np.inf, np.nan, 0, 3e38, 1e-42
    if N > 3:
        x[1, 7], x[2] = float("inf"), 0
        x[3] *= 1e-30
    xq, xs = i8.quantize(values(x))
    ref = i8.product(wq, ws, xq, xs).astype(np.float64)
    W = matrix(wq, ws)
    same(gq.gemm_i8(*W, *gq.quantize_i8(x)), ref, "gemm")
    if N <= 16:
        same(gq.gemv_i8(*W, x), ref, "gemv")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N", [1, 16, 50, 150])
def test_outputs_stay_in_bounds(N, t):
    """Outputs lie inside a larger buffer whose other values stay."""
    torch = torch_cuda()
    M, K = 77, 130
    wq, ws = i8.rows(16, M, K)
    xq, xs = i8.rows(17, N, K)
    W, X = matrix(wq, ws), matrix(xq, xs)
    up, us = i8.rows(18, M, K)
    U = matrix(up, us)
    dy, _ = floats(19, N, M, "bf16" if t == "f32" else t)

    def guarded(n, call, dtype):
        buf = torch.full((n + 64,), 5.0, dtype=dtype, device="cuda")
        off = 16
        call(buf[off:off + n])
        b = host(buf.float())
        assert (b[:off] == 5).all() and (b[off + n:] == 5).all()
        assert (b[off:off + n] != 5).any()

    guarded(N * M, lambda o: gq.gemm_i8(*W, *X, out=o.view(N, M)), ttype(t))
    guarded(N * M, lambda o: gq.gated_i8(W, U, *X, out=o.view(N, M)), ttype(t))
    if N <= 16:
        x, _ = floats(20, N, K, t)
        guarded(N * M, lambda o: gq.gemv_i8(*W, x, out=o.view(N, M)), ttype(t))
    guarded(N * K, lambda o: gq.gemm_i8_backward(*W, dy, out=o.view(N, K)), dy.dtype)
    guarded(N * K, lambda o: gq.gated_i8_backward(W, U, *X, dy, out=o.view(N, K)), dy.dtype)
    need = gq.gq_gated_i8_backward_workspace_bytes(N, K, M)
    ws = torch.full((need + 64,), 9, dtype=torch.uint8, device="cuda")
    gq.gated_i8_backward(W, U, *X, dy, ws=ws[:need])
    assert (host(ws)[need:] == 9).all()
    D = matrix(*i8.rows(21, K, M))
    xf, _ = floats(22, N, K, "bf16" if t == "f32" else t)
    need = gq.gq_ffn_i8_workspace_bytes(N, K, M)
    ws = torch.full((need + 64,), 9, dtype=torch.uint8, device="cuda")
    guarded(N * K, lambda o: gq.ffn_i8(W, U, D, xf, ws=ws[:need], out=o.view(N, K)), xf.dtype)
    assert (host(ws)[need:] == 9).all()


# -- the gated half ----------------------------------------------------------------

GATED = [  # I, H, N
    (1, 1, 1), (7, 16, 2), (16, 100, 1), (40, 64, 5), (33, 130, 16), (129, 200, 17), (64, 128, 64),
    (100, 127, 65), (128, 256, 33), (517, 1003, 77), (300, 384, 130), (257, 512, 300), (1030, 96, 3),
    (256, 640, 256), (2, 5000, 4),
]


def gated_reference(gate, up, xq, xs, kind):
    g = i8.product(*gate, xq, xs).astype(np.float64)
    u = i8.product(*up, xq, xs).astype(np.float64)
    return g, u, i8.act(g, kind)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("I,H,N", GATED)
def test_gated(I, H, N, t, kind):
    gate, up = i8.rows(30, I, H), i8.rows(31, I, H)
    xq, xs = i8.rows(32, N, H)
    g, u, (a, _, p) = gated_reference(gate, up, xq, xs, kind)
    h = a * u
    # sigmoid's error, two products and a quotient; below 2^-126 the sigmoid may be zero
    tol = np.abs(h) * i8.act_rel(p) + np.abs(g * u) * 2.0 ** -125 + 2.0 ** -149
    tol = tol + i8.half_step(np.abs(h) + tol, t)
    got = gq.gated_i8(matrix(*gate), matrix(*up, extra=1), *matrix(xq, xs), act=kind, dtype=ttype(t))
    near(got, h, tol, "gated")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_far_arguments(kind):
    """g from -1e6 to 1e6: the activation's ends, forward and backward, no NaN."""
    torch = torch_cuda()
    H = 16
    z = np.concatenate([np.linspace(-30, 30, 241), [-1e6, -1e4, -300, -90, -88, -87, 87, 300, 1e6, 0.0]])
    I = z.size
    gate = (np.eye(1, H, dtype=np.int8).repeat(I, 0), z.astype(np.float32))
    up = (np.eye(1, H, dtype=np.int8).repeat(I, 0), np.full(I, 1.0, np.float32))
    xq, xs = np.eye(1, H, dtype=np.int8), np.ones(1, np.float32)
    zz = z.astype(np.float32).astype(np.float64)[None]
    a, da, p = i8.act(zz, kind)
    tol = np.abs(a) * i8.act_rel(p) + np.abs(zz) * 2.0 ** -125 + 2.0 ** -149
    got = gq.gated_i8(matrix(*gate), matrix(*up), *matrix(xq, xs), act=kind)
    near(got, a, tol + i8.half_step(a, "f32"), "h")
    # one gradient at a time through the gate row: dx[0] = dh u act'(z) z + dh act(z)
    for i in list(range(0, I, 40)) + list(range(241, I)):
        dh = torch.zeros((1, I), dtype=torch.bfloat16, device="cuda")
        dh[0, i] = 1.0
        dx, _ = gq.gated_i8_backward(matrix(*gate), matrix(*up), *matrix(xq, xs), dh, act=kind)
        assert np.isfinite(values(dx)).all()
        want = da[0, i] * zz[0, i] + a[0, i]
        size = abs(da[0, i] * zz[0, i]) + abs(a[0, i])
        # dg and du rounded to bfloat16 each, and the result
        assert abs(values(dx)[0, 0] - want) <= size * 2.1 * 2.0 ** -8 + 1e-6, (z[i], values(dx)[0, 0], want)


# -- gradients -----------------------------------------------------------------

GRADS = [  # M, K, N
    (1, 1, 1), (8, 16, 2), (15, 17, 3), (16, 64, 16), (33, 130, 17), (64, 128, 64), (63, 127, 65),
    (100, 300, 33), (130, 64, 130), (257, 513, 257), (1003, 77, 40), (520, 256, 256), (77, 1003, 5),
    (2083, 100, 77), (128, 640, 300), (4096, 64, 1), (65, 2050, 1),
]


def grad_tolerance(size, rows, want, t):
    """size = sum |d||w16|: the sums' roundings (rows + 1 additions of binary32; subnormal
    operands' products down to 2^-149 each) and the result's."""
    e = size * (rows + 1) * 2.0 ** -24 + rows * 2.0 ** -149
    return e + i8.half_step(np.abs(want) + e, t)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", GRADS)
def test_gemm_backward(M, K, N, t):
    wq, ws = i8.rows(40, M, K, -128, 127)
    dy, d64 = floats(41, N, M, t)
    w = i8.weights16(wq, ws, t)
    want = d64 @ w
    tol = grad_tolerance(np.abs(d64) @ np.abs(w), M, want, t)
    near(gq.gemm_i8_backward(*matrix(wq, ws, extra=K % 2), dy), want, tol, "dX")


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("ld", [96, 104, 99, 101])
def test_gemm_backward_rows_apart(ld, t):
    """Rows of dY any distance apart, what lies between them NaN."""
    torch = torch_cuda()
    M, K, N = 93, 150, 37
    wq, ws = i8.rows(42, M, K)
    _, d64 = floats(43, N, M, t)
    buf = torch.full((N, ld), float("nan"), dtype=ttype(t), device="cuda")
    buf[:, :M] = dev(d64.astype(np.float32)).to(ttype(t))
    w = i8.weights16(wq, ws, t)
    want = d64 @ w
    tol = grad_tolerance(np.abs(d64) @ np.abs(w), M, want, t)
    near(gq.gemm_i8_backward(*matrix(wq, ws), buf[:, :M]), want, tol, "dX")


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_gemm_backward_nonfinite(t):
    """An infinite or NaN gradient stays in its row, an infinite weight scale reaches all rows
    with a gradient there."""
    M, K, N = 100, 70, 40
    wq, ws = i8.rows(44, M, K)
    wq[wq == 0] = 1
    dy, d64 = floats(45, N, M, t)
    dy[3, 7], dy[39, 99] = float("inf"), float("nan")
    got = values(gq.gemm_i8_backward(*matrix(wq, ws), dy))
    bad = ~np.isfinite(got)
    assert bad[3].all() and bad[39].all() and np.isnan(got[39]).all()
    assert not bad[np.setdiff1d(np.arange(N), [3, 39])].any()
    assert np.isinf(got[3]).all()
    ws[50] = np.inf
    got = values(gq.gemm_i8_backward(*matrix(wq, ws), floats(45, N, M, t)[0]))
    assert not np.isfinite(got).any()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("I,H,N", GATED)
def test_gated_backward(I, H, N, t, kind):
    gate, up = i8.rows(30, I, H), i8.rows(31, I, H)
    xq, xs = i8.rows(32, N, H)
    dh, d64 = floats(46, N, I, t)
    g, u, (a, da, p) = gated_reference(gate, up, xq, xs, kind)
    dg, du = d64 * u * da, d64 * a
    # act' = sig + z p' sig (1 - sig): the errors of its two terms, each relative
    sig = np.where(g != 0, a / np.where(g != 0, g, 1), 0.5)
    terms = np.abs(sig) + np.abs(da - sig) * 2
    eg = np.abs(d64 * u) * terms * (2 * i8.act_rel(p) + 8 * 2.0 ** -24) + 2.0 ** -120
    eu = np.abs(du) * i8.act_rel(p) + 2.0 ** -120
    # operands: the gradients times the scales' fractions, rounded; codes times powers of two
    (fg, pg), (fu, pu) = i8.split_scales(gate[1]), i8.split_scales(up[1])
    wg, wu = gate[0] * pg[:, None], up[0] * pu[:, None]
    dg, du, eg, eu = dg * fg, du * fu, eg * fg, eu * fu
    eg, eu = eg + i8.half_step(np.abs(dg) + eg, t), eu + i8.half_step(np.abs(du) + eu, t)
    want = dg @ wg + du @ wu
    size = (np.abs(dg) + eg) @ np.abs(wg) + (np.abs(du) + eu) @ np.abs(wu)
    tol = eg @ np.abs(wg) + eu @ np.abs(wu) + grad_tolerance(size, 2 * I, want, t)
    dx, _ = gq.gated_i8_backward(matrix(*gate, extra=1), matrix(*up), *matrix(xq, xs), dh, act=kind)
    near(dx, want, tol, "dX")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradient_against_differences(kind):
    """dX against central differences of the formula in binary64, along random directions of the
    token values."""
    I, H, N = 120, 90, 6
    gate, up = i8.rows(50, I, H), i8.rows(51, I, H)
    xq, xs = i8.rows(52, N, H)
    xs = xs * 4
    dh, d64 = floats(53, N, I, "f16")
    dx, _ = gq.gated_i8_backward(matrix(*gate), matrix(*up), *matrix(xq, xs), dh, act=kind)
    wg, wu = (m[0].astype(np.float64) * m[1].astype(np.float64)[:, None] for m in (gate, up))
    x = xq.astype(np.float64) * xs.astype(np.float64)[:, None]

    def loss(x):
        return ((i8.act(x @ wg.T, kind)[0] * (x @ wu.T)) * d64).sum(-1)

    g = np.random.default_rng(54)
    a, da, _ = i8.act(x @ wg.T, kind)
    # dg, du and the result are each rounded to 16 bits: a half step of every term and one of
    # the result, along v (and their binary32 errors, far smaller)
    size = np.abs(d64 * (x @ wu.T) * da) @ np.abs(wg) + np.abs(d64 * a) @ np.abs(wu)
    for _ in range(5):
        v = g.standard_normal((N, H))
        eps = 1e-5
        diff = (loss(x + eps * v) - loss(x - eps * v)) / (2 * eps)
        got = (values(dx) * v).sum(-1)
        tol = (size * np.abs(v)).sum(-1) * 2.5 * EPS2["f16"] + 1e-6 * np.abs(diff)
        assert (np.abs(got - diff) <= tol).all(), (got, diff, tol)


# -- the block -----------------------------------------------------------------

FFN = [  # T, H, I
    (1, 1, 1), (1, 64, 128), (1, 100, 77), (2, 256, 300), (4, 130, 515), (5, 1000, 64), (8, 96, 2100),
    (16, 128, 256), (17, 128, 256), (33, 200, 130), (64, 64, 512), (70, 300, 517), (130, 257, 384),
    (300, 512, 256), (3, 4096, 1030), (1, 1030, 14336), (16, 300, 9000),
]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,I", FFN)
def test_ffn_is_its_parts(T, H, I, t, kind):
    """The block equals quantiser, gated half, quantiser and product one after another, bit for
    bit; those are tested above."""
    G, U, D = (matrix(*i8.rows(60 + i, *s)) for i, s in enumerate([(I, H), (I, H), (H, I)]))
    x, _ = floats(63, T, H, t, 0.7)
    out, _ = gq.ffn_i8(G, U, D, x, act=kind)
    h = gq.gated_i8(G, U, *gq.quantize_i8(x), act=kind, dtype=x.dtype)
    want = gq.gemm_i8(*D, *gq.quantize_i8(h), dtype=x.dtype)
    same(out, values(want), "ffn")
    if T <= 16:
        same(gq.gemv_i8(*D, h), values(want), "gemv of h")


@pytest.mark.parametrize("T", [1, 3, 40])
def test_ffn_against_the_definition(T):
    """The block against its formula in binary64: with the codes of h free to move one step where
    h lies on a border."""
    H, I, t = 200, 300, "bf16"
    gate, up, down = i8.rows(64, I, H), i8.rows(65, I, H), i8.rows(66, H, I)
    x, x64 = floats(67, T, H, t)
    xq, xs = i8.quantize(x64)
    g, u, (a, _, _) = gated_reference(gate, up, xq, xs, "silu")
    h = i8.round_to((a * u).astype(np.float32), t)
    hq, hs = i8.quantize(h)
    want = i8.product(*down, hq, hs).astype(np.float64)
    out, _ = gq.ffn_i8(*(matrix(*m) for m in (gate, up, down)), x)
    # a value of h within binary32 error of a bfloat16 border may round to the next: 2^-8
    # relative, which moves its code by at most one (and its row's scale by 2^-7)
    edge = np.abs(h) * 2.0 ** -7 + hs[:, None] * 1.01
    near_border = np.abs(a * u - h) > i8.EPS2[t] * np.abs(h) * 0.99
    wabs = np.abs(down[0].astype(np.float64)) * down[1].astype(np.float64)[:, None]
    tol = (edge * near_border) @ wabs.T + i8.half_step(want, t) + np.abs(want) * 2.0 ** -20
    top = np.argmax(np.abs(h), -1)
    assert not near_border[np.arange(T), top].any()  # (the scales are exact for this seed)
    near(out, want, tol, "ffn")


@pytest.mark.parametrize("T", [2, 30, 100])
def test_ffn_nonfinite_token(T):
    """A token with an infinity gives NaN, the others what they give without it."""
    H, I = 130, 200
    G, U, D = (matrix(*i8.rows(70 + i, *s)) for i, s in enumerate([(I, H), (I, H), (H, I)]))
    x, _ = floats(73, T, H, "f16")
    ref = values(gq.ffn_i8(G, U, D, x)[0])
    x[1, 3] = float("inf")
    got = values(gq.ffn_i8(G, U, D, x)[0])
    assert np.isnan(got[1]).all()
    keep = np.arange(T) != 1
    assert (got[keep] == ref[keep]).all()


# -- how they are called -------------------------------------------------------------

def step(G, U, D, x, dh, ws, wb):
    """Operators together as a training step on frozen weights uses them."""
    q, s = gq.quantize_i8(x)
    h = gq.gated_i8(G, U, q, s, dtype=x.dtype)
    y = gq.gemm_i8(*D, *gq.quantize_i8(h), dtype=x.dtype)
    dhh = gq.gemm_i8_backward(*D, dh)
    dx, _ = gq.gated_i8_backward(G, U, q, s, dhh, ws=wb)
    o, _ = gq.ffn_i8(G, U, D, x, ws=ws)
    return h, y, dhh, dx, o, gq.gemv_i8(*G, x[:3])


def step_setup(T=70, H=200, I=300):
    torch = torch_cuda()
    G, U, D = (matrix(*i8.rows(80 + i, *s)) for i, s in enumerate([(I, H), (I, H), (H, I)]))
    ws = torch.empty(gq.gq_ffn_i8_workspace_bytes(T, H, I), dtype=torch.uint8, device="cuda")
    wb = torch.empty(gq.gq_gated_i8_backward_workspace_bytes(T, H, I), dtype=torch.uint8, device="cuda")
    return G, U, D, ws, wb


def test_captured_and_replayed():
    torch = torch_cuda()
    T, H, I = 70, 200, 300
    G, U, D, ws, wb = step_setup(T, H, I)
    x, _ = floats(83, T, H, "bf16")
    dh, _ = floats(84, T, H, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(G, U, D, x, dh, ws, wb)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(G, U, D, x, dh, ws, wb)
    for i in range(4):
        x.copy_(floats(85 + i, T, H, "bf16")[0])
        dh.copy_(floats(90 + i, T, H, "bf16")[0])
        graph.replay()
        torch.cuda.synchronize()
        eager = step(G, U, D, x, dh, torch.empty_like(ws), torch.empty_like(wb))
        for n, (a, b) in enumerate(zip(outs, eager)):
            same(a, values(b), "replay %d output %d" % (i, n))


def test_two_streams_at_once():
    torch = torch_cuda()
    G, U, D, _, _ = step_setup()
    ins = [(floats(100 + i, 70, 200, "bf16")[0], floats(110 + i, 70, 200, "bf16")[0]) for i in range(2)]
    want = [[values(o) for o in step(G, U, D, *v, None, None)] for v in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [None, None]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i] = step(G, U, D, *ins[i], None, None)
    torch.cuda.synchronize()
    for i in range(2):
        for n, o in enumerate(outs[i]):
            same(o, want[i][n], "stream %d output %d" % (i, n))


def test_helpers_stream_argument_and_no_rows():
    torch = torch_cuda()
    G, U, D, _, _ = step_setup()
    x, _ = floats(120, 5, 200, "f16")
    s1 = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, s = gq.quantize_i8(x, stream=s1)
    y = gq.gemm_i8(*G, q, s, dtype=torch.float16, stream=s1.cuda_stream)
    dx = gq.gemm_i8_backward(*G, y, stream=s1)
    db, _ = gq.gated_i8_backward(G, U, q, s, y, stream=s1)
    f, _ = gq.ffn_i8(G, U, D, x, stream=s1)
    v = gq.gemv_i8(*G, x.view(5, 1, 200), stream=s1)
    w = gq.dequant_i8(q, s, stream=s1)
    torch.cuda.synchronize()
    same(y, values(gq.gemm_i8(*G, *gq.quantize_i8(x), dtype=torch.float16)), "gemm")
    same(v, values(y), "gemv")
    same(dx, values(gq.gemm_i8_backward(*G, y)), "dX")
    same(db, values(gq.gated_i8_backward(G, U, q, s, y)[0]), "dX of the gated half")
    same(f, values(gq.ffn_i8(G, U, D, x)[0]), "ffn")
    e = x[:0]
    q0, s0 = gq.quantize_i8(e)
    assert q0.shape == (0, 200) and s0.shape == (0,)
    assert gq.gemm_i8(*G, q0, s0).shape == (0, 300)
    assert gq.gemv_i8(*G, e).shape == (0, 300)
    assert gq.dequant_i8(q0, s0).shape == (0, 200)
    assert gq.gated_i8(G, U, q0, s0).shape == (0, 300)
    assert gq.gemm_i8_backward(*G, y[:0]).shape == (0, 200)
    assert gq.gated_i8_backward(G, U, q0, s0, y[:0])[0].shape == (0, 200)
    assert gq.ffn_i8(G, U, D, e)[0].shape == (0, 200)
    torch.cuda.synchronize()


def test_helper_refusals():
    torch = torch_cuda()
    G, U, D, ws, wb = step_setup()
    x, _ = floats(121, 70, 200, "f16")
    q, s = gq.quantize_i8(x)
    dh = torch.zeros((70, 300), dtype=torch.float16, device="cuda")
    flat = torch.zeros((70, 200), dtype=torch.int8, device="cuda")
    short = torch.zeros(69 * 208 + 200, dtype=torch.int8, device="cuda").as_strided((70, 200), (208, 1))
    bad = [
        lambda: gq.quantize_i8(x.t()), lambda: gq.quantize_i8(x[0]), lambda: gq.quantize_i8(q),
        lambda: gq.quantize_i8(x, out=(flat, s)), lambda: gq.quantize_i8(x, out=(q[:5], s[:5])),
        lambda: gq.dequant_i8(q, s.double()), lambda: gq.dequant_i8(q, s[:5]),
        lambda: gq.dequant_i8(q.t(), s), lambda: gq.dequant_i8(short, s),
        lambda: gq.gemv_i8(*G, x[:4, :100]), lambda: gq.gemv_i8(*G, x[:4].cpu()),
        lambda: gq.gemm_i8(*G, flat, s), lambda: gq.gemm_i8(*G, q[:, :192], s),
        lambda: gq.gemm_i8(*G, q, s, dtype=torch.float64),
        lambda: gq.gemm_i8(*G, q, s, out=torch.empty((70, 299), device="cuda")),
        lambda: gq.gemm_i8_backward(*G, dh.float()), lambda: gq.gemm_i8_backward(*G, dh[:, :200]),
        lambda: gq.gemm_i8_backward(*G, dh.t()),
        lambda: gq.gated_i8(G, D, q, s), lambda: gq.gated_i8(G, U, q, s, act="relu"),
        lambda: gq.gated_i8_backward(G, U, q, s, dh[:5]),
        lambda: gq.ffn_i8(G, U, G, x), lambda: gq.ffn_i8(G, U, D, x.float()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("call %d was not refused" % i)
    for f in (lambda: gq.gemv_i8(*G, x), lambda: gq.ffn_i8(G, U, D, x, ws=ws[:-16]),
              lambda: gq.gated_i8_backward(G, U, q, s, dh, ws=wb[:-16]),
              lambda: gq.ffn_i8(G, U, D, x, ws=ws[1:])):
        with pytest.raises(gq.GQError):
            f()
    torch.cuda.synchronize()
