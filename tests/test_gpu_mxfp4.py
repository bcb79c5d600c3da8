"""MXFP4 operators on the GPU against plain numpy arithmetic in 64 bits.

Tolerances.  Codes, scales and dequantised values are compared exactly.  Products
of MXFP4 weights with activations are exact in the kernels and sums run in
binary32: at most K/8 roundings follow one another (a matrix instruction adds 32
products or more to an accumulator, K is split over waves and joined), 2^-23 of S
each at the worst, S = sum |w x|; with the signs of random data they add up as a
walk and 1e-5 S, the library's contract for binary32 sums, is held for every K
here.  A 16-bit result adds half a step of its type, relative to the value."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _mxfp4 as mx
from tests._gpu import dev, host, say, torch_cuda

pytestmark = pytest.mark.gpu

SUM = 1e-5


def as_type(x, t):
    """x rounded to type t: (device tensor, its exact binary64 values)."""
    torch = torch_cuda()
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[t]
    d = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dt)
    return d.cuda(), d.double().numpy()


def values64(t):
    torch = torch_cuda()
    torch.cuda.synchronize()
    return t.double().cpu().numpy()


def check(y, ref, S, t, what, extra=0.0):
    bound = mx.EPS2[t] * np.abs(ref) + mx.TINY[t] + SUM * S * (1 + mx.EPS2[t]) + extra
    err = np.abs(values64(y) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %g of its bound at %s" % (
        what, bad.sum(), bad.size, np.nanmax(err / bound), np.argwhere(bad)[0])
    say("  ", what, "max err/bound %.3f" % (err / bound).max())


def normal(seed, *shape):
    g = np.random.default_rng([seed, *shape])
    return g.standard_normal(shape)


# -- quantisation ---------------------------------------------------------------

@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,K", [(1, 32), (3, 96), (1, 4096), (17, 2080), (64, 14336), (1, 64)])
def test_quantize_exact(N, K, t):
    x = normal(1, N, K) * np.exp2(np.random.default_rng(2).integers(-12, 8, (N, 1)))
    x[0, :32] = 0.0  # a block of zeros
    x[-1, -1] = -0.0
    xd, x64 = as_type(x, t)
    q, s = gq.quantize_mxfp4(xd)
    qr, sr = mx.quantize(x64)
    assert np.array_equal(host(s), sr)
    assert np.array_equal(host(q), qr)
    for dt, name in ((None, "f32"), (torch_cuda().bfloat16, "bf16")):
        v = gq.dequant_mxfp4(q, s, dtype=dt)
        ref = mx.values(qr, sr)
        got = values64(v)
        assert np.array_equal(got, ref) and np.array_equal(np.signbit(got), np.signbit(ref)), name


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_quantize_borders(t):
    """Values on and next to every rounding border, at every exponent of the type."""
    lo, hi = {"f32": (-149, 127), "f16": (-24, 15), "bf16": (-133, 127)}[t]
    torch = torch_cuda()
    rows = []
    for e in range(lo, hi + 1, 1 if t != "f32" else 3):
        b = np.array([1.0, 1.25, 1.5, 1.75, 1.875, 0.0625, 0.1875, 0.3125, 0.4375, 0.625, 0.875,
                      0.03125, 0.5, 0.75, 1.125, 0.25])
        b = np.concatenate([b, -b]) * 2.0 ** e
        with np.errstate(over="ignore"):
            rows.append(b)
    x = np.array(rows)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[t]
    d0 = torch.from_numpy(x).to(dt)
    d0 = torch.where(torch.isfinite(d0), d0, torch.zeros_like(d0))
    # the neighbours above and below each value, as bit patterns
    it = torch.int32 if t == "f32" else torch.int16
    bits = d0.view(it)
    for step in (0, 1, -1):
        nb = torch.where((bits & (0x7FFFFFFF if t == "f32" else 0x7FFF)) != 0, bits + step, bits)
        d = nb.view(dt)
        d = torch.where(torch.isfinite(d), d, torch.zeros_like(d))
        q, s = gq.quantize_mxfp4(d.cuda())
        qr, sr = mx.quantize(d.double().numpy())
        assert np.array_equal(host(s), sr), step
        assert np.array_equal(host(q), qr), step


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_quantize_nonfinite_blocks(t):
    x = normal(3, 4, 160)
    x[0, 5] = np.inf
    x[1, 40] = np.nan
    x[2, 159] = -np.inf
    x[2, 96] = np.nan
    xd, x64 = as_type(x, t)
    q, s = gq.quantize_mxfp4(xd)
    qr, sr = mx.quantize(x64)
    assert (sr == 255).sum() == 4
    assert np.array_equal(host(s), sr) and np.array_equal(host(q), qr)
    v = values64(gq.dequant_mxfp4(q, s)).reshape(4, 5, 32)
    assert np.array_equal(np.isnan(v).all(-1), sr == 255) and np.array_equal(np.isnan(v).any(-1), sr == 255)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_quantize_strided_rows_and_bounds(t):
    torch = torch_cuda()
    xd, x64 = as_type(normal(4, 9, 256), t)
    view = xd[:, 64:160]
    q, s = gq.quantize_mxfp4(view)
    qr, sr = mx.quantize(np.ascontiguousarray(x64[:, 64:160]))
    assert np.array_equal(host(q), qr) and np.array_equal(host(s), sr)
    # one row of a wider matrix; every second row
    q, s = gq.quantize_mxfp4(xd[3:4, 32:64])
    qr, sr = mx.quantize(np.ascontiguousarray(x64[3:4, 32:64]))
    assert np.array_equal(host(q), qr) and np.array_equal(host(s), sr)
    q, s = gq.quantize_mxfp4(xd[::2])
    qr, sr = mx.quantize(np.ascontiguousarray(x64[::2]))
    assert np.array_equal(host(q), qr) and np.array_equal(host(s), sr)
    # nothing beyond the planes is written
    qb = torch.full((9 * 48 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sb = torch.full((9 * 3 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    gq.gq_quantize_mxfp4(view, {"f32": 0, "f16": 1, "bf16": 2}[t], 256, qb, sb, 9, 96)
    assert (host(qb)[9 * 48:] == 0xA5).all() and (host(sb)[27:] == 0xA5).all()
    # misaligned views and rows are refused
    with pytest.raises(gq.GQError):
        gq.quantize_mxfp4(xd[:, 1:33])
    with pytest.raises(ValueError):
        gq.quantize_mxfp4(xd.t())
    with pytest.raises(gq.GQError):
        gq.quantize_mxfp4(xd[:, :40])


def test_dequant_every_code_and_scale():
    torch = torch_cuda()
    q = np.repeat(np.arange(256, dtype=np.uint8).reshape(1, 16, 16), 256, 0)
    s = np.repeat(np.arange(256, dtype=np.uint8).reshape(256, 1, 1), 16, 1)
    ref = mx.values(q, s)
    qd, sd = dev(q), dev(s)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        got = values64(gq.dequant_mxfp4(qd, sd, dtype=dt))
        # rounded to the type: with s = 253 and 254 the codes 4 and 6 (and 2, 3 for
        # 254) are 2^128 or more, beyond binary32 and bfloat16, i.e. infinity
        with np.errstate(over="ignore"):
            want = ref.astype(np.float16 if dt == torch.float16 else np.float32).astype(np.float64)
        assert np.array_equal(got, want, equal_nan=True), dt
        ok = ~np.isnan(ref)
        assert np.array_equal(np.signbit(got)[ok], np.signbit(ref)[ok])


# -- products -------------------------------------------------------------------

def weights(seed, M, K):
    q, s = mx.weights(seed, M, K)
    return dev(q), dev(s), mx.values(q, s)


@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 6, 7, 8, 11, 15, 16])
@pytest.mark.parametrize("M,K", [(16, 32), (1, 96), (33, 2080), (100, 4096), (515, 160), (64, 14336),
                                 # several chunks of x, two and four tiles a workgroup
                                 (40, 16512), (4112, 1056), (8200, 160), (8209, 2080)])
def test_gemv(M, K, B):
    q, s, W = weights(5, M, K)
    x = normal(6, B, K).astype(np.float32)
    y = gq.gemv_mxfp4(q, s, dev(x))
    ref, S = mx.products(W, x.astype(np.float64))
    check(y, ref, S, "f32", "gemv %d %d %d" % (M, K, B))
    assert np.array_equal(host(gq.gemv_mxfp4(q, s, dev(x))), host(y))  # fixed order


@pytest.mark.parametrize("B", [1, 4, 16])
def test_gemv_wide_range_activations(B):
    """Whole activations at full binary32 precision: each row a mix of magnitudes
    whose low bits matter, and one huge or tiny row."""
    M, K = 48, 1056
    q, s, W = weights(7, M, K)
    g = np.random.default_rng(8)
    x = (normal(9, B, K) * np.exp2(g.integers(-20, 20, (B, K)))).astype(np.float32)
    x[0] *= np.float32(2.0 ** 60)
    if B > 1:
        x[1] *= np.float32(2.0 ** -60)
    y = gq.gemv_mxfp4(q, s, dev(x))
    ref, S = mx.products(W, x.astype(np.float64))
    check(y, ref, S, "f32", "gemv range %d" % B)
    # one-hot rows read single weights exactly
    x = np.zeros((B, K), np.float32)
    cols = g.integers(0, K, B)
    x[np.arange(B), cols] = np.float32(1.2345678)
    y = gq.gemv_mxfp4(q, s, dev(x))
    ref = W[:, cols].T * np.float64(np.float32(1.2345678))
    assert np.array_equal(host(y), ref.astype(np.float32))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(16, 32, 1), (1, 64, 5), (40, 96, 16), (130, 2080, 17), (65, 160, 33),
                                   (256, 512, 64), (300, 1056, 65), (257, 4096, 130),
                                   (128, 14336, 7), (515, 288, 300), (1024, 1024, 512),
                                   # each tile, each way of reading scales, K runs of one chunk
                                   (4100, 1024, 1030), (4100, 1568, 1030), (14300, 1024, 1030),
                                   (14300, 96, 1030), (4096, 4096, 130), (4100, 1152, 130),
                                   (4100, 2080, 130), (1000, 768, 40), (1000, 800, 40),
                                   (16500, 640, 1030), (1000, 1024, 40), (100, 992, 200),
                                   # the same of the larger tiles, in whole rounds and halves
                                   (16500, 96, 400), (16500, 96, 900), (6200, 640, 1300),
                                   (6200, 512, 1300), (16500, 512, 900), (16500, 640, 200),
                                   (16500, 512, 77), (16500, 288, 17), (16500, 512, 17),
                                   (16500, 1024, 40), (8200, 1024, 40), (1000, 288, 17), (70, 256, 20), (70, 2048, 20)])
def test_gemm(M, K, N, t):
    q, s, W = weights(10, M, K)
    xd, x64 = as_type(normal(11, N, K), t)
    y = gq.gemm_mxfp4(q, s, xd)
    ref, S = mx.products(W, x64)
    check(y, ref, S, t, "gemm %s %d %d %d" % (t, M, K, N))
    assert np.array_equal(values64(gq.gemm_mxfp4(q, s, xd)), values64(y))


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(16, 32, 1), (1, 64, 5), (40, 96, 16), (130, 2080, 17), (65, 160, 33),
                                   (256, 512, 64), (300, 1056, 65), (257, 4096, 130),
                                   (128, 14336, 7), (515, 288, 300), (1024, 1024, 512),
                                   # each tile size, with and without whole 512-column chunks
                                   (4100, 512, 1030), (4100, 1568, 1030), (14300, 1024, 1030),
                                   (14300, 96, 1030), (16500, 640, 1100),
                                   (16500, 96, 300), (16500, 512, 300), (8200, 2080, 77),
                                   (8200, 1536, 77), (16500, 96, 400), (16500, 512, 400)])
def test_mxgemm(M, K, N, t):
    torch = torch_cuda()
    q, s, W = weights(12, M, K)
    xq, xs, X = weights(13, N, K)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[t]
    y = gq.gemm_mxfp4_mxfp4(q, s, xq, xs, dtype=dt)
    ref, S = mx.products(W, X)
    check(y, ref, S, t, "mxgemm %s %d %d %d" % (t, M, K, N))
    assert np.array_equal(values64(gq.gemm_mxfp4_mxfp4(q, s, xq, xs, dtype=dt)), values64(y))


def test_products_far_scales():
    """Scales at both ends: exact powers of two through every product; binary16
    weights round as documented."""
    M, K, N = 32, 128, 3
    q = np.full((M, K // 2), 0x22, np.uint8)  # every weight 1.0 * scale
    for sc in (60, 104, 127, 140, 180):
        s = np.full((M, K // 32), sc, np.uint8)
        W = mx.values(q, s)
        xd, x64 = as_type(np.ones((N, K)), "bf16")
        ref = x64 @ W.T
        assert np.array_equal(values64(gq.gemm_mxfp4(dev(q), dev(s), xd)), ref)
        assert np.array_equal(values64(gq.gemv_mxfp4(dev(q), dev(s), xd.float())), ref)
        xq, xs = gq.quantize_mxfp4(xd)
        assert np.array_equal(values64(gq.gemm_mxfp4_mxfp4(dev(q), dev(s), xq, xs)), ref)
        with np.errstate(over="ignore"):
            w16 = W.astype(np.float16).astype(np.float64)
            want = (x64 @ w16.T).astype(np.float16).astype(np.float64)
        got = values64(gq.gemm_mxfp4(dev(q), dev(s), xd.half()))
        assert np.array_equal(got, want), sc


@pytest.mark.parametrize("N", [1, 40, 300])
def test_nan_and_infinity_stay_in_their_rows(N):
    torch = torch_cuda()
    M, K = 300, 416
    q, s = mx.weights(14, M, K)
    q |= 0x11  # no zero weights
    s[7, 3] = 255
    W = mx.values(q, s)
    rows = np.arange(M) != 7
    x = normal(15, N, K)
    xd, x64 = as_type(x, "bf16")
    ref, S = mx.products(W[rows], x64)
    ys = [gq.gemm_mxfp4(dev(q), dev(s), xd)]
    if N <= 16:
        ys.append(gq.gemv_mxfp4(dev(q), dev(s), xd.float()))
    xq, xs = gq.quantize_mxfp4(xd)
    ys.append(gq.gemm_mxfp4_mxfp4(dev(q), dev(s), xq, xs))
    for i, y in enumerate(ys):
        v = values64(y)
        assert np.isnan(v[:, 7]).all() and np.isfinite(v[:, rows]).all(), i
    s[7, 3] = 120
    x[N // 2, K - 1] = np.inf
    xd, _ = as_type(x, "f16")
    for y in [gq.gemm_mxfp4(dev(q), dev(s), xd)] + ([gq.gemv_mxfp4(dev(q), dev(s), xd.float())] if N <= 16 else []):
        v = values64(y)
        assert not np.isfinite(v[N // 2]).any()
        assert np.isfinite(np.delete(v, N // 2, 0)).all()
    xq, xs = gq.quantize_mxfp4(xd)
    v = values64(gq.gemm_mxfp4_mxfp4(dev(q), dev(s), xq, xs))
    assert np.isnan(v[N // 2]).all() and np.isfinite(np.delete(v, N // 2, 0)).all()


def test_outputs_stay_in_bounds():
    torch = torch_cuda()
    for M, K, N in ((17, 96, 3), (270, 288, 70), (300, 160, 260)):
        q, s, _ = weights(16, M, K)
        xd, _ = as_type(normal(17, N, K), "f16")
        y = torch.full((N * M + 512,), 7.0, dtype=torch.float16, device="cuda")
        gq.gq_gemm_mxfp4(q, s, xd, y, gq.GQ_F16, M, K, N)
        assert (values64(y)[N * M:] == 7.0).all()
        xq, xs = gq.quantize_mxfp4(xd)
        y = torch.full((N * M + 512,), 7.0, dtype=torch.float32, device="cuda")
        gq.gq_gemm_mxfp4_mxfp4(q, s, xq, xs, y, gq.GQ_F32, M, K, N)
        assert (values64(y)[N * M:] == 7.0).all()
        B = min(N, 16)
        y = torch.full((B * M + 512,), 7.0, dtype=torch.float32, device="cuda")
        gq.gq_gemv_mxfp4(q, s, xd[:B].float(), y, M, K, B)
        assert (values64(y)[B * M:] == 7.0).all()


# -- mixture of experts ------------------------------------------------------------

def silu64(z):
    return z / (1.0 + np.exp(-z))


def moe_case(seed, T, H, I, E, topk, t, ids=None):
    g = np.random.default_rng([seed, T, H, I, E])
    st = {}
    for n, r, k in (("g", I, H), ("u", I, H), ("d", H, I)):
        q, s = mx.weights(seed + ord(n), E * r, k, 118, 123)
        st[n] = (dev(q.reshape(E, r, k // 2)), dev(s.reshape(E, r, k // 32)))
        st["W" + n] = mx.values(q, s).reshape(E, r, k)
    st["x"], st["X"] = as_type(normal(seed + 1, T, H) * 0.25, t)
    if ids is None:
        ids = np.argsort(g.random((T, E)), -1)[:, :topk]
    st["ids"] = np.ascontiguousarray(ids, np.int32)
    st["wts"] = g.random((T, topk)).astype(np.float32)
    return st


def moe_check(st, T, H, I, E, topk, t, iw, ws=None):
    """Stage by stage through the workspace: h from x, d from the GPU's own h, the
    output from the GPU's own d.  h = silu(g) u with g, u off by SUM * S each:
    |silu'| <= 1.1, |silu(z)| <= |z|, the exponential and the arithmetic of the
    epilogue within 2^-19 of h, then half a step of its type."""
    out, ws = gq.moe_mxfp4(st["g"], st["u"], st["d"], st["x"], dev(st["ids"]), dev(st["wts"]),
                           ws=ws, input_weighted=iw)
    A = T * topk
    flat = st["ids"].reshape(-1)
    valid = (flat >= 0) & (flat < E)
    up = lambda v: (v + 255) // 256 * 256
    o = [0]
    for n in ((E + 3) * 4, A * 4, A * 4, 2 * (A + E) * 4, A * I * 2, A * H * 4):
        o.append(up(o[-1] + n))
    raw = host(ws)
    assert raw.nbytes >= o[6]
    offs = raw[:(E + 3) * 4].view(np.int32)
    assert offs[E] == valid.sum() and offs[E + 2] == (~valid).sum()
    order = raw[o[1]:o[1] + 4 * A].view(np.int32)[:valid.sum()]
    assert np.array_equal(order, np.argsort(np.where(valid, flat, E), kind="stable")[:valid.sum()])
    hb = raw[o[4]:o[4] + 2 * A * I].view(np.uint16).reshape(A, I)[:valid.sum()]
    h = (hb.view(np.float16) if t == "f16" else mx.from_bf16_bits(hb)).astype(np.float64)
    d = raw[o[5]:o[5] + 4 * A * H].view(np.float32).reshape(A, H)[:valid.sum()].astype(np.float64)
    worst = [0.0, 0.0, 0.0]
    pos = np.full(A, -1)
    pos[order] = np.arange(len(order))
    w16 = (lambda W: W.astype(np.float16).astype(np.float64)) if t == "f16" else (lambda W: W)
    for e in range(E):
        sel = np.nonzero(flat[order] == e)[0]
        if not len(sel):
            continue
        X = st["X"][order[sel] // topk]
        pw = st["wts"].reshape(-1)[order[sel]].astype(np.float64)[:, None] if iw else 1.0
        g, Sg = mx.products(w16(st["Wg"][e]), X)
        u, Su = mx.products(w16(st["Wu"][e]), X)
        g, u, Sg, Su = g * pw, u * pw, Sg * pw, Su * pw
        ref = silu64(g) * u
        dg, du = (SUM + 2.0 ** -24) * Sg, (SUM + 2.0 ** -24) * Su
        slack = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 2.0 ** -19 * np.abs(ref)
        bound = mx.EPS2[t] * (np.abs(ref) + slack) + slack + mx.TINY[t]
        worst[0] = max(worst[0], (np.abs(h[sel] - ref) / bound).max())
        ref, S = mx.products(w16(st["Wd"][e]), h[sel])
        worst[1] = max(worst[1], (np.abs(d[sel] - ref) / (SUM * S + 1e-30)).max())
    wt = np.ones((T, topk)) if iw else st["wts"].astype(np.float64)
    dd = np.where(pos[:, None] >= 0, d[np.maximum(pos, 0)] if len(d) else 0.0, 0.0)
    terms = dd.reshape(T, topk, H) * wt[..., None]
    ref = terms.sum(1)
    bound = mx.EPS2[t] * np.abs(ref) + mx.TINY[t] + (topk + 1) * 2.0 ** -23 * np.abs(terms).sum(1)
    worst[2] = (np.abs(values64(out) - ref) / bound).max()
    say("   moe", T, H, I, E, topk, t, iw, "err/bound h %.3f d %.3f out %.3f" % tuple(worst))
    assert max(worst) <= 1.0, worst
    return out, ws


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("iw", [False, True])
@pytest.mark.parametrize("T,H,I,E,topk", [(1, 256, 128, 8, 2), (1, 32, 32, 1, 1), (4, 160, 96, 16, 4),
                                          (33, 288, 224, 4, 3), (70, 256, 256, 2, 1), (150, 512, 96, 4, 2),
                                          (700, 128, 160, 3, 2),
                                          # tiles of 32, 128 and 256 tokens, each way of reading
                                          # scales, remainders of more and fewer than 64 tokens
                                          (24, 512, 640, 8, 3), (40, 1024, 512, 4, 1),
                                          (61, 288, 1024, 2, 2), (130, 1024, 512, 4, 2),
                                          (210, 640, 96, 3, 2), (330, 512, 1056, 2, 1)])
def test_moe(T, H, I, E, topk, t, iw):
    moe_check(moe_case(20, T, H, I, E, topk, t), T, H, I, E, topk, t, iw)


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_moe_one_expert_takes_all_and_invalid_ids(t):
    T, H, I, E, topk = 90, 128, 64, 8, 2
    ids = np.zeros((T, topk), np.int32)
    ids[:, 1] = 7
    moe_check(moe_case(21, T, H, I, E, topk, t, ids), T, H, I, E, topk, t, False)
    ids = np.argsort(np.random.default_rng(3).random((T, E)), -1)[:, :topk].astype(np.int32)
    ids[::3, 0] = -1
    ids[1::5, 1] = E
    ids[4] = [-5, 1000]  # a token without experts
    out, _ = moe_check(moe_case(22, T, H, I, E, topk, t, ids), T, H, I, E, topk, t, False)
    assert (values64(out)[4] == 0).all()
    # the same id twice in a token counts twice
    ids = np.full((T, topk), 3, np.int32)
    moe_check(moe_case(23, T, H, I, E, topk, t, ids), T, H, I, E, topk, t, True)


def test_moe_workspace_reused_by_another_size():
    torch = torch_cuda()
    need = max(gq.gq_moe_mxfp4_workspace_bytes(700, 128, 160, 3, 2),
               gq.gq_moe_mxfp4_workspace_bytes(33, 288, 224, 4, 3))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    moe_check(moe_case(24, 700, 128, 160, 3, 2, "f16"), 700, 128, 160, 3, 2, "f16", False, ws)
    moe_check(moe_case(25, 33, 288, 224, 4, 3, "bf16"), 33, 288, 224, 4, 3, "bf16", False, ws)


# -- as they are used ---------------------------------------------------------------

def test_quantize_then_product_then_experts():
    """A prompt's run: activations quantised, a projection in 4 bits, its output
    through the experts, the last token through the decode product; each stage
    checked on the values the stage before produced."""
    torch = torch_cuda()
    N, K, M = 70, 512, 256
    q, s, W = weights(30, M, K)
    xd, x64 = as_type(normal(31, N, K), "bf16")
    xq, xs = gq.quantize_mxfp4(xd)
    y = gq.gemm_mxfp4_mxfp4(q, s, xq, xs, dtype=torch.bfloat16)
    X = mx.values(host(xq), host(xs))
    assert np.array_equal(mx.quantize(x64)[0], host(xq))
    ref, S = mx.products(W, X)
    check(y, ref, S, "bf16", "projection")
    st = moe_case(32, N, M, 128, 8, 2, "bf16")
    st["x"], st["X"] = y, values64(y)
    ids, wts = gq.moe_route(torch.randn((N, 8), device="cuda"), 2)
    st["ids"], st["wts"] = host(ids), host(wts)
    out, _ = moe_check(st, N, M, 128, 8, 2, "bf16", False)
    q2, s2, W2 = weights(33, 100, M)
    last = out[-1:].float()
    z = gq.gemv_mxfp4(q2, s2, last)
    ref, S = mx.products(W2, values64(last))
    check(z, ref, S, "f32", "decode product")


def test_captured_and_replayed():
    torch = torch_cuda()
    M, K, N = 300, 416, 70
    q, s, _ = weights(40, M, K)
    st = moe_case(41, N, 256, 128, 4, 2, "f16")
    ids, wts = dev(st["ids"]), dev(st["wts"])
    x32 = torch.randn((4, K), device="cuda")
    x16 = torch.randn((N, K), device="cuda").half()
    xm = st["x"].clone()

    def run():
        xq, xs = gq.quantize_mxfp4(x16)
        return [gq.dequant_mxfp4(xq, xs), gq.gemv_mxfp4(q, s, x32), gq.gemm_mxfp4(q, s, x16),
                gq.gemm_mxfp4_mxfp4(q, s, xq, xs), gq.moe_mxfp4(st["g"], st["u"], st["d"], xm, ids, wts)[0]]

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run()
    for i in range(4):
        x32.copy_(torch.randn_like(x32))
        x16.copy_(torch.randn_like(x16))
        xm.copy_(torch.randn_like(xm) * 0.25)
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    torch = torch_cuda()
    M, K, N = 2048, 1024, 96
    q, s, _ = weights(42, M, K)
    xa = torch.randn((N, K), device="cuda").bfloat16()
    xb = torch.randn((N, K), device="cuda").bfloat16()
    want = [gq.gemm_mxfp4(q, s, x) for x in (xa, xb)]
    st = moe_case(43, 64, 256, 128, 4, 2, "bf16")
    ids, wts = dev(st["ids"]), dev(st["wts"])
    wm = gq.moe_mxfp4(st["g"], st["u"], st["d"], st["x"], ids, wts)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        outs.append((gq.gemm_mxfp4(q, s, xa, stream=s1), want[0]))
        outs.append((gq.gemm_mxfp4(q, s, xb, stream=s2.cuda_stream), want[1]))
        outs.append((gq.moe_mxfp4(st["g"], st["u"], st["d"], st["x"], ids, wts, stream=s1)[0], wm))
        outs.append((gq.moe_mxfp4(st["g"], st["u"], st["d"], st["x"], ids, wts, stream=s2)[0], wm))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, b)


def test_helpers_streams_shapes_and_no_rows():
    torch = torch_cuda()
    q, s, _ = weights(45, 40, 96)
    x = torch.randn((5, 96), device="cuda")
    want = gq.gemv_mxfp4(q, s, x)
    # the default stream by its handle, one row without a rows' dimension, a batch of rows
    assert torch.equal(gq.gemv_mxfp4(q, s, x, stream=0), want)
    assert torch.equal(gq.gemv_mxfp4(q, s, x[2]), gq.gemv_mxfp4(q, s, x[2:3]))
    a, b = gq.quantize_mxfp4(x)
    for got, ref in ((gq.quantize_mxfp4(x[3]), (a[3], b[3])),
                     (gq.quantize_mxfp4(x[:4].view(2, 2, 96)), (a[:4].view(2, 2, 48), b[:4].view(2, 2, 3)))):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    h = x.half()
    y = gq.gemm_mxfp4(q, s, h)
    assert torch.equal(gq.gemm_mxfp4(q, s, h.view(1, 5, 96)), y)
    # no rows
    none = torch.empty((0, 96), device="cuda")
    nq, ns = gq.quantize_mxfp4(none)
    assert nq.shape == (0, 48) and ns.shape == (0, 3)
    assert gq.dequant_mxfp4(nq, ns).shape == (0, 96)
    assert gq.gemv_mxfp4(q, s, none).shape == (0, 40)
    assert gq.gemm_mxfp4(q, s, none.half()).shape == (0, 40)
    assert gq.gemm_mxfp4_mxfp4(q, s, nq, ns).shape == (0, 40)
    # a pointer that is not 16-byte aligned
    with pytest.raises(gq.GQError) as e:
        gq.gemv_mxfp4(q, s, torch.randn(97, device="cuda")[1:])
    assert e.value.status == gq.GQ_EALIGN


def test_helper_refusals():
    torch = torch_cuda()
    q, s, _ = weights(44, 32, 64)
    x = torch.randn((2, 64), device="cuda")
    for call in (lambda: gq.gemv_mxfp4(q, s, x.half()),
                 lambda: gq.gemv_mxfp4(q, s[:, :1], x),
                 lambda: gq.gemm_mxfp4(q, s, x),
                 lambda: gq.gemm_mxfp4(q, s, x.half(), out=torch.empty((2, 32), device="cuda")),
                 lambda: gq.gemm_mxfp4_mxfp4(q, s, q[:, :16].contiguous(), s[:, :1].contiguous()),
                 lambda: gq.quantize_mxfp4(x.double()),
                 lambda: gq.dequant_mxfp4(q, s.float())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gq.GQError) as e:
        gq.gemv_mxfp4(q, s, torch.randn((17, 64), device="cuda"))
    assert e.value.status == gq.GQ_EINVAL
