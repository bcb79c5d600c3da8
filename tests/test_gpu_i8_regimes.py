"""The int8 operators where other kernels and paths run: each tile with full, ragged and halved
tiles, sums in runs, gradients in rows of any distance, and byte offsets past 32 bits."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _i8 as i8
from tests._gpu import dev, host, torch_cuda
from tests.test_gpu_i8 import (floats, gated_reference, grad_tolerance, matrix, near, same, ttype,
                               values)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def freed():
    torch_cuda().manual_seed(97)
    yield
    torch_cuda().cuda.empty_cache()


# 64-, 128- and 256-row tiles by their estimated time; 289 and 272 tiles of 256 are one round and
# some halves
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(500, 130, 300), (2050, 130, 2047), (2048, 256, 2048),
                                   (4096, 200, 4096), (4100, 128, 4097), (4095, 257, 4352),
                                   (20000, 64, 70), (70, 640, 20000), (1, 300, 3000), (3000, 300, 18)])
def test_product_tiles(M, K, N, t):
    wq, ws = i8.rows(200, M, K, -128, 127)
    xq, xs = i8.rows(201, N, K, -128, 127)
    same(gq.gemm_i8(*matrix(wq, ws), *matrix(xq, xs), dtype=ttype(t)),
         i8.round_to(i8.product(wq, ws, xq, xs), t), "gemm")


@pytest.mark.parametrize("M,K,N", [(8192, 200, 16), (8207, 1000, 5), (9000, 8200, 3), (8191, 8192, 2),
                                   (8300, 9001, 16)])
def test_streamed_products_of_tall_matrices(M, K, N):
    """Tiles of 16 and of 32 weight rows, eight and sixteen waves, ragged ends; gate and up."""
    wq, ws = i8.rows(214, M, K, -128, 127)
    xq, xs = i8.rows(215, N, K, -128, 127)
    W, X = matrix(wq, ws), matrix(xq, xs)
    ref = i8.product(wq, ws, xq, xs)
    same(gq.gemm_i8(*W, *X), ref.astype(np.float64), "gemm")
    U = matrix(wq[::-1].copy(), ws[::-1].copy())
    g, u = ref.astype(np.float64), ref[:, ::-1].astype(np.float64)
    a, _, p = i8.act(g, "silu")
    tol = np.abs(a * u) * (i8.act_rel(p) + 2.0 ** -22) + np.abs(g * u) * 2.0 ** -125 + 2.0 ** -149
    near(gq.gated_i8(W, U, *X), a * u, tol, "gated")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("I,H,N", [(300, 130, 300), (1030, 128, 2050), (2048, 100, 4096), (2100, 129, 4097),
                                   (4003, 64, 40), (9, 200, 5000)])
def test_gated_tiles(I, H, N, t, kind):
    gate, up = i8.rows(202, I, H), i8.rows(203, I, H)
    xq, xs = i8.rows(204, N, H)
    g, u, (a, da, p) = gated_reference(gate, up, xq, xs, kind)
    h = a * u
    tol = np.abs(h) * i8.act_rel(p) + np.abs(g * u) * 2.0 ** -125 + 2.0 ** -149
    tol = tol + i8.half_step(np.abs(h) + tol, t)
    G, U, X = matrix(*gate), matrix(*up, extra=2), matrix(xq, xs)
    near(gq.gated_i8(G, U, *X, act=kind, dtype=ttype(t)), h, tol, "gated")
    dh, d64 = floats(205, N, I, t)
    sig = np.where(g != 0, a / np.where(g != 0, g, 1), 0.5)
    eg = np.abs(d64 * u) * (np.abs(sig) + 2 * np.abs(da - sig)) * (2 * i8.act_rel(p) + 2.0 ** -21) + 2.0 ** -120
    dg, du = d64 * u * da, d64 * a
    eu = np.abs(du) * i8.act_rel(p) + 2.0 ** -120
    (fg, pg), (fu, pu) = i8.split_scales(gate[1]), i8.split_scales(up[1])
    wg, wu = gate[0] * pg[:, None], up[0] * pu[:, None]
    dg, du, eg, eu = dg * fg, du * fu, eg * fg, eu * fu
    eg, eu = eg + i8.half_step(np.abs(dg) + eg, t), eu + i8.half_step(np.abs(du) + eu, t)
    want = dg @ wg + du @ wu
    size = (np.abs(dg) + eg) @ np.abs(wg) + (np.abs(du) + eu) @ np.abs(wu)
    tol = eg @ np.abs(wg) + eu @ np.abs(wu) + grad_tolerance(size, 2 * I, want, t)
    near(gq.gated_i8_backward(G, U, *X, dh, act=kind)[0], want, tol, "dX")


# large tiles, 128-row ones, small ones; one run of the sum and several, of unequal length
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(96, 4096, 4096), (70, 4100, 4090), (64, 2048, 700), (1000, 300, 300),
                                   (4096, 130, 33), (5000, 70, 260), (9001, 16, 3), (640, 2000, 130),
                                   (72, 100, 1), (8200, 257, 70), (129, 8200, 8)])
def test_gradient_tiles_and_runs(M, K, N, t):
    wq, ws = i8.rows(206, M, K, -128, 127)
    dy, d64 = floats(207, N, M, t)
    w = i8.weights16(wq, ws, t)
    want = d64 @ w
    tol = grad_tolerance(np.abs(d64) @ np.abs(w), M, want, t)
    W = matrix(wq, ws, extra=1)
    a = gq.gemm_i8_backward(*W, dy)
    near(a, want, tol, "dX")
    b = gq.gemm_i8_backward(*W, dy)
    assert (values(a) == values(b)).all()  # (no order varies from call to call)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("M,ld", [(104, 112), (104, 104), (8, 4096), (200, 203), (201, 208), (64, 65)])
@pytest.mark.parametrize("N", [1, 2, 70, 300])
def test_gradient_rows_apart(M, ld, N, t):
    """NaN between dY's rows and behind the last one."""
    torch = torch_cuda()
    K = 150
    wq, ws = i8.rows(208, M, K)
    _, d64 = floats(209, N, M, t)
    buf = torch.full((N + 1, ld), float("nan"), dtype=ttype(t), device="cuda")
    buf[:N, :M] = dev(d64.astype(np.float32)).to(ttype(t))
    w = i8.weights16(wq, ws, t)
    want = d64 @ w
    tol = grad_tolerance(np.abs(d64) @ np.abs(w), M, want, t)
    near(gq.gemm_i8_backward(*matrix(wq, ws, fill=-128), buf[:N, :M]), want, tol, "dX")


@pytest.mark.parametrize("N", [1, 7, 40, 200, 1000])
def test_a_row_does_not_depend_on_the_others(N):
    """Products and gradients of a row alone and among others: the whole-number products are the
    same, gradients within the order of their sums."""
    M, K = 300, 500
    wq, ws = i8.rows(210, M, K)
    xq, xs = i8.rows(211, N, K)
    W = matrix(wq, ws)
    y = values(gq.gemm_i8(*W, *matrix(xq, xs)))
    n = N // 2
    one = values(gq.gemm_i8(*W, *matrix(xq[n:n + 1], xs[n:n + 1])))
    assert (y[n] == one[0]).all()


def test_extreme_scales_in_gradients():
    """Scales at the ends of the types: binary16 weights below 2^-24 and above 65504, subnormal
    and huge ones in bfloat16."""
    M, K, N = 64, 40, 20
    for t, exps in (("f16", (-30, -24, -10, 8, 12)), ("bf16", (-130, -120, 0, 100, 118))):
        for e in exps:
            wq, _ = i8.rows(212, M, K)
            ws = np.full(M, 1.37 * 2.0 ** e, np.float32)
            dy, d64 = floats(213, N, M, t, 2.0 ** -8)
            w = i8.weights16(wq, ws, t)
            with np.errstate(all="ignore"):
                want = d64 @ w
                size = np.abs(d64) @ np.abs(w)
            got = values(gq.gemm_i8_backward(*matrix(wq, ws), dy))
            big = 65504.0 if t == "f16" else 3.3e38
            ok = np.isfinite(want) & (size < big / 2)
            tol = grad_tolerance(size, M, want, t)
            assert (np.abs(got - want)[ok] <= tol[ok]).all(), (t, e)
            assert not np.isfinite(got[~np.isfinite(want)]).any(), (t, e)


def some(n):
    return np.unique(np.clip([0, 1, n // 2, n - 17, n - 2, n - 1], 0, n - 1))


def codes(rows, K):
    torch = torch_cuda()
    ld = (K + 15) // 16 * 16
    q = torch.empty((rows, ld), dtype=torch.int8, device="cuda").random_(-128, 128)
    return q[:, :K], torch.empty(rows, device="cuda").uniform_(2.0 ** -12, 2.0 ** -9)


def part(m, i):
    return host(m[0][i]), host(m[1][i])


def test_products_of_many_weight_rows():
    """4.4 GB of codes."""
    M, K = 2_150_003, 2050
    W = codes(M, K)
    assert W[0].untyped_storage().nbytes() > 1 << 32
    r = some(M)
    ri = dev(r)
    w = part(W, ri)
    for N in (1, 3, 16, 20):
        x, x64 = floats(220, N, K, "bf16")
        xq, xs = i8.quantize(x64)
        ref = i8.product(*w, xq, xs)
        X = gq.quantize_i8(x)
        same(gq.gemm_i8(*W, *X)[:, ri], ref.astype(np.float64), "gemm %d" % N)
        if N <= 16:
            same(gq.gemv_i8(*W, x)[:, ri], i8.round_to(ref, "bf16"), "gemv %d" % N)
        h = values(gq.gated_i8(W, W, *X)[:, ri])
        g = ref.astype(np.float64)
        a, _, p = i8.act(g, "silu")
        assert (np.abs(h - a * g) <= np.abs(a * g) * (i8.act_rel(p) + 2.0 ** -22) + 2.0 ** -120).all()


def test_products_of_many_tokens_and_outputs():
    """Codes of tokens and outputs past 4 GiB."""
    torch = torch_cuda()
    M, K, N = 2300, 4100, (1 << 20) + 5
    W, X = codes(M, K), codes(N, K)
    assert X[0].untyped_storage().nbytes() > 1 << 32
    n, m = some(N), some(M)
    ni, mi = dev(n), dev(m)
    ref = i8.product(*part(W, mi), *part(X, ni))
    y = gq.gemm_i8(*W, *X, dtype=torch.bfloat16)
    assert 2 * y.numel() > 1 << 32
    same(y[ni][:, mi], i8.round_to(ref, "bf16"), "gemm")
    del y
    h = gq.gated_i8(W, W, *X, dtype=torch.bfloat16)[ni][:, mi]
    g = ref.astype(np.float64)
    a, _, p = i8.act(g, "silu")
    tol = np.abs(a * g) * (i8.act_rel(p) + 2.0 ** -22) + 2.0 ** -120
    near(h, a * g, tol + i8.half_step(np.abs(a * g) + tol, "bf16"), "gated")


def test_gradients_of_many_rows():
    """dY, dX and the weights' codes past 4 GiB, in turn."""
    torch = torch_cuda()
    for M, K, N in ((2056, 520, (1 << 20) + 3), (40, 4104, (1 << 19) + 9), (1 << 20, 4160, 5)):
        W = codes(M, K)
        dy = torch.empty((N, M), dtype=torch.bfloat16, device="cuda").normal_()
        n = some(N)
        ni = dev(n)
        d64 = values(dy[ni])
        dx = gq.gemm_i8_backward(*W, dy)[ni]
        if M < 1 << 16:
            w = i8.weights16(*part(W, dev(np.arange(M))), "bf16")
            want, size = d64 @ w, np.abs(d64) @ np.abs(w)
        else: # few columns of it
            c = np.arange(0, K, 256)
            q = host(W[0][:, dev(c)].contiguous())
            w = i8.weights16(q, host(W[1]), "bf16")
            want, size = d64 @ w, np.abs(d64) @ np.abs(w)
            dx = dx[:, dev(c)]
        near(dx, want, grad_tolerance(size, M, want, "bf16"), "dX")
        del W, dy, dx
        torch.cuda.empty_cache()


def test_quantise_many_values():
    """4.4e9 values; rows far apart."""
    torch = torch_cuda()
    N, K = 1_100_001, 4000
    x = torch.empty((N, K + 8), dtype=torch.float16, device="cuda").normal_()[:, :K]
    q, s = gq.quantize_i8(x)
    assert q.untyped_storage().nbytes() > 1 << 32
    i = dev(some(N))
    rq, rs = i8.quantize(values(x[i]))
    same(q[i], rq.astype(np.float64), "codes")
    same(s[i], rs.astype(np.float64), "scales")
    v = gq.dequant_i8(q, s, torch.float16)
    same(v[i], i8.round_to(rq.astype(np.float32) * rs[:, None], "f16"), "values")


def test_block_of_many_tokens():
    """h of 4.3 GB; against its parts."""
    torch = torch_cuda()
    T, H, I = 70_001, 64, 32_000
    G, U, D = codes(I, H), codes(I, H), codes(H, I)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_()
    out, _ = gq.ffn_i8(G, U, D, x)
    i = dev(some(T))
    h = gq.gated_i8(G, U, *gq.quantize_i8(x[i]), dtype=x.dtype)
    want = gq.gemm_i8(*D, *gq.quantize_i8(h), dtype=x.dtype)
    same(out[i], values(want), "ffn")


def test_codes_of_a_wider_matrix():
    """Columns of a wider matrix as weights and tokens: gate and up side by side."""
    torch = torch_cuda()
    I, H, N = 130, 160, 50
    wide = torch.empty((I, 512), dtype=torch.int8, device="cuda").random_(-128, 128)
    tok = torch.empty((N, 400), dtype=torch.int8, device="cuda").random_(-128, 128)
    s = torch.rand(I, device="cuda") + 0.5
    xs = torch.rand(N, device="cuda") * 2.0 ** -12
    a, b = (wide[:, 32:32 + H], s), (wide[:, 256:256 + H], s)
    x = (tok[:, 64:64 + H], xs)
    apart = [(m[0].contiguous(), m[1]) for m in (a, b, x)]
    for dt in (torch.float32, torch.bfloat16):
        same(gq.gated_i8(a, b, *x, dtype=dt), values(gq.gated_i8(apart[0], apart[1], *apart[2], dtype=dt)), "h")
        same(gq.gemm_i8(*a, *x, dtype=dt), values(gq.gemm_i8(*apart[0], *apart[2], dtype=dt)), "y")
    dh = torch.randn((N, I), device="cuda").half()
    same(gq.gated_i8_backward(a, b, *x, dh)[0],
         values(gq.gated_i8_backward(apart[0], apart[1], *apart[2], dh)[0]), "dX")
    # 16-byte aligned views of rows
    same(gq.gemm_i8(a[0][4:20], s[4:20], *x), values(gq.gemm_i8(*a, *x))[:, 4:20], "rows")
