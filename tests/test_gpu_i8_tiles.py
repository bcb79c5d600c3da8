"""Every form of the int8 tile kernels at ordinary values: each tile with a whole and a cut last stage,
whole tiles, halves and both in one launch, and each tile of the gradients in one run of the sum and
in several.  tests/test_i8_plan.py checks on the CPU that the sizes below take what they are said
to take."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _i8 as i8
from tests._gpu import dev, torch_cuda
from tests.test_gpu_i8 import (floats, gated_reference, grad_tolerance, matrix, near, same, ttype,
                               values)
from tests.test_gpu_i8_gated_gradients import want_and_tolerance

pytestmark = pytest.mark.gpu

# (M, K, N): tile, K a multiple of a stage's 128 columns, how the tiles of 256 rows lie
PRODUCTS = {
    (700, 300, 77): (64, False, None), (513, 512, 99): (64, True, None),
    (772, 100, 4111): (128, False, None), (8885, 128, 323): (128, True, None),
    (8613, 200, 403): (256, False, "halves"), (8282, 128, 399): (256, True, "halves"),
    (8371, 300, 770): (256, False, "whole"), (8209, 384, 769): (256, True, "whole"),
    (7605, 130, 2053): (256, False, "both"), (8203, 128, 1835): (256, True, "both"),
}
# (I, H, N): the same of gate and up, forward and gradients
GATED = {
    (300, 200, 40): (64, False, None), (257, 256, 33): (64, True, None),
    (4039, 405, 461): (128, False, None), (7559, 640, 193): (128, True, None),
    (6307, 200, 465): (256, False, "halves"), (7047, 256, 395): (256, True, "halves"),
    (8613, 130, 405): (256, False, "whole"), (8967, 128, 323): (256, True, "whole"),
    (8371, 77, 770): (256, False, "both"), (8209, 128, 769): (256, True, "both"),
    (14336, 4096, 1024): (256, True, "whole"),
}
# (M, K, N): the tile's number, M a multiple of a stage's 64 rows, several runs
GRADIENTS = {
    (97, 1562, 4711): (0, False, False), (64, 10863, 655): (0, True, False),
    (2211, 11277, 150): (0, False, True), (2240, 11277, 150): (0, True, True),
    (70, 11299, 130): (1, False, False), (64, 11299, 129): (1, True, False),
    (4231, 6613, 283): (1, False, True), (4224, 6613, 283): (1, True, True),
    (93, 300, 130): (2, False, False), (512, 1003, 517): (2, True, False),
    (700, 500, 300): (2, False, True), (448, 300, 19): (2, True, True),
    (4096, 14336, 2048): (0, True, False), (5835, 11995, 189): (0, False, True),
}
# (I, H, N): the same of the gated half's backward pass, two parts of the sum
GATED_GRADIENTS = {
    (45, 1562, 4710): (0, False, False), (64, 10863, 655): (0, True, False),
    (981, 11397, 141): (0, False, True), (14336, 4096, 1024): (0, True, True),
    (130, 11299, 131): (1, False, False), (1024, 4001, 1501): (1, True, False),
    (2600, 4096, 517): (1, False, True), (2560, 4096, 517): (1, True, True),
    (33, 130, 40): (2, False, False), (64, 300, 30): (2, True, False),
    (300, 200, 40): (2, False, True), (960, 2048, 300): (2, True, True),
}


def sample(n):
    """Up to 40 of n rows: both ends, tiles' borders, some between."""
    edges = [0, 1, 31, 32, 63, 64, 127, 128, 255, 256, n - 257, n - 129, n - 65, n - 33, n - 2, n - 1]
    some = np.random.default_rng(n).integers(0, n, 24)
    return np.unique([i for i in [*edges, *some] if 0 <= i < n])


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,N", PRODUCTS)
def test_products(M, K, N, t):
    wq, ws = i8.rows(300, M, K, -128, 127)
    xq, xs = i8.rows(301, N, K, -128, 127)
    n = sample(N)
    y = gq.gemm_i8(*matrix(wq, ws, extra=1), *matrix(xq, xs), dtype=ttype(t))
    same(y[dev(n)], i8.round_to(i8.product(wq, ws, xq[n], xs[n]), t), "gemm")


@pytest.mark.parametrize("t,kind", [("f32", "silu"), ("f16", "gelu"), ("bf16", "silu")])
@pytest.mark.parametrize("I,H,N", GATED)
def test_gated(I, H, N, t, kind):
    gate, up = i8.rows(302, I, H), i8.rows(303, I, H)
    xq, xs = i8.rows(304, N, H)
    n = sample(N)
    g, u, (a, _, p) = gated_reference(gate, up, xq[n], xs[n], kind)
    h = a * u
    tol = np.abs(h) * i8.act_rel(p) + np.abs(g * u) * 2.0 ** -125 + 2.0 ** -149
    tol = tol + i8.half_step(np.abs(h) + tol, t)
    got = gq.gated_i8(matrix(*gate), matrix(*up, extra=1), *matrix(xq, xs), act=kind, dtype=ttype(t))
    near(got[dev(n)], h, tol, "gated")


@pytest.mark.parametrize("t,kind", [("f16", "gelu"), ("bf16", "silu")])
@pytest.mark.parametrize("I,H,N", {**GATED, **GATED_GRADIENTS})
def test_gated_backward(I, H, N, t, kind):
    gate, up = i8.rows(305, I, H), i8.rows(306, I, H)
    xq, xs = i8.rows(307, N, H)
    dh, d64 = floats(308, N, I, t, 2.0 ** -4)
    n = sample(N)
    want, tol, _ = want_and_tolerance(gate, up, xq[n], xs[n], d64[n], kind, t)
    # the workspace holds what the last call left: numbers that would show
    ws = torch_cuda().full((gq.gq_gated_i8_backward_workspace_bytes(N, H, I),), 0x7e,
                           dtype=torch_cuda().uint8, device="cuda")
    got, _ = gq.gated_i8_backward(matrix(*gate, extra=1), matrix(*up), *matrix(xq, xs), dh, act=kind, ws=ws)
    near(got[dev(n)], want, tol, "dX")
    again, _ = gq.gated_i8_backward(matrix(*gate, extra=1), matrix(*up), *matrix(xq, xs), dh, act=kind, ws=ws)
    assert bool((got == again).all())


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", GRADIENTS)
def test_gemm_backward(M, K, N, t):
    wq, ws = i8.rows(309, M, K, -128, 127)
    dy, d64 = floats(310, N, M, t)
    n = sample(N)
    w = i8.weights16(wq, ws, t)
    want = d64[n] @ w
    tol = grad_tolerance(np.abs(d64[n]) @ np.abs(w), M, want, t)
    got = gq.gemm_i8_backward(*matrix(wq, ws, extra=1), dy)
    near(got[dev(n)], want, tol, "dX")
    assert bool((got == gq.gemm_i8_backward(*matrix(wq, ws, extra=1), dy)).all())


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("N", [1, 7, 40, 200, 1000])
def test_gradients_of_a_row_alone(N, t):
    """A token's gradients alone and among others: the same but for the order of the sums, and with
    others' infinities beside it not different at all."""
    M, K = 300, 500
    wq, ws = i8.rows(311, M, K)
    W, dy = matrix(wq, ws), floats(312, N, M, t)[0]
    gate, up = matrix(*i8.rows(313, M, K)), matrix(*i8.rows(314, M, K))
    xq, xs = i8.rows(315, N, K)
    n = N // 2
    w = i8.weights16(wq, ws, t)
    d64 = values(dy)
    all_ = values(gq.gemm_i8_backward(*W, dy))
    one = values(gq.gemm_i8_backward(*W, dy[n:n + 1].clone()))[0]
    want = d64[n] @ w
    # each within its tolerance of the formula
    tol = grad_tolerance(np.abs(d64[n]) @ np.abs(w), M, want, t)
    assert (np.abs(all_[n] - want) <= tol).all() and (np.abs(one - want) <= tol).all()
    X = matrix(xq, xs)
    gall = values(gq.gated_i8_backward(gate, up, *X, dy)[0])
    gone = values(gq.gated_i8_backward(gate, up, *matrix(xq[n:n + 1], xs[n:n + 1]), dy[n:n + 1].clone())[0])
    gw, gt, _ = want_and_tolerance(i8.rows(313, M, K), i8.rows(314, M, K), xq[n:n + 1], xs[n:n + 1],
                                   d64[n:n + 1], "silu", t)
    assert (np.abs(gall[n] - gw[0]) <= gt[0]).all() and (np.abs(gone - gw) <= gt).all()
    if N > 1:
        others = dy.clone()
        others[n + 1:] = float("inf")
        others[:n] = float("nan")
        assert (values(gq.gemm_i8_backward(*W, others))[n] == all_[n]).all()
        assert (values(gq.gated_i8_backward(gate, up, *X, others)[0])[n] == gall[n]).all()


def test_gradients_past_4_gib_of_codes():
    """Gradients of a few weight rows at both ends of a matrix and around its 2^32-byte border, zeros
    elsewhere: a wrong address shows whole, sums of a million rows do not hide it."""
    torch = torch_cuda()
    M, K, N = 1 << 20, 4160, 5
    W = torch.empty((M, K), dtype=torch.int8, device="cuda").random_(-128, 128)
    s = torch.empty(M, device="cuda").uniform_(2.0 ** -12, 2.0 ** -9)
    border = (1 << 32) // K
    rows = np.unique([*range(8), *range(border - 8, border + 9), *range((1 << 31) // K - 4, (1 << 31) // K + 5),
                      *range(M // 2, M // 2 + 3), *range(M - 8, M)])
    at = dev(rows)
    for t in ("f16", "bf16"):
        dy = torch.zeros((N, M), dtype=ttype(t), device="cuda")
        d, d64 = floats(316, N, rows.size, t)
        dy[:, at] = d
        w = i8.weights16(W[at].cpu().numpy(), s[at].cpu().numpy(), t)
        want, size = d64 @ w, np.abs(d64) @ np.abs(w)
        tol = grad_tolerance(size, rows.size, want, t) # (products with zero add nothing)
        assert (tol < np.abs(want)).mean() > 0.9 # (a result of zeros would fail)
        near(gq.gemm_i8_backward(W, s, dy), want, tol, "dX")
        # one row at a time, one token each: the row itself
        for r in (0, border, border + 1, M - 1):
            dy.zero_()
            dy[3, r] = 1.0
            got = values(gq.gemm_i8_backward(W, s, dy))
            i = int(np.searchsorted(rows, r))
            assert (got[3] == w[i]).all() and (got[[0, 1, 2, 4]] == 0).all(), r
    del W, dy
    torch.cuda.empty_cache()
