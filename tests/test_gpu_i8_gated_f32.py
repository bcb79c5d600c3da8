"""binary32 results of the gated half carry binary32's precision for every argument of the
activation, on the streaming kernels and on tiles."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _i8 as i8
from tests.test_gpu_i8 import gated_reference, matrix, near

pytestmark = pytest.mark.gpu


def tolerance(g, u, kind):
    """exp to two units in the last place (2^-22, where the sigmoid is small enough for it to count),
    1 + e, the quotient and two products half a unit each (4 2^-24): 2^-21 with room.  GELU's p is
    off by five half steps (its constants, three products, two fused sums), which the sigmoid passes
    on times 1 - sigmoid.  A sigmoid below 2^-126 is a multiple of 2^-149."""
    a, _, p = i8.act(g, kind)
    rel = 2.0 ** -21
    if kind == "gelu":
        sig = np.where(g != 0, a / np.where(g != 0, g, 1), 0.5)
        rel = rel + np.abs(p) * (1 - sig) * 5 * 2.0 ** -24
    return a * u, np.abs(a * u) * rel + (2 * np.abs(g * u) + 1) * 2.0 ** -149


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("I,H,N", [(300, 100, 1), (257, 64, 7), (8300, 96, 16), (40, 9000, 3), (130, 128, 70),
                                   (1030, 200, 700), (2100, 128, 2100)])
def test_binary32_results(I, H, N, kind):
    """g from -110 to 110 (for GELU -12 to 12: p of 1.6 z + 0.07 z^3), u large where g is far below."""
    gate, up = i8.rows(1, I, H), i8.rows(2, I, H)
    xq, xs = i8.rows(3, N, H)
    spread = np.abs(i8.product(*gate, xq, xs)).max()
    xs = (xs * ((110 if kind == "silu" else 12) / spread)).astype(np.float32)
    up[1][::3] *= np.float32(2.0 ** 100)
    g, u, _ = gated_reference(gate, up, xq, xs, kind)
    h, tol = tolerance(g, u, kind)
    got = gq.gated_i8(matrix(*gate), matrix(*up), *matrix(xq, xs), act=kind)
    near(got, h, tol, "h")


def test_far_below_zero():
    """Sigmoids below 2^-126 times large values of u."""
    H, z = 16, np.array([-87.0, -88.5, -90.0, -95.0, -100.0, -103.0, -110.0, 88.0, 110.0, 0.0], np.float32)
    I = z.size
    one = np.eye(1, H, dtype=np.int8)
    gate, up = (one.repeat(I, 0), z), (one.repeat(I, 0), np.full(I, 2.0 ** 100, np.float32))
    for N in (1, 40):
        xq, xs = one.repeat(N, 0), np.ones(N, np.float32)
        g, u, _ = gated_reference(gate, up, xq, xs, "silu")
        h, tol = tolerance(g, u, "silu")
        got = gq.gated_i8(matrix(*gate), matrix(*up), *matrix(xq, xs))
        near(got, h, tol, "h by %d rows" % N)
        assert (np.abs(h[0, :6]) > 0).all()
