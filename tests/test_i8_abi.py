"""The int8 entry points on the CPU: refusals on the host, before any launch, calls without
work, and the test oracle's own checks."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from tests import _i8 as i8

P = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
BAD = ctypes.c_void_p(0x10008)
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from quantized_unpack_q4_amd import gq
    return gq.lib()


def refused(L, st, code, *words):
    msg = L.gq_last_error().decode()
    assert L.gq_status_str(st).decode() == code, (st, msg)
    for w in words:
        assert w in msg, msg


def test_quantize_refusals(L):
    f = L.gq_quantize_i8

    def call(x=P, t=F32, ldx=64, q=P, ldq=64, s=P, N=2, K=64):
        return f(x, t, ldx, q, ldq, s, N, K, None)

    refused(L, call(t=3), "GQ_EINVAL", "x_type = 3")
    refused(L, call(N=-1), "GQ_EINVAL", "N = -1")
    refused(L, call(K=0), "GQ_EINVAL", "K = 0")
    refused(L, call(ldx=63), "GQ_ESHAPE", "ldx = 63")
    refused(L, call(ldx=-64), "GQ_ESHAPE", "ldx = -64")
    refused(L, call(ldx=(1 << 40) + 1), "GQ_ESHAPE", "ldx")
    refused(L, call(ldq=48), "GQ_ESHAPE", "ldq = 48")
    refused(L, call(ldq=72), "GQ_EALIGN", "ldq = 72")
    refused(L, call(ldq=(1 << 40) + 16), "GQ_ESHAPE", "ldq")
    refused(L, call(N=(1 << 14) + 1, K=1 << 20, ldx=1 << 20, ldq=1 << 20), "GQ_ESHAPE", "2^34")
    refused(L, call(x=None), "GQ_EINVAL", "x is NULL")
    refused(L, call(q=BAD), "GQ_EALIGN", " q ")
    refused(L, call(s=None), "GQ_EINVAL", "s is NULL")
    assert call(N=0, x=None, q=None, s=None) == 0


def test_dequant_refusals(L):
    f = L.gq_dequant_i8
    refused(L, f(P, 64, P, P, 3, 2, 64, None), "GQ_EINVAL", "out_type = 3")
    refused(L, f(P, 60, P, P, F32, 2, 60, None), "GQ_EALIGN", "ldq = 60")
    refused(L, f(P, 64, P, P, F32, 2, 65, None), "GQ_ESHAPE", "ldq = 64")
    refused(L, f(P, 64, P, P, F32, (1 << 28) + 1, 64, None), "GQ_ESHAPE", "2^34")
    refused(L, f(P, 64, P, BAD, F32, 2, 64, None), "GQ_EALIGN", "out")
    assert f(None, 64, None, None, F32, 0, 64, None) == 0


def test_gemv_refusals(L):
    f = L.gq_gemv_i8

    def call(wq=P, ldw=64, ws=P, x=P, y=P, t=F32, M=8, K=64, B=1, wsp=None, n=0):
        return f(wq, ldw, ws, x, y, t, M, K, B, wsp, n, None)

    for B in (-1, 17):
        refused(L, call(B=B), "GQ_EINVAL", "B = %d" % B)
    refused(L, call(t=9), "GQ_EINVAL", "type = 9")
    refused(L, call(M=-1), "GQ_EINVAL", "M = -1")
    refused(L, call(M=(1 << 26) + 1), "GQ_ESHAPE", "M = ")
    refused(L, call(K=0), "GQ_EINVAL", "K = 0")
    refused(L, call(K=131072, ldw=131072), "GQ_ESHAPE", "K = 131072", "131071")
    refused(L, call(ldw=48), "GQ_ESHAPE", "ldw = 48")
    refused(L, call(ldw=65), "GQ_EALIGN", "ldw = 65")
    refused(L, call(ldw=(1 << 22) + 16), "GQ_ESHAPE", "ldw")
    refused(L, call(ws=BAD), "GQ_EALIGN", "ws")
    refused(L, call(x=None), "GQ_EINVAL", "x is NULL")
    from quantized_unpack_q4_amd import gq
    for K, B in ((16384, 1), (8192, 2), (4096, 3), (4096, 4)):
        assert gq.gq_gemv_i8_workspace_bytes(K, B) == 0
        assert gq.gq_gemv_i8_workspace_bytes(K + 1, B) > B * (K + 1)
    need = gq.gq_gemv_i8_workspace_bytes(1025, 16)
    assert need >= 16 * (1040 + 4)
    refused(L, call(K=1025, ldw=1040, B=16), "GQ_EWORKSPACE", str(need))
    refused(L, call(K=1025, ldw=1040, B=16, wsp=P, n=need - 1), "GQ_EWORKSPACE", str(need))
    refused(L, call(K=1025, ldw=1040, B=16, wsp=BAD, n=need), "GQ_EALIGN", "ws")
    for args, why in (((0, 1), "K = 0"), ((131072, 1), "K = 131072"), ((64, 17), "B = 17"), ((64, -1), "B = -1")):
        assert gq.gq_gemv_i8_workspace_bytes(*args) == 0 and why in gq.last_error()
    assert call(M=0, wq=None, ws=None, x=None, y=None) == 0
    assert call(B=0, wq=None, ws=None, x=None, y=None) == 0


def test_gemm_refusals(L):
    f = L.gq_gemm_i8

    def call(wq=P, ldw=64, ws=P, xq=P, ldx=64, xs=P, y=P, t=F32, M=8, K=64, N=2):
        return f(wq, ldw, ws, xq, ldx, xs, y, t, M, K, N, None)

    refused(L, call(t=-1), "GQ_EINVAL", "y_type = -1")
    refused(L, call(N=(1 << 21) + 1), "GQ_ESHAPE", "N = ")
    refused(L, call(N=-3), "GQ_EINVAL", "N = -3")
    refused(L, call(M=1 << 26, N=1 << 12), "GQ_ESHAPE", "outputs")
    refused(L, call(K=65), "GQ_ESHAPE", "ldw = 64")
    refused(L, call(ldx=72), "GQ_EALIGN", "ldx = 72")
    refused(L, call(ldx=16), "GQ_ESHAPE", "ldx = 16")
    refused(L, call(xs=None), "GQ_EINVAL", "xs is NULL")
    refused(L, call(xq=BAD), "GQ_EALIGN", "xq")
    refused(L, call(y=BAD), "GQ_EALIGN", " y ")
    assert call(N=0, wq=None, xq=None, y=None) == 0
    assert call(M=0, wq=None, xq=None, y=None) == 0


def test_gemm_backward_refusals(L):
    f = L.gq_gemm_i8_backward

    from quantized_unpack_q4_amd import gq
    size = gq.gq_gemm_i8_backward_workspace_bytes
    # (8 weight rows are one run of the sum)
    assert size(8, 64, 2, 16) == 0 and size(8, 64, 1, 3) == 0 and size(8, 64, 0, 8) == 0
    need = size(8, 64, 2, 9)
    assert need >= 2 * 8 * 2 and size(9, 64, 2, 16) >= 2 * 16 * 2 and size(9, 64, 1, 0) >= 32
    assert size(4096, 4096, 130, 4096) % (130 * 4096 * 4) == 0
    assert size(8, 64, 2, 7) == 0 and "ldd = 7" in gq.last_error()

    def call(wq=P, ldw=64, ws=P, dy=P, ldd=8, dx=P, t=F16, M=8, K=64, N=2, wsp=None, n=0):
        return f(wq, ldw, ws, dy, ldd, dx, t, M, K, N, wsp, n, None)

    refused(L, call(ldd=9), "GQ_EWORKSPACE", "wsp", str(need))
    refused(L, call(ldd=9, wsp=P, n=need - 1), "GQ_EWORKSPACE", str(need))
    refused(L, call(ldd=9, wsp=BAD, n=need), "GQ_EALIGN", "wsp")

    refused(L, call(t=F32), "GQ_EINVAL", "type = 0")
    refused(L, call(M=0), "GQ_EINVAL", "M = 0")
    refused(L, call(M=(1 << 22) + 1, ldd=(1 << 22) + 1), "GQ_ESHAPE", "M = ")
    refused(L, call(K=131072, ldw=131072), "GQ_ESHAPE", "K = 131072")
    refused(L, call(ldd=7), "GQ_ESHAPE", "ldd = 7")
    refused(L, call(ldd=(1 << 22) + 1), "GQ_ESHAPE", "ldd")
    refused(L, call(ldw=100), "GQ_EALIGN", "ldw = 100")
    refused(L, call(K=131071, ldw=131072, N=1 << 21), "GQ_ESHAPE", "outputs")
    refused(L, call(dy=BAD), "GQ_EALIGN", "dy")
    refused(L, call(dx=None), "GQ_EINVAL", "dx is NULL")
    assert call(N=0, wq=None, ws=None, dy=None, dx=None) == 0


def test_gated_refusals(L):
    f = L.gq_gated_i8

    def call(g=P, ldg=64, gs=P, u=P, ldu=64, us=P, xq=P, ldx=64, xs=P, h=P, t=F32, act=0, I=8, H=64,
             N=2):
        return f(g, ldg, gs, u, ldu, us, xq, ldx, xs, h, t, act, I, H, N, None)

    refused(L, call(t=4), "GQ_EINVAL", "h_type = 4")
    refused(L, call(act=2), "GQ_EINVAL", "act = 2")
    refused(L, call(I=-1), "GQ_EINVAL", "I = -1")
    refused(L, call(H=131072, ldg=131072, ldu=131072, ldx=131072), "GQ_ESHAPE", "H = ")
    refused(L, call(ldg=60), "GQ_ESHAPE", "ld_gate")
    refused(L, call(ldu=66), "GQ_EALIGN", "ld_up")
    refused(L, call(us=None), "GQ_EINVAL", "ws_up is NULL")
    refused(L, call(h=BAD), "GQ_EALIGN", " h ")
    assert call(I=0, g=None, h=None) == 0
    assert call(N=0, g=None, h=None) == 0


def test_gated_backward_refusals(L):
    from quantized_unpack_q4_amd import gq
    f = L.gq_gated_i8_backward
    need = gq.gq_gated_i8_backward_workspace_bytes(2, 64, 8)
    assert need >= 2 * 2 * 8 * 2
    assert gq.gq_gated_i8_backward_workspace_bytes(2, 0, 8) == 0 and "H = 0" in gq.last_error()
    assert gq.gq_gated_i8_backward_workspace_bytes(2, 64, (1 << 21) + 1) == 0

    def call(g=P, ldg=64, gs=P, u=P, ldu=64, us=P, xq=P, ldx=64, xs=P, dh=P, dx=P, t=F16, act=1, I=8,
             H=64, N=2, ws=P, n=need):
        return f(g, ldg, gs, u, ldu, us, xq, ldx, xs, dh, dx, t, act, I, H, N, ws, n, None)

    refused(L, call(t=F32), "GQ_EINVAL", "type = 0")
    refused(L, call(act=-1), "GQ_EINVAL", "act = -1")
    refused(L, call(I=0), "GQ_EINVAL", "I = 0")
    refused(L, call(I=(1 << 21) + 1, n=1 << 60), "GQ_ESHAPE", "I = ")
    refused(L, call(H=131071, ldg=131072, ldu=131072, ldx=131072, N=1 << 21, n=1 << 60), "GQ_ESHAPE",
            "N*H")
    refused(L, call(dh=None), "GQ_EINVAL", "dh is NULL")
    refused(L, call(dx=BAD), "GQ_EALIGN", "dx")
    refused(L, call(ws=None), "GQ_EWORKSPACE", str(need))
    refused(L, call(ws=BAD), "GQ_EALIGN", "ws")
    refused(L, call(n=need - 1), "GQ_EWORKSPACE", str(need))
    assert call(N=0, g=None, dh=None, ws=None, n=0) == 0


def test_ffn_refusals(L):
    from quantized_unpack_q4_amd import gq
    f = L.gq_ffn_i8
    T, H, I = 3, 64, 80
    need = gq.gq_ffn_i8_workspace_bytes(T, H, I)
    assert need >= T * (64 + 4 + 160 + 80 + 4)
    assert gq.gq_ffn_i8_workspace_bytes(1 << 20, 1 << 15, 16) == 0 and "2^34" in gq.last_error()
    assert gq.gq_ffn_i8_workspace_bytes(1, 131072, 16) == 0

    def call(g=P, ldg=64, gs=P, u=P, ldu=64, us=P, d=P, ldd=80, ds=P, x=P, out=P, t=F16, act=0, T=T,
             H=H, I=I, ws=P, n=need):
        return f(g, ldg, gs, u, ldu, us, d, ldd, ds, x, out, t, act, T, H, I, ws, n, None)

    refused(L, call(t=F32), "GQ_EINVAL", "type = 0")
    refused(L, call(act=7), "GQ_EINVAL", "act = 7")
    refused(L, call(T=-1), "GQ_EINVAL", "T = -1")
    refused(L, call(I=0), "GQ_EINVAL", "I = 0")
    refused(L, call(I=131072, ldd=131072, n=1 << 60), "GQ_ESHAPE", "I = ")
    refused(L, call(ldd=64), "GQ_ESHAPE", "ld_down")
    refused(L, call(ldu=72), "GQ_EALIGN", "ld_up")
    refused(L, call(d=None), "GQ_EINVAL", "wq_down is NULL")
    refused(L, call(x=BAD), "GQ_EALIGN", " x ")
    refused(L, call(ws=None), "GQ_EWORKSPACE", str(need))
    refused(L, call(n=need - 1), "GQ_EWORKSPACE", str(need))
    assert call(T=0, g=None, x=None, out=None, ws=None, n=0) == 0


def test_helpers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    from quantized_unpack_q4_amd import gq
    q, s = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    x = torch.zeros((4, 64))
    for call in (lambda: gq.quantize_i8(x), lambda: gq.dequant_i8(q, s), lambda: gq.gemv_i8(q, s, x),
                 lambda: gq.gemm_i8(q, s, q, s), lambda: gq.gemm_i8_backward(q, s, x[:, :4].half()),
                 lambda: gq.gated_i8((q, s), (q, s), q, s),
                 lambda: gq.gated_i8_backward((q, s), (q, s), q, s, x[:, :4].half()),
                 lambda: gq.ffn_i8((q, s), (q, s), (q, s), x.half())):
        with pytest.raises(ValueError):
            call()


def test_oracle_codes_are_the_nearest():
    """The oracle's codes against exact fractions, ties and their neighbours among them."""
    g = np.random.default_rng(4)
    x = g.standard_normal((40, 24)).astype(np.float32)
    x[:, 1] = x[:, 0] / 2  # where column 0 is the largest: the tie at 63.5
    x[:20, 0] = np.float32(4.0) * np.sign(x[:20, 0])
    x[:20, 1] = np.where(np.arange(20) % 2 == 0, 2.0, np.nextafter(np.float32(2.0), np.float32(0)))
    x[7, :4] = [127.0, 2.5, 3.5, -0.5]
    x[8] *= np.float32(1e-38)
    x[9] = 0
    q, s = i8.quantize(x.astype(np.float64))
    for n in range(x.shape[0]):
        top = Fraction(float(np.abs(x[n]).max()))
        for k in range(x.shape[1]):
            if top == 0:
                assert q[n, k] == 0 and s[n] == 0
                continue
            t = Fraction(float(x[n, k])) * 127 / top
            assert q[n, k] == round(t), (n, k)  # Python rounds fractions half to even
    assert q[0, 1] == 64 * np.sign(x[0, 1]) and abs(q[1, 1]) == 63
