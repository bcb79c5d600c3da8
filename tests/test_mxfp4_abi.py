"""The MXFP4 entry points on the CPU: refusals on the host, before any launch,
calls without work, and the test oracle's own checks."""
import ctypes

import numpy as np
import pytest

from tests import _mxfp4 as mx

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
    f = L.gq_quantize_mxfp4
    refused(L, f(P, 3, 64, P, P, 2, 64, None), "GQ_EINVAL", "x_type = 3")
    refused(L, f(P, F32, 64, P, P, -1, 64, None), "GQ_EINVAL", "N = -1")
    refused(L, f(P, F32, 64, P, P, 2, 48, None), "GQ_ESHAPE", "K = 48", "multiple")
    refused(L, f(P, F32, 64, P, P, 2, 0, None), "GQ_EINVAL", "K = 0")
    refused(L, f(P, F32, 32, P, P, 2, 64, None), "GQ_ESHAPE", "ldx = 32")
    refused(L, f(P, F32, -64, P, P, 2, 64, None), "GQ_ESHAPE", "ldx = -64")
    refused(L, f(P, F32, 66, P, P, 2, 64, None), "GQ_EALIGN", "66")
    refused(L, f(P, F16, 68, P, P, 2, 64, None), "GQ_EALIGN", "68")
    refused(L, f(P, F32, 1 << 41, P, P, 2, 64, None), "GQ_ESHAPE", "ldx")
    refused(L, f(P, F32, 1 << 20, P, P, (1 << 14) + 1, 1 << 20, None), "GQ_ESHAPE", "2^34")
    refused(L, f(None, F32, 64, P, P, 2, 64, None), "GQ_EINVAL", "x is NULL")
    refused(L, f(P, F32, 64, BAD, P, 2, 64, None), "GQ_EALIGN", " q ")
    refused(L, f(P, F32, 64, P, None, 2, 64, None), "GQ_EINVAL", "s is NULL")
    assert f(None, F16, 0, None, None, 0, 64, None) == 0


def test_dequant_refusals(L):
    f = L.gq_dequant_mxfp4
    refused(L, f(P, P, P, -1, 2, 64, None), "GQ_EINVAL", "out_type")
    refused(L, f(P, P, P, F32, 2, 40, None), "GQ_ESHAPE", "K = 40")
    refused(L, f(P, P, P, F32, (1 << 30) + 1, 32, None), "GQ_ESHAPE", "M = ")
    refused(L, f(P, P, P, F32, (1 << 29) + 1, 32, None), "GQ_ESHAPE", "2^34")
    refused(L, f(P, P, BAD, F32, 2, 64, None), "GQ_EALIGN", "out")
    assert f(None, None, None, F32, 0, 64, None) == 0


def test_gemv_refusals(L):
    f = L.gq_gemv_mxfp4
    for B in (-1, 17):
        refused(L, f(P, P, P, P, 8, 64, B, None), "GQ_EINVAL", "B = %d" % B)
    refused(L, f(P, P, P, P, 8, 72, 1, None), "GQ_ESHAPE", "K = 72")
    refused(L, f(P, P, P, P, (1 << 26) + 1, 64, 1, None), "GQ_ESHAPE", "M = ")
    refused(L, f(P, BAD, P, P, 8, 64, 1, None), "GQ_EALIGN", "ws")
    refused(L, f(P, P, None, P, 8, 64, 1, None), "GQ_EINVAL", "x is NULL")
    assert f(None, None, None, None, 0, 64, 1, None) == 0
    assert f(None, None, None, None, 8, 64, 0, None) == 0


def test_gemm_refusals(L):
    f = L.gq_gemm_mxfp4
    refused(L, f(P, P, P, P, F32, 8, 64, 2, None), "GQ_EINVAL", "type = 0", "GQ_BF16")
    refused(L, f(P, P, P, P, F16, 8, 16, 2, None), "GQ_ESHAPE", "K = 16")
    refused(L, f(P, P, P, P, F16, 8, 64, (1 << 21) + 1, None), "GQ_ESHAPE", "N = ")
    refused(L, f(P, P, P, P, F16, -8, 64, 1, None), "GQ_EINVAL", "M = -8")
    refused(L, f(P, P, P, P, F16, 8, (1 << 22) + 32, 1, None), "GQ_ESHAPE", "K = ")
    refused(L, f(P, P, P, BAD, BF16, 8, 64, 1, None), "GQ_EALIGN", " y ")
    assert f(None, None, None, None, F16, 8, 64, 0, None) == 0
    g = L.gq_gemm_mxfp4_mxfp4
    refused(L, g(P, P, P, P, P, 7, 8, 64, 2, None), "GQ_EINVAL", "y_type = 7")
    refused(L, g(P, P, P, P, P, F32, 8, 100, 2, None), "GQ_ESHAPE", "K = 100")
    refused(L, g(P, P, P, None, P, F32, 8, 64, 2, None), "GQ_EINVAL", "xs is NULL")
    refused(L, g(P, P, P, P, P, F32, 1 << 20, 64, 1 << 18, None), "GQ_ESHAPE", "M*N")
    assert g(None, None, None, None, None, F32, 0, 64, 2, None) == 0


def test_moe_refusals(L):
    from quantized_unpack_q4_amd import gq
    f = L.gq_moe_gemm_mxfp4
    w = [P] * 6
    T, H, I, E, k = 5, 96, 160, 4, 2
    need = gq.gq_moe_mxfp4_workspace_bytes(T, H, I, E, k)
    assert need > T * k * (2 * I + 4 * H)
    assert gq.gq_moe_mxfp4_workspace_bytes(T, 100, I, E, k) == 0
    assert gq.gq_moe_mxfp4_workspace_bytes(T, H, I, 257, k) == 0

    def call(type=F16, T=T, H=H, I=I, E=E, k=k, w=w, x=P, ws=P, n=need):
        return f(*w, x, P, P, P, type, T, H, I, E, k, 0, ws, n, None)

    refused(L, call(type=F32), "GQ_EINVAL", "type = 0")
    refused(L, call(H=80), "GQ_ESHAPE", "H = 80")
    refused(L, call(I=1000), "GQ_ESHAPE", "I = 1000")
    refused(L, call(k=5), "GQ_EINVAL", "topk = 5")
    refused(L, call(E=300), "GQ_ESHAPE", "E = 300")
    refused(L, call(T=1 << 20), "GQ_ESHAPE", "T*topk")
    refused(L, call(T=1 << 18, H=1 << 13, n=1 << 62), "GQ_ESHAPE", "T*H")
    refused(L, call(H=(1 << 22) + 32, n=1 << 62), "GQ_ESHAPE", "H = ")
    refused(L, call(w=[P, P, P, None, P, P]), "GQ_EINVAL", "ws_up is NULL")
    refused(L, call(x=BAD), "GQ_EALIGN", " x ")
    refused(L, call(ws=None), "GQ_EWORKSPACE", str(need))
    refused(L, call(ws=BAD), "GQ_EALIGN", " ws ")
    refused(L, call(n=need - 1), "GQ_EWORKSPACE", str(need))
    assert call(T=0, w=[None] * 6, x=None, ws=None, n=0) == 0


def test_helpers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    from quantized_unpack_q4_amd import gq
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    x = torch.zeros((1, 64))
    for call in (lambda: gq.quantize_mxfp4(x), lambda: gq.dequant_mxfp4(q, s),
                 lambda: gq.gemv_mxfp4(q, s, x), lambda: gq.gemm_mxfp4(q, s, x.half()),
                 lambda: gq.gemm_mxfp4_mxfp4(q, s, q, s),
                 lambda: gq.moe_mxfp4((q[None], s[None]), (q[None], s[None]), (q[None], s[None]),
                                      x.half(), s[:1, :1].int(), x[:1, :1])):
        with pytest.raises(ValueError):
            call()


def test_oracle_grid_and_ties():
    # every tie between neighbours goes to the even code; above 6 saturates
    x = np.zeros((1, 32))
    x[0, :12] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 7.9, -0.0]
    q, s = mx.quantize(x)
    assert s[0, 0] == 127
    v = mx.values(q, s)[0]
    assert list(v[:12]) == [6, 0, 1, 1, 2, 2, 4, 4, 0, -4, 6, 0]
    assert np.signbit(v[11]) and np.signbit(v[8])
    # every (code, scale) is its own quantisation when the block spans its binade
    for sc in (1, 2, 100, 127, 200, 252):
        q = np.arange(256, dtype=np.uint8).reshape(16, 16)
        q[:, 0] = 0x77
        s = np.full((16, 1), sc, np.uint8)
        q2, s2 = mx.quantize(mx.values(q, s))
        assert np.array_equal(q, q2) and np.array_equal(s, s2)
