"""The workspace of the MXFP4 expert layer, asked for on the CPU: its size answers for what
the layer accepts and leaves the reason where it does not."""
import pytest

from quantized_unpack_q4_amd import gq


@pytest.fixture(scope="module")
def L():
    return gq.lib()


# sizes the layer refuses: (T, H, I, E, topk), a word of the reason
REFUSED = [((1 << 18, 1 << 13, 32, 8, 1), "T*H"), ((4, (1 << 22) + 32, 32, 8, 1), "H = "),
           ((4, 32, (1 << 22) + 32, 8, 1), "I = "), ((4, 48, 32, 8, 1), "H = 48"),
           ((4, 32, 32, 8, 9), "topk = 9"), ((1 << 20, 32, 32, 8, 2), "T*topk"), ((-1, 32, 32, 8, 1), "T = -1")]


@pytest.mark.parametrize("size,word", REFUSED)
def test_no_size_for_what_the_layer_refuses(L, size, word):
    P = 0x10000  # aligned, never dereferenced
    st = L.gq_moe_gemm_mxfp4(*[P] * 10, gq.GQ_F16, *size, 0, P, 1 << 62, None)
    assert st != 0 and word in L.gq_last_error().decode()
    L.gq_gemv_mxfp4(P, P, P, P, 8, 64, 17, None)  # another message in between
    assert gq.gq_moe_mxfp4_workspace_bytes(*size) == 0
    msg = L.gq_last_error().decode()
    assert word in msg and "gq_moe_mxfp4_workspace_bytes" in msg


def test_a_size_leaves_the_last_message(L):
    L.gq_gemv_mxfp4(None, None, None, None, 8, 64, 17, None)
    before = L.gq_last_error()
    assert b"B = 17" in before
    assert gq.gq_moe_mxfp4_workspace_bytes(4, 64, 32, 8, 2) > 0
    # the largest sizes the layer takes
    assert gq.gq_moe_mxfp4_workspace_bytes((1 << 20) - 1, 2048 - 32, 32, 8, 1) > 0
    assert gq.gq_moe_mxfp4_workspace_bytes(1, 1 << 22, 1 << 22, 8, 1) > 0
    assert L.gq_last_error() == before
