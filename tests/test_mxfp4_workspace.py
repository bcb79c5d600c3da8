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


@pytest.mark.parametrize("size", [(5, 96, 160, 4, 2), (1, 32, 32, 1, 1), (256, 2048, 1024, 64, 8)])
def test_offsets_for_multiples_of_32(L, size):
    T, H, I, E, k = size
    A = T * k
    off = gq.gq_moe_mxfp4_workspace_offsets(*size)
    assert off[0] == 0 and off == sorted(off) and all(o % 256 == 0 for o in off)
    # regions hold what gq.h says of them, and follow one another
    need = [4 * (E + 3), 4 * A, 4 * A, 8 * (A + E), 2 * A * I, 4 * A * H]
    assert all(0 <= off[i + 1] - off[i] - need[i] < 256 for i in range(6))
    assert off[6] == gq.gq_moe_mxfp4_workspace_bytes(*size)
    if H % 256 == 0 and I % 256 == 0:
        assert off == gq.gq_moe_workspace_offsets(*size)


@pytest.mark.parametrize("size,word", REFUSED)
def test_no_offsets_for_what_the_layer_refuses(L, size, word):
    with pytest.raises(gq.GQError) as e:
        gq.gq_moe_mxfp4_workspace_offsets(*size)
    assert word in str(e.value)
    assert L.gq_moe_mxfp4_workspace_offsets(4, 64, 32, 8, 2, None) == gq.GQ_EINVAL
