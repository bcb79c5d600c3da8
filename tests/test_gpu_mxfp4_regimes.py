"""MXFP4 operators on the GPU at the sizes that choose each form of a kernel: the tile or
the number of row tiles of a workgroup, how the scales are read, whole rounds of tiles and
halves.  Tolerances and the plain arithmetic are those of test_gpu_mxfp4."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _mxfp4 as mx
from tests._gpu import dev, host, say, torch_cuda
from tests.test_gpu_mxfp4 import moe_case, moe_check

pytestmark = pytest.mark.gpu


# -- mixture of experts ------------------------------------------------------------

@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("topk", [1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 12, 16])
def test_moe_combines_any_number_of_slots(topk, t):
    """The combine step takes slots by eights, fours, twos and ones."""
    T, H, I, E = 5, 96, 32, 16
    ids = np.argsort(np.random.default_rng(topk).random((T, E)), -1)[:, :topk].astype(np.int32)
    ids[1, 0] = -1
    ids[2, topk - 1] = E
    for iw in (False, True):
        moe_check(moe_case(50, T, H, I, E, topk, t, ids), T, H, I, E, topk, t, iw)


@pytest.mark.parametrize("topk", [2, 3, 8])
def test_moe_combines_many_tokens(topk):
    """More workgroups than the device holds: one slot after another."""
    T, H, I, E = 2100, 64, 32, 8
    moe_check(moe_case(51, T, H, I, E, topk, "bf16"), T, H, I, E, topk, "bf16", False)
