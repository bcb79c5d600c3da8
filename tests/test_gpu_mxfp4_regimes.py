"""MXFP4 operators on the GPU at the sizes that choose each form of a kernel: the tile or
the number of row tiles of a workgroup, how the scales are read, whole rounds of tiles and
halves.  Tolerances and the plain arithmetic are those of test_gpu_mxfp4."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _mxfp4 as mx
from tests._gpu import dev, host, torch_cuda
from tests.test_gpu_mxfp4 import as_type, check, moe_case, moe_check, normal, values64, weights

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


def token_tile(ws, ids, E, H, I):
    """Tokens of a tile of the expert products, from the tile list the layer left in its
    workspace: checked against the counts for that tile."""
    A = ids.size
    up = lambda v: (v + 255) // 256 * 256
    raw = host(ws)
    o3 = up((E + 3) * 4) + 2 * up(A * 4)
    ntiles = raw[:(E + 3) * 4].view(np.int32)[E + 1]
    count = np.bincount(ids.reshape(-1), minlength=E)
    fits = [bn for bn in (16, 64, 128, 256) if sum(-(-c // bn) for c in count) == ntiles]
    # distinct counts of tiles tell the sizes apart
    assert len(fits) == 1, (ntiles, count, fits)
    first = raw[o3:o3 + 8 * (A + E)].view(np.int32)
    assert sorted(first[:ntiles]) == sorted(np.repeat(np.arange(E), -(-count // fits[0])))
    return fits[0]


def counts_to_ids(seed, count, topk):
    """Expert ids [T][topk] with so many slots of each expert, in a random order."""
    ids = np.repeat(np.arange(len(count)), count)
    return np.random.default_rng(seed).permutation(ids).reshape(-1, topk).astype(np.int32)


# H and I choose how each product reads its scales: 16 bytes at a time (a multiple of 512), by
# dwords (of 128) or byte by byte; 1536 is three chunks of 512 columns, both places in turn
HI = [(1024, 1536), (512, 512), (1536, 640), (384, 2048), (160, 1056)]


@pytest.mark.parametrize("t,iw", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("H,I", HI)
@pytest.mark.parametrize("tile,count,topk", [
    (16, [20, 7, 1, 0, 16, 2], 2),   # the weight-streaming kernel
    (64, [70, 1, 33, 24], 2),        # a full tile and a rest, one token, half a tile, less
    (64, [64, 65, 3, 0, 28], 1),
    (128, [150, 64, 65, 129], 2),    # rests of 22, 64, 65 and 1
    (128, [128, 192, 40], 1),
    (256, [296, 356], 1),            # rests of 40 and 100
    (256, [320, 257, 576], 1),       # 64, 1 and 64 after two whole tiles
    (256, [321, 512, 7], 2),         # 65, none, one short tile
])
def test_moe_tiles(tile, count, topk, H, I, iw, t):
    E = len(count)
    ids = counts_to_ids(1, count, topk)
    T = len(ids)
    _, ws = moe_check(moe_case(60, T, H, I, E, topk, t, ids), T, H, I, E, topk, t, iw)
    assert token_tile(ws, ids, E, H, I) == tile


# -- products ------------------------------------------------------------------------

def cus():
    return torch_cuda().cuda.get_device_properties(0).multi_processor_count


# one row tile of 16 a workgroup up to one per CU, two up to two per CU, then four; a wave
# takes one step of 128 columns at a time below 16 steps, two below 32, then four
FEW_ROWS = [(tiles, K) for tiles in (1, 2, 4) for K in (160, 2080, 4128)]


def few_rows_m(tiles):
    """A number of weight rows for so many tiles a workgroup, no tile or workgroup whole."""
    return {1: 16 * cus() - 19, 2: 16 * cus() + 17, 4: 32 * cus() + 41}[tiles]


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("N", [1, 5, 16])
@pytest.mark.parametrize("tiles,K", FEW_ROWS)
def test_gemm_few_rows(tiles, K, N, t):
    M = few_rows_m(tiles)
    q, s, W = weights(61, M, K)
    xd, x64 = as_type(normal(62, N, K), t)
    y = gq.gemm_mxfp4(q, s, xd)
    ref, S = mx.products(W, x64)
    check(y, ref, S, t, "gemm %s %d %d %d" % (t, M, K, N))


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [1, 5, 16])
@pytest.mark.parametrize("tiles,K", FEW_ROWS)
def test_mxgemm_few_rows(tiles, K, N, t):
    torch = torch_cuda()
    M = few_rows_m(tiles)
    q, s, W = weights(63, M, K)
    xq, xs, X = weights(64, N, K)
    y = gq.gemm_mxfp4_mxfp4(q, s, xq, xs, dtype={"f32": torch.float32, "f16": torch.float16,
                                                 "bf16": torch.bfloat16}[t])
    ref, S = mx.products(W, X)
    check(y, ref, S, t, "mxgemm %s %d %d %d" % (t, M, K, N))


@pytest.mark.parametrize("K", [512, 1536, 544])
def test_mxgemm_whole_and_half_tiles(K):
    """18 x 16 tiles of 256 x 256 (on 256 CUs): 256 whole ones and 32 in halves, one launch."""
    torch = torch_cuda()
    M, N = 4500, 4000
    q, s, W = weights(65, M, K)
    xq, xs, X = weights(66, N, K)
    y = gq.gemm_mxfp4_mxfp4(q, s, xq, xs, dtype=torch.bfloat16)
    ref, S = mx.products(W, X)
    check(y, ref, S, "bf16", "mxgemm whole and halves %d" % K)


@pytest.mark.parametrize("K", [512, 1536, 640, 544])
def test_gemm_whole_and_half_tiles(K):
    M, N = 4500, 4000
    q, s, W = weights(67, M, K)
    xd, x64 = as_type(normal(68, N, K), "f16")
    y = gq.gemm_mxfp4(q, s, xd)
    ref, S = mx.products(W, x64)
    check(y, ref, S, "f16", "gemm whole and halves %d" % K)


# -- activations' range --------------------------------------------------------------

@pytest.mark.parametrize("B", [1, 3, 5, 6, 16])
@pytest.mark.parametrize("ex", [-149, -140, -133, -126, -120, -112, -60, 0, 60, 100])
def test_gemv_whole_vectors_of_a_magnitude(ex, B):
    """Activations from the smallest subnormal on, weights that bring the results to about
    2^-20 or, for 1e-40 and the like, as near as scales go.  GQ_GEMV_ACCURACY: 1e-5 S, and a
    few multiples of 2^-149 for results in the subnormal range: here one for every wave's
    sum and every part (16 waves, 3 parts).  Of an activation 2^-149 may be lost: its third part
    ends at 2^-148."""
    M, K = 48, 1056
    lo = int(np.clip(127 - 20 - ex, 1, 240))
    q, s = mx.weights(69, M, K, lo, lo + 8)
    W = mx.values(q, s)
    x = np.ldexp(normal(70, B, K), ex).astype(np.float32)
    x[:, ::7] = 0.0
    y = values64(gq.gemv_mxfp4(dev(q), dev(s), dev(x)))
    ref, S = mx.products(W, x.astype(np.float64))
    bound = 1e-5 * S + 48 * 2.0 ** -149 + mx.EPS2["f32"] * np.abs(ref) + 2.0 ** -149 * np.abs(W).sum(1)
    assert np.isfinite(y).all() and (np.abs(y - ref) <= bound).all(), (np.abs(y - ref) / bound).max()


@pytest.mark.parametrize("B", [1, 3, 5, 6, 16])
def test_gemv_results_in_the_subnormal_range(B):
    """Products and sums below 2^-126: multiples of 2^-149, off by a rounding at each of the
    additions that follow one another (K / 8 and the joins)."""
    M, K = 48, 1056
    q, s = mx.weights(71, M, K, 127 - 70, 127 - 66)
    W = mx.values(q, s)
    x = np.ldexp(normal(72, B, K), -66).astype(np.float32)
    y = values64(gq.gemv_mxfp4(dev(q), dev(s), dev(x)))
    ref, S = mx.products(W, x.astype(np.float64))
    assert (np.abs(y - ref) <= 1e-5 * S + (K // 8 + 48) * 2.0 ** -149).all()


def test_gemv_near_the_largest_activations():
    """The scaled parts stay finite: 2^127 and neighbours, weights far below one."""
    M, K = 16, 64
    q, s = mx.weights(73, M, K, 40, 44)
    W = mx.values(q, s)
    x = np.full((6, K), np.float32(3.4028235e38))
    x[1] = np.nextafter(np.float32(2.0 ** 127), np.float32(0))
    x[2] = -np.float32(1.2345678 * 2.0 ** 126)
    for B in (1, 3, 6):
        y = values64(gq.gemv_mxfp4(dev(q), dev(s), dev(x[:B])))
        ref, S = mx.products(W, x[:B].astype(np.float64))
        assert (np.abs(y - ref) <= 1e-5 * S).all()


@pytest.mark.parametrize("B", [1, 3, 5, 6, 16])
@pytest.mark.parametrize("value", [2.0 ** 126 * (1 + 2.0 ** -7 - 2.0 ** -22), 2.0 ** 126 * (1 + 2.0 ** -8 - 2.0 ** -22),
                                   2.0 ** 126 * (2 - 2.0 ** -22), 2.0 ** 126 * (1 + 2.0 ** -15 - 2.0 ** -22)])
def test_gemv_results_in_the_highest_binade(value, B):
    """Sums just below the largest number: the parts' sums stay below them.  Three weights of
    one (a single one where three would pass it)."""
    M, K = 16, 64
    n = 3 if 3 * value < 3.4e38 else 1
    q = np.zeros((M, K // 2), np.uint8)
    q[:, :n] = 0x02
    s = np.full((M, K // 32), 127, np.uint8)
    x = np.zeros((B, K), np.float32)
    x[:, :2 * n:2] = np.float32(value)
    x[:, 1::2] = np.float32(-value)  # against zero weights
    y = values64(gq.gemv_mxfp4(dev(q), dev(s), dev(x)))
    ref = n * np.float64(np.float32(value))
    assert (np.abs(y - ref) <= 1e-5 * ref).all()


# -- weights' range --------------------------------------------------------------------

@pytest.mark.parametrize("N", [1, 6, 40])
def test_weights_beyond_a_type_reach_their_rows_only(N):
    """Row 3 has a block of infinite weights of the type (bfloat16, binary32: s = 253 with codes
    of 4; binary16: s = 141 with codes of 4): its results are infinite or NaN, the others
    and the product of two MXFP4 matrices are right."""
    torch = torch_cuda()
    M, K = 40, 160
    q, s = mx.weights(74, M, K, 110, 120)
    q[3, 16:32] = 0x66
    rows = np.arange(M) != 3
    x = np.abs(normal(75, N, K)) + 0.5
    for t, sc in (("bf16", 253), ("f16", 141)):
        s[3, 1] = sc
        W = mx.values(q, s)
        xd, x64 = as_type(x, t)
        ys = [gq.gemm_mxfp4(dev(q), dev(s), xd)]
        if t == "bf16" and N <= 16:
            ys.append(gq.gemv_mxfp4(dev(q), dev(s), xd.float()))
        ref, S = mx.products(W, x64)
        for y in ys:
            v = values64(y)
            assert not np.isfinite(v[:, 3]).any()
            f = "f32" if y.dtype == torch.float32 else t
            bound = mx.EPS2[f] * np.abs(ref) + mx.TINY[f] + 1e-5 * S * (1 + mx.EPS2[f])
            assert (np.abs(v - ref) <= bound)[:, rows].all()
    # scales up to 254, against activations small enough for the results
    s[3, 1] = 254
    W = mx.values(q, s)
    xq, xs = mx.weights(76, N, K, 20, 24)
    ref, S = mx.products(W, mx.values(xq, xs))
    v = values64(gq.gemm_mxfp4_mxfp4(dev(q), dev(s), dev(xq), dev(xs)))
    assert (np.abs(v - ref) <= 1e-5 * S + mx.EPS2["f32"] * np.abs(ref)).all()


@pytest.mark.parametrize("N", [1, 6, 40])
@pytest.mark.parametrize("lo", [0, 1, 3])
def test_smallest_weights(lo, N):
    """Scales from 2^-127 on: subnormal numbers of bfloat16, exact like all others."""
    M, K = 40, 160
    q, s = mx.weights(77, M, K, lo, lo + 2)
    W = mx.values(q, s)
    xd, x64 = as_type(np.ldexp(normal(78, N, K), 100), "bf16")
    ref, S = mx.products(W, x64)
    check(gq.gemm_mxfp4(dev(q), dev(s), xd), ref, S, "bf16", "smallest weights")
    if N <= 16:
        check(gq.gemv_mxfp4(dev(q), dev(s), xd.float()), ref, S, "f32", "smallest weights")
    xq, xs = mx.weights(79, N, K, 220, 224)
    ref, S = mx.products(W, mx.values(xq, xs))
    check(gq.gemm_mxfp4_mxfp4(dev(q), dev(s), dev(xq), dev(xs)), ref, S, "f32", "smallest weights")
    # subnormal activations against large weights
    q, s = mx.weights(80, M, K, 200, 204)
    xd, x64 = as_type(np.ldexp(normal(81, N, K), -130), "bf16")
    ref, S = mx.products(mx.values(q, s), x64)
    check(gq.gemm_mxfp4(dev(q), dev(s), xd), ref, S, "bf16", "subnormal activations")


@pytest.mark.parametrize("tokens", [4, 60, 300])
def test_moe_h_beyond_binary16(tokens):
    """h of one token above 65504: infinite in binary16, and with it that token's outputs;
    the others as ever, and all of them finite in bfloat16."""
    H, I, E, topk = 128, 96, 2, 1
    for t in ("bf16", "f16"):
        st = moe_case(82, tokens, H, I, E, topk, t)
        x = st["x"].clone()
        x[1] *= 8192.0
        st["x"], st["X"] = x, values64(x)
        flat = st["ids"].reshape(-1)
        W = [st["W" + n][flat[1]] for n in "gu"]
        g, u = (st["X"][1] @ w.T for w in W)
        assert np.abs(g / (1 + np.exp(-np.clip(g, -700, 700))) * u).max() > 2 * 65504
        if t == "bf16":
            out, _ = moe_check(st, tokens, H, I, E, topk, t, False)
            assert np.isfinite(values64(out)).all()
        else:
            out, _ = gq.moe_mxfp4(st["g"], st["u"], st["d"], st["x"], dev(st["ids"]), dev(st["wts"]))
            v = values64(out)
            assert not np.isfinite(v[1]).any() and np.isfinite(np.delete(v, 1, 0)).all()
            x[1] = 0.0  # the other tokens' outputs do not depend on it
            alone, _ = gq.moe_mxfp4(st["g"], st["u"], st["d"], x, dev(st["ids"]), dev(st["wts"]))
            assert np.array_equal(np.delete(values64(alone), 1, 0), np.delete(v, 1, 0))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("count", [[3, 9, 4, 2], [70, 1, 33, 24], [150, 64, 65, 129], [321, 512, 7, 300]])
def test_moe_nan_and_infinity_stay_with_their_token_and_expert(count, t):
    """The streaming kernel and each token tile: a NaN or infinity in a token, a block of NaN
    weights in an expert."""
    H, I, E = 160, 96, len(count)
    ids = counts_to_ids(2, count, 1)
    T = len(ids)
    st = moe_case(83, T, H, I, E, 1, t, ids)
    clean, _ = moe_check(st, T, H, I, E, 1, t, False)
    clean = values64(clean)
    x = st["x"].clone()
    x[T // 2, H - 1] = float("nan")
    x[T - 1, 0] = float("inf")
    out, _ = gq.moe_mxfp4(st["g"], st["u"], st["d"], x, dev(st["ids"]), dev(st["wts"]))
    v = values64(out)
    hit = np.isin(np.arange(T), [T // 2, T - 1])
    assert not np.isfinite(v[hit]).any() and np.array_equal(v[~hit], clean[~hit])
    st["d"][1][1, 5, I // 32 - 1] = 255  # the last block of row 5 of expert 1's down matrix
    out, _ = gq.moe_mxfp4(st["g"], st["u"], st["d"], st["x"], dev(st["ids"]), dev(st["wts"]))
    v = values64(out)
    hit = np.zeros(v.shape, bool)
    hit[ids[:, 0] == 1, 5] = True
    assert np.isnan(v[hit]).all() and np.array_equal(v[~hit], clean[~hit])
