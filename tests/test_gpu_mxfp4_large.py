"""MXFP4 operators on matrices whose byte offsets pass 32 bits, against the plain arithmetic
on their first, middle and last rows.  Codes and scales are made on the device."""
import numpy as np
import pytest

from quantized_unpack_q4_amd import gq
from tests import _mxfp4 as mx
from tests._gpu import dev, host, torch_cuda
from tests.test_gpu_mxfp4 import as_type, check, normal, silu64, values64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded_and_freed():
    torch_cuda().manual_seed(89)
    yield
    torch_cuda().cuda.empty_cache()


def planes(shape, K, lo=112, hi=124):
    torch = torch_cuda()
    q = torch.empty((*shape, K // 2), dtype=torch.uint8, device="cuda").random_(0, 256)
    s = torch.empty((*shape, K // 32), dtype=torch.uint8, device="cuda").random_(lo, hi)
    return q, s


def some_rows(n):
    return np.unique(np.clip([0, 1, n // 2, n - 17, n - 2, n - 1], 0, n - 1))


def test_products_of_many_rows():
    """4.4 GiB of codes: 2.3 million rows of 4096."""
    torch = torch_cuda()
    M, K = 2_300_003, 4096
    q, s = planes((M,), K)
    assert q.numel() > 1 << 32
    r = some_rows(M)
    ri = dev(r)
    W = mx.values(host(q[ri]), host(s[ri]))
    for N in (1, 7, 20):
        xd, x64 = as_type(normal(90, N, K), "bf16")
        ref, S = mx.products(W, x64)
        check(gq.gemm_mxfp4(q, s, xd)[:, ri], ref, S, "bf16", "gemm %d" % N)
        if N <= 16:
            check(gq.gemv_mxfp4(q, s, xd.float())[:, ri], ref, S, "f32", "gemv %d" % N)
        xq, xs = gq.quantize_mxfp4(xd)
        ref, S = mx.products(W, mx.values(host(xq), host(xs)))
        check(gq.gemm_mxfp4_mxfp4(q, s, xq, xs)[:, ri], ref, S, "f32", "mxgemm %d" % N)


def test_products_of_many_activation_rows_and_outputs():
    """Activations of 4.6 GB and outputs of 9 GB, few weight rows."""
    torch = torch_cuda()
    M, K, N = 4400, 2240, (1 << 20) + 5
    q, s = planes((M,), K)
    x = torch.empty((N, K), dtype=torch.bfloat16, device="cuda").normal_()
    assert 2 * x.numel() > 1 << 32 and N * M > 1 << 32
    n, m = some_rows(N), some_rows(M)
    ni, mi = dev(n), dev(m)
    W = mx.values(host(q[mi]), host(s[mi]))
    ref, S = mx.products(W, values64(x[ni]))
    check(gq.gemm_mxfp4(q, s, x)[ni][:, mi], ref, S, "bf16", "gemm")
    xq, xs = gq.quantize_mxfp4(x)
    X = mx.values(host(xq[ni]), host(xs[ni]))
    assert np.array_equal(np.stack(mx.quantize(values64(x[ni]))[:1]), np.stack([host(xq[ni])]))
    del x
    ref, S = mx.products(W, X)
    check(gq.gemm_mxfp4_mxfp4(q, s, xq, xs, dtype=torch.bfloat16)[ni][:, mi], ref, S, "bf16", "mxgemm")


def test_quantise_and_back_beyond_32_bits():
    torch = torch_cuda()
    N, K = (1 << 19) + 3, 16384  # 8.6e9 values
    x = torch.empty((N, K), dtype=torch.float16, device="cuda").normal_()
    q, s = gq.quantize_mxfp4(x)
    ni = dev(some_rows(N))
    qr, sr = mx.quantize(values64(x[ni]))
    assert np.array_equal(host(q[ni]), qr) and np.array_equal(host(s[ni]), sr)
    del x
    v = gq.dequant_mxfp4(q, s, dtype=torch.bfloat16)
    assert np.array_equal(values64(v[ni]), mx.values(qr, sr))
    # three rows far apart
    ldx = (1 << 31) + 8
    flat = v.view(-1)
    rows = flat.as_strided((3, 96), (ldx, 1))
    rows.copy_(torch.randn((3, 96), device="cuda"))
    q, s = gq.quantize_mxfp4(rows)
    qr, sr = mx.quantize(values64(rows.contiguous()))
    assert np.array_equal(host(q), qr) and np.array_equal(host(s), sr)


def expert_layer(T, H, I, E, topk, t, experts):
    """The layer on expert stacks made on the device, every token to one of `experts`; rows of
    some tokens against the formula, h rounded as the layer rounds it."""
    torch = torch_cuda()
    g, u, d = planes((E, I), H, 116, 121), planes((E, I), H, 116, 121), planes((E, H), I, 116, 121)
    dt = torch.float16 if t == "f16" else torch.bfloat16
    x = (torch.empty((T, H), dtype=torch.float32 if T * H < 1 << 28 else dt, device="cuda").normal_() * 0.25).to(dt)
    ids = torch.tensor(experts, dtype=torch.int32, device="cuda")[
        torch.randint(0, len(experts), (T, topk), device="cuda")].contiguous()
    wts = torch.rand((T, topk), device="cuda")
    out, ws = gq.moe_mxfp4(g, u, d, x, ids, wts)
    del ws
    tok = some_rows(T)
    got = values64(out[dev(tok)])
    eid, w = host(ids[dev(tok)]), host(wts[dev(tok)]).astype(np.float64)
    X = values64(x[dev(tok)])
    ref, bound = np.zeros_like(got), np.zeros_like(got)
    val = lambda p, e: mx.values(host(p[0][e]), host(p[1][e]))
    for e in set(eid.reshape(-1).tolist()):
        Wg, Wu, Wd = val(g, e), val(u, e), val(d, e)
        for i, k in zip(*np.nonzero(eid == e)):
            (gv, Sg), (uv, Su) = (mx.products(W_, X[i:i + 1]) for W_ in (Wg, Wu))
            h = silu64(gv) * uv
            # h: its two sums (|silu'| <= 1.1), the epilogue's arithmetic, half a step of the type
            slack = 1.1 * 1e-5 * Sg * (np.abs(uv) + 1e-5 * Su) + np.abs(gv) * 1e-5 * Su + 2.0 ** -19 * np.abs(h)
            slack = slack + mx.EPS2[t] * (np.abs(h) + slack) + mx.TINY[t]
            y, S = mx.products(Wd, h)
            ref[i] += w[i, k] * y[0]
            bound[i] += w[i, k] * (1e-5 * S[0] + (1 + 1e-5) * (slack @ np.abs(Wd).T)[0] + 2.0 ** -23 * (topk + 1) * np.abs(y[0]))
    bound += mx.EPS2[t] * (np.abs(ref) + bound) + mx.TINY[t]
    assert (np.abs(got - ref) <= bound).all(), (np.abs(got - ref) / bound).max()


@pytest.mark.parametrize("T", [3, 200])
def test_expert_stacks_beyond_32_bits(T):
    """256 experts, 4.6 GB of codes a stack; the tokens go to the first and the last ones."""
    expert_layer(T, 8192, 4352, 256, 2, "bf16", [0, 1, 131, 254, 255])


def test_expert_layer_h_beyond_32_bits():
    expert_layer(1 << 17, 32, 16384, 2, 2, "f16", [0, 1])


def test_expert_layer_activations_up_to_32_bits():
    """T*H just under 2^31: 4.3 GB of activations, 8.6 GB of expert outputs."""
    expert_layer((1 << 18) + 900, 8160, 32, 3, 1, "bf16", [0, 1, 2])
