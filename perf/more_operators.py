"""The 8-bit integer (int8) operators with a scale per row, case by case.

A matrix is int8 codes [rows][K] and one binary32 scale per row: a row of
activations is a token, a row of weights an output channel; the value is
scale * code.  Rows of codes are a multiple of 16 bytes apart.

  quantize  x -> codes and scales, and back to the values they stand for
  gemv      y[B][M] = x[B][K] W^T, float activations quantised per token on the way
  gemm      Y[N][M] = X W^T, both matrices int8
  ffn       the gated feed-forward block: quantise, gate and up products with
            the activation, quantise, down product
  gated     the gate and up half with its backward pass: h, and the gradient of
            the token values for a given gradient of h (weights are frozen)
  grad      the gradient of the product's token values: dX = dY W

Scales are max|row| / 127, codes 127 x / max|row| to the nearest whole number
(ties to even).  Gradients pass the rounding of the codes unchanged.

`run` computes them in plain torch operations, or, where `own` is true, with
the calls a user of quantized_unpack_q4_amd makes.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
GELU_C = math.sqrt(2.0 / math.pi)
GELU_A = 0.044715


# -- cases ---------------------------------------------------------------------

def listed():
    return [
        # one token's activations on their way into the products of a layer
        dict(name="quantize_token", op="quantize", N=1, K=4096, dtype="bf16"),
        # the activations of a 4096-token prompt entering the down product
        dict(name="quantize_prompt", op="quantize", N=4096, K=14336, dtype="f16"),
        # one token against the q or o projection: the smallest product of a decode step
        dict(name="gemv_token", op="gemv", M=4096, K=4096, B=1, dtype="bf16"),
        # sixteen sequences decoded together, the down projection
        dict(name="gemv_batch16_down", op="gemv", M=4096, K=14336, B=16, dtype="f16"),
        # a small product of odd size: no tile, vector or step divides it
        dict(name="gemm_odd", op="gemm", M=1003, K=2083, N=77, dtype="f32"),
        # prompt processing: 4096 tokens through the gate or up projection
        dict(name="gemm_prompt", op="gemm", M=14336, K=4096, N=4096, dtype="bf16"),
        # the feed-forward block of a decode step, one token
        dict(name="ffn_token", op="ffn", T=1, H=4096, I=14336, dtype="bf16", act="silu"),
        # the block in prompt processing
        dict(name="ffn_prompt", op="ffn", T=2048, H=4096, I=14336, dtype="f16", act="silu"),
        # training on top of frozen weights: 1024 tokens through gate and up and back
        dict(name="gated_train", op="gated", N=1024, H=4096, I=14336, dtype="bf16", act="silu"),
        # a small block of odd size with the other activation
        dict(name="gated_train_odd", op="gated", N=77, H=1003, I=517, dtype="f16", act="gelu"),
        # the gradient of 2048 tokens through the down projection
        dict(name="grad_prompt", op="grad", M=4096, K=14336, N=2048, dtype="bf16"),
        # the gradient of a short sequence through the q or o projection
        dict(name="grad_short", op="grad", M=4096, K=4096, N=130, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size between lo and hi: half of them whole multiples of 16."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.5 else max(lo, n // 16 * 16)


def draw(rng):
    op = rng.choice(["quantize", "gemv", "gemm", "ffn", "gated", "grad"])
    any_type, half = rng.choice(["f32", "f16", "bf16"]), rng.choice(["f16", "bf16"])
    act = rng.choice(["silu", "gelu"])
    if op == "quantize":
        return dict(op=op, N=_log_int(rng, 1, 4096), K=_size(rng, 16, 14336), dtype=any_type)
    if op == "gemv":
        return dict(op=op, M=_size(rng, 16, 14336), K=_size(rng, 16, 14336),
                    B=rng.randint(1, 16), dtype=any_type)
    if op == "gemm":
        M, K = _size(rng, 16, 14336), _size(rng, 16, 14336)
        top = min(4096, 14336 * 4096 * 4096 // (M * K))
        return dict(op=op, M=M, K=K, N=_log_int(rng, 1, max(1, top)), dtype=any_type)
    if op == "grad":
        M, K = _size(rng, 16, 14336), _size(rng, 16, 14336)
        top = min(2048, 14336 * 4096 * 2048 // (M * K))
        return dict(op=op, M=M, K=K, N=_log_int(rng, 1, max(1, top)), dtype=half)
    H, I = _size(rng, 64, 4096), _size(rng, 64, 14336)
    if op == "ffn":
        return dict(op=op, T=_log_int(rng, 1, 2048), H=H, I=I, dtype=half, act=act)
    return dict(op=op, N=_log_int(rng, 1, 1024), H=H, I=I, dtype=half, act=act)


# -- inputs --------------------------------------------------------------------

def _normal(gen, shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _row_codes(rows, K):
    """Storage for codes whose rows start 16-byte aligned."""
    return torch.empty((rows, (K + 15) // 16 * 16), dtype=torch.int8, device="cuda")[:, :K]


def _weights(gen, rows, K):
    """Codes and scales of a trained layer's look: normal, each row of its own spread."""
    q, s = _row_codes(rows, K), torch.empty(rows, device="cuda")
    step = max(1, (1 << 25) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        spread = 0.02 * torch.exp2(torch.rand((n, 1), generator=gen, device="cuda") * 2.0 - 1.0)
        w = _normal(gen, (n, K)) * spread
        top = w.abs().amax(-1, keepdim=True)
        q[r:r + n] = torch.round(w * (127.0 / top)).to(torch.int8)
        s[r:r + n] = (top / 127.0).squeeze(-1)
    return q, s


def _activations(gen, rows, K, dtype):
    """Normal, with one channel in 64 about eight times the others."""
    x = _normal(gen, (rows, K))
    big = torch.rand((K,), generator=gen, device="cuda") < 1.0 / 64.0
    return (x * torch.where(big, 8.0, 1.0)).to(dtype)


def _tokens(gen, rows, K):
    """Activations as the quantiser leaves them: codes and scales."""
    q, s = _row_codes(rows, K), None
    q0, s = _quantize_plain(_activations(gen, rows, K, torch.bfloat16))
    q.copy_(q0)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        st["x"] = _activations(gen, case["N"], case["K"], dtype)
    elif op == "gemv":
        st["w"] = _weights(gen, case["M"], case["K"])
        st["x"] = _activations(gen, case["B"], case["K"], dtype)
    elif op == "gemm":
        st["w"] = _weights(gen, case["M"], case["K"])
        st["x"] = _tokens(gen, case["N"], case["K"])
    elif op == "grad":
        st["w"] = _weights(gen, case["M"], case["K"])
        st["dy"] = (0.01 * _normal(gen, (case["N"], case["M"]))).to(dtype)
    else:
        H, I = case["H"], case["I"]
        st["gate"], st["up"] = _weights(gen, I, H), _weights(gen, I, H)
        if op == "gated":
            st["x"] = _tokens(gen, case["N"], H)
            st["dh"] = (0.01 * _normal(gen, (case["N"], I))).to(dtype)
        else:
            st["down"] = _weights(gen, H, I)
            st["x"] = _activations(gen, case["T"], H, dtype)
        if own:
            from quantized_unpack_q4_amd import gq
            n = (gq.gq_gated_i8_backward_workspace_bytes(case["N"], H, I) if op == "gated"
                 else gq.gq_ffn_i8_workspace_bytes(case["T"], H, I))
            st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


# -- one pass ------------------------------------------------------------------

def _quantize_plain(x):
    """(codes as int8, scales) of finite x.  The quotients in 64 bits: half of the
    largest magnitude lies on the border between two codes."""
    top = x.float().abs().amax(-1, keepdim=True)
    t = x.double() * 127.0 / torch.where(top > 0, top, 1.0).double()
    return torch.round(t).to(torch.int8), (top / 127.0).squeeze(-1)


def _product_plain(x, w):
    """X W^T in 32 bits of two matrices (codes, scales)."""
    return (x[0].float() @ w[0].float().t()) * x[1][:, None] * w[1][None, :]


def _act_plain(z, act):
    """act(z) and its derivative: z sigmoid(p(z)), p = z or the tanh form of GELU."""
    if act == "silu":
        p, dp = z, 1.0
    else:
        p = 2.0 * GELU_C * (z + GELU_A * z * z * z)
        dp = 2.0 * GELU_C * (1.0 + 3.0 * GELU_A * z * z)
    sig = 1.0 / (1.0 + torch.exp(-p))
    return z * sig, sig + z * sig * (1.0 - sig) * dp


def run(st):
    case = st["case"]
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if own:
        from quantized_unpack_q4_amd import gq
        if op == "quantize":
            return gq.dequant_i8(*gq.quantize_i8(st["x"]))
        if op == "gemv":
            return gq.gemv_i8(*st["w"], st["x"])
        if op == "gemm":
            return gq.gemm_i8(*st["w"], *st["x"], dtype=dtype)
        if op == "grad":
            return gq.gemm_i8_backward(*st["w"], st["dy"])
        if op == "gated":
            h = gq.gated_i8(st["gate"], st["up"], *st["x"], act=case["act"], dtype=dtype)
            dx, _ = gq.gated_i8_backward(st["gate"], st["up"], *st["x"], st["dh"],
                                         act=case["act"], ws=st["ws"])
            return h, dx
        return gq.ffn_i8(st["gate"], st["up"], st["down"], st["x"], act=case["act"],
                         ws=st["ws"])[0]
    if op == "quantize":
        q, s = _quantize_plain(st["x"])
        return q.float() * s[:, None]
    if op == "gemv":
        return _product_plain(_quantize_plain(st["x"]), st["w"]).to(dtype)
    if op == "gemm":
        return _product_plain(st["x"], st["w"]).to(dtype)
    if op == "grad":
        w = st["w"][0].float() * st["w"][1][:, None]
        return (st["dy"].float() @ w).to(dtype)
    x = st["x"] if op == "gated" else _quantize_plain(st["x"])
    g, u = _product_plain(x, st["gate"]), _product_plain(x, st["up"])
    a, da = _act_plain(g, case["act"])
    h = (a * u).to(dtype)
    if op == "ffn":
        return _product_plain(_quantize_plain(h), st["down"]).to(dtype)
    dh = st["dh"].float()
    dg, du = dh * u * da, dh * a
    dx = (dg @ (st["gate"][0].float() * st["gate"][1][:, None])
          + du @ (st["up"][0].float() * st["up"][1][:, None]))
    return h, dx.to(dtype)


# -- what a pass cannot do without ----------------------------------------------

def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op == "quantize":
        n = case["N"] * case["K"]
        # x in, codes and scales out, the values they stand for out in binary32
        return dict(bytes=n * (b + 1 + 4) + 4 * case["N"], flops=2 * n)
    if op in ("gemv", "gemm", "grad"):
        M, K, N = case["M"], case["K"], case["B"] if op == "gemv" else case["N"]
        x = N * K * (1 if op == "gemm" else b)
        return dict(bytes=M * K + 4 * M + x + b * N * M, flops=2 * M * K * N)
    H, I = case["H"], case["I"]
    if op == "ffn":
        T = case["T"]
        return dict(bytes=3 * H * I + 4 * (2 * I + H) + 2 * b * T * H, flops=6 * T * H * I)
    N = case["N"]
    # forward: two products; backward: two products of their gradients
    return dict(bytes=2 * H * I + 8 * I + N * H * (1 + b) + 2 * b * N * I, flops=8 * N * H * I)


# -- the definition in 64 bits ---------------------------------------------------

def _codes64(x):
    """Codes and scales of x as binary64 numbers, from whole numbers: every x is a
    whole multiple of a power of two, and so is the quotient's remainder."""
    v = x.double()
    top = v.abs().max(-1, keepdim=True).values
    safe = torch.where(top > 0, top, torch.ones_like(top))
    n = torch.floor(254.0 * v.abs() / safe)           # in half steps
    n = n - (n * safe > 254.0 * v.abs()).double() + ((n + 1) * safe <= 254.0 * v.abs()).double()
    on = (n * safe == 254.0 * v.abs())                # the quotient is n half steps exactly
    k = torch.floor((n + 1) / 2)                      # nearest, halves up
    odd_tie = on & (n.remainder(2) == 1) & (k.remainder(2) == 1)
    k = torch.where(odd_tie, k - 1, k)                # halves to even
    return torch.where(v < 0, -k, k), top / 127.0


def _dense64(m):
    return m[0].double() * m[1].double().unsqueeze(-1)


def _times64(a, b):
    return torch.matmul(a, b.t().contiguous())


def exact(case, seed):
    st = prepare(case, seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "quantize":
        k, s = _codes64(st["x"])
        return k * s
    if op == "gemv":
        k, s = _codes64(st["x"])
        return _times64(k * s, _dense64(st["w"]))
    if op == "gemm":
        return _times64(_dense64(st["x"]), _dense64(st["w"]))
    if op == "grad":
        return torch.matmul(st["dy"].double(), _dense64(st["w"]))
    if op == "gated":
        x = _dense64(st["x"])
    else:
        k, s = _codes64(st["x"])
        x = k * s
    wg, wu = _dense64(st["gate"]), _dense64(st["up"])
    g, u = _times64(x, wg), _times64(x, wu)
    if case["act"] == "silu":
        gate = torch.sigmoid(g)
        slope = gate * (1.0 + g * (1.0 - gate))
    else:
        th = torch.tanh(GELU_C * (g + GELU_A * g ** 3))
        gate = 0.5 * (1.0 + th)
        slope = gate + 0.5 * g * (1.0 - th * th) * GELU_C * (1.0 + 3.0 * GELU_A * g ** 2)
    h = g * gate * u
    if op == "ffn":
        k, s = _codes64(h.to(dtype))                  # h is held in the type of x
        return _times64(k * s, _dense64(st["down"]))
    dh = st["dh"].double()
    return h, torch.matmul(dh * u * slope, wg) + torch.matmul(dh * g * gate, wu)
