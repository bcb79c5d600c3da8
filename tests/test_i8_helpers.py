"""The Python helpers of the int8 operators on the CPU, against a stand-in for the library: what
they allocate lives until the entry point has returned.  An entry launches several kernels and
other threads run meanwhile: memory given back before could be theirs by then."""
import weakref

import pytest

from quantized_unpack_q4_amd import gq


class Entries:
    """Every entry point succeeds; workspace queries ask for 4096 bytes."""

    def __init__(self, made):
        self.made, self.called = made, []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("_workspace_bytes"):
                return 4096
            gone = [shape for shape, ref in self.made if ref() is None]
            assert not gone, (name, gone)
            addresses = {a for a in args if isinstance(a, int)}
            for shape, ref in self.made: # and what was made is what is used
                assert ref().data_ptr() in addresses, (name, shape)
            self.called.append(name)
            return 0
        return entry


@pytest.fixture
def entries(monkeypatch):
    torch = pytest.importorskip("torch")
    made = []

    def new(shape, dtype, like, stream):
        t = torch.zeros(shape, dtype=dtype)
        made.append((tuple(shape), weakref.ref(t)))
        return t

    e = Entries(made)
    monkeypatch.setattr(gq, "_torch", torch)
    monkeypatch.setattr(gq, "_mx_codes", {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    monkeypatch.setattr(gq, "_mx_enter", lambda name, t: (torch, -1))
    monkeypatch.setattr(gq, "_mx_stream", lambda stream, dev: 0)
    monkeypatch.setattr(gq, "_mx_new", new)
    monkeypatch.setattr(gq, "lib", lambda: e)
    return e


@pytest.mark.parametrize("call", ["quantize", "dequant", "gemv", "gemm", "gemm_backward", "gated",
                                  "gated_backward", "ffn"])
def test_new_tensors_live_through_the_call(entries, call):
    import torch
    q, s = torch.zeros((8, 64), dtype=torch.int8), torch.zeros(8)
    d, ds = torch.zeros((64, 16), dtype=torch.int8)[:, :8], torch.zeros(64)
    x, dy = torch.zeros((16, 64), dtype=torch.float16), torch.zeros((16, 8), dtype=torch.float16)
    xq, xs = torch.zeros((16, 64), dtype=torch.int8), torch.zeros(16)
    {"quantize": lambda: gq.quantize_i8(x), "dequant": lambda: gq.dequant_i8(q, s),
     "gemv": lambda: gq.gemv_i8(q, s, x), "gemm": lambda: gq.gemm_i8(q, s, xq, xs),
     "gemm_backward": lambda: gq.gemm_i8_backward(q, s, dy),
     "gated": lambda: gq.gated_i8((q, s), (q, s), xq, xs),
     "gated_backward": lambda: gq.gated_i8_backward((q, s), (q, s), xq, xs, dy),
     "ffn": lambda: gq.ffn_i8((q, s), (q, s), (d, ds), x)}[call]()
    assert len(entries.called) == 1 and entries.made
