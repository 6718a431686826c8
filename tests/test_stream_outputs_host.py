"""Which stream a wrapper's own tensors belong to (no GPU: stand-ins for CUDA tensors, streams and the library).  The caching
allocator may hand out memory that work queued on the allocating stream still uses, so a call on another stream has its
outputs and workspaces allocated for that stream, and marked in use by the stream they are read on."""
import contextlib

import pytest
import torch

from moe_linear_layers_b200 import q4

HERE = "the current stream"


class Stream:
    cuda_stream = 7
    device = torch.device("cuda:0")

    def __repr__(self):
        return "the side stream"


SIDE = Stream()


class Cuda(torch.Tensor):
    """A host tensor that answers like one on cuda:0, and notes the streams it is marked in use by."""
    is_cuda = True
    device = torch.device("cuda:0")

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.__dict__.setdefault("marks", []).append(stream)


def cuda(t):
    return t.as_subclass(Cuda)


class Library:
    """Every call succeeds and does nothing; every workspace is 64 bytes."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("workspace_size") or "workspace_size_" in name:
            return lambda *a: 64
        if name == "q4_linear_w4a16_max_gemv_m":
            return lambda: 4

        def call(*a):
            self.streams.append(a[-1])
            return 0
        return call


@pytest.fixture
def made(monkeypatch):
    """[(tensor, the current stream when it was allocated)], by the wrapper under test alone."""
    made, at = [], [HERE]

    @contextlib.contextmanager
    def stream(s):
        at.append(s)
        yield
        at.pop()

    real = torch.empty

    def empty(*shape, dtype=None, device=None):
        t = cuda(real(*shape, dtype=dtype))
        made.append((t, at[-1]))
        return t

    lib = Library()
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at[-1])
    monkeypatch.setattr(q4, "_raw_current_stream", lambda d: 5)
    monkeypatch.setattr(q4, "_current_device", lambda: 0)
    monkeypatch.setattr(q4, "_lib", lib)
    monkeypatch.setattr(q4, "_SPLIT_WS", {})
    made_lib = (made, lib)
    weights = _weights()
    monkeypatch.setattr(torch, "empty", empty)
    return (*made_lib, weights)


def _weights():
    def w4(n, k):
        return q4.Q4Weight(cuda(torch.zeros((n, k // 2), dtype=torch.uint8)), cuda(torch.zeros((n, k // 32), dtype=torch.float16)),
                           None, n, k, 32, True)
    return {"w": w4(8, 64), "gate": w4(4 * 32, 64), "up": w4(4 * 32, 64), "down": w4(4 * 64, 32)}


def bf16(*s):
    return cuda(torch.zeros(s, dtype=torch.bfloat16))


def f32(*s):
    return cuda(torch.zeros(s))


def i8(*s):
    return cuda(torch.zeros(s, dtype=torch.int8))


def i32(*s):
    return cuda(torch.zeros(s, dtype=torch.int32))


def _experts(W):
    return (W["gate"], W["up"], W["down"])


CALLS = {
    "q8_linear_w8a8": lambda W, **k: q4.q8_linear_w8a8(i8(3, 64), f32(3), i8(8, 64), f32(8), **k),
    "q8_linear_w8a8 bf16": lambda W, **k: q4.q8_linear_w8a8(i8(3, 64), f32(3), i8(8, 64), f32(8), out_dtype=torch.bfloat16, **k),
    "q8_linear_w8a8_gated": lambda W, **k: q4.q8_linear_w8a8_gated(i8(3, 64), f32(3), i8(8, 64), f32(8), i8(8, 64), f32(8), **k),
    "block_norm": lambda W, **k: q4.block_norm(bf16(3, 64), bf16(3, 64), f32(64), quant=True, **k),
    "q4_quantize_pack": lambda W, **k: q4.q4_quantize_pack(f32(8, 64), 32, False, **k),
    "q4_linear_w4a16": lambda W, **k: q4.q4_linear_w4a16(bf16(16, 64), W["w"], **k),
    "q4_linear_w4a16_swiglu": lambda W, **k: q4.q4_linear_w4a16_swiglu(f32(2, 64), f32(2, 64), W["w"], **k),
    "act_quant_per_token": lambda W, **k: q4.act_quant_per_token(bf16(3, 64), **k),
    "q4_linear_w4a8": lambda W, **k: q4.q4_linear_w4a8(i8(3, 64), f32(3), W["w"], **k),
    "moe_q4_forward": lambda W, **k: q4.moe_q4_forward(bf16(3, 64), f32(4, 64), None, 2, _experts(W), 32, want_routing=True, **k),
    "moe_q4_forward a8": lambda W, **k: q4.moe_q4_forward(bf16(3, 64), f32(4, 64), None, 2, _experts(W), 32, a8_mask=1, **k),
    "moe_q4_forward_classes": lambda W, **k: q4.moe_q4_forward_classes(bf16(3, 64), f32(4, 64), None, 2, [0, 4], [_experts(W)], 32,
                                                                       want_routing=True, **k),
    "moe_q4_forward_range": lambda W, **k: q4.moe_q4_forward_range(bf16(3, 64), f32(4, 64), None, 2, 0, 4, _experts(W), 32, **k),
    "moe_q4_forward_noalloc": lambda W, **k: q4.moe_q4_forward_noalloc(bf16(3, 64), f32(4, 64), None, 2, _experts(W), 32, **k),
    "moe_q4_route": lambda W, **k: q4.moe_q4_route(bf16(3, 64), f32(4, 64), None, 2, **k),
    "moe_q4_forward_rows": lambda W, **k: q4.moe_q4_forward_rows(bf16(6, 64), i32(6), 0, _experts(W), 32, **k),
    "moe_q4_combine": lambda W, **k: q4.moe_q4_combine(f32(6, 64), i32(6), f32(3, 2), **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_made_for_the_stream_of_the_call(made, name):
    tensors, lib, W = made
    CALLS[name](W, stream=SIDE)
    assert tensors and lib.streams == [SIDE.cuda_stream]
    for t, at in tensors:
        assert at is SIDE, f"{name}: a tensor of {tuple(t.shape)} was allocated for {at}"
        assert HERE in t.marks, f"{name}: a tensor of {tuple(t.shape)} may be reused while {HERE} reads it"


@pytest.mark.parametrize("name", CALLS)
def test_made_for_the_current_stream(made, name):
    tensors, lib, W = made
    CALLS[name](W)
    assert tensors and lib.streams == [5]
    assert all(at is HERE and not hasattr(t, "marks") for t, at in tensors)


def test_shared_workspace_grows_behind_its_users(made, monkeypatch):
    """A larger workspace takes the place of one whose last call may still be queued: the smaller one is marked in use by the
    stream of the call that comes after it."""
    tensors, lib, W = made
    size = [64]
    monkeypatch.setattr(Library, "q4_linear_workspace_size", lambda self, *a: size[0], raising=False)
    dev = torch.device("cuda:0")
    a = q4.linear_workspace(16, W["w"], dev)
    size[0] = 128
    b = q4.linear_workspace(16, W["w"], dev, SIDE)
    assert a.marks == [SIDE] and b is not a and [at for _, at in tensors] == [HERE, SIDE]
    size[0] = 256
    q4.linear_workspace(16, W["w"], dev)
    assert HERE in b.marks


@pytest.mark.parametrize("capturing", [False, True])
def test_chain_counters_are_zero_before_any_call(made, monkeypatch, capturing):
    """A chain's stage counters are zeroed on the stream that builds it, and its calls may go to any: the zeros are waited for
    once, where the chain is built (never inside a capture, which may not wait)."""
    tensors, lib, W = made
    waited = []

    class Current:
        def synchronize(self):
            waited.append(len(lib.streams))

    monkeypatch.setattr(torch, "zeros", lambda *s, dtype=None, device=None: torch.ones(*s, dtype=dtype).mul(0).as_subclass(Cuda))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Current())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(Library, "q4_linear_w4a16_chain_sync_bytes", lambda self, n: 64, raising=False)
    w = W["w"]
    x, y = torch.ones(w.k, dtype=torch.bfloat16).as_subclass(Cuda), torch.ones(w.n).as_subclass(Cuda)
    chain = q4.GemvChain([[(x, w, y)]])
    assert waited == ([] if capturing else [0])
    chain(stream=SIDE)
    assert lib.streams == [SIDE.cuda_stream] and waited == ([] if capturing else [0])
