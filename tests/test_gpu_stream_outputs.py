"""Calls on a stream other than the current one: memory that queued work on the current stream still uses is not written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    from moe_linear_layers_b200 import q4 as mod
    assert torch.cuda.is_available()
    return mod


def _calls(q4):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((600, 1024), device="cuda", generator=g).bfloat16()
    w = (0.05 * torch.randn((1024, 1024), device="cuda", generator=g))
    q, sa = q4.act_quant_per_token(x)
    wq, sw = q4.act_quant_per_token(w.bfloat16())
    w4 = q4.q4_quantize_pack(w, 64, True)
    ones = torch.ones(1024, device="cuda")
    return [lambda **k: [q4.q8_linear_w8a8(q, sa, wq, sw, **k)], lambda **k: [q4.q8_linear_w8a8_gated(q, sa, wq, sw, wq, sw, **k)],
            lambda **k: list(q4.block_norm(x, x, ones, quant=True, **k)), lambda **k: list(q4.act_quant_per_token(x, **k)),
            lambda **k: [q4.q4_linear_w4a16(x, w4, **k)], lambda **k: [q4.q4_linear_w4a8(q, sa, w4, **k)]]


def test_memory_of_queued_work_is_not_taken(q4):
    """A temporary of each output's size is dropped while the work that fills and reads it is still queued; the call on the side
    stream runs meanwhile."""
    side = torch.cuda.Stream()
    for call in _calls(q4):
        want = call()
        torch.cuda.synchronize()
        for _ in range(3):
            temps = [torch.empty_like(t) for t in want]
            at = {t.data_ptr() for t in temps}
            copies = [torch.empty_like(t) for t in want]
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)        # some 10 ms
            for t, c in zip(temps, copies):
                t.fill_(7)
                c.copy_(t)
            del temps, t
            got = call(stream=side)
            assert not at & {t.data_ptr() for t in got}
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(bool((c == 7).all()) for c in copies)
            del got, copies


def test_outputs_read_and_dropped_on_the_current_stream(q4):
    """The caller orders the current stream behind the side stream, reads an output there and drops it: later calls on the side
    stream do not write that memory before it is read."""
    side = torch.cuda.Stream()
    for call in _calls(q4):
        want = call()
        torch.cuda.synchronize()
        kept = []
        for _ in range(6):
            got = call(stream=side)
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda._sleep(5_000_000)
            kept.append([t.clone() for t in got])
            del got
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for out in kept for a, b in zip(out, want))


def test_captured_with_a_forked_stream(q4):
    """The same calls on a stream that a capture forks: outputs from the graph's own pool, the same bits at every replay."""
    for call in _calls(q4):
        want = call()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            got = call(stream=side)
            torch.cuda.current_stream().wait_stream(side)
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        del graph


def test_chain_built_behind_queued_work(q4):
    """A chain built while the current stream is busy, called at once on another: its stage counters are zero by then."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn(1024, device="cuda", generator=g).bfloat16()
    w1, w2 = (q4.q4_quantize_pack(0.05 * torch.randn((1024, 1024), device="cuda", generator=g), 64, True) for _ in range(2))
    mid, out = torch.empty(1024, dtype=torch.bfloat16, device="cuda"), torch.empty(1024, dtype=torch.bfloat16, device="cuda")
    stages = [[(x, w1, mid)], [(mid, w2, out)]]
    q4.GemvChain(stages)()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(5):
        out.zero_()
        torch.cuda.synchronize()
        junk = torch.full((4096,), 7, dtype=torch.int32, device="cuda")   # memory the counters may be given
        del junk
        torch.cuda._sleep(10_000_000)
        q4.GemvChain(stages)(dev_status=st, stream=side)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.equal(out, want)
