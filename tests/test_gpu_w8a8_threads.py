"""The INT8 products and the block norm called from several host threads at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

# pairs of block-norm shapes that one kernel instance of the persistent form serves with different amounts of shared memory:
# rows of whole 2048s, of other widths on 16 bytes, and of odd widths; one warp a row and 8 (odd: 16)
PAIRS = [((7200, 2048), (600, 16384)), ((7200, 2000), (600, 15000)), ((1800, 1001), (600, 16383))]


@pytest.mark.parametrize("shapes", PAIRS)
def test_two_shapes_of_one_kernel(shapes):
    """Two threads a shape, each on a stream of its own, launch over and over; every call is accepted and gives the bits that the
    call alone gives."""
    from moe_linear_layers_b200 import q4
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    cases = []
    for T, H in shapes:
        x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
        r = torch.randn((T, H), device="cuda", generator=g).bfloat16()
        w = torch.rand(H, device="cuda", generator=g) + 0.5
        want = q4.block_norm(x, r, w, quant=True, want_y=False)
        outs = [torch.empty_like(want[0]), torch.empty_like(want[2]), torch.empty_like(want[3])]
        cases.append((x, r, w, want, outs))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2 * len(cases))

    def work(case):
        x, r, w, _, (ro, xq, sa) = case
        T, H = x.shape
        stream = torch.cuda.Stream()
        bf16 = q4._NORM_DTYPES[torch.bfloat16]
        d = q4._pack_block_norm(x.data_ptr(), r.data_ptr(), 0, 0, w.data_ptr(), ro.data_ptr(), 0, xq.data_ptr(), sa.data_ptr(),
                                bf16, bf16, q4._NORM_DTYPES[torch.float32], 0, bf16, 1, 1e-5, 1.0, 1.0)
        start.wait(30)
        # the library's call alone: the threads meet inside it, not at the interpreter
        for _ in range(60):
            bad = [rc for rc in [q4._lib.block_norm(d, T, H, None, stream.cuda_stream) for _ in range(300)] if rc]
            stream.synchronize()
            if bad:
                failed.append(q4.status_string(bad[0]))
                break

    threads = [threading.Thread(target=work, args=(c,)) for c in cases * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for _, _, _, want, (ro, xq, sa) in cases:
        assert torch.equal(ro, want[0]) and torch.equal(xq, want[2]) and torch.equal(sa, want[3])
