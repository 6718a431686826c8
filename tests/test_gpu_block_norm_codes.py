"""block_norm's codes and scales are those that elementary tensor operations on the GPU make of the normed rows, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1, 2048), (300, 1001), (2500, 2048), (4096, 1024), (600, 8192), (5001, 513), (5, 32768)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_codes_of_tensor_operations(T, H, dt):
    from moe_linear_layers_b200 import q4
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    x, r = (torch.randn((T, H), device="cuda", generator=g).to(dt) for _ in range(2))
    w = torch.rand(H, device="cuda", generator=g) + 0.5
    _, y, xq, sa = q4.block_norm(x, r, w, out_dtype=dt, quant=True)
    v = y.float()
    scale = v.abs().amax(-1) / 127
    assert torch.equal(sa, scale) and torch.equal(xq, (v / scale[:, None]).round().clamp(-128, 127).to(torch.int8))
