"""Refusals of the INT8 x INT8 products and of the block norm that need no GPU: the library's checks come before any
CUDA call, and the binding refuses host tensors and unknown options."""
import ctypes

import pytest
import torch

from moe_linear_layers_b200 import q4

FAKE = 0x10000  # never dereferenced: every call below fails validation first
L = q4._lib


@pytest.mark.parametrize("change,expect", [
    (dict(m=-1), q4.Q4_ERR_SHAPE),
    (dict(n=-1), q4.Q4_ERR_SHAPE),
    (dict(m=q4.Q8_MAX_ROWS + 1), q4.Q4_ERR_SHAPE),
    (dict(n=q4.Q8_MAX_ROWS + 1), q4.Q4_ERR_SHAPE),
    (dict(k=0), q4.Q4_ERR_SHAPE),
    (dict(k=24), q4.Q4_ERR_SHAPE),                       # rows would not start on 16 bytes
    (dict(k=q4.Q8_MAX_K + 16), q4.Q4_ERR_SHAPE),         # the sum could leave int32
    (dict(out_dtype=2), q4.Q4_ERR_UNSUPPORTED),
    (dict(xq=None), q4.Q4_ERR_NULL),
    (dict(scale_a=None), q4.Q4_ERR_NULL),
    (dict(wq=None), q4.Q4_ERR_NULL),
    (dict(scale_w=None), q4.Q4_ERR_NULL),
    (dict(y=None), q4.Q4_ERR_NULL),
    (dict(xq=FAKE + 8), q4.Q4_ERR_ALIGN),
    (dict(wq=FAKE + 4), q4.Q4_ERR_ALIGN),
    (dict(y=FAKE + 4), q4.Q4_ERR_ALIGN),
    (dict(scale_a=FAKE + 2), q4.Q4_ERR_ALIGN),
    (dict(scale_w=FAKE + 1), q4.Q4_ERR_ALIGN),
    (dict(bias=FAKE + 2), q4.Q4_ERR_ALIGN),
    (dict(m=0, xq=None, scale_a=None, y=None), q4.Q4_OK),
    (dict(n=0, wq=None, scale_w=None, y=None), q4.Q4_OK),
])
def test_linear_w8a8_validation(change, expect):
    a = dict(xq=FAKE, scale_a=FAKE, m=4, wq=FAKE, scale_w=FAKE, n=8, k=64, bias=None, y=FAKE, out_dtype=0)
    a.update(change)
    assert L.q8_linear_w8a8(*a.values(), None, None) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(act=2), q4.Q4_ERR_UNSUPPORTED),
    (dict(act=-1), q4.Q4_ERR_UNSUPPORTED),
    (dict(wu=None), q4.Q4_ERR_NULL),
    (dict(su=None), q4.Q4_ERR_NULL),
    (dict(wg=None), q4.Q4_ERR_NULL),
    (dict(wu=FAKE + 8), q4.Q4_ERR_ALIGN),
    (dict(su=FAKE + 2), q4.Q4_ERR_ALIGN),
    (dict(k=40), q4.Q4_ERR_SHAPE),
    (dict(m=0, xq=None, scale_a=None, h=None), q4.Q4_OK),
])
def test_gated_validation(change, expect):
    a = dict(xq=FAKE, scale_a=FAKE, m=4, wg=FAKE, sg=FAKE, wu=FAKE, su=FAKE, n=8, k=64, act=0, h=FAKE, out_dtype=1)
    a.update(change)
    assert L.q8_linear_w8a8_gated(*a.values(), None, None) == expect


@pytest.mark.parametrize("y", ["xq", "scale_a", "wq", "scale_w", "bias"])
def test_output_over_an_input_is_refused(y):
    a = dict(xq=1 << 20, scale_a=2 << 20, m=4, wq=3 << 20, scale_w=4 << 20, n=8, k=64, bias=5 << 20)
    assert L.q8_linear_w8a8(*a.values(), a[y], 0, None, None) == q4.Q4_ERR_UNSUPPORTED
    assert L.q8_linear_w8a8(*a.values(), a[y] - 64, 0, None, None) == q4.Q4_ERR_UNSUPPORTED   # y is 128 bytes
    g = (1 << 20, 2 << 20, 4, 3 << 20, 4 << 20, 6 << 20, 7 << 20, 8, 64, 0)
    for up in (6 << 20, 7 << 20):
        assert L.q8_linear_w8a8_gated(*g, up, 0, None, None) == q4.Q4_ERR_UNSUPPORTED


def test_max_k_is_the_last_exact_sum():
    assert q4.Q8_MAX_K % 16 == 0
    assert 128 * 128 * q4.Q8_MAX_K < 2 ** 31 <= 128 * 128 * (q4.Q8_MAX_K + 16)


BIG = 1 << 20


@pytest.mark.parametrize("change,T,H,expect", [
    (dict(), -1, 64, q4.Q4_ERR_SHAPE),
    (dict(), 4, 0, q4.Q4_ERR_SHAPE),
    (dict(), 4, q4.Q4_BLOCK_NORM_MAX_H + 1, q4.Q4_ERR_SHAPE),
    (dict(), 0, 64, q4.Q4_OK),
    (dict(x=None, residual=None), 0, 64, q4.Q4_OK),
    (dict(x_dtype=3), 4, 64, q4.Q4_ERR_UNSUPPORTED),
    (dict(y_dtype=-1), 4, 64, q4.Q4_ERR_UNSUPPORTED),
    (dict(eps=-1e-6), 4, 64, q4.Q4_ERR_SHAPE),
    (dict(eps=float("nan")), 4, 64, q4.Q4_ERR_SHAPE),
    (dict(eps=float("inf")), 4, 64, q4.Q4_ERR_SHAPE),
    (dict(x=None, residual=None), 4, 64, q4.Q4_ERR_NULL),
    (dict(x=None, gate=9 * BIG, gate_rows=1), 4, 64, q4.Q4_ERR_NULL),
    (dict(x=None, post_w=9 * BIG), 4, 64, q4.Q4_ERR_NULL),
    (dict(residual_out=None, y=None), 4, 64, q4.Q4_ERR_NULL),
    (dict(xq=9 * BIG), 4, 64, q4.Q4_ERR_NULL),                    # codes without scales
    (dict(scale_a=9 * BIG), 4, 64, q4.Q4_ERR_NULL),
    (dict(gate=9 * BIG, gate_rows=0), 4, 64, q4.Q4_ERR_SHAPE),
    (dict(gate=9 * BIG, gate_rows=3), 4, 64, q4.Q4_ERR_SHAPE),    # 3 does not divide 4 tokens
    (dict(x=BIG + 2), 4, 64, q4.Q4_ERR_ALIGN),                    # fp32 on 2 bytes
    (dict(residual=2 * BIG + 1), 4, 64, q4.Q4_ERR_ALIGN),
    (dict(y=4 * BIG + 1), 4, 64, q4.Q4_ERR_ALIGN),
    (dict(y=BIG), 4, 64, q4.Q4_ERR_UNSUPPORTED),                  # bf16 over the fp32 x: other rows are hit
    (dict(residual_out=2 * BIG + 4), 4, 64, q4.Q4_ERR_UNSUPPORTED),   # shifted against the residual
    (dict(y=3 * BIG), 4, 64, q4.Q4_ERR_UNSUPPORTED),              # both outputs in one place
    (dict(y=5 * BIG), 4, 64, q4.Q4_ERR_UNSUPPORTED),              # over the weights
])
def test_block_norm_validation(change, T, H, expect):
    f = dict(x=BIG, residual=2 * BIG, pre_w=5 * BIG, residual_out=3 * BIG, y=4 * BIG, x_dtype=0, residual_dtype=1,
             w_dtype=0, gate_dtype=0, y_dtype=1, gate_rows=1, eps=1e-5, res_scale=1.0, branch_scale=1.0)
    f.update(change)
    d = q4.q4_block_norm(**f)
    assert L.block_norm(ctypes.byref(d), T, H, None, None) == expect


def test_packed_descriptor_is_the_structure():
    """The binding's one-call packing and the ctypes structure lay out the same bytes."""
    vals = [*range(101, 110), 0, 1, 2, 0, 1, 5, 1e-5, 0.5, 0.25]
    packed = q4._pack_block_norm(*vals)
    d = q4.q4_block_norm(*vals)
    assert packed == bytes(d) and len(packed) == ctypes.sizeof(d) == 112


def test_block_norm_null_descriptor():
    assert L.block_norm(None, 4, 64, None, None) == q4.Q4_ERR_NULL


def test_binding_refuses_host_tensors_and_unknown_options():
    xq, w = torch.zeros((4, 64), dtype=torch.int8), torch.zeros((8, 64), dtype=torch.int8)
    s4, s8 = torch.ones(4), torch.ones(8)
    with pytest.raises(TypeError):
        q4.q8_linear_w8a8(xq, s4, w, s8)
    with pytest.raises(TypeError):
        q4.q8_linear_w8a8_gated(xq, s4, w, s8, w, s8)
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8_gated(xq, s4, w, s8, w, s8, act="relu")
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8(xq, s4, w[0], s8)
    with pytest.raises(TypeError):
        q4.block_norm(torch.zeros((4, 64)), None, None)
    with pytest.raises(TypeError):
        q4.block_norm(None, None, None)


def test_kernel_choice():
    """Which kernel a size takes (148 SMs: also what the library assumes without a GPU): the three regimes, and sizes that launch
    nothing."""
    for m, n, k, want in ((1, 2048, 2048, "stream"), (8, 2048, 8192, "stream"), (200, 1024, 2048, "split"), (333, 1003, 1040, "split"),
                          (4096, 8192, 2048, "pair"), (2048, 2048, 131056, "pair")):
        assert q4.q8_linear_w8a8_kernel(m, n, k) == q4.q8_linear_w8a8_kernel(m, n, k, gated=True) == want
    for sizes in ((0, 8, 64), (8, 0, 64), (8, 8, 24), (8, 8, q4.Q8_MAX_K + 16), (-1, 8, 64)):
        with pytest.raises(q4.Q4Error):
            q4.q8_linear_w8a8_kernel(*sizes)
