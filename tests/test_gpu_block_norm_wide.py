"""block_norm on rows of more than 16384 values: many of them (the persistent form, up to twenty warps a row, one or two slots
of its ring) and few (a CTA a row), against the same steps as the narrower rows; what a row can hold and what a call can
leave out.  Bit for bit, so there is no tolerance but the one of the formula in 64 bits (see test_gpu_block_norm.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import test_gpu_block_norm as base
from test_gpu_block_norm import BF16, F16, F32, q4  # noqa: F401 (q4: the fixture)

pytestmark = pytest.mark.gpu


def _codes_only(q4, T, H, post=False, gates=0, rd=BF16, **kw):
    """Residual and codes without y, on bf16 rows: the fewest bytes a value, so the persistent form from two rows an SM on."""
    c = base._case(T, H, BF16, rd, F32, F32, post, gates, **kw)
    t = base._cuda(c, BF16, rd, F32, F32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r, y, xq, sa = q4.block_norm(t["x"], t["residual"], t["pre_w"], post_w=t["post_w"], gate=t["gate"], quant=True, want_y=False,
                                 dev_status=st)
    rr, _, qq, ss = base._steps(c, 1e-5, 1.0, 1.0, BF16)
    assert y is None and int(st.item()) == 0 and base._equal(r, rr, rd if c["residual"] is not None else BF16)
    assert np.array_equal(xq.cpu().numpy(), qq) and np.array_equal(sa.cpu().numpy(), ss)


@pytest.mark.parametrize("T,H", [(300, 18432), (301, 24576), (297, 17408), (310, 16400), (300, 32768), (295, 18432)])
def test_many_rows(q4, T, H):
    _codes_only(q4, T, H)
    _codes_only(q4, T, H, post=True, with_res=False)
    base._check(q4, T, H, post=False, gates=0, with_res=False)
    base._check(q4, T, H, xd=F16, yd=F16, post=True, gates=0, with_res=False, pre=False)


@pytest.mark.parametrize("T,H", [(600, 16385), (601, 20479), (592, 18001), (600, 20481), (591, 16385)])
def test_many_odd_rows(q4, T, H):
    """Odd widths: the persistent form a value at a time up to 20480, from four rows an SM on and where the shared vectors leave
    room for a row; a CTA a row otherwise."""
    _codes_only(q4, T, H)
    _codes_only(q4, T, H, post=True, gates=1)
    base._check(q4, T, H, xd=F16, rd=F16, yd=F16, post=False, gates=0, quant=False)


@pytest.mark.parametrize("T,H", [(3, 16385), (5, 16386), (4, 16392), (3, 20000), (2, 32766), (2, 32767), (3, 32768)])
def test_few_rows(q4, T, H):
    base._check(q4, T, H, rs=0.9, bs=0.25, gates=T)
    base._check(q4, T, H, xd=F16, rd=F32, yd=F32, wd=BF16, gd=F16, gates=1, quant=H % 2 == 0)
    base._check(q4, T, H, with_res=False, gates=0)
    base._check(q4, T, H, with_x=False, post=False, gates=0, rs=0.7)
    base._check(q4, T, H, pre=False, post=False, gates=1, eps=0.0)


@pytest.mark.parametrize("H", [16385, 16400, 32767, 32768])
def test_zero_and_non_finite_rows(q4, H):
    base.test_zero_and_non_finite_rows(q4, H, 400)


@pytest.mark.parametrize("T,H", [(300, 18432), (300, 24576), (600, 16385)])
def test_zero_and_non_finite_rows_persistent(q4, T, H):
    c = base._case(T, H, BF16, BF16, F32, F32, False, 0)
    for k in ("x", "residual"):
        c[k][[1, 200, T - 1]] = 0
    c["residual"][5, H // 2] = np.inf
    c["x"][6, H - 1] = np.nan
    c["residual"][7] = base._rnd(np.full(H, 3e38, np.float32), BF16)   # squares that leave fp32, not fp64
    t = base._cuda(c, BF16, BF16, F32, F32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r, _, xq, sa = q4.block_norm(t["x"], t["residual"], t["pre_w"], quant=True, want_y=False, dev_status=st)
    assert int(st.item()) == q4.Q4_ERR_NONFINITE
    rr, _, qq, ss = base._steps(c, 1e-5, 1.0, 1.0, BF16)
    ok = np.ones(T, bool)
    ok[[5, 6]] = False
    assert np.array_equal(r.float().cpu().numpy()[ok], base._rnd(rr, BF16)[ok])
    assert np.array_equal(xq.cpu().numpy()[ok], qq[ok]) and np.array_equal(sa.cpu().numpy()[ok], ss[ok])
    for row in (1, 200, T - 1):
        assert not xq[row].any() and float(sa[row]) == 0.0
    assert not bool(torch.isfinite(sa[[5, 6]]).any())


@pytest.mark.parametrize("T,H", [(3, 16385), (4, 16392), (2, 32767), (3, 32768), (300, 18432), (600, 16385)])
def test_in_place_and_single_outputs(q4, T, H):
    base.test_in_place_and_single_outputs(q4, T, H)
    # in place with the codes and without y, where many rows take the persistent form
    c = base._case(T, H, BF16, BF16, F32, F32, False, 0)
    t = base._cuda(c, BF16, BF16, F32, F32)
    r, _, xq, sa = q4.block_norm(t["x"], t["residual"], t["pre_w"], quant=True, want_y=False)
    for name in ("residual", "x"):
        buf = {k: None if v is None else v.clone() for k, v in t.items()}
        out, _, q, s = q4.block_norm(buf["x"], buf["residual"], buf["pre_w"], quant=True, want_y=False, residual_out=buf[name])
        assert out is buf[name] and torch.equal(out, r) and torch.equal(q, xq) and torch.equal(s, sa)


@pytest.mark.parametrize("T,H", [(3, 16385), (3, 16392), (2, 32768), (300, 18432), (600, 16385)])
def test_offset_views(q4, T, H):
    """Rows that start off 16 bytes, and the memory around the outputs."""
    c = base._case(T, H, BF16, F16, F32, F32, False, 0)
    t = {k: v for k, v in base._cuda(c, BF16, F16, F32, F32).items() if v is not None}
    want = q4.block_norm(t["x"], t["residual"], t["pre_w"], quant=True)
    for off in (1, 8, 16):
        shift = {k: torch.cat([torch.zeros(off, dtype=v.dtype, device="cuda"), v.reshape(-1)])[off:].view(v.shape) for k, v in t.items()}
        bufs = [torch.full((T * H + 2 * off,), 7, dtype=d, device="cuda") for d in (F16, BF16, torch.int8)]
        views = [b[off:off + T * H].view(T, H) for b in bufs]
        got = q4.block_norm(shift["x"], shift["residual"], shift["pre_w"], quant=True, residual_out=views[0], y=views[1], xq=views[2])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for b in bufs:
            assert bool((b[:off] == 7).all()) and bool((b[off + T * H:] == 7).all())


@pytest.mark.parametrize("T,H", [(2, 20000), (300, 18432), (600, 16385)])
def test_graph_and_side_stream(q4, T, H):
    base.test_graph_and_side_stream(q4, T, H)


SCRIPT = r'''
import torch
from moe_linear_layers_b200 import q4
assert q4.LIB_PATH.endswith("libq4_debug.so") and q4._lib.q4_build_flags() & 1
st = torch.zeros(1, dtype=torch.int32, device="cuda")
g = torch.Generator(device="cuda"); g.manual_seed(1)
for T, H in ((1, 32768), (3, 16385), (2, 20000), (300, 18432), (300, 24576), (600, 16385), (600, 20479)):
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    r = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    w = torch.rand(H, device="cuda", generator=g) + 0.5
    for want_y in (True, False):
        out, y, xq, sa = q4.block_norm(x, r, w, quant=True, want_y=want_y, dev_status=st)
        assert int(st.item()) == 0, (T, H, int(st.item()))
        b = x.double() + r.double()
        n = b * torch.rsqrt((b * b).mean(1, keepdim=True) + 1e-5) * w.double()
        assert float((out.double() - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())
        # codes of n rounded to bf16 (2^-8 of it), half a step of the code
        assert float((xq.double() * sa.double()[:, None] - n).abs().max()) <= 0.51 * float(sa.max()) + 2.0 ** -7 * float(n.abs().max())
print("ok")
'''


def test_debug_build_checks_stay_silent():
    env = dict(os.environ, Q4_DEBUG_LIBRARY="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
