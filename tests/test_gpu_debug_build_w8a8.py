"""The bounds-checked build (libq4_debug.so) on the INT8 x INT8 products and the block norm: in a process of its own, a case
of every kernel and store path runs without a check firing, with the results the formula gives."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r'''
import torch
from moe_linear_layers_b200 import q4
assert q4.LIB_PATH.endswith("libq4_debug.so") and q4._lib.q4_build_flags() & 1
st = torch.zeros(1, dtype=torch.int32, device="cuda")
g = torch.Generator(device="cuda"); g.manual_seed(1)
codes = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device="cuda", generator=g)
for m, n, k in ((1, 33, 64), (12, 200, 2048), (60, 2048, 2064), (100, 1003, 1040), (333, 512, 2048), (600, 5000, 256), (600, 5001, 256)):
    xq, w, u = codes(m, k), codes(n, k), codes(n, k)
    sa, sw = torch.rand(m, device="cuda") + 0.1, (torch.rand(n, device="cuda") + 0.1) / k
    ref = xq.double() @ w.double().t() * sw.double() * sa.double()[:, None]
    for dt, tol in ((torch.float32, 2.0 ** -21), (torch.bfloat16, 2.0 ** -7)):
        y = q4.q8_linear_w8a8(xq, sa, w, sw, out_dtype=dt, dev_status=st)
        assert int(st.item()) == 0, (m, n, k, int(st.item()))
        assert bool(((y.double() - ref).abs() <= tol * ref.abs()).all()), (m, n, k)
        q4.q8_linear_w8a8_gated(xq, sa, w, sw, u, sw, out_dtype=dt, dev_status=st)
        assert int(st.item()) == 0, (m, n, k, int(st.item()))
for T, H in ((1, 2048), (5, 100), (40, 64), (9, 12000), (3000, 1024), (2500, 2048), (3000, 1001), (3001, 770), (2500, 1000)):
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    r = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    w = torch.rand(H, device="cuda", generator=g) + 0.5
    out, y, xq, sa = q4.block_norm(x, r, w, post_w=w, quant=True, dev_status=st)
    assert int(st.item()) == 0, (T, H, int(st.item()))
    b = x.double(); b = b * torch.rsqrt((b * b).mean(1, keepdim=True) + 1e-5) * w.double() + r.double()
    n = b * torch.rsqrt((b * b).mean(1, keepdim=True) + 1e-5) * w.double()
    assert float((out.double() - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())
    assert float((y.double() - n).abs().max()) <= 2.0 ** -7 * float(n.abs().max())
    assert float((xq.double() * sa.double()[:, None] - y.double()).abs().max()) <= 0.51 * float(sa.max())
print("ok")
'''


def test_debug_build_checks_stay_silent():
    env = dict(os.environ, Q4_DEBUG_LIBRARY="1")
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
