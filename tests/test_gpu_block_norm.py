"""GPU parity of block_norm: bit for bit against its steps taken in numpy (fp32 operations in the documented order, sums
of squares in fp64), and against the formula in 64 bits.

Tolerance of the second, with e = 2^-24: b takes five fp32 roundings at most (rstd and four products), the scaled residual
one, their sum one: tol_r = 5.01 e |b| + e |a r| + e |r'|.  n = r' rstd w adds three, and rstd moves by the relative
2-norm of r's error: tol_n = |rstd w| tol_r + |n| (norm(tol_r) / norm(r') + 3.01 e).  A 16-bit store adds half a step
(2^-8 bf16, 2^-11 fp16, and half the smallest fp16 number, 2^-25)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E = 2.0 ** -24
HALF = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}


@pytest.fixture(scope="module")
def q4():
    from moe_linear_layers_b200 import q4 as mod
    assert torch.cuda.is_available()
    return mod


def _rnd(a, dt):
    """fp32 numpy -> the values a tensor of dtype dt holds, as fp32 numpy."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(dt).float().numpy()


def _case(T, H, xd, rd, wd, gd, post, gates, seed=0, with_x=True, with_res=True, pre=True):
    g = np.random.default_rng(seed + T * 7 + H)
    f = lambda *s: g.standard_normal(s).astype(np.float32)  # noqa: E731
    return {"x": _rnd(3 * f(T, H), xd) if with_x else None, "residual": _rnd(8 * f(T, H), rd) if with_res else None,
            "post_w": _rnd(1 + 0.3 * f(H), wd) if post else None, "pre_w": _rnd(1 + 0.3 * f(H), wd) if pre else None,
            "gate": _rnd(f(gates, H), gd) if gates else None}


def _steps(c, eps, rs, bs, ydt):
    """The documented steps: one fp32 operation each."""
    one = np.float32
    rstd = lambda v: (1.0 / np.sqrt(np.square(v.astype(np.float64)).mean(1, keepdims=True) + eps)).astype(one)  # noqa: E731
    with np.errstate(all="ignore"):
        b = c["x"]
        if b is not None:
            if c["post_w"] is not None:
                b = (b * rstd(b)) * c["post_w"]
            b = b * one(bs)
            if c["gate"] is not None:
                b = b * np.repeat(c["gate"], b.shape[0] // c["gate"].shape[0], 0)
        r = c["residual"]
        if r is not None:
            r = r * one(rs)
            r = r + b if b is not None else r
        else:
            r = b
        n = r * rstd(r)
        if c["pre_w"] is not None:
            n = n * c["pre_w"]
        n = _rnd(n, ydt)
        scale = np.abs(n).max(1) * (one(1) / one(127))
        q = np.where(scale[:, None] > 0, np.clip(np.rint(n / scale[:, None]), -128, 127), 0).astype(np.int8)
    return r, n, q, scale


def _cuda(c, xd, rd, wd, gd):
    t = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in c.items()}
    for k, d in (("x", xd), ("residual", rd), ("post_w", wd), ("pre_w", wd), ("gate", gd)):
        t[k] = None if t[k] is None else t[k].to(d)
    return t


def _equal(got, want, dt):
    return np.array_equal(got.float().cpu().numpy(), _rnd(want, dt))


def _check(q4, T, H, xd=BF16, rd=BF16, wd=F32, gd=F32, yd=BF16, post=True, gates=1, rs=1.0, bs=1.0, quant=True, eps=1e-5, **kw):
    c = _case(T, H, xd, rd, wd, gd, post, gates, **kw)
    t = _cuda(c, xd, rd, wd, gd)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r, y, xq, sa = q4.block_norm(t["x"], t["residual"], t["pre_w"], post_w=t["post_w"], gate=t["gate"], eps=eps, res_scale=rs,
                                 branch_scale=bs, out_dtype=yd, quant=quant, dev_status=st)
    assert int(st.item()) == 0
    rr, nn, qq, ss = _steps(c, eps, rs, bs, yd)
    r_dt = rd if c["residual"] is not None else xd
    assert r.dtype == r_dt and y.dtype == yd
    assert _equal(r, rr, r_dt) and _equal(y, nn, yd)
    if quant:
        assert np.array_equal(xq.cpu().numpy(), qq) and np.array_equal(sa.cpu().numpy(), ss)
        if yd != F32 and H % 8 == 0:
            # the quantizer of 16-bit rows divides by 127: scales within an ulp, and codes that differ only next to a border
            xq2, sa2 = q4.act_quant_per_token(y)
            assert bool(((sa2 - sa).abs() <= 2.0 ** -23 * sa2).all())
            off = (xq2.int() - xq.int()).abs()
            frac = (y.double() / sa2.double()[:, None].clamp_min(1e-300)).frac().abs()
            assert int(off.max()) <= 1 and bool(((off == 0) | ((frac - 0.5).abs() < 127 * 2.0 ** -22)).all())
    else:
        assert xq is None and sa is None
    # the formula in 64 bits
    d = {k: None if v is None else v.astype(np.float64) for k, v in c.items()}
    rstd = lambda v: 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)  # noqa: E731
    b = np.zeros((T, H))
    if d["x"] is not None:
        b = d["x"] * (rstd(d["x"]) * d["post_w"] if post else 1.0) * float(np.float32(bs))
        if gates:
            b = b * np.repeat(d["gate"], T // gates, 0)
    ar = d["residual"] * float(np.float32(rs)) if d["residual"] is not None else np.zeros((T, H))
    r64 = ar + b
    tol_r = 5.01 * E * np.abs(b) + E * np.abs(ar) + E * np.abs(r64)
    assert (np.abs(r.double().cpu().numpy() - r64) <= tol_r + HALF[r_dt] * (np.abs(r64) + tol_r) + 2.0 ** -25).all()
    w = d["pre_w"] if d["pre_w"] is not None else np.ones(H)
    s = rstd(r64)
    n64 = r64 * s * w
    moved = np.linalg.norm(tol_r, axis=1, keepdims=True) / np.maximum(np.linalg.norm(r64, axis=1, keepdims=True), 1e-300)
    tol_n = np.abs(s * w) * tol_r + np.abs(n64) * (moved + 3.01 * E)
    assert (np.abs(y.double().cpu().numpy() - n64) <= tol_n + HALF[yd] * (np.abs(n64) + tol_n) + 2.0 ** -25).all()


@pytest.mark.parametrize("T", [1, 2, 3, 37, 300, 1500])
@pytest.mark.parametrize("H", [1, 8, 64, 100, 1000, 1001, 2048])
def test_sizes(q4, T, H):
    _check(q4, T, H, post=T % 2 == 1, gates=(0, 1, T)[(T + H) % 3])


@pytest.mark.parametrize("T,H", [(5, 8192), (3, 8200), (2, 16384), (3, 16385), (2, 32760), (2, 32767), (1, 32768), (170, 8192),
                                 (400, 5120), (300, 4097), (2500, 256), (3, 12000)])
def test_wide_rows(q4, T, H):
    _check(q4, T, H, rs=0.9, bs=0.25)
    _check(q4, T, H, xd=F32, rd=F32, yd=F32, gates=0)


@pytest.mark.parametrize("T,H", [(5000, 64), (5003, 1), (5001, 3), (6000, 17), (5200, 130), (5111, 511), (5000, 512), (5001, 513),
                                 (4800, 1000), (5001, 1001), (4999, 1024), (3000, 1026), (2500, 2047), (2500, 2048), (1300, 4095),
                                 (1300, 4096), (1201, 4097), (700, 8192), (701, 8190), (601, 8193), (600, 12288), (601, 16383)])
def test_many_rows(q4, T, H):
    """Rows enough for the persistent form: every width of access, one to sixteen warps a row, last rows that end inside a
    16-byte piece, gates that change with the token."""
    _check(q4, T, H, gates=1, rs=0.9, bs=0.25)
    _check(q4, T, H, xd=F32, rd=F16, yd=F32, gates=T, quant=H % 2 == 0)
    div = next(g for g in (500, 100, 11, 7, 3, 2, 1) if T % g == 0)
    _check(q4, T, H, xd=F16, rd=BF16, yd=F16, gd=BF16, gates=div, post=False)


@pytest.mark.parametrize("xd", [F32, BF16, F16])
@pytest.mark.parametrize("rd", [F32, BF16, F16])
@pytest.mark.parametrize("yd", [F32, BF16, F16])
def test_types(q4, xd, rd, yd):
    _check(q4, 21, 256, xd=xd, rd=rd, yd=yd, wd=BF16, gd=F16, gates=3, rs=0.5, bs=0.22)
    _check(q4, 21, 255, xd=xd, rd=rd, yd=yd, wd=F16, gd=BF16, gates=7, rs=0.5, bs=0.22, post=False)
    _check(q4, 5000, 512, xd=xd, rd=rd, yd=yd, gates=0, post=xd != rd)
    _check(q4, 5000, 254, xd=xd, rd=rd, yd=yd, gates=1, post=xd != rd)


@pytest.mark.parametrize("T,H", [(7, 512), (7, 129), (900, 2048), (5000, 257), (2600, 2048)])
def test_parts_left_out(q4, T, H):
    _check(q4, T, H, with_res=False, gates=0)
    _check(q4, T, H, with_x=False, post=False, gates=0, rs=0.7)
    _check(q4, T, H, pre=False, post=False, gates=1)
    _check(q4, T, H, quant=False, gates=T, eps=0.0)


@pytest.mark.parametrize("T,H", [(33, 256), (6, 100), (5000, 1024), (4999, 333)])
def test_in_place_and_single_outputs(q4, T, H):
    c = _case(T, H, BF16, BF16, F32, F32, True, 1)
    t = _cuda(c, BF16, BF16, F32, F32)
    args = dict(post_w=t["post_w"], gate=t["gate"])
    r, y, xq, sa = q4.block_norm(t["x"], t["residual"], t["pre_w"], quant=True, **args)
    r2, y2, _, _ = q4.block_norm(t["x"], t["residual"], t["pre_w"], want_residual=False, **args)
    assert r2 is None and torch.equal(y2, y)
    r3, y3, _, _ = q4.block_norm(t["x"], t["residual"], t["pre_w"], want_y=False, **args)
    assert y3 is None and torch.equal(r3, r)
    _, _, q, s = q4.block_norm(t["x"], t["residual"], t["pre_w"], want_y=False, want_residual=False, quant=True, **args)
    assert torch.equal(q, xq) and torch.equal(s, sa)
    res, x = t["residual"].clone(), t["x"].clone()
    out, yy, q, s = q4.block_norm(x, res, t["pre_w"], residual_out=res, y=x, quant=True, **args)
    assert out is res and yy is x and torch.equal(res, r) and torch.equal(x, y) and torch.equal(q, xq) and torch.equal(s, sa)


def test_eps_in_64_bits(q4):
    """eps counts with all its digits: a mean square next to a rounding border of rstd shows one rounded to fp32."""
    H, eps = 128, 1e-5
    g = np.random.default_rng(7)
    x = g.standard_normal((200000, H)).astype(np.float32)
    ms = np.square(x.astype(np.float64)).mean(1)
    off = (1 / np.sqrt(ms + eps)).astype(np.float32) != (1 / np.sqrt(ms + float(np.float32(eps)))).astype(np.float32)
    rows = np.concatenate([x[off], x[:50]])
    assert off.any()
    _, y, _, _ = q4.block_norm(torch.from_numpy(rows).cuda(), None, None, eps=eps, out_dtype=F32, want_residual=False)
    want = rows * (1 / np.sqrt(np.square(rows.astype(np.float64)).mean(1, keepdims=True) + eps)).astype(np.float32)
    assert np.array_equal(y.cpu().numpy(), want)


def test_rows_past_32_bits(q4):
    """More than 2^31 values: the last rows are where they belong."""
    T, H = 270000, 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    some = torch.randn((5, H), device="cuda", generator=g)
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    x[-5:] = some.to(BF16)
    _, y, xq, sa = q4.block_norm(x, None, None, quant=True, want_residual=False)
    _, y5, xq5, sa5 = q4.block_norm(x[-5:].clone(), None, None, quant=True, want_residual=False)
    assert torch.equal(y[-5:], y5) and torch.equal(xq[-5:], xq5) and torch.equal(sa[-5:], sa5)
    assert not bool(y[: T - 5].any()) and not bool(sa[: T - 5].any())


def test_offset_views(q4):
    """Rows that start off 16 bytes, and the memory around the outputs."""
    T, H = 19, 64
    c = _case(T, H, BF16, F32, F32, F32, True, 1)
    t = _cuda(c, BF16, F32, F32, F32)
    want = q4.block_norm(t["x"], t["residual"], t["pre_w"], post_w=t["post_w"], gate=t["gate"], quant=True)
    for off in (1, 3, 8):
        shift = {k: torch.cat([torch.zeros(off, dtype=v.dtype, device="cuda"), v.reshape(-1)])[off:].view(v.shape) for k, v in t.items()}
        bufs = [torch.full((T * H + 2 * off,), 7, dtype=d, device="cuda") for d in (F32, BF16, torch.int8)]
        views = [b[off:off + T * H].view(T, H) for b in bufs]
        got = q4.block_norm(shift["x"], shift["residual"], shift["pre_w"], post_w=shift["post_w"], gate=shift["gate"], quant=True,
                            residual_out=views[0], y=views[1], xq=views[2])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for b in bufs:
            assert bool((b[:off] == 7).all()) and bool((b[off + T * H:] == 7).all())


@pytest.mark.parametrize("H,T", [(64, 400), (65, 400), (2048, 400), (64, 5000), (65, 5000), (2048, 2500)])
def test_zero_and_non_finite_rows(q4, H, T):
    c = _case(T, H, F32, F32, F32, F32, True, 1)
    c["x"][1] = 0
    c["residual"][1] = 0
    c["residual"][5, H // 2] = np.inf
    c["x"][6, 3] = np.nan
    c["residual"][399] = np.finfo(np.float32).max      # squares that leave fp32, not fp64
    c["x"][8] = 1e-38                                    # squares below fp32's smallest
    t = _cuda(c, F32, F32, F32, F32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r, y, xq, sa = q4.block_norm(t["x"], t["residual"], t["pre_w"], post_w=t["post_w"], gate=t["gate"], out_dtype=F32, quant=True,
                                 dev_status=st)
    assert int(st.item()) == q4.Q4_ERR_NONFINITE
    rr, nn, qq, ss = _steps(c, 1e-5, 1.0, 1.0, F32)
    ok = np.ones(T, bool)
    ok[[5, 6]] = False
    assert np.array_equal(r.cpu().numpy(), rr, equal_nan=True)
    assert np.array_equal(y.cpu().numpy()[ok], nn[ok]) and np.isnan(y.cpu().numpy()[6]).all()
    assert np.array_equal(xq.cpu().numpy()[ok], qq[ok]) and np.array_equal(sa.cpu().numpy()[ok], ss[ok])
    assert not xq[1].any() and float(sa[1]) == 0.0
    # without codes nothing is reported, and the other rows do not see the bad ones
    st.zero_()
    _, y2, _, _ = q4.block_norm(t["x"], t["residual"], t["pre_w"], post_w=t["post_w"], gate=t["gate"], out_dtype=F32, dev_status=st)
    assert int(st.item()) == 0 and np.array_equal(y2.cpu().numpy(), y.cpu().numpy(), equal_nan=True)


def test_empty(q4):
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    r, y, xq, sa = q4.block_norm(e, e, None, quant=True, gate=torch.empty((0, 64), device="cuda"))
    assert r.shape == y.shape == xq.shape == (0, 64) and sa.shape == (0,)


@pytest.mark.parametrize("T,H", [(4, 2048), (1200, 1024), (5000, 1024), (2500, 2045)])
def test_graph_and_side_stream(q4, T, H):
    c = _case(T, H, BF16, BF16, F32, F32, True, 1)
    t = _cuda(c, BF16, BF16, F32, F32)
    args = dict(post_w=t["post_w"], gate=t["gate"], quant=True)
    want = q4.block_norm(t["x"], t["residual"], t["pre_w"], **args)
    torch.cuda.synchronize()
    x = torch.zeros_like(t["x"])
    outs = [torch.empty_like(v) for v in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            q4.block_norm(x, t["residual"], t["pre_w"], residual_out=outs[0], y=outs[1], xq=outs[2], scale_a=outs[3], **args)
    for _ in range(3):
        x.copy_(t["x"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [q4.block_norm(t["x"], t["residual"], t["pre_w"], stream=s, **args) for s in (s1, s2) * 6]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in got for a, b in zip(out, want))


def test_refusals(q4):
    x, r = torch.zeros((6, 64), device="cuda"), torch.zeros((6, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        q4.block_norm(x, r[:5], w)
    with pytest.raises(ValueError):
        q4.block_norm(x, r, w[:63])
    with pytest.raises(ValueError):
        q4.block_norm(x, r, w, gate=torch.ones((4, 64), device="cuda"))
    with pytest.raises(ValueError):
        q4.block_norm(x.t().contiguous().t(), r, w)
    with pytest.raises(TypeError):
        q4.block_norm(x.double(), r, w)
    with pytest.raises(TypeError):
        q4.block_norm(x, r, w, post_w=w.bfloat16())
    with pytest.raises(TypeError):
        q4.block_norm(x, r, w, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        q4.block_norm(x, r.cpu(), w)
    for bad in (dict(gate=w, x=None), dict(post_w=w, x=None)):
        with pytest.raises(q4.Q4Error):
            q4.block_norm(bad.pop("x"), r, w, **bad)
    with pytest.raises(q4.Q4Error) as e:
        q4.block_norm(x, r, w, y=x[:, :].view(-1).view(BF16)[:384].view(6, 64))
    assert e.value.status == q4.Q4_ERR_UNSUPPORTED
    with pytest.raises(q4.Q4Error):
        q4.block_norm(x, r, w, want_y=False, want_residual=False)
    with pytest.raises(q4.Q4Error):
        q4.block_norm(x, r, w, eps=-1.0)
