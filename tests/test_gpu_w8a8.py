"""GPU parity of the INT8 x INT8 products (q8_linear_w8a8, q8_linear_w8a8_gated) against the formula in 64 bits.

Tolerances.  The sum is exact, so with unit scales the fp32 output is the sum itself (below 2^24: bit for bit).  In
general y = (float(acc) * sw) * sa makes three roundings of at most 2^-24 of the product, a bias one more of the result,
and a bf16 output one of 2^-8.  The gated form adds, per value with z the exponent's argument: z itself to
7 * 2^-23 of its magnitude (three roundings of g, threefold in the cubic term, and the polynomial's own), e^-z to that times |z| plus
(2 + 1.173 |z|) * 2^-23, one addition, a division of 2 ulp and the products with g and u (1.5 ulp each of their own):
(8.2 |z| + 8) * 2^-23 in all."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24


@pytest.fixture(scope="module")
def q4():
    from moe_linear_layers_b200 import q4 as mod
    assert torch.cuda.is_available()
    return mod


def _inputs(m, n, k, seed=0, mats=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + m + 31 * n + 17 * k)
    xq = torch.randint(-128, 128, (m, k), dtype=torch.int8, device="cuda", generator=g)
    sa = torch.rand(m, device="cuda", generator=g) * 0.05 + 1e-3
    ws = []
    for _ in range(mats):
        ws.append(torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda", generator=g))
        ws.append((torch.rand(n, device="cuda", generator=g) * 0.01 + 1e-4) / math.sqrt(k))
    bias = torch.randn(n, device="cuda", generator=g)
    return xq, sa, ws, bias


def _prod(xq, sa, w, sw):
    acc = xq.double() @ w.double().t()           # exact: below 2^53
    return acc * sw.double() * sa.double()[:, None]


def _check(y, ref, tol, what):
    bad = (y.double() - ref).abs() > tol
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


def _check_linear(q4, m, n, k, out, with_bias, seed=0):
    xq, sa, (w, sw), bias = _inputs(m, n, k, seed)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = q4.q8_linear_w8a8(xq, sa, w, sw, bias=bias if with_bias else None, out_dtype=out, dev_status=st)
    assert int(st.item()) == 0 and y.shape == (m, n) and y.dtype == out
    prod = _prod(xq, sa, w, sw)
    ref = prod + bias.double() if with_bias else prod
    tol = 3.01 * U24 * prod.abs()
    if with_bias:
        tol = tol + U24 * (ref.abs() + tol)
    if out == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    _check(y, ref, tol, f"m={m} n={n} k={k} {out} bias={with_bias}")


# every width of kernel, ragged and whole tiles, one and many rows, lengths on and off the 128-code blocks
SHAPES = [
    (1, 1, 16), (1, 16, 64), (1, 2048, 2048), (2, 17, 48), (4, 512, 2048), (5, 33, 1040), (8, 100, 8192),
    (9, 128, 128), (16, 2048, 8192), (17, 255, 272), (31, 64, 4096), (33, 1003, 1040), (64, 512, 512), (77, 129, 144),
    (100, 2048, 2048), (128, 128, 16), (129, 257, 112), (200, 1024, 2048), (255, 8192, 512), (256, 256, 256),
    (333, 1003, 1040), (512, 2048, 2048), (513, 40, 8192), (1000, 8, 2048), (1025, 1025, 1024), (2048, 512, 2048),
    (2049, 4100, 528), (3, 128256, 256), (300, 70001, 64), (70000, 48, 32), (40, 6000, 4096), (600, 640, 4112),
]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_linear(q4, m, n, k, out):
    _check_linear(q4, m, n, k, out, with_bias=(m + n) % 2 == 1)


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act,out", [("silu", torch.float32), ("silu", torch.bfloat16), ("gelu", torch.float32)])
def test_gated(q4, m, n, k, act, out):
    xq, sa, (wg, sg, wu, su), _ = _inputs(m, n, k, mats=2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = q4.q8_linear_w8a8_gated(xq, sa, wg, sg, wu, su, act=act, out_dtype=out, dev_status=st)
    assert int(st.item()) == 0 and h.shape == (m, n) and h.dtype == out
    g, u = _prod(xq, sa, wg, sg), _prod(xq, sa, wu, su)
    z = g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    ref = g * torch.sigmoid(z) * u
    tol = (8.2 * z.abs() + 8) * 2.0 ** -23 * ref.abs() + (g * u).abs() * 2.0 ** -126
    if out == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    _check(h, ref, tol, f"gated m={m} n={n} k={k} {act} {out}")


@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (16, 128, 1008), (70, 40, 96), (130, 300, 1024), (600, 520, 1024)])
def test_sums_are_exact(q4, m, n, k):
    """Unit scales: every sum of magnitude below 2^24 comes back as the integer itself."""
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    xq = torch.randint(-128, 128, (m, k), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda", generator=g)
    y = q4.q8_linear_w8a8(xq, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"))
    assert torch.equal(y.double(), xq.double() @ w.double().t())


@pytest.mark.parametrize("m", [1, 40, 300])
def test_extreme_sums(q4, m):
    """The largest sums int32 has to hold: all codes -128 (and one row of +127) at the longest k."""
    k, n = q4.Q8_MAX_K, 130
    xq = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    y = q4.q8_linear_w8a8(xq, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"))
    ref = torch.full((m, n), 128.0 * 128 * k, dtype=torch.float64, device="cuda")
    ref[:, 1] = -128.0 * 127 * k
    _check(y, ref, U24 * ref.abs(), "extreme")


@pytest.mark.parametrize("m,n,k", [(3, 40, 64), (48, 130, 160), (300, 700, 256), (2000, 1999, 128)])
def test_neighbouring_memory_stays(q4, m, n, k):
    """The memory before and behind the output is left as it was."""
    xq, sa, (wg, sg, wu, su), _ = _inputs(m, n, k, mats=2)
    for out in (torch.float32, torch.bfloat16):
        buf = torch.full((m * n + 256,), 7.0, dtype=out, device="cuda")
        y = buf[128:128 + m * n].view(m, n)
        q4.q8_linear_w8a8(xq, sa, wg, sg, y=y)
        assert bool((buf[:128] == 7).all()) and bool((buf[128 + m * n:] == 7).all())
        q4.q8_linear_w8a8_gated(xq, sa, wg, sg, wu, su, h=y)
        assert bool((buf[:128] == 7).all()) and bool((buf[128 + m * n:] == 7).all())


def test_outputs_past_32_bits(q4):
    """More than 2^31 outputs: the last rows are where they belong, on both kernels' store paths (n off and on 16 bytes)."""
    for m, n in ((33000, 66001), (33000, 66000)):
        xq, sa, (w, sw), _ = _inputs(m, n, 16)
        y = q4.q8_linear_w8a8(xq, sa, w, sw, out_dtype=torch.bfloat16)
        for rows in (slice(0, 3), slice(m // 2, m // 2 + 3), slice(m - 3, m)):
            ref = _prod(xq[rows], sa[rows], w, sw)
            _check(y[rows], ref, (3.01 * U24 + 2.0 ** -8 * (1 + 4 * U24)) * ref.abs(), f"rows {rows}")
        del y, xq, w


def test_zero_scales_and_codes(q4):
    """A row of zeros as act_quant_per_token codes it (scale 0) gives zeros, plus the bias."""
    xq, sa, (w, sw), bias = _inputs(20, 24, 64)
    xq[3] = 0
    sa[3] = 0
    y = q4.q8_linear_w8a8(xq, sa, w, sw, bias=bias)
    assert torch.equal(y[3], bias)


@pytest.mark.parametrize("m", [0, 1, 50, 400])
def test_empty_sides(q4, m):
    e8 = torch.empty((0, 64), dtype=torch.int8, device="cuda")
    e = torch.empty(0, device="cuda")
    xq, sa, (w, sw), _ = _inputs(max(m, 1), 24, 64)
    assert q4.q8_linear_w8a8(e8, e, w, sw).shape == (0, 24)
    assert q4.q8_linear_w8a8_gated(e8, e, w, sw, w, sw).shape == (0, 24)
    assert q4.q8_linear_w8a8(xq[:m], sa[:m], e8, e).shape == (m, 0)


@pytest.mark.parametrize("m,n,k", [(1, 512, 2048), (24, 300, 2048), (700, 1500, 512)])
def test_graph_and_side_stream(q4, m, n, k):
    """Captured calls replay on new inputs; two streams run the same call side by side; results do not vary."""
    xq, sa, (wg, sg, wu, su), bias = _inputs(m, n, k, mats=2)
    want = q4.q8_linear_w8a8(xq, sa, wg, sg, bias=bias)
    want_h = q4.q8_linear_w8a8_gated(xq, sa, wg, sg, wu, su)
    torch.cuda.synchronize()
    xs, ys, hs = torch.zeros_like(xq), torch.empty_like(want), torch.empty_like(want_h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            q4.q8_linear_w8a8(xs, sa, wg, sg, bias=bias, y=ys)
            q4.q8_linear_w8a8_gated(xs, sa, wg, sg, wu, su, h=hs)
    for _ in range(3):
        xs.copy_(xq)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys, want) and torch.equal(hs, want_h)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[q4.q8_linear_w8a8(xq, sa, wg, sg, bias=bias, stream=s) for s in (s1, s2)] for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for pair in got for t in pair)


def test_feed_forward_in_sequence(q4):
    """A layer's feed-forward on 8-bit weights as a user runs it: norm with codes, gate and up, codes of h, down, the next
    norm -- launched back to back, against the same steps taken one at a time with a synchronisation between."""
    T, H, inter = 96, 512, 1024
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    res = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    nw = (1 + 0.1 * torch.randn(H, device="cuda", generator=g))
    quant = [q4.act_quant_per_token((0.05 * torch.randn(s, device="cuda", generator=g)).bfloat16())
             for s in ((inter, H), (inter, H), (H, inter))]

    def step(sync):
        r, _, xq, sa = q4.block_norm(x, res, nw, quant=True, want_y=False)
        sync()
        h = q4.q8_linear_w8a8_gated(xq, sa, *quant[0], *quant[1], out_dtype=torch.bfloat16)
        sync()
        hq, hs = q4.act_quant_per_token(h)
        sync()
        y = q4.q8_linear_w8a8(hq, hs, *quant[2], out_dtype=torch.bfloat16)
        sync()
        out = q4.block_norm(y, r, nw, quant=True)
        sync()
        return (r, h, y, *out)

    want = step(torch.cuda.synchronize)
    got = [step(lambda: None) for _ in range(10)]
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    # and the whole against fp64 on the weights the codes stand for: four 8-bit roundings of rows and one 16-bit a step
    wg, wu, wd = (q.double() * s.double()[:, None] for q, s in quant)
    r = res.double() + x.double()
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-5) * nw.double()
    gg, uu = n @ wg.t(), n @ wu.t()
    y = (gg * torch.sigmoid(gg) * uu) @ wd.t()
    err = (want[2].double() - y).norm() / y.norm()
    assert float(err) < 0.05


@pytest.mark.parametrize("m,n,k", [(2, 1024, 1024), (30, 2048, 2048), (150, 1024, 2048), (900, 2048, 1024)])
def test_buffers_rewritten_in_sequence(q4, m, n, k):
    """Weights, codes and output buffers that each step rewrites, steps launched back to back: every product reads what
    the quantizers two launches before it wrote, and none overwrites what an earlier one still reads."""
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    ws = [(0.05 * torch.randn((n, k), device="cuda", generator=g)).bfloat16() for _ in range(6)]
    xs = [torch.randn((m, k), device="cuda", generator=g).bfloat16() for _ in range(6)]
    wq, sw = torch.empty((n, k), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    xq, sa = torch.empty((m, k), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    y = torch.empty((m, n), device="cuda")

    def steps(sync):
        out = []
        for w, x in zip(ws, xs):
            q4.act_quant_per_token(w, xq=wq, scale_a=sw)
            sync()
            q4.act_quant_per_token(x, xq=xq, scale_a=sa)
            sync()
            q4.q8_linear_w8a8(xq, sa, wq, sw, y=y)
            sync()
            out.append(y.clone())
            sync()
        return out

    want = steps(torch.cuda.synchronize)
    for _ in range(5):
        got = steps(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(q4):
    xq, sa, (w, sw), bias = _inputs(6, 24, 64)
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8(xq, sa[:5], w, sw)
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8(xq, sa, w, sw[:23])
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8(xq, sa, w, sw, bias=bias[:5])
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8(xq[:, :48], sa, w, sw)
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8(xq, sa, w.t().contiguous().t(), sw)
    with pytest.raises(TypeError):
        q4.q8_linear_w8a8(xq.float(), sa, w, sw)
    with pytest.raises(TypeError):
        q4.q8_linear_w8a8(xq, sa.double(), w, sw)
    with pytest.raises(TypeError):
        q4.q8_linear_w8a8(xq, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8(xq, sa, w.cpu(), sw)
    with pytest.raises(ValueError):
        q4.q8_linear_w8a8_gated(xq, sa, w, sw, w[:8], sw)
    with pytest.raises(TypeError):
        q4.q8_linear_w8a8(xq, sa, w, sw, dev_status=torch.zeros(1, device="cuda"))
    buf = torch.zeros(6 * 64 + 8, dtype=torch.int8, device="cuda")
    with pytest.raises(q4.Q4Error) as e:
        q4.q8_linear_w8a8(buf[8:].view(6, 64), sa, w, sw)
    assert e.value.status == q4.Q4_ERR_ALIGN
    with pytest.raises(q4.Q4Error) as e:
        q4.q8_linear_w8a8(torch.zeros((6, 72), dtype=torch.int8, device="cuda"), sa,
                          torch.zeros((24, 72), dtype=torch.int8, device="cuda"), sw)
    assert e.value.status == q4.Q4_ERR_SHAPE
