"""The W8A8 products on CTA pairs: exact sums up to the longest K, ragged token counts, the memory around the output, on sizes
that are asserted to take that kernel.

Tolerances as in the other W8A8 tests: a sum is exact, fp32 rounds it once and each scale once more (3 * 2^-24 of the product,
3.01 with the cross terms).  A gated value whose e^-z is below 2^-100 is g * u up to the roundings of g and u (6 * 2^-24), a
division off by at most 2 ulp (2^-22) and two products (2 * 2^-24): 12 * 2^-24, 12.01 with the cross terms."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24


@pytest.fixture(scope="module")
def q4():
    from moe_linear_layers_b200 import q4 as mod
    assert torch.cuda.is_available()
    return mod


def _pair(q4, m, n, k, gated=False):
    assert q4.q8_linear_w8a8_kernel(m, n, k, gated) == "pair"


def _codes(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-128, 128, shape, dtype=torch.int8, device="cuda", generator=g)


def _inside(y, ref, tol):
    bad = (y.double() - ref).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("m,n,k", [(2048, 2048, 1024), (1999, 2300, 1008), (1281, 8191, 16), (4097, 4104, 240)])
def test_sums_are_exact(q4, m, n, k):
    """Unit scales: every sum (below 2^24 in magnitude) comes back as the integer itself, on each store path."""
    _pair(q4, m, n, k)
    xq, w = _codes(m, m, k), _codes(n, n, k)
    y = q4.q8_linear_w8a8(xq, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"))
    assert torch.equal(y.double(), xq.double() @ w.double().t())


@pytest.mark.parametrize("m,n", [(2048, 2304), (1800, 2049)])
def test_longest_sums(q4, m, n):
    """The longest K: random codes, a token and a weight row of -128 (the largest sum int32 has to hold) and a row of +127."""
    k = q4.Q8_MAX_K
    _pair(q4, m, n, k)
    xq, w = _codes(m, m, k), _codes(n, n, k)
    xq[5] = w[7] = -128
    w[9] = 127
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = q4.q8_linear_w8a8(xq, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"), dev_status=st)
    wd = w.double().t()
    for r in range(0, m, 256):
        ref = xq[r:r + 256].double() @ wd
        _inside(y[r:r + 256], ref, U24 * ref.abs())
    assert float(y[5, 7]) == float(torch.tensor(128.0 * 128 * k, dtype=torch.float64).float())
    assert int(st.item()) == 0


def test_longest_sums_gated(q4):
    """Both accumulator halves at the longest K: constant codes, whose products are known, with scales that keep g large and
    positive (act(g) is g there) and u of either sign."""
    m, n, k = 2048, 1160, q4.Q8_MAX_K
    _pair(q4, m, n, k, gated=True)
    xq = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    wg = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    wu = torch.full((n, k), -127, dtype=torch.int8, device="cuda")
    wg[1], wg[n - 1], wu[3], wu[n - 2] = -126, -100, 127, 1
    sa, s = torch.full((m,), 2.0 ** -12, device="cuda"), torch.full((n,), 2.0 ** -11, device="cuda")
    h = q4.q8_linear_w8a8_gated(xq, sa, wg, s, wu, s)
    g, u = (w[:, 0].double() * -128.0 * k * 2.0 ** -23 for w in (wg, wu))
    assert float(g.min()) > 100      # e^-z below 2^-100
    ref = (g * u).expand(m, n)
    _inside(h, ref, 12.01 * U24 * ref.abs())


@pytest.mark.parametrize("m,n,k", [(2001, 2008, 128), (1793, 4104, 64), (2001, 2009, 128), (2001, 2010, 128)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_neighbouring_memory_stays(q4, m, n, k, out):
    """Rows on 16 bytes (stored by TMA) and off, a last tile with few tokens and columns: the memory before and behind the output
    is left as it was, and the output is the formula's."""
    _pair(q4, m, n, k)
    _pair(q4, m, n, k, gated=True)
    xq, wg, wu = _codes(m, m, k), _codes(n, n, k), _codes(n + 1, n, k)
    sa = torch.rand(m, device="cuda") * 0.05 + 1e-3
    sw = (torch.rand(n, device="cuda") + 0.1) * 0.01
    buf = torch.full((m * n + 4096,), 7.0, dtype=out, device="cuda")
    y = buf[2048:2048 + m * n].view(m, n)
    q4.q8_linear_w8a8(xq, sa, wg, sw, y=y)
    ref = xq.double() @ wg.double().t() * sw.double() * sa.double()[:, None]
    _inside(y, ref, ((3.01 * U24) if out == torch.float32 else 3.01 * U24 + 2.0 ** -8 * (1 + 4 * U24)) * ref.abs())
    assert bool((buf[:2048] == 7).all()) and bool((buf[2048 + m * n:] == 7).all())
    q4.q8_linear_w8a8_gated(xq, sa, wg, sw, wu, sw, h=y)
    assert bool((buf[:2048] == 7).all()) and bool((buf[2048 + m * n:] == 7).all())


@pytest.mark.parametrize("m,n,k", [(1999, 2304, 2064), (2048, 2048, 8192)])
def test_pair_kernel_against_others(q4, m, n, k):
    """An output does not depend on the kernel: a few tokens' rows alone take another one and give the same bits."""
    _pair(q4, m, n, k)
    xq, w, u = _codes(m, m, k), _codes(n, n, k), _codes(n + 1, n, k)
    sa = torch.rand(m, device="cuda") * 0.05 + 1e-3
    sw = (torch.rand(n, device="cuda") + 0.1) / k
    y, h = q4.q8_linear_w8a8(xq, sa, w, sw), q4.q8_linear_w8a8_gated(xq, sa, w, sw, u, sw)
    for rows, kernel in ((slice(m - 7, m), "stream"), (slice(250, 350), "split")):
        c = rows.stop - rows.start
        assert q4.q8_linear_w8a8_kernel(c, n, k) == q4.q8_linear_w8a8_kernel(c, n, k, True) == kernel
        x1, s1 = xq[rows].clone(), sa[rows].clone()
        assert torch.equal(q4.q8_linear_w8a8(x1, s1, w, sw), y[rows])
        assert torch.equal(q4.q8_linear_w8a8_gated(x1, s1, w, sw, u, sw), h[rows])
