"""The experts' products on the GPU where activations or sizes lie at their
limits, against their definitions in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

import redzones  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24                     # half a step of binary32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    epl.load()


@pytest.fixture(autouse=True)
def _red_zones():
    yield
    redzones.check()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def every_bf16(low, high):
    """All bf16 values of magnitude between low and high, of both signs."""
    bits = torch.arange(0x7f80, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[(v >= low) & (v <= high)]
    return torch.cat([v, -v])


def gelu_parts(z):
    z = z.double()
    return 0.5 * torch.erfc(-z / math.sqrt(2)), \
        torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("expected", [1, 0])
def test_gelu_in_its_tails(expected, out):
    """GELU and its slope relative to their own size, from zero to where they
    leave binary32. The distribution function is a polynomial in t = 1 / (1 +
    p |z|) times exp(-z^2 / 2): t is off by 3 u, which the polynomial passes on
    three times at most and adds 6 u of its own, the exponential 4 u, products
    4 u. In the slope the exponential stands by itself: the binary32 constant
    log2(e) / 2 is off by 1.4e-8 of itself, 19 u of exp(-z^2 / 2) at 13. 32 u
    are asked for."""
    z = every_bf16(2.0 ** -12, 13.0)
    n = len(z)
    cdf, pdf = gelu_parts(z)
    one = torch.zeros(n, 8).bfloat16()
    one[:, 0] = z
    w = torch.ones(1, 8, 8).bfloat16().to(DEV)
    half = 0.0 if out == torch.float32 else 2.0 ** -8
    for act, ref, mag in (("gelu", z.double() * cdf, z.double().abs() * cdf),
                          ("gelu_grad", cdf + z.double() * pdf, cdf + z.double().abs() * pdf)):
        grad = act == "gelu_grad"
        if grad:
            one[:, 0] = 1.0
        pre = z[:, None].expand(n, 8).contiguous().to(DEV) if grad else None
        y = redzones.poisoned((n, 8), out, 0x5A, DEV)
        p = epl.Product(n, expected, 1, 8, 8, 0, 5 if grad else 2, int(out == torch.bfloat16), 0)
        epl.epl_expert_product(p, one.to(DEV), w, None, None, i32([0]), i32([n]), pre, y)
        got = y.cpu().double()
        assert (got == got[:, :1]).all()
        tol = 32 * U * mag + half * ref.abs() + 2.0 ** -126
        off = (got[:, 0] - ref).abs()
        assert (off <= tol).all(), (act, float((off / mag).max() / U), z[(off / mag).argmax()])


@pytest.mark.parametrize("N,K", [(256, 512), (64, 1032)])
def test_weight_gradient_of_a_large_buffer(N, K):
    """Few rows in a buffer of many: with the rows expected, the bits that the
    rows by themselves give, whatever lies behind them."""
    counts = [300, 0, 41, 700]
    rows, cap = sum(counts), 20000
    g = torch.Generator().manual_seed(N)
    d = torch.full((cap, N), float("nan")).bfloat16()
    x = torch.full((cap, K), float("nan")).bfloat16()
    d[:rows] = torch.randn(rows, N, generator=g).bfloat16()
    x[:rows] = torch.randn(rows, K, generator=g).bfloat16()
    d, x = d.to(DEV), x.to(DEV)
    at, n = i32([0, 300, 300, 341]), i32(counts)
    kw = dict(out_dtype=torch.float32)
    want = epl.expert_weight_grad(d[:rows], x[:rows], at, n, **kw)
    assert torch.equal(epl.expert_weight_grad(d, x, at, n, expected_rows=rows, **kw), want)
    start = 0
    for e, c in enumerate(counts):
        de, xe = d[start:start + c].cpu().double(), x[start:start + c].cpu().double()
        for got in (want, epl.expert_weight_grad(d, x, at, n, **kw),
                    epl.expert_weight_grad(d, x, at, n, expected_rows=4, **kw)):
            tol = 2 * (c + 1) * U * (de.abs().t() @ xe.abs())
            assert ((got[e].cpu().double() - de.t() @ xe).abs() <= tol).all()
        start += c
