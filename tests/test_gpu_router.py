"""The router and its gradient on the GPU against their definitions in 64 bits.

Tolerances (u = 2^-24, half a step of binary32). Indices are exact. Weights:
renormalised ones and those of a biased choice are computed in binary64 and
rounded once (2 u asked for); the rest take binary32 exponentials, each off
by at most (2 |x| + 4) u for arguments |x| (the product with log2(e) is
rounded, the instruction is good to about a step), and a sum of at most 2048
terms added at most 38 deep; with |x| <= 30 below that is 102 u, and 128 u
is asked for. Gradients are binary32 throughout: per element (2 |x| + 64) u
of the sum of the magnitudes that enter it covers the exponentials, the
quotients and the sums over at most 64 slots; outputs in bf16 add half a step
of it, 2^-8.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

import redzones  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    epl.load()


@pytest.fixture(autouse=True)
def _red_zones():
    yield
    redzones.check()


def reference(logits, bias, K, score, G, TG, top, renorm, scale, mask):
    """The definition, in 64 bits."""
    x = np.minimum(np.asarray(logits, dtype=np.float64), np.finfo(np.float32).max)
    x = np.where(x > -np.inf, x, -np.inf)
    T, E = x.shape
    b = np.zeros(E) if bias is None else np.minimum(bias.astype(np.float64),
                                                    np.finfo(np.float32).max)
    out = ~(x > -np.inf) | ~(b > -np.inf)[None]
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "softmax":
            m = x.max(1, keepdims=True)
            p = np.where(x > -np.inf, np.exp(x - np.where(np.isfinite(m), m, 0.0)), 0.0)
            total = p.sum(1, keepdims=True)
            p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
        else:
            p = np.where(x > -np.inf, 1.0 / (1.0 + np.exp(-x)), 0.0)
        sums = bias is not None or (TG < G and top == 2)
        c = np.where(out, -np.inf, p + b if sums else x)
    if TG < G:
        g = np.sort(c.reshape(T, G, E // G), axis=2)[:, :, ::-1]
        s = g[:, :, 0].copy()
        if top == 2 and E // G > 1:
            with np.errstate(invalid="ignore"):
                s = np.where(g[:, :, 1] > -np.inf, s + g[:, :, 1], s)
        if sums:
            # Two groups may hold the same scores and biases paired otherwise:
            # equal sums, which binary64 rounds apart by some 2^-52. With 40
            # bits they are equal again (sums that differ do so by far more).
            finite = np.isfinite(s)
            part, power = np.frexp(np.where(finite, s, 0.0))
            s = np.where(finite, np.ldexp(np.round(part * 2.0 ** 40) * 2.0 ** -40, power), s)
        order = np.argsort(-s, axis=1, kind="stable")
        for t in range(T):
            for o in order[t, TG:]:
                c[t, o * (E // G):(o + 1) * (E // G)] = -np.inf
    idx = np.argsort(-c, axis=1, kind="stable")[:, :K]
    live = np.take_along_axis(c, idx, 1) > -np.inf
    if mask is not None:
        live &= mask[:, None] != 0
    if score == "softmax" and renorm:       # ratios: from the chosen alone, so they cannot underflow
        xs = np.where(live, np.take_along_axis(x, idx, 1), -np.inf)
        m = xs.max(1, keepdims=True)
        w = np.where(live, np.exp(xs - np.where(np.isfinite(m), m, 0.0)), 0.0)
    else:
        w = np.where(live, np.take_along_axis(p, idx, 1), 0.0)
    if renorm:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return np.where(live, idx, -1), w * scale


def check(logits, bias, K, score="softmax", G=1, TG=1, top=1, renorm=False, scale=1.0, mask=None):
    T, E = logits.shape
    code = epl.EPL_OUT_BF16 if logits.dtype == torch.bfloat16 else epl.EPL_OUT_F32
    p = epl.Router(T, K, E, {"softmax": 0, "sigmoid": 1}[score], G, TG, top, int(renorm), code,
                   scale, 0)
    idx = redzones.poisoned((T, K), torch.int64, 0x5A, DEV)
    w = redzones.poisoned((T, K), torch.float32, 0x5A, DEV)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    epl.epl_route(p, d(logits), d(bias), d(mask), idx, w)
    ri, rw = reference(logits.float().numpy(), None if bias is None else bias.numpy(), K, score, G,
                       TG, top, renorm, scale, None if mask is None else mask.numpy())
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    got = w.cpu().double().numpy()
    u = (2 if renorm else 128) * U
    assert (np.abs(got - rw) <= u * np.abs(rw) + 1e-37).all(), np.abs(got - rw).max()
    return idx, w


def logits_of(T, E, dtype, seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).clamp(-12, 12).to(dtype)


# Experts on both sides of every kernel's reach, odd counts, one token to several workgroups.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (3, 7, 3), (33, 60, 8), (64, 64, 6),
                                   (65, 72, 1), (31, 128, 7), (17, 200, 8), (9, 256, 8),
                                   (5, 257, 8), (7, 512, 8), (3, 1000, 5), (2, 2048, 8),
                                   (6, 96, 9), (4, 160, 64), (2, 2048, 33)])
def test_plain_choice(T, E, K, dtype):
    x = logits_of(T, E, dtype, seed=E)
    check(x, None, K, "softmax")
    check(x, None, K, "sigmoid", renorm=True, scale=2.5)
    b = torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.1
    check(x, b, K, "sigmoid", renorm=True)
    check(x, b, K, "softmax", renorm=False, scale=-0.5)


@pytest.mark.parametrize("T", [4097, 5000])
@pytest.mark.parametrize("E", [60, 128, 250, 256, 512])
def test_many_tokens(T, E):
    x = logits_of(T, E, torch.float32, seed=T + E)
    mask = (torch.arange(T) % 7 != 3).to(torch.uint8)
    check(x, None, 8, "softmax", mask=mask)
    check(x, torch.linspace(-0.2, 0.2, E), 8, "sigmoid", renorm=True, mask=mask)


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T,E,G,TG,K", [(65, 256, 8, 4, 8), (4100, 256, 8, 4, 8), (5, 256, 4, 1, 8),
                                        (9, 256, 32, 3, 6), (7, 160, 8, 3, 6), (5, 60, 4, 2, 4),
                                        (3, 2048, 2, 1, 8), (4, 2048, 64, 5, 8), (6, 64, 64, 9, 8),
                                        (4100, 512, 8, 2, 8), (33, 128, 2, 1, 8),
                                        (11, 256, 8, 8, 8), (5, 256, 8, 4, 20)])
def test_groups(T, E, G, TG, K, top):
    x = logits_of(T, E, torch.float32, seed=G + T)
    b = torch.randn(E, generator=torch.Generator().manual_seed(2)) * 0.05
    check(x, b, K, "sigmoid", G, TG, top, renorm=True, scale=2.5)
    check(x, None, K, "softmax", G, TG, top)
    check(x.bfloat16(), None, K, "sigmoid", G, TG, top, renorm=True)


@pytest.mark.parametrize("T", [3, 5000])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G,TG", [(1, 1), (8, 4)])
def test_ties_go_to_the_lower_index(T, biased, G, TG):
    """Logits of three values only: nearly everything ties."""
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-1, 2, (T, 256), generator=g).float()
    b = torch.zeros(256) if biased else None
    for score in ("softmax", "sigmoid"):
        check(x, b, 8, score, G, TG, 2, renorm=True)
        check(torch.zeros(T, 256), b, 8, score, G, TG, 2, renorm=True)


@pytest.mark.parametrize("T,E,G,TG", [(3, 64, 1, 1), (40, 128, 4, 2), (5, 256, 8, 4),
                                      (5000, 256, 8, 4), (7, 512, 1, 1), (3, 1024, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biased_choice_of_coarse_logits(T, E, G, TG, score):
    """Logits of few values and a bias of few: many scores tie or nearly do,
    among tokens where none does, in every kernel."""
    g = torch.Generator().manual_seed(E + T)
    x = torch.randn(T, E, generator=g) * 1.5
    x[::3] = (x[::3] * 2).round() / 2
    b = torch.randint(-2, 3, (E,), generator=g) * 2.0 ** -5
    mask = (torch.rand(T, generator=g) > 0.2).to(torch.uint8)
    check(x, b, 8, score, G, TG, 2, renorm=True, mask=mask)
    check(x, b, 3, score, G, TG, 1, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("K", [8, 12])
def test_neighbours_in_the_last_place(score, biased, K):
    """Logits one step of binary32 apart are told apart, with a bias too."""
    x = torch.full((9, 128), 0.7).numpy()
    steps = np.random.default_rng(3).permuted(np.tile(np.arange(128), (9, 1)), axis=1)
    x = (x.view(np.int32) + steps.astype(np.int32)).view(np.float32)
    check(torch.from_numpy(x), torch.full((128,), 0.25) if biased else None, K, score, renorm=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,K", [(64, 8), (256, 8), (96, 16)])
def test_masked_experts_and_special_values(score, renorm, E, K):
    inf, low = float("inf"), torch.finfo(torch.float32).min
    x = logits_of(12, E, torch.float32, seed=9)
    x[0] = -inf                                  # nothing to choose
    x[1, 3:] = -inf                              # three candidates
    x[2, ::2] = float("nan")
    x[3, 5] = inf
    x[4, [7, 9]] = inf                           # two infinities tie
    x[5] = low                                   # the lowest value: candidates like any other
    x[6, 4:] = low
    x[7, 0] = -inf
    x[7, 1] = float("nan")
    x[8] = -80.0
    x[9, :2] = torch.tensor([60.0, -60.0])
    x[10] = float("nan")
    x[11] = -0.0
    x[11, ::3] = 0.0                             # zeros of both signs tie
    b = torch.zeros(E)
    b[1], b[2], b[6] = -inf, float("nan"), 0.5
    check(x, None, K, score, renorm=renorm)
    check(x, b, K, score, renorm=renorm)
    if E == 256:
        check(x, None, K, score, 8, 2, 2, renorm=renorm)
        check(x, b, K, score, 8, 2, 1, renorm=renorm)


def test_logits_of_one_are_not_wide_rows():
    """Rows that start off a 16-byte boundary (an odd number of experts, or a
    tensor that starts inside another)."""
    base = logits_of(1, 41 * 101 + 1, torch.float32, seed=4)[0]
    x = base[1:].view(41, 101)
    dev = base.to(DEV)[1:].view(41, 101)
    idx, w = epl.route(dev, 4, renormalize=True)
    ri, _ = reference(x.numpy(), None, 4, "softmax", 1, 1, 1, True, 1.0, None)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)


# ------------------------------------------------------------- gradient --

def grad_reference(logits, idx, g, score, renorm, scale):
    x = np.minimum(logits.astype(np.float64), np.finfo(np.float32).max)
    x = np.where(x > -np.inf, x, -np.inf)
    T, E = x.shape
    K = idx.shape[1]
    live = (idx >= 0) & (idx < E)
    at = np.where(live, idx, 0)
    g = np.where(live, g.astype(np.float64), 0.0) * scale
    if score == "softmax":
        m = x.max(1, keepdims=True)
        if renorm:
            m = np.where(live, np.take_along_axis(x, at, 1), -np.inf).max(1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        with np.errstate(over="ignore"):
            p = np.where(x > -np.inf, np.exp(x - m), 0.0)
        if not renorm:
            s = p.sum(1, keepdims=True)
            p = np.divide(p, s, out=np.zeros_like(p), where=s > 0)
    else:
        p = np.where(x > -np.inf, 1 / (1 + np.exp(-np.maximum(x, -700))), 0.0)
    pk = np.where(live, np.take_along_axis(p, at, 1), 0.0)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    if renorm:
        D = pk.sum(1, keepdims=True)
        over = np.divide(1.0, D, out=np.zeros_like(D), where=D > 0)
        share = pk * over
        h = share * (g - (share * g).sum(1, keepdims=True))
        hm = share * (np.abs(g) + (share * np.abs(g)).sum(1, keepdims=True))
    else:
        h, hm = pk * g, pk * np.abs(g)
    if score == "sigmoid":
        tail = 1 / (1 + np.exp(np.maximum(np.minimum(np.take_along_axis(x, at, 1), 700), -700)))
        h, hm = h * tail, hm * tail
    for k in range(K):
        rows = np.flatnonzero(live[:, k])
        out[rows, at[rows, k]] += h[rows, k]
        mag[rows, at[rows, k]] += hm[rows, k]
    if score == "softmax" and not renorm:
        out -= p * h.sum(1, keepdims=True)
        mag += p * hm.sum(1, keepdims=True)
    return out, mag


def check_grad(x, idx, g, score, renorm, scale=1.0):
    T, E = x.shape
    dev = x.to(DEV)
    p = epl.Router(T, idx.shape[1], E, {"softmax": 0, "sigmoid": 1}[score], 1, 1, 1, int(renorm),
                   1 if x.dtype == torch.bfloat16 else 0, scale, 0)
    out = redzones.poisoned((T, E), x.dtype, 0x5A, DEV)
    epl.epl_route_backward(p, dev, idx.to(DEV), g.to(DEV), out)
    ref, mag = grad_reference(x.float().numpy(), idx.numpy(), g.numpy(), score, renorm, scale)
    got = out.cpu().double().numpy()
    finite = np.where(np.isfinite(x.float().numpy()), np.abs(x.float().numpy()), 0.0)
    big = np.minimum(finite, 30).max()
    tol = (4 * big + 64) * U * mag + 1e-37
    if x.dtype == torch.bfloat16:
        tol = tol + np.abs(ref) * 2.0 ** -8 + 2.0 ** -134     # the smallest bf16 step, halved
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) - tol).max()


def choice_of(T, E, K, seed, empty=0.1):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :K]
    return idx.masked_fill(torch.rand(T, K, generator=g) < empty, -1).contiguous(), \
        torch.randn(T, K, generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (65, 16, 2), (33, 60, 8), (40, 128, 7),
                                   (9, 250, 8), (300, 256, 8), (5, 512, 64), (3, 2048, 33),
                                   (4, 1001, 5)])
def test_gradient(T, E, K, score, renorm, dtype):
    x = logits_of(T, E, dtype, seed=E + K)
    idx, g = choice_of(T, E, K, seed=T)
    check_grad(x, idx, g, score, renorm, 2.5)


def test_empty_batches_and_refusals():
    for E in (16, 256):
        idx, w = epl.route(torch.zeros(0, E, device=DEV), 4)
        assert idx.shape == w.shape == (0, 4)
        assert epl.route_backward(torch.zeros(0, E, device=DEV), idx, w).shape == (0, E)
    x = torch.zeros(4, 32, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        epl.route(x[:, ::2], 2)
    with pytest.raises(ValueError, match="bias must have shape"):
        epl.route(x, 2, bias=torch.zeros(16, device=DEV))
    with pytest.raises(TypeError, match="token_mask"):
        epl.route(x, 2, token_mask=torch.ones(4, dtype=torch.bool, device=DEV))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        epl.route(x, 2, bias=torch.zeros(32))
    idx, w = epl.route(x, 2)
    with pytest.raises(ValueError, match="grad_weights"):
        epl.route_backward(x, idx, w[:2].contiguous())


def test_router_captured_and_on_another_stream():
    x = logits_of(4100, 256, torch.float32, seed=1).to(DEV)
    b = torch.linspace(-0.1, 0.1, 256, device=DEV)
    rules = dict(score="sigmoid", bias=b, num_groups=8, topk_groups=4, group_top=2,
                 renormalize=True, scale=2.5)
    g = torch.randn(4100, 8, device=DEV)

    def run():
        idx, w = epl.route(x, 8, **rules)
        return idx, w, epl.route_backward(x, idx, g, score="sigmoid", renormalize=True, scale=2.5)

    eager = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other = run()
    side.synchronize()
    for a, c in zip(other, eager):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for n in range(4):
        x.add_(0.25 * x.flip(1))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(kept, run()):
            assert torch.equal(a, c)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_odd_choices(score, renorm):
    """The same expert twice, empty tokens, ids out of range, NaN gradients in
    empty slots, unavailable logits."""
    x = logits_of(6, 64, torch.float32, seed=3)
    idx, g = choice_of(6, 64, 4, seed=2, empty=0.0)
    idx[0] = torch.tensor([5, 5, 7, 5])
    idx[1] = -1
    idx[2, 1], idx[2, 2] = 64, -9
    g[1] = float("nan")
    g[2, 1:3] = float("nan")
    x[3, :10] = -float("inf")
    idx[3, 0] = 2
    x[4, 60] = torch.finfo(torch.float32).min
    idx[5] = torch.tensor([-1, 3, -1, -1])
    check_grad(x, idx, g, score, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    """The definition's gradient is the slope of the definition's weights:
    central differences in 64 bits, with step h off by O(h^2) = 1e-8 and
    rounding 1e-16 / h = 1e-12."""
    x = logits_of(4, 24, torch.float32, seed=8).numpy().astype(np.float64)
    idx, _ = reference(x, None, 4, score, 1, 1, 1, renorm, 2.5, None)
    g = np.random.default_rng(0).standard_normal((4, 4))

    def loss(v):
        if score == "softmax":
            p = np.exp(v - v.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
        else:
            p = 1 / (1 + np.exp(-v))
        w = np.take_along_axis(p, idx, 1)
        w = w / w.sum(1, keepdims=True) if renorm else w
        return 2.5 * (w * g).sum()

    ref, _ = grad_reference(x, idx, g, score, renorm, 2.5)
    for t in range(4):
        for e in range(24):
            d = np.zeros_like(x)
            d[t, e] = 1e-4
            assert abs((loss(x + d) - loss(x - d)) / 2e-4 - ref[t, e]) < 1e-7
    check_grad(torch.from_numpy(x).float(), torch.from_numpy(idx), torch.from_numpy(g).float(),
               score, renorm, 2.5)
