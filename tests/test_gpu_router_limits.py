"""The router and its gradient on the GPU where scores, biases or logits lie at
the limits of their types, against their definitions in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

import redzones  # noqa: E402
import test_gpu_router as router  # noqa: E402

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


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


def group_scores(s, G):
    """Sums of two of [T, E] sigmoids, to 40 bits, and whether a rounding of
    the sum in 64 bits (some 2^-52 of it) cannot change that."""
    sums = np.sort(s.reshape(len(s), G, -1), axis=2)[:, :, -2:].sum(2)
    part, power = np.frexp(sums)
    scaled = part * 2.0 ** 40
    clear = np.abs(scaled - np.floor(scaled) - 0.5) > 2.0 ** -8
    return np.ldexp(np.round(scaled) * 2.0 ** -40, power), clear.all(1)


@pytest.mark.parametrize("E,G,TG,K", [
    (64, 8, 1, 8), (64, 8, 4, 8), (128, 8, 4, 8), (32, 8, 3, 4), (64, 8, 4, 32), (256, 8, 3, 48),
    (60, 12, 5, 25)])
@pytest.mark.parametrize("T", [300, 4500])
def test_saturated_groups(T, E, G, TG, K):
    """Sigmoids next to 1, whose sums over groups lie close together: exactly
    TG groups stay, those of the largest sums, ties to the lower one."""
    x = torch.empty(T, E).uniform_(24, 28, generator=torch.Generator().manual_seed(E + TG))
    idx, _ = epl.route(x.to(DEV), K, score="sigmoid", num_groups=G, topk_groups=TG, group_top=2,
                       renormalize=True)
    idx = idx.cpu().numpy()
    assert (idx >= 0).all()
    assert (np.diff(np.sort(idx, axis=1), axis=1) > 0).all()
    size = E // G
    scores, clear = group_scores(sigmoid(x.numpy()), G)
    assert clear.mean() > 0.8
    stay = np.sort(np.argsort(-scores, axis=1, kind="stable")[:, :TG], axis=1)
    for t in np.flatnonzero(clear):
        assert np.isin(idx[t] // size, stay[t]).all(), t
        if K == TG * size:
            np.testing.assert_array_equal(np.unique(idx[t] // size), stay[t])


@pytest.mark.parametrize("T", [1, 5000])
def test_a_chain_of_near_groups(T):
    """Each group's score within 2^-38 of the next one's, the ends further apart."""
    x = torch.tensor([25.55, 26.02, 26.94]).repeat_interleave(8).repeat(T, 1)
    for order, best in (([0, 1, 2], 2), ([2, 1, 0], 0), ([1, 2, 0], 1)):
        v = x.view(T, 3, 8)[:, order].reshape(T, 24).contiguous().to(DEV)
        idx, w = epl.route(v, 8, score="sigmoid", num_groups=3, topk_groups=1, group_top=2,
                           renormalize=True)
        assert torch.equal(idx.cpu(), torch.arange(best * 8, best * 8 + 8).expand(T, 8))
        assert ((w - 0.125).abs() <= 2 * U * 0.125).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [64, 256])
@pytest.mark.parametrize("B", [16.0, 50.0, 200.0, 1000.0])
def test_groups_of_cancelling_biases(B, E, score):
    """A group's two best lie B above and B below the rest: their scores round
    by steps of B in binary32, which their small sum does not show."""
    T, G = 4500, 8
    g = torch.Generator().manual_seed(int(B) + E)
    x = torch.full((T, G, E // G), -float("inf"))
    x[:, :, :2] = torch.randn(T, 1, 1, generator=g) + 3e-5 * torch.randn(T, G, 2, generator=g)
    b = torch.zeros(G, E // G)
    b[:, 0], b[:, 1] = B, -B
    idx, _ = epl.route(x.view(T, E).to(DEV), 2, score=score, bias=b.view(E).to(DEV), num_groups=G,
                       topk_groups=1, group_top=2)
    s = x[:, :, :2].double()
    p = torch.sigmoid(s) if score == "sigmoid" else torch.softmax(s.view(T, -1), 1).view(T, G, 2)
    at = p.sum(2).argmax(1) * (E // G)
    assert torch.equal(idx.cpu(), torch.stack([at, at + 1], 1))


def test_groups_of_the_smallest_logits():
    """Denormal logits one step apart order the groups, empty groups last."""
    step = 2.0 ** -149
    x = torch.full((4, 64), -float("inf"))
    x[0, ::8] = step * torch.tensor([3.0, 1, 2, 4, 0, 5, 7, 6])
    x[1, ::8] = step * torch.tensor([-3.0, -1, -2, -4, 0, -5, -7, -6])
    x[2, 8:16] = -step
    idx, _ = epl.route(x.to(DEV), 2, score="sigmoid", num_groups=8, topk_groups=2, renormalize=True)
    assert idx.tolist() == [[48, 56], [32, 8], [8, 9], [-1, -1]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [1, 2, 8])
@pytest.mark.parametrize("base", [-87.0, -100.0, -300.0, -600.0, 0.0, 60.0])
def test_gradient_of_far_sigmoids(base, K, dtype):
    """Chosen logits far below zero: their sigmoids leave binary32, the ratios
    of renormalised ones do not. The chosen lie within 30 of each other, so the
    exponentials' (2 |x| + 4) u of them and of their sum stay below the 184 u
    that check_grad allows at these sizes."""
    E, T = 64, 200
    g = torch.Generator().manual_seed(K)
    x = (base + 30 * torch.rand(T, E, generator=g) - 15).to(dtype)
    idx, grad = router.choice_of(T, E, K, seed=K)
    router.check_grad(x, idx, grad * 20, "sigmoid", True, 2.5)
    assert not (router.grad_reference(x.float().numpy(), idx.numpy(), grad.numpy() * 20, "sigmoid",
                                      True, 2.5)[0] == 0).all() or base == 60 or K == 1


def test_sigmoids_that_are_zero():
    """Below -700 a sigmoid counts as 0: so do weights of nothing else, and
    their gradients."""
    x = torch.full((3, 64), -2000.0)
    x[1] = torch.finfo(torch.float32).min
    x[2, 5] = -690.0
    idx, w = epl.route(x.to(DEV), 4, score="sigmoid", renormalize=True)
    assert (w[:2] == 0).all() and w[2].tolist() == [1, 0, 0, 0] and idx[2, 0] == 5
    g = torch.randn(3, 4, generator=torch.Generator().manual_seed(0)).to(DEV)
    dx = epl.route_backward(x.to(DEV), idx, g, score="sigmoid", renormalize=True)
    assert (dx[:2] == 0).all() and (dx[2].abs() <= 4 * U * g[2, 0].abs()).all()


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T", [100, 5000])
@pytest.mark.parametrize("E", [128, 256, 512])
def test_softmax_weights_are_rounded_once(E, T, biased):
    """Weights of a softmax over all experts. Their rounding is off by u at
    most, u / sqrt 3 as a root mean square; the row's sum, of exponentials each
    good to about a step, whose errors average out over some hundred equal
    terms, may add 0.45 u to that: 0.75 u together."""
    g = torch.Generator().manual_seed(E)
    x = torch.rand(T, E, generator=g) - 0.5
    b = torch.linspace(-0.2, 0.2, E) if biased else None
    idx, w = epl.route(x.to(DEV), 8, bias=None if b is None else b.to(DEV))
    ref = torch.softmax(x.double(), 1).gather(1, idx.cpu())
    off = (w.cpu().double() - ref) / ref
    assert off.square().mean().sqrt() < 0.75 * U, float(off.square().mean().sqrt() / U)
