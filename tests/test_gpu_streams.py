"""Calls with stream= on a stream of their own, while the current stream is
still busy, against the same calls on the current stream."""
import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    epl.load()


def busy(n=60):
    """Some milliseconds of work on the current stream."""
    a = torch.randn(4096, 4096, device=DEV, dtype=torch.bfloat16)
    for _ in range(n):
        a = a @ a
    return a


def beside(call):
    """call(stream=) on a side stream behind a busy current one, and its result."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    work = busy()
    out = call(stream=side)
    side.synchronize()
    early = not torch.cuda.current_stream().query()
    out = [t.clone() for t in (out if isinstance(out, tuple) else (out,))]
    torch.cuda.synchronize()
    del work
    return early, out


def test_dispatch_backward_beside_the_current_stream():
    T, K, H = 300, 4, 256
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(T * K, H, generator=g).bfloat16().to(DEV)
    at = torch.randperm(T * K, generator=g).int().view(T, K).to(DEV)
    want = rows.float()[at.long()].sum(1)
    beside_it = []
    for _ in range(3):
        early, (dx,) = beside(lambda stream: epl.dispatch_backward(rows, at, stream=stream))
        beside_it.append(early)
        assert (dx - want).abs().max() <= 4 * 2.0 ** -23 * rows.float()[at.long()].abs().sum(1).max()
    assert any(beside_it)                  # it did not wait for the current stream
    assert torch.equal(dx, epl.dispatch_backward(rows, at))


def test_split_products_back_to_back_on_two_streams():
    """A product on the current stream frees its workspace while its kernels
    are pending; one on a named stream, started at once, takes another."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(300, 8192, generator=g).bfloat16().to(DEV)
    w = (torch.randn(1, 256, 8192, generator=g) / 90).bfloat16().to(DEV)
    d = torch.randn(300, 256, generator=g).bfloat16().to(DEV)
    start = torch.zeros(1, dtype=torch.int32, device=DEV)
    count = torch.full((1,), 300, dtype=torch.int32, device=DEV)
    product = lambda **kw: epl.expert_product(x, w, start, count, activation="silu",  # noqa: E731
                                              out_dtype=torch.float32, **kw)
    grad = lambda **kw: epl.expert_weight_grad(d, x, start, count,  # noqa: E731
                                               out_dtype=torch.float32, **kw)
    want, want_grad = product(), grad()
    p = epl.Product(300, 0, 1, 8192, 256, 0, 1, 0, 0)
    assert epl.epl_product_workspace_bytes(p) > 0
    side = torch.cuda.Stream()
    for _ in range(10):
        torch.cuda.synchronize()
        work = busy(4)
        outs = [product(), product(stream=side), grad(), grad(stream=side.cuda_stream), product(),
                product(stream=side)]
        torch.cuda.synchronize()
        del work
        for n, out in enumerate(outs):
            assert torch.equal(out, want_grad if n in (2, 3) else want), n


def test_layer_on_a_stream_beside_the_current_one():
    """Routing, dispatch, product, combine and their gradients, each with
    stream=, behind a busy current stream."""
    T, E, K, H, F = 400, 16, 4, 256, 64
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(T, E, generator=g).to(DEV)
    x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    w = (torch.randn(E, 2 * F, H, generator=g) / 16).bfloat16().to(DEV)
    w2 = (torch.randn(E, H, F, generator=g) / 8).bfloat16().to(DEV)
    dy = torch.randn(T, H, generator=g).to(DEV)

    def layer(stream=None):
        kw = dict(stream=stream)
        idx, wt = epl.route(logits, K, renormalize=True, **kw)
        r = epl.dispatch(x, idx, E, 4, **kw)
        at = (r.expert_start_loc, r.num_tokens_per_expert)
        h = epl.expert_product(r.out, w, *at, activation="swiglu", **kw)
        v = epl.expert_product(h, w2, *at, **kw)
        y = epl.combine(v, r.output_index, wt, **kw)
        dv, dw = epl.combine_backward(dy, v, r.output_index, wt, **kw)
        dw2 = epl.expert_weight_grad(dv, h, *at, **kw)
        dx = epl.dispatch_backward(dv, r.output_index, **kw)
        return idx, wt, y, dw, dw2, dx, epl.route_backward(logits, idx, dw, renormalize=True, **kw)

    want = layer()
    for _ in range(3):
        _, got = beside(layer)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_the_null_stream_by_its_address():
    x = torch.randn(64, 32, device=DEV)
    torch.cuda.synchronize()
    idx, w = epl.route(x, 4, stream=0)
    torch.cuda.synchronize()
    for a, b in zip((idx, w), epl.route(x, 4)):
        assert torch.equal(a, b)
