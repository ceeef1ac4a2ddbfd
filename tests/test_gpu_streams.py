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
