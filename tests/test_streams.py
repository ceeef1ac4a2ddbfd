"""Calls with stream=: what they allocate and fill inside belongs to the stream
that they launch on, whatever the current one. On the host, against a stand-in
for torch's streams and for the library's entry points that only notes who
ordered what."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU, and which stream it came from."""
    is_cuda = True
    device = property(lambda t: torch.device("cuda:0"))

    def record_stream(self, s):
        self.kept = getattr(self, "kept", []) + [s]


class Pinned(torch.Tensor):
    def is_pinned(self):
        return True


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


class Streams:
    """Stands in for torch and for libepl: tensors remember the stream that was
    current when they were made, launches the raw stream they went to."""

    def __init__(self, lib):
        self.lib, self.made, self.launches = lib, [], []
        self.now = self.default = Stream(0)
        self.cuda, self._C = self, object()

    def __getattr__(self, name):
        return getattr(torch, name)

    # torch.cuda
    def current_device(self):
        return 0

    def current_stream(self, device=None):
        return self.now

    def ExternalStream(self, raw, device=None):
        return Stream(raw)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    # torch
    def _make(self, make, *args, device=None, pin_memory=False, **kw):
        t = make(*args, **kw)
        if pin_memory:
            return t.as_subclass(Pinned)
        t = t.as_subclass(OnGpu)
        t.owner = self.now
        self.made.append(t)
        return t

    def empty(self, *args, **kw):
        return self._make(torch.empty, *args, **kw)

    def ones(self, *args, **kw):
        return self._make(torch.ones, *args, **kw)

    def zeros(self, *args, **kw):
        return self._make(torch.zeros, *args, **kw)

    def empty_like(self, t):
        return self._make(torch.empty, t.shape, dtype=t.dtype)

    # libepl
    def entry(self, name):
        if name.endswith(("_validate", "_bytes", "_rows")) or name == "epl_strerror":
            return getattr(self.lib, name)

        def call(*args):
            self.launches.append((name, args[-1]))
            return 0
        return call


class Library:
    def __init__(self, streams):
        self.streams = streams

    def __getattr__(self, name):
        return self.streams.entry(name)


@pytest.fixture
def streams(monkeypatch):
    epl.ensure_built()
    s = Streams(epl.load())
    monkeypatch.setattr(epl, "_TORCH", s)
    monkeypatch.setattr(epl, "_LIB", Library(s))
    return s


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


T, K, E, H, F, ROWS = 6, 2, 4, 128, 32, 2048
BF16, I32 = torch.bfloat16, torch.int32


def _result():
    return epl.DispatchResult(gpu(ROWS, H, dtype=BF16), None, gpu(ROWS, dtype=I32), None, None, None,
                              None, None, None, None, gpu(1 << 20, dtype=torch.uint8),
                              epl.Problem.make(T, K, E, 2, H))


# sizes whose products split their contraction, so that they take a workspace
DEEP = 4096

CALLS = {
    "dispatch": lambda **kw: epl.dispatch(
        gpu(T, H, dtype=BF16), gpu(T, K, dtype=torch.int64), E, 2, **kw),
    "combine": lambda **kw: epl.combine(
        gpu(ROWS, H, dtype=BF16), gpu(T, K, dtype=I32), gpu(T, K), **kw),
    "expert_scale": lambda **kw: epl.expert_scale(_result(), **kw),
    "route": lambda **kw: epl.route(gpu(T, E), K, **kw),
    "route_backward": lambda **kw: epl.route_backward(
        gpu(T, E), gpu(T, K, dtype=torch.int64), gpu(T, K), **kw),
    "expert_product": lambda **kw: epl.expert_product(
        gpu(ROWS, DEEP, dtype=BF16), gpu(E, F, DEEP, dtype=BF16), gpu(E, dtype=I32),
        gpu(E, dtype=I32), **kw),
    "expert_weight_grad": lambda **kw: epl.expert_weight_grad(
        gpu(ROWS, F, dtype=BF16), gpu(ROWS, H, dtype=BF16), gpu(E, dtype=I32), gpu(E, dtype=I32),
        **kw),
    "combine_backward": lambda **kw: epl.combine_backward(
        gpu(T, H), gpu(ROWS, H, dtype=BF16), gpu(T, K, dtype=I32), gpu(T, K), **kw),
    "dispatch_backward": lambda **kw: epl.dispatch_backward(
        gpu(ROWS, H, dtype=BF16), gpu(T, K, dtype=I32), **kw),
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_what_a_call_makes_belongs_to_its_stream(streams, name, raw):
    out = CALLS[name](stream=0x77 if raw else Stream(0x77))
    assert streams.now is streams.default
    assert streams.launches and all(s == 0x77 for _, s in streams.launches), streams.launches
    assert streams.made and all(t.owner.cuda_stream == 0x77 for t in streams.made)
    # what the caller gets may be used, and dropped, on the stream it was on
    for t in out if isinstance(out, tuple) else (out,):
        if isinstance(t, OnGpu):
            assert streams.default in t.kept


@pytest.mark.parametrize("name", list(CALLS))
def test_without_a_stream_the_current_one(streams, name):
    with streams.stream(Stream(0x55)):
        CALLS[name]()
    assert streams.made and all(s == 0x55 for _, s in streams.launches)
    assert all(t.owner.cuda_stream == 0x55 for t in streams.made)


def test_products_here_take_a_workspace(streams):
    """(else the calls above would not show where it comes from)"""
    for name in ("expert_product", "expert_weight_grad"):
        CALLS[name]()
        assert any(t.dtype == torch.uint8 for t in streams.made)
        streams.made.clear()


class OnSecond(OnGpu):
    device = property(lambda t: torch.device("cuda:1"))


def test_dispatch_backward_off_the_current_gpu(streams, monkeypatch):
    """Kernels are launched on the current GPU: the tensors' has to be it."""
    at = [0]

    @contextlib.contextmanager
    def device(index):
        before, at[0] = at[0], index
        yield
        at[0] = before

    where = []
    inner = streams.entry

    def entry(name):
        call = inner(name)
        return lambda *args: (where.append((name, at[0])), call(*args))[1]

    monkeypatch.setattr(streams, "device", device, raising=False)
    monkeypatch.setattr(streams, "current_device", lambda: at[0])
    monkeypatch.setattr(streams, "entry", entry)
    monkeypatch.setattr(streams, "_make", lambda make, *args, device=None, **kw:
                        make(*args, **kw).as_subclass(OnSecond))
    epl.dispatch_backward(torch.zeros(ROWS, H, dtype=BF16).as_subclass(OnSecond),
                          torch.zeros(T, K, dtype=I32).as_subclass(OnSecond))
    assert ("epl_combine", 1) in where and at[0] == 0, where
