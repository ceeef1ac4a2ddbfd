"""The experts' products, their weight gradients and the combine's gradient on
the GPU against their definitions in 64 bits.

Tolerances. A product sums K exact products in binary32: whatever the order,
each of its at most K additions is off by at most one step of the running sum
(2^-23, a full step, so that an adder that truncates is covered too), so |z -
z64| <= K 2^-23 B with B = sum |x||w| (+ |bias|). An activation passes that on
times its steepest slope (1.13 for the smooth ones) and adds its own error,
32 u of the larger of |z|, 1 (u = 2^-24; exp's argument is below 40 wherever
the result is not flat). The output's rounding adds half a step of its type.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

import redzones  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
ACTS = {"none": 0, "silu": 1, "gelu": 2, "swiglu": 3, "silu_grad": 4, "gelu_grad": 5,
        "swiglu_grad": 6}
SLOPE = 1.13


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    epl.load()


@pytest.fixture(autouse=True)
def _red_zones():
    yield
    redzones.check()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def randn(*shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).mul_(std).bfloat16()


def silu(z):
    return z * torch.sigmoid(z)


def silu_slope(z):
    p = torch.sigmoid(z)
    return p + z * p * torch.sigmoid(-z)


def gelu(z):
    return 0.5 * z * torch.erfc(-z / math.sqrt(2))


def gelu_slope(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2)) + \
        z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def blocks(counts, gap=0):
    """Starts of blocks with `gap` unowned rows after each, and the rows' count."""
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += c + gap
    return starts, at


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def filled(shape, dtype, seed):
    """An output buffer between red zones that holds known values."""
    t = redzones.poisoned(shape, dtype, 0x5A, DEV)
    t.copy_(torch.randn(shape, generator=torch.Generator().manual_seed(seed)))
    return t


def workspace(nbytes):
    return redzones.poisoned(nbytes, torch.uint8, 0x5A, DEV) if nbytes else None


def check_product(counts, K, N, act="none", bias=False, residual=False, pre=False,
                  transposed=False, out=torch.bfloat16, gap=0, expected=0, seed=0, rows=None,
                  starts=None, in_place=False, split=True):
    E = len(counts)
    made, total = blocks(counts, gap)
    starts = made if starts is None else starts
    total = total if rows is None else rows
    grad = act.endswith("_grad")
    cols = N // 2 if act == "swiglu" else 2 * N if act == "swiglu_grad" else N
    x = randn(total, K, seed=seed)
    w = randn(E, K, N, seed=seed + 1, std=K ** -0.5) if transposed else \
        randn(E, N, K, seed=seed + 1, std=K ** -0.5)
    b = torch.randn(E, N, generator=torch.Generator().manual_seed(seed + 2)) if bias else None
    res = randn(total, cols, seed=seed + 3) if residual else None
    saved = randn(total, cols, seed=seed + 4, std=2.0) if grad else None
    owned = torch.zeros(total, dtype=torch.bool)
    for s, c in zip(starts, counts):
        owned[max(s, 0):max(min(s + c, total), 0)] = True
    x[~owned] = float("nan")                    # rows of no expert are not read
    y = filled((total, cols), out, seed + 5)
    if in_place:
        y.copy_(res)
    before = y.cpu().clone()
    z_out = None
    if grad:
        z_out = saved.to(DEV)
    elif pre:
        z_out = filled((total, N), torch.bfloat16, seed + 6)
    z_before = None if z_out is None else z_out.cpu().clone()
    p = epl.Product(total, expected, E, K, N, int(transposed), ACTS[act],
                    1 if out == torch.bfloat16 else 0, 0)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    epl.epl_expert_product(p, d(x), d(w), d(b), y if in_place else d(res), i32(starts),
                           i32(counts), z_out, y, workspace(epl.epl_product_workspace_bytes(p)) if split else None)
    got = y.cpu()
    assert torch.equal(got[~owned].view(torch.int16 if out == torch.bfloat16 else torch.int32),
                       before[~owned].view(torch.int16 if out == torch.bfloat16 else torch.int32))
    z_got = None if z_out is None else z_out.cpu()
    if grad:
        assert torch.equal(z_got, saved)
    for e in range(E):
        lo, hi = max(starts[e], 0), max(min(starts[e] + counts[e], total), 0)
        if hi <= lo:
            continue
        xe, we = x[lo:hi].double(), w[e].double()
        we = we if transposed else we.t()
        z, B = xe @ we, xe.abs() @ we.abs()
        if bias:
            z, B = z + b[e].double(), B + b[e].abs().double()
        err = K * 2 * U * B
        if pre and not grad:
            tol = err + half_step(torch.bfloat16) * (z.abs() + err)
            assert ((z_got[lo:hi].double() - z).abs() <= tol).all()
        own = lambda v: 32 * U * v.abs().clamp(min=1)  # noqa: E731
        if act == "none":
            ref, tol = z, err
        elif act == "silu":
            ref, tol = silu(z), SLOPE * err + own(z)
        elif act == "gelu":
            ref, tol = gelu(z), SLOPE * err + own(z)
        elif act == "swiglu":
            (g, u), (eg, eu) = z.chunk(2, 1), err.chunk(2, 1)
            ref = silu(g) * u
            tol = (SLOPE * eg + own(g)) * (u.abs() + eu) + silu(g).abs() * eu + 2 * U * ref.abs()
        elif act == "swiglu_grad":
            g, u = saved[lo:hi].double().chunk(2, 1)
            ref = torch.cat([z * u * silu_slope(g), z * silu(g)], 1)
            tol = torch.cat([err * u.abs() * SLOPE + 40 * U * (z * u).abs() * g.abs().clamp(min=1),
                             err * silu(g).abs() + z.abs() * own(g)], 1)
        else:
            s = saved[lo:hi].double()
            slope = silu_slope(s) if act == "silu_grad" else gelu_slope(s)
            ref = z * slope
            tol = err * SLOPE + 40 * U * z.abs() * s.abs().clamp(min=1)
        if residual:
            ref = ref + res[lo:hi].double()
            tol = tol + 2 * U * (ref.abs() + res[lo:hi].abs())
        tol = tol + half_step(out) * (ref.abs() + tol) + 1e-37
        diff = (got[lo:hi].double() - ref).abs()
        assert (diff <= tol).all(), (e, float((diff - tol).max()), torch.nonzero(diff > tol)[:4])
    return y


# Blocks around the edges of pieces (16), tiles (128, 256) and their kernels,
# which follow the rows expected for an expert.
FEW = [0, 1, 15, 16, 17, 33, 64, 65, 3]
MANY = [0, 1, 127, 128, 129, 255, 256, 257, 300]
SIZES = [(8, 8), (64, 16), (72, 264), (200, 256), (520, 48), (1024, 528)]


@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("expected", [9, 9 * 100, 0])
def test_forward_sizes(K, N, expected):
    counts = FEW if expected == 9 else MANY
    if expected == 0:
        counts = MANY + [700] * 3          # about 250 rows an expert
    check_product(counts, K, N, expected=expected, seed=K)


@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("expected", [9, 0])
def test_transposed_sizes(K, N, expected):
    counts = FEW if expected else MANY + [700] * 3
    check_product(counts, K, N, transposed=True, expected=expected, seed=K + 1)


# Sums split over workgroups and joined: one tile to several rounds and a few
# tiles left, odd numbers of stages, parts of different length, tiles without
# rows; and the same without a workspace.
@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,K,N,act", [
    ([300], 4096, 256, "none"), ([129], 2056, 128, "swiglu"), ([70, 0, 300, 200], 1288, 520, "gelu"),
    ([256] * 3, 520, 1024, "silu"), ([140] * 40, 1032, 1808, "none"),
    ([5000], 1160, 3600, "swiglu_grad"), ([100, 90], 8200, 64, "silu_grad")])
def test_split_contraction(counts, K, N, act, transposed, split):
    grad = act.endswith("_grad")
    check_product(counts, K, N, act, transposed=transposed, bias=not grad, residual=not grad,
                  pre=True, seed=11, split=split)


@pytest.mark.parametrize("counts,N,K,accumulate", [
    ([4000], 64, 72, False), ([3000, 0, 1500], 272, 520, True), ([700, 900], 1040, 264, False),
    ([20000], 512, 128, True), ([513] * 12, 528, 1032, False)])
def test_split_rows(counts, N, K, accumulate):
    check_weight_grad(counts, N, K, accumulate=accumulate, seed=5)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,K,act", [
    ([300, 10, 260, 700, 257] * 4, 136, "silu"),
    ([512, 400, 511, 512] * 4 + [500], 1032, "gelu"),  # 272 tiles of 256 x 256, 16 of them split
    ([100, 30, 128, 129, 0] * 8, 72, "swiglu"),        # 640 of 128 x 128
])
def test_products_of_many_tiles(counts, K, act, transposed):
    """Workgroups that make several tiles, one after the other."""
    check_product(counts, K, 2048, act=act, bias=True, residual=True, pre=True,
                  transposed=transposed, seed=K)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("expected", [4, 4 * 100, 0])
@pytest.mark.parametrize("act", list(ACTS))
def test_epilogues(act, expected, transposed, out):
    counts = [5, 0, 50, 20] if expected == 4 else [300, 0, 129, 400]
    grad = act.endswith("_grad")
    for extra in ({},) if grad else ({}, dict(bias=True, residual=True, pre=True)):
        check_product(counts, 136, 288, act, transposed=transposed, out=out, expected=expected,
                      seed=7, **extra)


@pytest.mark.parametrize("expected", [3, 0])
def test_rows_of_no_expert_stay(expected):
    """Padding between blocks, capacity behind the last, an empty layer."""
    check_product([40, 0, 17], 64, 32, "swiglu", pre=True, gap=13, expected=expected)
    check_product([300, 0, 170], 64, 32, "gelu", bias=True, gap=13, rows=900, expected=expected)
    check_product([0, 0], 64, 32, rows=10, expected=expected)


@pytest.mark.parametrize("expected", [3, 0])
def test_blocks_are_cut_to_the_buffer(expected):
    """Counts beyond the buffer (slots that found no room), blocks outside it."""
    check_product([30, 50, 10], 64, 32, rows=60, expected=expected)
    check_product([300, 500, 10], 64, 32, rows=600, expected=expected, starts=[0, 300, 800])
    check_product([20, -5, 7], 64, 32, rows=40, starts=[-8, 20, 35], expected=expected)
    check_product([20, 2 ** 31 - 1], 64, 32, rows=40, starts=[0, 20], expected=expected)


def test_rectangle_of_equal_blocks():
    """The low-latency layout: expert e's rows from e * cap on."""
    check_product([3, 0, 128, 60], 128, 64, "silu", rows=512, starts=[0, 128, 256, 384],
                  expected=191)


def test_residual_in_place():
    check_product([40, 90], 64, 40, "silu", residual=True, in_place=True, expected=2)
    check_product([300, 290], 64, 40, "silu", residual=True, in_place=True)


def test_many_experts():
    g = np.random.default_rng(0)
    check_product([int(v) for v in g.integers(0, 4, 2048)], 16, 16, expected=3000)
    check_product([int(v) for v in g.integers(0, 4, 2048)], 16, 16, transposed=True)
    check_product([int(v) for v in g.integers(0, 90, 257)], 24, 16, expected=257 * 100)


def test_one_row():
    check_product([0, 1, 0], 4096, 512, "swiglu", expected=1)
    check_product([1], 2048, 8)


@pytest.mark.parametrize("expected", [2, 0])
def test_special_values_stay_in_their_rows(expected):
    """A row with NaN or infinity leaves the others alone; saturated gates."""
    K, N = 64, 32
    counts, total = [200, 210], 410
    x, w = randn(total, K, seed=1), randn(2, N, K, seed=2, std=0.125)
    clean = epl.expert_product(x.to(DEV), w.to(DEV), i32([0, 200]), i32(counts),
                               activation="silu", expected_rows=expected)
    bad = x.clone()
    bad[3] = float("nan")
    bad[205, 5] = float("inf")
    y = epl.expert_product(bad.to(DEV), w.to(DEV), i32([0, 200]), i32(counts), activation="silu",
                           expected_rows=expected)
    keep = [r for r in range(total) if r not in (3, 205)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[205]).all()
    # z = +-inf: silu is inf and 0, gelu likewise, slopes 1 and 0
    one = torch.zeros(1, 8).bfloat16()
    one[0, 0] = 1.0
    wt = torch.zeros(1, 8, 8).bfloat16()
    wt[0, 0, 0], wt[0, 1, 0], wt[0, 2, 0] = float("inf"), -float("inf"), 3e38
    for act in ("silu", "gelu"):
        v = epl.expert_product(one.to(DEV), wt.to(DEV), i32([0]), i32([1]), activation=act,
                               expected_rows=expected)
        assert v[0, 0] == float("inf") and v[0, 1] == 0 and v[0, 2] > 2.9e38
    far = torch.tensor([[float("inf"), -float("inf"), 1e30, -1e30, 200.0, -200.0, 0.0, 20.0]])
    wt = torch.ones(1, 8, 8).bfloat16()
    for act in ("silu_grad", "gelu_grad"):
        v = epl.expert_product(one.to(DEV), wt.to(DEV), i32([0]), i32([1]), activation=act,
                               pre=far.bfloat16().to(DEV))
        assert v[0].tolist() == [1, 0, 1, 0, 1, 0, 0.5, 1]


def test_repeats_bit_for_bit_and_streams():
    """Twice the same bits; on a stream of its own; two streams at once."""
    x, w = randn(900, 256, seed=1).to(DEV), randn(3, 512, 256, seed=2, std=0.06).to(DEV)
    start, count = i32([0, 300, 600]), i32([300, 290, 300])
    run = lambda **kw: epl.expert_product(x, w, start, count, activation="swiglu",  # noqa: E731
                                          out=torch.zeros(900, 256, device=DEV), **kw)
    a, b = run(), run()
    few = run(expected_rows=3)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        c = run()
    with torch.cuda.stream(s2):
        d = run(expected_rows=3)
    dw = epl.expert_weight_grad(x[:, :64].contiguous(), x, start, count, out_dtype=torch.float32)
    dw2 = epl.expert_weight_grad(x[:, :64].contiguous(), x, start, count,
                                 out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(few, d)
    assert torch.equal(dw, dw2)


def test_split_products_on_two_streams_and_in_a_graph():
    """Calls that split their sums, each with a workspace of its own: at once
    on two streams, and captured, replayed against the eager result."""
    x, w = randn(300, 4096, seed=1).to(DEV), randn(1, 256, 4096, seed=2, std=0.02).to(DEV)
    g = randn(300, 256, seed=3).to(DEV)
    start, count = i32([0]), i32([300])

    def run():
        y = epl.expert_product(x, w, start, count, activation="silu", out_dtype=torch.float32)
        dx = epl.expert_product(g, w, start, count, transposed=True)
        return y, dx, epl.expert_weight_grad(g, x, start, count, out_dtype=torch.float32)

    eager = run()
    p = epl.Product(300, 0, 1, 4096, 256, 0, 1, 0, 0)
    assert epl.epl_product_workspace_bytes(p) > 0
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for s in streams * 3:
        with torch.cuda.stream(s):
            outs.append(run())
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
    # a stream named in the call
    y = epl.expert_product(x, w, start, count, activation="silu", out_dtype=torch.float32,
                           stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(y, eager[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for n in range(4):
        for t in kept:
            t.zero_()
        keep = x.clone()
        x.mul_(2.0 if n % 2 else 1.0)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)
        x.copy_(keep)


def test_workspace_is_checked():
    x, w = randn(300, 4096, seed=1).to(DEV), randn(1, 256, 4096, seed=2).to(DEV)
    p = epl.Product(300, 0, 1, 4096, 256, 0, 0, 1, 0)
    y = torch.zeros(300, 256, dtype=torch.bfloat16, device=DEV)
    need = epl.epl_product_workspace_bytes(p)
    small = torch.zeros(need - 256, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="workspace holds"):
        epl.epl_expert_product(p, x, w, None, None, i32([0]), i32([300]), None, y, small)
    odd = torch.zeros(need + 16, dtype=torch.uint8, device=DEV)[16:]
    with pytest.raises(epl.EplError):
        epl.epl_expert_product(p, x, w, None, None, i32([0]), i32([300]), None, y, odd)
    with pytest.raises(ValueError, match="contiguous"):
        epl.expert_product(x[:, ::2], w[:, :, ::2].contiguous(), i32([0]), i32([300]))
    with pytest.raises(TypeError, match="num_tokens_per_expert"):
        epl.expert_product(x, w, i32([0]), i32([300]).long())
    with pytest.raises(epl.EplError):                 # x off a 16-byte boundary
        flat = torch.zeros(300 * 4096 + 4, dtype=torch.bfloat16, device=DEV)
        epl.expert_product(flat[4:].view(300, 4096), w, i32([0]), i32([300]))


# ------------------------------------------------------- weight gradient --

def check_weight_grad(counts, N, K, out=torch.float32, bias=True, accumulate=False, gap=0, rows=None,
                      starts=None, seed=0):
    E = len(counts)
    made, total = blocks(counts, gap)
    starts = made if starts is None else starts
    total = total if rows is None else rows
    d, x = randn(total, N, seed=seed), randn(total, K, seed=seed + 1)
    owned = torch.zeros(total, dtype=torch.bool)
    for s, c in zip(starts, counts):
        owned[max(s, 0):max(min(s + c, total), 0)] = True
    d[~owned] = float("nan")
    x[~owned] = float("nan")
    dw = filled((E, N, K), out, seed + 2)
    db = filled((E, N), torch.float32, seed + 3) if bias else None
    w0, b0 = dw.cpu().double(), None if db is None else db.cpu().double()
    p = epl.Product(total, 0, E, K, N, 0, 0, 1 if out == torch.bfloat16 else 0, 0)
    epl.epl_expert_weight_grad(p, d.to(DEV), x.to(DEV), i32(starts), i32(counts), accumulate, dw,
                               db, workspace(epl.epl_weight_grad_workspace_bytes(p)))
    for e in range(E):
        lo, hi = max(starts[e], 0), max(min(starts[e] + counts[e], total), 0)
        hi = max(hi, lo)
        de, xe = d[lo:hi].double(), x[lo:hi].double()
        ref, B = de.t() @ xe, de.abs().t() @ xe.abs()
        if accumulate:
            ref, B = ref + w0[e], B + w0[e].abs()
        tol = (hi - lo + 1) * 2 * U * B
        tol = tol + half_step(out) * (ref.abs() + tol)
        diff = (dw[e].cpu().double() - ref).abs()
        assert (diff <= tol).all(), (e, float((diff - tol).max()), torch.nonzero(diff > tol)[:4])
        if bias:
            ref, B = de.sum(0), de.abs().sum(0)
            if accumulate:
                ref, B = ref + b0[e], B + b0[e].abs()
            assert ((db[e].cpu().double() - ref).abs() <= (hi - lo + 1) * U * B).all()


@pytest.mark.parametrize("N,K", [(8, 8), (16, 264), (264, 72), (256, 512), (520, 40)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_grad(N, K, out, accumulate):
    check_weight_grad([0, 1, 63, 64, 65, 130, 300], N, K, out, accumulate=accumulate, seed=N)


@pytest.mark.parametrize("counts,N,K", [
    ([100, 40, 0, 130, 64], 2048, 4096),
    ([100, 40, 0, 130], 2048, 4096),             # 512 tiles of 256 x 256
    ([20, 70] * 20, 384, 1024),                  # 960 of 128 x 128
])
def test_weight_grad_of_many_tiles(counts, N, K):
    """Workgroups that make several tiles, one after the other."""
    check_weight_grad(counts, N, K, out=torch.bfloat16, seed=K)


def test_weight_grad_blocks():
    check_weight_grad([20, 0, 33], 32, 64, gap=11)
    check_weight_grad([300, 500, 10], 32, 64, rows=600, starts=[0, 300, 800])
    check_weight_grad([20, -5, 7], 32, 64, rows=40, starts=[-8, 20, 35], bias=False)
    check_weight_grad([0, 0], 32, 64, rows=5)
    check_weight_grad([2] * 300, 16, 24)


def test_weight_grad_of_nothing():
    """No rows at all: zeros, or what was there."""
    empty = torch.zeros(0, 16, dtype=torch.bfloat16, device=DEV)
    out = torch.ones(2, 16, 16, device=DEV)
    epl.expert_weight_grad(empty, empty, i32([0, 0]), i32([0, 0]), out=out, accumulate=True)
    assert (out == 1).all()
    epl.expert_weight_grad(empty, empty, i32([0, 0]), i32([0, 0]), out=out)
    assert (out == 0).all()


# ------------------------------------------------------ combine gradient --

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (1, 8, 7168), (64, 2, 128), (33, 7, 1032),
                                   (5, 64, 520), (300, 9, 2056), (17, 3, 1024)])
def test_combine_backward(T, K, H, dtype):
    g = torch.Generator().manual_seed(T + H)
    rows = T * K + 5
    place = torch.randperm(rows, generator=g)[:T * K].int().view(T, K)
    place = place.masked_fill(torch.rand(T, K, generator=g) < 0.2, -1)
    if T > 1:
        place[1] = -1
    w = torch.randn(T, K, generator=g)
    w[place < 0] = float("nan")                       # not used
    v = randn(rows, H, seed=1)
    dy = torch.randn(T, H, generator=g).to(dtype)
    dv = filled((rows, H), torch.bfloat16, 3)
    dw = redzones.poisoned((T, K), torch.float32, 0x5A, DEV)
    before = dv.cpu().clone()
    p = epl.Problem.make(T, K, 1, 1, H)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    epl.epl_combine_backward(p, dy.to(DEV), v.to(DEV), rows, place.to(DEV), w.to(DEV), dv, dw, ws)
    assert epl.epl_status(ws) == epl.EPL_OK
    t, k = torch.nonzero(place >= 0, as_tuple=True)
    at = place[t, k].long()
    want = before.clone()
    want[at] = (w[t, k][:, None] * dy[t].float()).bfloat16()     # one product, one rounding
    assert torch.equal(dv.cpu().view(torch.int16), want.view(torch.int16))
    ref, mag = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    prod = v[at].double() * dy[t].double()
    ref[t, k], mag[t, k] = prod.sum(1), prod.abs().sum(1)
    assert ((dw.cpu().double() - ref).abs() <= H * U * mag).all()


def test_combine_backward_flags_rows_beyond_the_buffer():
    place = torch.tensor([[0, 9], [3, -4]], dtype=torch.int32, device=DEV)
    v = torch.ones(4, 16, dtype=torch.bfloat16, device=DEV)
    dv = filled((4, 16), torch.bfloat16, 1)
    before = dv.clone()
    dy = torch.full((2, 16), 2.0, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    _, dw = epl.combine_backward(dy, v, place, torch.ones(2, 2, device=DEV), dv, ws)
    assert epl.epl_status(ws) == epl.EPL_ERANGE
    assert dw.tolist() == [[32, 0], [32, 0]]
    assert (dv[[0, 3]] == 2).all() and torch.equal(dv[1:3], before[1:3])


def test_gradients_against_differences():
    """The definitions' gradients are slopes: central differences in 64 bits
    of silu, gelu and the gated product."""
    z = torch.linspace(-6, 6, 25, dtype=torch.float64)
    h = 1e-5
    for f, df in ((silu, silu_slope), (gelu, gelu_slope)):
        assert ((f(z + h) - f(z - h)) / (2 * h) - df(z)).abs().max() < 1e-8
