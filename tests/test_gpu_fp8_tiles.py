"""The tile kernels of the products on 8-bit rows, at sizes that reach every one of
them: large (256 x 256) and small (128 x 128) tiles, both weight layouts, with and
without the cast of the result, in one round and in several, with last rounds whole
and shared by workgroups.

Codes are 0, +-1 and +-2 and scales powers of two within 2^2 of each other, so that
every sum is a whole number below 2^24 times one power of two: z is exact in
binary32 in any order, and results without an activation have to be equal bit for
bit, whether contractions are shared or not. Bounds of the activations are those of
test_gpu_fp8.py: 32 u of the larger of |z|, 1 (u = 2^-24) for silu and gelu of a
given z, a slope of at most 1.13, and half a step for each rounding.

Each case says which tiles it reaches, and the test holds it to that: by the bytes of
its workspace, and by the plan that the kernel makes of its tiles.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

import fp8_reference as ref  # noqa: E402
import redzones  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
SLOPE = 1.13
ACTS = {"none": 0, "silu": 1, "gelu": 2, "swiglu": 3, "silu_grad": 4, "gelu_grad": 5,
        "swiglu_grad": 6}
FORMATS = {"f32": 1, "ue8m0": 2, "rect": 3}
CUS = 256


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    epl.load()


@pytest.fixture(autouse=True)
def _red_zones():
    yield
    redzones.check()


# ------------------------------------------------- which tiles a case takes --

def most_parts(K):
    return min(16, K // 512)


def bound_of_tiles(p, side):
    return (p.num_rows // side + p.num_experts) * -(-p.out_cols // side)


def held(side):
    """Tiles of a round."""
    return CUS * (1 if side == 256 else 2)


def side_of(p):
    """The tiles' side, by the workspace: partial tiles of as many workgroups as there may be."""
    made = epl.epl_product_fp8_workspace_bytes(p)
    bytes_of = {side: 256 + min(held(side), bound_of_tiles(p, side) * most_parts(p.in_cols)) *
                side * side * 4 for side in (256, 128)}
    assert most_parts(p.in_cols) > 1 and bytes_of[256] != bytes_of[128]
    assert made in bytes_of.values()
    return 256 if made == bytes_of[256] else 128


def plan_of(p, counts, side):
    """(tiles are more than workgroups, parts of the last round's tiles) with a workspace."""
    tiles = sum(-(-c // side) for c in counts) * -(-p.out_cols // side)
    most = most_parts(p.in_cols)
    grid = min(bound_of_tiles(p, side) * most, held(side))
    left, stages = tiles % grid, -(-p.in_cols // 128)
    parts = min(grid // left, most) if left else 1
    if parts > 1 and stages * (parts - 1) * (17 if side == 256 else 42) <= left * parts * parts:
        parts = 1
    return tiles > grid, parts


# ----------------------------------------------------------------- the case --

def codes_at(shape, seed):
    pick = torch.tensor([0x00, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    return pick[torch.randint(0, 5, shape, generator=g, device=DEV)]


def normal(*shape, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * std


def exponents(shape, low, seed):
    """Exponent bytes of 2^low .. 2^(low + 2)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(127 + low, 130 + low, shape, generator=g, device=DEV).to(torch.uint8)


def silu(z):
    return z * torch.sigmoid(z)


def silu_slope(z):
    p = torch.sigmoid(z)
    return p + z * p * torch.sigmoid(-z)


def gelu(z):
    return 0.5 * z * torch.erfc(-z / math.sqrt(2))


def own(z):
    return 32 * U * z.abs().clamp(min=1)


def raw(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def poison(shape, dtype):
    return redzones.poisoned(shape, dtype, 0x5A, DEV)


def check(counts, K, N, act="none", transposed=False, quantized=None, out=torch.float32, fmt="f32",
          w_fmt="f32", whole_epilogue=False, side=None, several=None, parts=None, seed=0):
    E = len(counts)
    grad = act.endswith("_grad")
    cols = N // 2 if act == "swiglu" else 2 * N if act == "swiglu_grad" else N
    gap, cap = 5, 0
    starts, total = [], 3                                # rows of no expert before, between, behind
    for c in counts:
        starts.append(total)
        total += c + gap
    if fmt == "rect":
        cap = max(counts) + gap
        starts, total = [e * cap for e in range(E)], E * cap
    owned = torch.zeros(total, dtype=torch.bool, device=DEV)
    for s, c in zip(starts, counts):
        owned[s:s + c] = True

    x = codes_at((total, K), seed)
    x[~owned] = 0x7F                                     # (not read)
    xb = exponents((total, ref.groups(K)), 0, seed + 1)
    shape = (E, K, N) if transposed else (E, N, K)
    w = codes_at(shape, seed + 2)
    wb = exponents((E, ref.groups(shape[1]), ref.groups(shape[2])), -8, seed + 3)
    numbers = lambda b: torch.exp2(b.double() - 127)  # noqa: E731
    laid = ref.pack(xb.cpu()).to(DEV) if fmt == "ue8m0" else \
        ref.lay(numbers(xb).float(), fmt, cap)
    ws = wb if w_fmt == "ue8m0" else numbers(wb).float()
    b = normal(E, N, seed=seed + 4) if whole_epilogue else None
    res = normal(total, cols, seed=seed + 5).bfloat16() if whole_epilogue else None
    saved = normal(total, cols, seed=seed + 6, std=2.0).bfloat16() if grad else None
    keep = act in ("swiglu", "silu", "gelu")

    p = epl.ProductFp8(total, sum(counts), E, K, N, int(transposed), ACTS[act],
                       0 if out == torch.float32 else 1, FORMATS[fmt], cap, FORMATS[w_fmt],
                       FORMATS[quantized] if quantized else 0, 0, 0)
    assert side_of(p) == side and plan_of(p, counts, side) == (several, parts)
    at, n = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (starts, counts))

    def run(split, with_y=True):
        y = poison((total, cols), out) if with_y else None
        pre = saved.clone() if grad else poison((total, N), torch.bfloat16) if keep else None
        codes = scale = None
        if quantized:
            s = ref.groups(cols)
            codes = poison((total, cols), torch.uint8)
            scale = poison(((s + 3) // 4, total), torch.int32) if quantized == "ue8m0" else \
                poison((total, s), torch.float32)
        space = poison(epl.epl_product_fp8_workspace_bytes(p), torch.uint8) if split else None
        epl.epl_expert_product_fp8(p, x, laid, w, ws, b, res, at, n, pre, y, codes, scale, space)
        return y, pre, codes, scale

    y, pre, codes, scale = made = run(True)
    for again in (run(True), run(False)):                # z is exact, shared or not
        for got, want in zip(again, made):
            assert got is None or torch.equal(raw(got), raw(want))
    if quantized:
        for got, want in zip(run(True, with_y=False)[2:], made[2:]):
            assert torch.equal(raw(got), raw(want))

    assert (y.view(torch.uint8).view(total, -1)[~owned] == 0x5A).all()
    if grad:
        assert torch.equal(raw(pre), raw(saved))
    elif keep:
        assert (pre.view(torch.uint8).view(total, -1)[~owned] == 0x5A).all()
    xv = x.view(torch.float8_e4m3fn).double() * numbers(xb).repeat_interleave(128, 1)[:, :K]
    for e in range(E):
        lo, hi = starts[e], starts[e] + counts[e]
        if lo == hi:
            continue
        wide = numbers(wb[e]).repeat_interleave(128, 0)[:shape[1]].repeat_interleave(128, 1)[:, :shape[2]]
        wv = w[e].view(torch.float8_e4m3fn).double() * wide
        z = xv[lo:hi] @ (wv if transposed else wv.t().contiguous())
        assert float(z.abs().max()) * 2.0 ** 8 < 2.0 ** 24
        tol = torch.zeros_like(z)
        if b is not None:
            z = z + b[e].double()
            tol = U * z.abs()
        if keep:
            if b is None:
                assert torch.equal(raw(pre[lo:hi]), raw(z.bfloat16()))
            else:
                assert ((pre[lo:hi].double() - z).abs() <= tol + 2.0 ** -8 * (z.abs() + tol)).all()
        if act == "none":
            v, vt = z, tol
        elif act == "gelu":
            v, vt = gelu(z), SLOPE * tol + own(z)
        elif act == "silu":
            v, vt = silu(z), SLOPE * tol + own(z)
        elif act == "swiglu":
            g, u = z.chunk(2, 1)
            tg, tu = tol.chunk(2, 1)
            v = silu(g) * u
            vt = (SLOPE * tg + own(g)) * (u.abs() + tu) + silu(g).abs() * tu + 2 * U * v.abs()
        else:
            g, u = saved[lo:hi].double().chunk(2, 1)
            f = torch.cat([u * silu_slope(g), silu(g)], 1)
            fe = torch.cat([u.abs() * 64 * U, own(g)], 1)
            z = torch.cat([z, z], 1)
            v, vt = z * f, z.abs() * fe + 4 * U * (z * f).abs()
        if res is not None:
            r = res[lo:hi].double()
            v = v + r
            vt = vt + U * (v.abs() + r.abs())
        if act == "none" and b is None:
            assert torch.equal(raw(y[lo:hi]), raw(v.to(out)))
        else:
            assert ((y[lo:hi].double() - v).abs() <=
                    vt + torch.finfo(out).eps / 2 * (v.abs() + vt)).all()
    if quantized:
        made_scale = scale.cpu()
        if quantized == "ue8m0":
            made_scale = made_scale.t().reshape(-1).view(torch.uint8).view(total, -1)
            made_scale = made_scale[:, :ref.groups(cols)].contiguous()
        mine = owned.cpu()
        assert (codes[~owned] == 0x5A).all()
        assert (raw(made_scale)[~mine] == (0x5A if quantized == "ue8m0" else 0x5A5A5A5A)).all()
        if out == torch.float32:
            want, want_scale = ref.cast_rows(y[owned].cpu(), quantized)
            assert torch.equal(codes.cpu()[mine], want)
            assert torch.equal(raw(made_scale)[mine], raw(want_scale))


def uneven(experts, mean):
    return [int(mean * f) for f in ([1.7, 0, 0.6, 1.7] * experts)[:experts]]


LARGE, SMALL = 256, 128

# counts, K, N, tiles, more of them than workgroups, parts of the last round's tiles
SIZES = {
    "large, one round": ([300] * 12, 1040, 2048, LARGE, False, 1),
    "large, one round, shared": (uneven(40, 150), 4112, 1024, LARGE, False, 2),
    "large, two rounds": (uneven(12, 2100), 1040, 1024, LARGE, True, 1),
    "large, two rounds, second shared": (uneven(12, 1500), 2064, 1024, LARGE, True, 4),
    "small, one round, shared": ([520], 1040, 1152, SMALL, False, 2),
    "small, two rounds": (uneven(40, 300), 1040, 1024, SMALL, True, 1),
    "small, two rounds, second shared": ([2100] * 2, 2064, 2048, SMALL, True, 4),
    "small, four rounds, last shared": (uneven(40, 300), 1040, 2048, SMALL, True, 2),
}
ODD = {
    "large, one round": ([260] * 12, 1040, 2064, LARGE, False, 1),
    "large, two rounds, second shared": (uneven(12, 500), 1040, 2064, LARGE, True, 2),
    "small, two rounds": (uneven(40, 150), 1040, 1552, SMALL, True, 1),
    "small, two rounds, second shared": ([900] * 4, 2064, 2064, SMALL, True, 4),
}
GATED = {
    "one round": ([300] * 4, 1040, 2048, LARGE, False, 1),
    "one round, shared": ([850, 0, 300, 850], 1168, 1024, LARGE, False, 2),
    "two rounds": ([260] * 40, 1040, 1024, LARGE, True, 1),
    "two rounds, second shared": ([520] * 12, 1040, 2048, LARGE, True, 2),
}


def reach(size, **kw):
    counts, K, N, side, several, parts = size
    check(counts, K, N, side=side, several=several, parts=parts, **kw)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("quantized", [None, "f32", "ue8m0"])
@pytest.mark.parametrize("size", list(SIZES))
def test_tiles(size, quantized, transposed):
    reach(SIZES[size], quantized=quantized, transposed=transposed)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("size", list(ODD))
def test_tiles_that_end_inside(size, transposed):
    """Columns that end inside a tile and inside a block of scales."""
    reach(ODD[size], transposed=transposed, out=torch.bfloat16)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("quantized", ["f32", "ue8m0"])
@pytest.mark.parametrize("size", list(SIZES))
def test_tiles_gated_gradient_and_its_cast(size, quantized, transposed):
    reach(SIZES[size], act="swiglu_grad", quantized=quantized, transposed=transposed)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("quantized", ["f32", "ue8m0"])
@pytest.mark.parametrize("size", list(GATED))
def test_tiles_gated_activation_and_its_cast(size, quantized, transposed):
    reach(GATED[size], act="swiglu", quantized=quantized, transposed=transposed)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("size", list(SIZES))
def test_tiles_gated_activation(size, transposed):
    reach(SIZES[size], act="swiglu", transposed=transposed, out=torch.bfloat16)


@pytest.mark.parametrize("act,quantized", [("silu", None), ("gelu", None), ("swiglu", None),
                                           ("silu", "f32"), ("gelu", "f32")])
@pytest.mark.parametrize("size", ["large, one round, shared", "large, two rounds, second shared",
                                  "small, two rounds, second shared"])
def test_tiles_whole_epilogue(size, act, quantized):
    reach(SIZES[size], act=act, quantized=quantized, whole_epilogue=True)


@pytest.mark.parametrize("size", ["one round, shared", "two rounds, second shared"])
def test_tiles_gated_whole_epilogue_and_its_cast(size):
    reach(GATED[size], act="swiglu", quantized="f32", whole_epilogue=True)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("fmt,w_fmt", [("ue8m0", "f32"), ("ue8m0", "ue8m0"), ("rect", "f32"),
                                       ("rect", "ue8m0"), ("f32", "ue8m0")])
@pytest.mark.parametrize("size", ["large, one round, shared", "small, one round, shared"])
def test_tiles_scale_formats(size, fmt, w_fmt, transposed):
    reach(SIZES[size], fmt=fmt, w_fmt=w_fmt, transposed=transposed, out=torch.bfloat16)
