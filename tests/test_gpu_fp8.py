"""Casts to 8 bits and back and the experts' products on 8-bit rows, on the
GPU, against their definitions (fp8_reference.py).

Casts of values that are given exactly have to equal the binary32 steps of
their definition, bit for bit. Where an activation comes first, its result v is
off by at most 32 u of the larger of |v|, 1 (u = 2^-24, as for the bf16
products), the scale by 4 u of itself, and a code rounds by half a step: 2^-4
of the value, or half of the smallest step 2^-9 of a scale.

Products: z is within the bound that fp8_reference.product derives; an
activation passes that on times its steepest slope 1.13 and adds its own 32 u
of the larger of |z|, 1; the output's rounding adds half a step of its type.
The cast of a result starts from the same binary32 values as y, so that codes
and scales are those of the cast of an fp32 y, bit for bit.
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
ACTS = {"none": 0, "silu": 1, "gelu": 2, "swiglu": 3, "silu_grad": 4, "gelu_grad": 5,
        "swiglu_grad": 6}
FORMATS = {"f32": 1, "ue8m0": 2, "rect": 3}
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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(*shape, seed, std=1.0):
    return torch.randn(*shape, generator=gen(seed)) * std


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def bytes_buffer(shape, dtype=torch.uint8):
    return redzones.poisoned(shape, dtype, 0x5A, DEV)


def raw(t):
    """The bits of a tensor, on the CPU."""
    t = t.cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same_codes(got, want):
    """Equal codes; NaNs of either sign are one."""
    got, want = got.cpu(), want.cpu()
    nan = (want & 0x7F) == 0x7F
    assert torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, want))


def scale_buffer(rows, cols, fmt, cap=0):
    s = ref.groups(cols)
    if fmt == "ue8m0":
        return bytes_buffer(((s + 3) // 4, rows), torch.int32)
    if fmt == "rect":
        return bytes_buffer((rows // cap, s, cap), torch.float32)
    return bytes_buffer((rows, s), torch.float32)


def by_row(scale, fmt, cols):
    """Scales in a buffer's layout -> [rows, groups] (fp32, or uint8 exponents)."""
    scale, s = scale.cpu(), ref.groups(cols)
    if fmt == "ue8m0":
        return scale.t().reshape(-1).view(torch.uint8).view(scale.shape[1], -1)[:, :s].contiguous()
    if fmt == "rect":
        return scale.transpose(1, 2).reshape(-1, s).contiguous()
    return scale


def owned_rows(total, starts, counts):
    if starts is None:
        return torch.ones(total, dtype=torch.bool)
    o = torch.zeros(total, dtype=torch.bool)
    for s, c in zip(starts, counts):
        o[max(s, 0):max(min(s + c, total), 0)] = True
    return o


# ------------------------------------------------------------------ casts --

def hard_values(rows, cols, seed):
    """Normal rows of differing size, among them groups of zeros, of values
    below and near binary32's smallest, of ties and of single large values."""
    x = randn(rows, cols, seed=seed) * torch.exp(randn(cols, seed=seed + 1, std=2.0))
    flat = x.view(-1)
    for i, v in enumerate((0.0, 1e-38, 3e-41, 2.0 ** -126, 3e38, 1e-30)):
        a = (i * 128) % max(flat.numel() - 128, 1)
        flat[a:a + 128] = v * torch.randint(-3, 4, (min(128, flat.numel() - a),),
                                            generator=gen(seed + 2 + i)).clamp(-1, 1)
    return x


@pytest.mark.parametrize("rows,cols,fmt,dtype,blocks", [
    (1, 16, "f32", "bf16", None), (1, 7168, "f32", "bf16", None), (3, 144, "ue8m0", "f32", None),
    (130, 1280, "f32", "f32", None), (257, 528, "ue8m0", "bf16", None),
    (64, 2048, "f32", "bf16", ([0, 10, 10, 50], [7, 0, 30, 9])),
    (90, 640, "ue8m0", "f32", ([60, 0, 40], [40, 17, 0])),     # cut to the buffer, out of order
    (60, 256, "rect", "bf16", ([0, 20, 40], [20, 0, 3])),
    (33, 1152, "rect", "f32", None), (5, 128, "f32", "f32", ([-3, 4], [5, 9])),
])
def test_quantize_equals_its_steps(rows, cols, fmt, dtype, blocks):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = hard_values(rows, cols, seed=rows).to(dt)
    starts, counts = blocks if blocks else (None, None)
    owned = owned_rows(rows, starts, counts)
    x[~owned] = float("nan")
    cap = rows // 3 if fmt == "rect" else 0
    codes, scale = bytes_buffer((rows, cols)), scale_buffer(rows, cols, fmt, cap)
    p = epl.Cast(rows, len(starts) if starts else 0, cols, int(dtype == "bf16"), 0, FORMATS[fmt],
                 cap, 0, 0)
    epl.epl_quantize(p, x.to(DEV), i32(starts) if starts else None,
                     i32(counts) if starts else None, codes, scale)
    want, want_scale = ref.cast_rows(x.float(), fmt)
    same_codes(codes[owned], want[owned])
    got = by_row(scale, fmt, cols)
    assert torch.equal(raw(got)[owned], raw(want_scale)[owned])
    assert (codes.cpu()[~owned] == 0x5A).all()
    assert (raw(got)[~owned] == (0x5A if fmt == "ue8m0" else 0x5A5A5A5A)).all()
    if fmt == "ue8m0":
        rest = scale.cpu().t().reshape(-1).view(torch.uint8).view(rows, -1)[:, ref.groups(cols):]
        assert (rest[owned] == 0).all() and (rest[~owned] == 0x5A).all()


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_quantize_infinities_and_nans(fmt):
    x = randn(4, 384, seed=0)
    x[0, 5], x[1, 130], x[2, 300], x[2, 301] = float("inf"), float("nan"), float("-inf"), 7.0
    x[3, :128] = float("nan")
    codes, scale = epl.quantize(x.to(DEV), scale_format=fmt)
    want, want_scale = ref.cast_rows(x, fmt)
    same_codes(codes, want)
    assert torch.equal(raw(by_row(scale, fmt, 384)), raw(want_scale))
    back = epl.dequantize(codes, scale, out_dtype=torch.float32).cpu()
    assert torch.isnan(back[0, 5]) and torch.isnan(back[1, 130]) and torch.isnan(back[2, 300])
    assert torch.isfinite(back[1, :128]).all() and torch.isfinite(back[0, 128:]).all()
    assert torch.isfinite(back[1, 131:256]).all()        # a NaN leaves its group's others alone


def test_quantize_is_the_low_latency_cast():
    T, H, E, cap = 40, 640, 2, 64
    x = hard_values(T, H, seed=4).bfloat16()
    x[torch.isinf(x)] = 0
    p = epl.Problem.make(T, 1, E, 1, H, H // 128)
    d = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    idx = (torch.arange(T) % E)[:, None].to(DEV)
    out, sc, oi = d(E, cap, H, t=torch.uint8), d(E, H // 128, cap, t=torch.float32), d(T, 1)
    cnt = d(E)
    epl.epl_ll_dispatch(p, T, cap, idx, x.to(DEV), out, sc, cnt, d(E, cap), d(E, 1, 2), oi,
                        d(epl.epl_ll_workspace_bytes(p, T), t=torch.uint8))
    codes, scale = epl.quantize(x.to(DEV))
    at = oi[:, 0].long()
    assert torch.equal(codes, out.view(-1, H)[at])
    assert torch.equal(scale, sc.transpose(1, 2).reshape(-1, H // 128)[at])
    # and its rectangle is read where it lies
    starts = torch.arange(E, device=DEV, dtype=torch.int32) * cap
    y = epl.dequantize(out.view(-1, H), sc, starts, cnt, out=d(E * cap, H, t=torch.float32))
    assert torch.equal(y[at], epl.dequantize(codes, scale, out_dtype=torch.float32))
    assert int((y != 0).any(1).sum()) <= T


@pytest.mark.parametrize("rows,f,fmt,dtype", [(1, 16, "f32", "bf16"), (37, 400, "f32", "f32"),
                                              (300, 2048, "ue8m0", "bf16")])
def test_quantize_gated(rows, f, fmt, dtype):
    x = randn(rows, 2 * f, seed=rows, std=2.0).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    codes, scale = epl.quantize(x.to(DEV), activation="swiglu", scale_format=fmt)
    g, u = x.double().chunk(2, 1)
    v = g * torch.sigmoid(g) * u
    s = ref.numbers(by_row(scale, fmt, f))
    wide = s.repeat_interleave(128, 1)[:, :f]
    own = 32 * U * v.abs().clamp(min=1)
    off = (ref.decode(codes.cpu()) * wide - v).abs()
    assert (off <= 2.0 ** -4 * (v.abs() + own) + 2.0 ** -10 * wide + own + 4 * U * v.abs()).all()
    pad = torch.nn.functional.pad(v, (0, -f % 128)).view(rows, -1, 128).abs().amax(2)
    tol = 32 * U * pad.clamp(min=1) + 4 * U * pad
    if fmt == "f32":
        assert ((s * 448 - pad).abs() <= tol).all()
    else:                                           # the least power of two that holds them
        assert (pad - tol <= s * 448).all() and (pad + tol >= s * 224).all()


@pytest.mark.parametrize("rows,cols,fmt,dtype,blocks", [
    (1, 16, "f32", "bf16", None), (70, 1408, "ue8m0", "bf16", ([5, 40], [30, 40])),
    (129, 272, "f32", "f32", None), (48, 640, "rect", "bf16", ([0, 16, 32], [16, 0, 7])),
    (1000, 128, "ue8m0", "f32", None),
])
def test_dequantize(rows, cols, fmt, dtype, blocks):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = gen(rows)
    codes = torch.randint(0, 256, (rows, cols), generator=g, dtype=torch.uint8)
    s = ref.groups(cols)
    scale = torch.randint(0, 256, (rows, s), generator=g, dtype=torch.uint8) if fmt == "ue8m0" else \
        torch.exp(randn(rows, s, seed=1, std=3.0))
    cap = 16 if fmt == "rect" else 0
    starts, counts = blocks if blocks else (None, None)
    owned = owned_rows(rows, starts, counts)
    y = bytes_buffer((rows, cols), dt)
    epl.dequantize(codes.to(DEV), ref.lay(scale, fmt, cap).to(DEV),
                   i32(starts) if starts else None, i32(counts) if starts else None, out=y)
    # a code has 4 significant bits: the product is rounded once, to fp32, and fp32 to bf16
    wide = ref.numbers(scale).repeat_interleave(128, 1)[:, :cols]
    want = (ref.decode(codes) * wide).float().to(dt)
    got = y.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got[owned]), nan[owned])
    assert torch.equal(torch.where(nan, 0, got)[owned], torch.where(nan, 0, want)[owned])
    assert (y.view(torch.uint8).view(rows, -1).cpu()[~owned] == 0x5A).all()


@pytest.mark.parametrize("E,N,K,fmt,dtype", [
    (1, 1, 16, "f32", "f32"), (2, 300, 400, "f32", "bf16"), (3, 128, 1152, "ue8m0", "bf16"),
    (1, 1000, 1040, "ue8m0", "f32"), (5, 257, 128, "f32", "f32"),
])
def test_quantize_weight_equals_its_steps(E, N, K, fmt, dtype):
    w = hard_values(E * N, K, seed=N).view(E, N, K)
    w = w.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    codes = bytes_buffer((E, N, K))
    scale = bytes_buffer((E, ref.groups(N), ref.groups(K)),
                         torch.uint8 if fmt == "ue8m0" else torch.float32)
    epl.quantize_weight(w.to(DEV), out=codes, out_scale=scale)
    want, want_scale = ref.cast_weight(w.float(), fmt)
    same_codes(codes, want)
    assert torch.equal(raw(scale), raw(want_scale))
    made = epl.quantize_weight(w.to(DEV), scale_format=fmt)
    assert torch.equal(raw(made[0]), raw(codes)) and torch.equal(raw(made[1]), raw(scale))


# --------------------------------------------------------------- products --

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


def blocks(counts, gap):
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += c + gap
    return starts, at


def codes_of(x, fmt):
    codes, scale = ref.cast_rows(x, "ue8m0" if fmt == "ue8m0" else "f32")
    return codes, scale


def check_product(counts, K, N, act="none", fmt="f32", w_fmt="f32", out=torch.bfloat16, bias=False,
                  residual=False, pre=False, transposed=False, quantized=None, gap=0, expected=0,
                  rows=None, starts=None, in_place=False, split=True, seed=0, spread=1.0):
    E = len(counts)
    made, total = blocks(counts, gap)
    cap = 0
    if fmt == "rect":
        cap = max(max(counts), 1) + gap
        made, total = [e * cap for e in range(E)], E * cap
    starts = made if starts is None else starts
    total = total if rows is None else rows
    grad = act.endswith("_grad")
    cols = N // 2 if act == "swiglu" else 2 * N if act == "swiglu_grad" else N
    x = randn(total, K, seed=seed) * torch.exp(randn(K, seed=seed + 1, std=spread))
    xc, xs = codes_of(x, fmt)
    shape = (E, K, N) if transposed else (E, N, K)
    wc, ws = ref.cast_weight(randn(*shape, seed=seed + 2, std=K ** -0.5), w_fmt)
    b = randn(E, N, seed=seed + 3) if bias else None
    res = randn(total, cols, seed=seed + 4).bfloat16() if residual else None
    saved = randn(total, cols, seed=seed + 5, std=2.0).bfloat16() if grad else None
    owned = owned_rows(total, starts, counts)
    xc[~owned] = 0x7F                            # rows of no expert are not read
    y = None
    if out is not None:
        y = bytes_buffer((total, cols), out)
        if in_place:
            y.copy_(res)
    before = None if y is None else raw(y).clone()
    z_out = saved.to(DEV) if grad else bytes_buffer((total, N), torch.bfloat16) if pre else None
    codes = codes_scale = None
    if quantized:
        codes, codes_scale = bytes_buffer((total, cols)), scale_buffer(total, cols, quantized)
    p = epl.ProductFp8(total, expected, E, K, N, int(transposed), ACTS[act],
                       0 if out == torch.float32 else 1, FORMATS[fmt], cap, FORMATS[w_fmt],
                       FORMATS[quantized] if quantized else 0, 0, 0)
    nbytes = epl.epl_product_fp8_workspace_bytes(p)
    ws_buffer = bytes_buffer(nbytes) if nbytes and split else None
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    args = (p, d(xc), d(ref.lay(xs, fmt, cap)), d(wc), d(ws), d(b), y if in_place else d(res),
            i32(starts), i32(counts), z_out, y, codes, codes_scale, ws_buffer)
    epl.epl_expert_product_fp8(*args)
    if y is not None:
        got = y.cpu()
        assert torch.equal(raw(got)[~owned], before[~owned])
    if codes is not None:
        assert (codes.cpu()[~owned] == 0x5A).all()
        got_scale = by_row(codes_scale, quantized, cols)
        assert (raw(got_scale)[~owned] == (0x5A if quantized == "ue8m0" else 0x5A5A5A5A)).all()
    if grad:
        assert torch.equal(raw(z_out), raw(saved))
    xnum, wnum = ref.numbers(xs), ref.weight_scales(ws, *shape[1:])
    for e in range(E):
        lo, hi = max(starts[e], 0), max(min(starts[e] + counts[e], total), 0)
        if hi <= lo:
            continue
        w, s = (wc[e].t().contiguous(), wnum[e].t()) if transposed else (wc[e], wnum[e])
        z, tol = ref.product(xc[lo:hi], xnum[lo:hi], w, s[:, ::128])
        if b is not None:
            z = z + b[e].double()
            tol = tol + U * (z.abs() + b[e].double().abs())
        if pre and not grad:
            err = (z_out[lo:hi].cpu().double() - z).abs()
            assert (err <= tol + 2.0 ** -8 * (z.abs() + tol)).all()
        own = lambda v: 32 * U * v.abs().clamp(min=1)  # noqa: E731
        if act == "none":
            v, vt = z, tol
        elif act in ("silu", "gelu"):
            v = silu(z) if act == "silu" else gelu(z)
            vt = SLOPE * tol + own(z)
        elif act == "swiglu":
            g, u = z.chunk(2, 1)
            tg, tu = tol.chunk(2, 1)
            v = silu(g) * u
            h = silu(g).abs()
            tg = SLOPE * tg + own(g)
            vt = tg * (u.abs() + tu) + h * tu + 2 * U * v.abs()
        else:
            kept = saved[lo:hi].double()
            if act == "swiglu_grad":
                g, u = kept.chunk(2, 1)
                f = torch.cat([u * silu_slope(g), silu(g)], 1)
                fe = torch.cat([u.abs() * 32 * U * 2, own(g)], 1)
                z, tol = torch.cat([z, z], 1), torch.cat([tol, tol], 1)
            else:
                f = silu_slope(kept) if act == "silu_grad" else gelu_slope(kept)
                fe = 64 * U * torch.ones_like(f)
            v = z * f
            vt = tol * (f.abs() + fe) + z.abs() * fe + 4 * U * v.abs()
        if res is not None:
            r = res[lo:hi].double()
            v = v + r
            vt = vt + U * (v.abs() + r.abs())
        if y is not None:
            err = (got[lo:hi].double() - v).abs()
            lim = vt + torch.finfo(out).eps / 2 * (v.abs() + vt)
            assert (err <= lim).all(), (e, float((err - lim).max()))
        if codes is not None:
            if out == torch.float32:
                want, want_scale = ref.cast_rows(got[lo:hi], quantized)
                same_codes(codes[lo:hi], want)
                assert torch.equal(raw(got_scale)[lo:hi], raw(want_scale))
            wide = ref.numbers(got_scale[lo:hi]).repeat_interleave(128, 1)
            err = (ref.decode(codes[lo:hi].cpu()) * wide - v).abs()
            assert (err <= 2.0 ** -4 * (v.abs() + vt) + 2.0 ** -10 * wide + vt + 4 * U * v.abs()).all()
    return args


@pytest.mark.parametrize("counts,K,N", [
    ([1], 16, 16), ([3], 128, 128), ([0, 5, 0, 17], 144, 48), ([40, 1, 70], 272, 336),
    ([300], 640, 272), ([130, 0, 260], 1040, 144), ([2] * 33, 512, 64),
])
@pytest.mark.parametrize("transposed", [False, True])
def test_product_sizes(counts, K, N, transposed):
    check_product(counts, K, N, transposed=transposed, gap=1)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("counts", [[4, 0, 9], [150, 0, 45]])
def test_product_activations(act, counts):
    grad = act.endswith("_grad")
    for transposed in (False, True):
        check_product(counts, 400, 288, act=act, transposed=transposed, bias=not grad,
                      residual=not grad, pre=not grad, out=torch.float32, gap=3)


@pytest.mark.parametrize("fmt,w_fmt", [("f32", "ue8m0"), ("ue8m0", "f32"), ("ue8m0", "ue8m0"),
                                       ("rect", "f32"), ("rect", "ue8m0")])
@pytest.mark.parametrize("counts", [[5, 0, 11], [200, 31, 0]])
def test_product_scale_formats(fmt, w_fmt, counts):
    for transposed in (False, True):
        check_product(counts, 1168, 176, fmt=fmt, w_fmt=w_fmt, transposed=transposed, gap=2)


@pytest.mark.parametrize("act,N", [("none", 384), ("gelu", 128), ("swiglu", 768),
                                   ("swiglu_grad", 256), ("silu_grad", 128)])
@pytest.mark.parametrize("quantized", ["f32", "ue8m0"])
@pytest.mark.parametrize("counts", [[3, 0, 12], [129, 0, 40]])
def test_product_cast_of_its_result(act, N, quantized, counts):
    grad = act.endswith("_grad")
    for out in (None, torch.float32, torch.bfloat16):
        check_product(counts, 528, N, act=act, quantized=quantized, out=out, transposed=grad,
                      pre=grad or act == "swiglu", residual=act == "gelu", gap=1)


def test_product_blocks_that_leave_the_buffer():
    check_product([5, 20, 9], 128, 64, starts=[-2, 10, 36], rows=40)
    check_product([0, 0], 128, 64, starts=[0, 0], rows=7)


def test_product_in_place_residual():
    check_product([60, 7], 256, 128, residual=True, in_place=True, bias=True)


@pytest.mark.parametrize("split", [False, True])
def test_product_long_contraction(split):
    check_product([33, 5], 4096, 256, split=split)
    check_product([33, 5], 4096, 256, split=split, transposed=True, quantized="f32",
                  out=torch.float32, expected=38)


def test_product_expected_rows_change_nothing_but_the_kernel():
    for expected in (1, 40, 10 ** 6):
        check_product([3, 0, 64, 1], 512, 256, rows=900, expected=expected, act="swiglu",
                      quantized="f32", out=torch.float32)


def test_product_nan_codes_stay_in_their_row_and_column():
    x, w = randn(20, 256, seed=0), randn(1, 128, 256, seed=1)
    xc, xs = ref.cast_rows(x, "f32")
    wc, ws = ref.cast_weight(w, "f32")
    xc[4, 200], wc[0, 9, 3] = 0x7F, 0xFF
    y = epl.expert_product_fp8(xc.to(DEV), xs.to(DEV), wc.to(DEV), ws.to(DEV), i32([0]), i32([20]))
    bad = torch.isnan(y.cpu())
    want = torch.zeros(20, 128, dtype=torch.bool)
    want[4], want[:, 9] = True, True
    assert torch.equal(bad, want)


def test_python_call_returns_what_it_is_asked_for():
    x = randn(24, 256, seed=0).to(DEV)
    w = randn(2, 256, 256, seed=1, std=1 / 16).to(DEV)
    xc, xs = epl.quantize(x)
    wc, ws = epl.quantize_weight(w)
    at, n = i32([0, 10]), i32([10, 14])
    y = epl.expert_product_fp8(xc, xs, wc, ws, at, n)
    assert y.dtype == torch.bfloat16 and y.shape == (24, 256)
    y32, c, s = epl.expert_product_fp8(xc, xs, wc, ws, at, n, out_dtype=torch.float32,
                                       quantized="f32")
    assert torch.equal(y32.bfloat16(), y)
    c2, s2 = epl.expert_product_fp8(xc, xs, wc, ws, at, n, quantized="f32")
    assert torch.equal(c, c2) and torch.equal(s, s2)
    c3, s3 = epl.quantize(y32)
    assert torch.equal(c, c3) and torch.equal(s, s3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = epl.expert_product_fp8(xc, xs, wc, ws, at, n, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, y)
    with pytest.raises(ValueError, match="x_scale must have shape"):
        epl.expert_product_fp8(xc, xs[:, :1].contiguous(), wc, ws, at, n)
    with pytest.raises(ValueError, match="weight_scale must have shape"):
        epl.expert_product_fp8(xc, xs, wc, ws[:, :1].contiguous(), at, n)
    with pytest.raises(ValueError, match="contiguous"):
        epl.expert_product_fp8(xc[:, :128], xs, wc, ws, at, n)
    empty = epl.expert_product_fp8(xc[:0], xs[:0], wc, ws, i32([0, 0]), i32([0, 0]))
    assert empty.shape == (0, 256)


# ------------------------------------------------------------ gated block --

def block_inputs(counts, H, F, fmt, seed=0):
    E, total = len(counts), sum(counts)
    starts = [sum(counts[:e]) for e in range(E)]
    x = randn(total, H, seed=seed)
    w1, w2 = randn(E, 2 * F, H, seed=seed + 1, std=H ** -0.5), randn(E, H, F, seed=seed + 2, std=F ** -0.5)
    dy = randn(total, H, seed=seed + 3).bfloat16()
    w_fmt = "ue8m0" if fmt == "ue8m0" else "f32"
    return starts, x, ref.cast_weight(w1, w_fmt), ref.cast_weight(w2, w_fmt), dy


def block_in_64_bits(starts, counts, x, w1, w2, dy):
    """The block on the weights' and rows' values without its inner casts, and its gradients."""
    def values(w):
        codes, scale = w
        return ref.decode(codes) * ref.weight_scales(scale, *codes.shape[1:])
    w1, w2 = values(w1), values(w2)
    x = x.clone().requires_grad_(True)
    z = torch.cat([x[s:s + c] @ w1[e].t() for e, (s, c) in enumerate(zip(starts, counts))])
    z.retain_grad()
    g, u = z.chunk(2, 1)
    h = silu(g) * u
    y = torch.cat([h[s:s + c] @ w2[e].t() for e, (s, c) in enumerate(zip(starts, counts))])
    y.backward(dy.double())
    return y.detach(), z.detach(), x.grad, z.grad


def far(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


# The 2-norm of the error over the result's: a cast rounds each value by at most
# 2^-4 of it (and values below 2^-6 scales, 2^-10 of a group's largest over 448,
# by far less than that in norm), and the sums of a product pass relative
# errors of its rows on as they are where their signs are independent; y has
# one cast before it (h), grad_pre one (dy), grad_x two (dy, dz): 2^-4 each,
# with all of a value's error against it, besides a few steps of bf16.
TOL = 2.0 ** -4 + 4 * 2.0 ** -8


@pytest.mark.parametrize("counts,H,F,fmt", [
    ([1], 128, 128, "f32"), ([5, 0, 9], 256, 384, "f32"), ([200, 31, 0, 64], 384, 128, "ue8m0"),
    ([300, 40], 1024, 256, "f32"),
])
def test_block_forwards_and_back(counts, H, F, fmt):
    starts, x, w1, w2, dy = block_inputs(counts, H, F, fmt)
    xc, xs = ref.cast_rows(x, fmt)
    d = lambda t: t.to(DEV)  # noqa: E731
    xv = ref.decode(xc) * ref.numbers(xs).repeat_interleave(128, 1)
    z = torch.empty(x.shape[0], 2 * F, dtype=torch.bfloat16, device=DEV)
    w = [d(t) for t in (*w1, *w2)]
    y = epl.gated_block_fp8(d(xc), d(ref.lay(xs, fmt)), *w, i32(starts), i32(counts), pre=z,
                            scale_format=fmt)
    gx, gz = epl.gated_block_fp8_backward(d(dy), z, *w, i32(starts), i32(counts), scale_format=fmt)
    ry, rz, rgx, rgz = block_in_64_bits(starts, counts, xv, w1, w2, dy)
    assert far(z, rz) < 2.0 ** -8 and far(y, ry) < TOL
    assert far(gz, rgz) < TOL and far(gx, rgx) < 2 * TOL


def test_block_gradient_against_differences():
    """The formula that the gradients are held to above, by central differences in 64 bits."""
    counts = [3, 2]
    starts, x, w1, w2, dy = block_inputs(counts, 128, 128, "f32")
    x = x.double()
    _, _, gx, _ = block_in_64_bits(starts, counts, x, w1, w2, dy)
    v = randn(*x.shape, seed=9).double()
    step = 1e-5
    up, down = (block_in_64_bits(starts, counts, x + k * step * v, w1, w2, dy)[0] for k in (1, -1))
    slope = float(((up - down) * dy.double()).sum() / (2 * step))
    # the differences' own error: step^2 of the third derivative, and 2^-53 / step of the values
    assert abs(slope - float((gx * v).sum())) < 1e-6 * float((gx.abs() * v.abs()).sum())


def test_block_as_a_layer_serves_and_trains_it():
    """Router, cast, dispatch of 8-bit rows, block, combine; back: combine's gradient, the
    block's, the weights' from rows made bf16 again, the dispatch's. Against the same layer in
    64 bits with the choice that the router made."""
    T, H, F, E, K = 150, 256, 128, 8, 2
    x = randn(T, H, seed=0)
    _, _, w1, w2, _ = block_inputs([1] * E, H, F, "f32", seed=5)
    logits = randn(T, E, seed=7).to(DEV)
    dy = randn(T, H, seed=8).to(DEV)
    idx, wt = epl.route(logits, K, renormalize=True)
    codes, scale = epl.quantize(x.to(DEV))
    p = epl.Problem.make(T, K, E, 1, H, H // 128)
    cap = epl.epl_capacity_rows(p)
    e32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    cnt, per_rank, at, oi, m = e32(E), e32(1), e32(E), e32(T, K), e32(cap)
    in_rank = torch.empty(T, 1, dtype=torch.uint8, device=DEV)
    rows = torch.zeros(cap, H, dtype=torch.uint8, device=DEV)
    rows_scale = torch.zeros(cap, H // 128, device=DEV)
    epl.epl_dispatch_fp8(p, idx, codes, scale, epl.EPL_SCALE_F32, cap, cnt, per_rank, None, in_rank,
                         at, None, rows, rows_scale, m, oi,
                         torch.empty(epl.epl_workspace_bytes(p), dtype=torch.uint8, device=DEV))
    w = [t.to(DEV) for t in (*w1, *w2)]
    z = torch.zeros(cap, 2 * F, dtype=torch.bfloat16, device=DEV)
    o = epl.gated_block_fp8(rows, rows_scale, *w, at, cnt, pre=z, expected_rows=T * K)
    y = epl.combine(o, oi, wt)
    do, dwt = epl.combine_backward(dy, o, oi, wt)
    drows, dz = epl.gated_block_fp8_backward(do, z, *w, at, cnt, expected_rows=T * K)
    dx = epl.dispatch_backward(drows, oi)
    rows16 = epl.dequantize(rows, rows_scale, at, cnt)
    dw1 = epl.expert_weight_grad(dz, rows16, at, cnt, out_dtype=torch.float32)

    cc, cs = codes.cpu(), scale.cpu()
    xv = ref.decode(cc) * cs.double().repeat_interleave(128, 1)
    v1 = ref.decode(w1[0]) * ref.weight_scales(w1[1], 2 * F, H)
    v2 = ref.decode(w2[0]) * ref.weight_scales(w2[1], H, F)
    xv.requires_grad_(True)
    v1.requires_grad_(True)
    wv = wt.cpu().double().requires_grad_(True)
    out = torch.zeros(T, H).double()
    for k in range(K):
        e = idx[:, k].cpu()
        g, u = (xv[:, None, :] * v1[e]).sum(2).chunk(2, 1)
        out = out + wv[:, k][:, None] * ((silu(g) * u)[:, None, :] * v2[e]).sum(2)
    out.backward(dy.cpu().double())
    assert far(y, out.detach()) < TOL and far(dwt, wv.grad) < 2 * TOL
    assert far(dx, xv.grad) < 2 * TOL and far(dw1, v1.grad) < 2 * TOL


def test_captured_block_replays_like_eager():
    counts, H, F = [60, 0, 130, 10], 512, 256
    starts, x, w1, w2, dy = block_inputs(counts, H, F, "f32")
    total = sum(counts)
    w = [t.to(DEV) for t in (*w1, *w2)]
    xin, dyin = x.to(DEV), dy.to(DEV)
    at, n = i32(starts), i32(counts)
    y = torch.zeros(total, H, dtype=torch.bfloat16, device=DEV)
    z, dz = (torch.zeros(total, 2 * F, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dx = torch.zeros_like(y)

    def step():
        c, s = epl.quantize(xin, expert_start_loc=at, num_tokens_per_expert=n)
        epl.gated_block_fp8(c, s, *w, at, n, pre=z, out=y)
        epl.gated_block_fp8_backward(dyin, z, *w, at, n, grad_x=dx, grad_pre=dz)

    outs, made = (y, z, dx, dz), []
    for seed in (11, 12, 13):
        xin.copy_(randn(total, H, seed=seed))
        step()
        made.append([o.clone() for o in outs])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for k in range(6):
        for o in outs:
            o.zero_()
        xin.copy_(randn(total, H, seed=11 + k % 3))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, made[k % 3]):
            assert torch.equal(got, want)
        _ = (xin @ xin.t()).sum()                       # the program's own work between


def test_two_streams_at_once():
    """Calls that overlap share nothing but their inputs."""
    counts, H, F = [70, 30, 0, 200], 640, 256
    starts, x, w1, w2, _ = block_inputs(counts, H, F, "f32")
    w = [t.to(DEV) for t in (*w1, *w2)]
    xc, xs = epl.quantize(x.to(DEV))
    at, n = i32(starts), i32(counts)
    want = epl.gated_block_fp8(xc, xs, *w, at, n)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [epl.gated_block_fp8(xc, xs, *w, at, n, stream=streams[k % 3]) for k in range(12)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for g in got:
        assert torch.equal(g, want)


@pytest.mark.parametrize("act,K,N,quantized,out", [
    ("none", 8240, 48, None, torch.bfloat16), ("swiglu", 4096, 80, None, torch.float32),
    ("swiglu", 4240, 400, None, torch.bfloat16), ("swiglu", 4096, 256, "f32", torch.float32),
    ("swiglu_grad", 4112, 128, "ue8m0", torch.float32), ("gelu", 6160, 128, "f32", None),
])
@pytest.mark.parametrize("split", [False, True])
def test_product_few_rows_long_contraction(act, K, N, quantized, out, split):
    """The contraction shared by workgroups and joined, but for the expert of
    more than 32 rows; without a workspace, taken in segments of it."""
    counts, grad = [1, 40, 0, 17, 32], act.endswith("_grad")
    p = epl.ProductFp8(sum(counts) + 5, 0, 5, K, N, 0, ACTS[act], 1, 1, 0, 1,
                       FORMATS[quantized] if quantized else 0, 0, 0)
    assert epl.epl_product_fp8_workspace_bytes(p) > 256
    check_product(counts, K, N, act=act, quantized=quantized, out=out, split=split, gap=1,
                  bias=not grad, residual=not grad, pre=not grad)


@pytest.mark.parametrize("counts", [[3], [24], [150]])
@pytest.mark.parametrize("blocks_of_k", [1, 3, 8])
def test_product_infinite_scales(counts, blocks_of_k):
    """An infinite scale over finite codes of one sign: infinities, and none of
    them times a padded zero."""
    K, rows = 128 * blocks_of_k, counts[0]
    one = torch.full((rows, K), 0x38, dtype=torch.uint8, device=DEV)
    scale = torch.ones(rows, blocks_of_k, device=DEV)
    scale[1, blocks_of_k - 1], scale[2, 0] = math.inf, math.inf
    w = torch.full((1, 144, K), 0x38, dtype=torch.uint8, device=DEV)
    ws = torch.ones(1, 2, blocks_of_k, device=DEV)
    want = torch.full((rows, 144), float(K))
    want[1:3] = math.inf
    assert torch.equal(epl.expert_product_fp8(one, scale, w, ws, i32([0]), i32(counts)).cpu(),
                       want.bfloat16())
    ws[0, 1, 0] = math.inf
    want[:, 128:] = math.inf
    assert torch.equal(epl.expert_product_fp8(one, scale, w, ws, i32([0]), i32(counts)).cpu(),
                       want.bfloat16())


@pytest.mark.parametrize("rows", [5, 150])
def test_product_exponents_at_their_ends(rows):
    """A byte of 255 makes its row, or its block's columns, NaN; 0 is 2^-127."""
    K = 256
    one = torch.full((rows, K), 0x38, dtype=torch.uint8, device=DEV)
    w = torch.full((1, 256, K), 0x38, dtype=torch.uint8, device=DEV)
    power = torch.full((rows, 4), 127, dtype=torch.uint8)
    power[:, 2:] = 0
    power[1, 1], power[2, :2] = 255, 0
    scale = power.view(torch.int32).t().contiguous().to(DEV)
    ws = torch.full((1, 2, 2), 127, dtype=torch.uint8, device=DEV)
    ws[0, 1, 0] = 255
    y = epl.expert_product_fp8(one, scale, w, ws, i32([0]), i32([rows]),
                               out_dtype=torch.float32).cpu()
    want = torch.full((rows, 256), 256.0)
    want[2] = 256 * 2.0 ** -127
    want[1], want[:, 128:] = math.nan, math.nan
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    # 2^-119 is a normal number, and every step to it is exact
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))


def test_no_rows():
    none = torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV)
    w1 = epl.quantize_weight(randn(2, 512, 256, seed=0).to(DEV))
    w2 = epl.quantize_weight(randn(2, 256, 256, seed=1).to(DEV))
    at = i32([0, 0])
    for fmt in ("f32", "ue8m0"):
        codes, scale = epl.quantize(none, scale_format=fmt)
        assert epl.dequantize(codes, scale).shape == (0, 256)
        assert epl.expert_product_fp8(codes, scale, *w1, at, at).shape == (0, 512)
        assert epl.gated_block_fp8(codes, scale, *w1, *w2, at, at).shape == (0, 256)
    dx, dz = epl.gated_block_fp8_backward(none, torch.zeros(0, 512, dtype=torch.bfloat16, device=DEV),
                                          *w1, *w2, at, at)[:2]
    assert dx.shape == (0, 256) and dz.shape == (0, 512)


def test_two_captured_graphs_share_a_workspace():
    """Replayed in turn, in one stream's order: neither finds what the other left."""
    made = []
    for counts, K, N, act, seed in [([1, 20, 9], 4096, 256, "swiglu", 0), ([130, 0, 260], 1040, 144, "none", 3)]:
        args = list(check_product(counts, K, N, act=act, seed=seed))
        made.append((args, args[10].clone()))
    size = max(a[13].numel() for a, _ in made)
    shared = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
    graphs = []
    for args, _ in made:
        args[13] = shared
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            epl.epl_expert_product_fp8(*args)
        graphs.append(g)
    for k in range(6):
        for (args, want), g in zip(made, graphs):
            args[10].zero_()
            g.replay()
            assert torch.equal(args[10], want)
        shared.fill_(0x11 * k)                          # the program's own work between
        torch.cuda.synchronize()


def close_to_product(y, xc, xs, wc, ws):
    """A bf16 result against the sums and their bound (fp8_reference.product)."""
    z, tol = ref.product(xc, xs, wc, ref.weight_scales(ws[None], *wc.shape)[0][:, ::128])
    assert ((y.cpu().double() - z).abs() <= tol + 2.0 ** -8 * (z.abs() + tol)).all()


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_rows_past_32_bits(fmt):
    rows, K = 300_001, 7168                              # 2.15e9 codes
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-200:] = randn(200, K, seed=0).to(DEV)
    codes, scale = epl.quantize(x, scale_format=fmt)
    last = x[-200:].cpu().float()
    want, want_scale = ref.cast_rows(last, fmt)
    same_codes(codes[-200:], want)
    got_scale = by_row(scale[:, -200:] if fmt == "ue8m0" else scale[-200:], fmt, K)
    assert torch.equal(raw(got_scale), raw(want_scale))
    assert not codes[:-200].any()
    x.fill_(1)
    epl.dequantize(codes, scale, out=x)
    wide = (ref.decode(want) * ref.numbers(want_scale).repeat_interleave(128, 1)).float().bfloat16()
    assert torch.equal(raw(x[-200:]), raw(wide)) and not x[:-200].any()
    del x
    wc, ws = ref.cast_weight(randn(1, 48, K, seed=1, std=K ** -0.5), "f32")
    for count in (3, 200):
        y = epl.expert_product_fp8(codes, scale, wc.to(DEV), ws.to(DEV), i32([rows - count]),
                                   i32([count]), expected_rows=count)
        close_to_product(y[-count:], want[-count:], ref.numbers(want_scale)[-count:], wc[0], ws[0])


def test_weights_past_32_bits():
    E, N, K = 2048, 1024, 1040                           # 2.18e9 codes
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    w[-1] = randn(N, K, seed=0, std=K ** -0.5).to(DEV)
    codes, scale = epl.quantize_weight(w)
    want, want_scale = ref.cast_weight(w[-1:].cpu().float(), "f32")
    del w
    same_codes(codes[-1:], want)
    assert torch.equal(raw(scale[-1:]), raw(want_scale)) and not codes[:-1].any()
    counts = [0] * (E - 1) + [150]
    for transposed in (False, True):
        xc, xs = ref.cast_rows(randn(150, N if transposed else K, seed=1), "f32")
        y = epl.expert_product_fp8(xc.to(DEV), xs.to(DEV), codes, scale, i32([0] * E), i32(counts),
                                   transposed=transposed)
        if transposed:
            full = ref.weight_scales(want_scale, N, K)[0].t()
            z, tol = ref.product(xc, ref.numbers(xs), want[0].t().contiguous(), full[:, ::128])
            assert ((y.cpu().double() - z).abs() <= tol + 2.0 ** -8 * (z.abs() + tol)).all()
        else:
            close_to_product(y, xc, ref.numbers(xs), want[0], want_scale[0])
