"""The gated block on 8-bit rows, its gradient and a layer around it, row by row: a
norm over a whole tensor does not see one wrong row."""
import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

import fp8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    epl.load()


def randn(*shape, seed, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def raw(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def filled(shape, dtype):
    """Every byte 0x5A."""
    n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
    return torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV).view(dtype).view(shape)


def case(counts, H, F, fmt, gap):
    """Blocks with `gap` rows of no expert behind each, whose codes and values are NaN."""
    starts, total = [], 0
    for c in counts:
        starts.append(total)
        total += c + gap
    owned = torch.zeros(total, dtype=torch.bool)
    for s, c in zip(starts, counts):
        owned[s:s + c] = True
    E, w_fmt = len(counts), "ue8m0" if fmt == "ue8m0" else "f32"
    xc, xs = ref.cast_rows(randn(total, H, seed=0), fmt)
    xc[~owned] = 0x7F
    w1 = ref.cast_weight(randn(E, 2 * F, H, seed=1, std=H ** -0.5), w_fmt)
    w2 = ref.cast_weight(randn(E, H, F, seed=2, std=F ** -0.5), w_fmt)
    dy = randn(total, H, seed=3).bfloat16()
    dy[~owned] = float("nan")
    on = lambda *t: [v.to(DEV) for v in t]  # noqa: E731
    return dict(x=on(xc, ref.lay(xs, fmt)), w=on(*w1, *w2), dy=dy.to(DEV), owned=owned.to(DEV),
                at=i32(starts), n=i32(counts), total=total, cpu=(xc, xs, w1, w2, starts))


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
@pytest.mark.parametrize("counts,H,F", [
    ([1], 128, 128), ([5, 0, 20, 1], 1040, 384), ([1, 20, 9], 4096, 256),  # few rows, shared
    ([200, 31, 0, 64], 400, 128),                                         # tiles
    ([850, 0, 300, 850], 1168, 512),                                      # the first product shared
    ([300] * 4, 1040, 1024), ([520] * 12, 1040, 1024),
])
def test_block_equals_its_products_and_casts(counts, H, F, fmt):
    """Bit for bit, with h, dy and dz in hand: the products' own tests hold each of them, with
    its cast, to its definition."""
    c = case(counts, H, F, fmt, gap=3)
    w1, w1s, w2, w2s = c["w"]
    at, n, owned, total = c["at"], c["n"], c["owned"], c["total"]
    rows = dict(expert_start_loc=at, num_tokens_per_expert=n, expected_rows=sum(counts))
    pre, y = filled((total, 2 * F), torch.bfloat16), filled((total, H), torch.bfloat16)
    epl.gated_block_fp8(*c["x"], *c["w"], **rows, pre=pre, out=y, scale_format=fmt)
    z = filled((total, 2 * F), torch.bfloat16)
    h, hc, hs = epl.expert_product_fp8(*c["x"], w1, w1s, **rows, activation="swiglu", pre=z,
                                       out_dtype=torch.float32, quantized=fmt)
    want, want_scale = ref.cast_rows(h[owned].cpu(), fmt)
    assert torch.equal(hc[owned].cpu(), want)
    got = epl.dequantize(hc, hs, out_dtype=torch.float32)[owned].cpu()
    wide = ref.numbers(want_scale).repeat_interleave(128, 1)
    assert torch.equal(got, (ref.decode(want) * wide).float())
    assert torch.equal(raw(pre), raw(z))
    y2 = filled((total, H), torch.bfloat16)
    epl.expert_product_fp8(hc, hs, w2, w2s, **rows, out=y2)
    assert torch.equal(raw(y), raw(y2))
    assert (raw(y)[~owned] == 0x5A5A).all() and (raw(pre)[~owned] == 0x5A5A).all()
    assert torch.isfinite(y[owned].float()).all()

    gx, gz = filled((total, H), torch.bfloat16), filled((total, 2 * F), torch.bfloat16)
    epl.gated_block_fp8_backward(c["dy"], pre, *c["w"], **rows, grad_x=gx, grad_pre=gz,
                                 scale_format=fmt)
    dc, ds = epl.quantize(c["dy"], scale_format=fmt, expert_start_loc=at, num_tokens_per_expert=n)
    dz, zc, zs = epl.expert_product_fp8(dc, ds, w2, w2s, **rows, activation="swiglu_grad", pre=pre,
                                        out_dtype=torch.float32, quantized=fmt, transposed=True)
    want, want_scale = ref.cast_rows(dz[owned].cpu(), fmt)
    assert torch.equal(zc[owned].cpu(), want)
    assert torch.equal(raw(gz)[owned], raw(dz.bfloat16())[owned])
    x2 = filled((total, H), torch.bfloat16)
    epl.expert_product_fp8(zc, zs, w1, w1s, **rows, out=x2, transposed=True)
    assert torch.equal(raw(gx), raw(x2))
    assert (raw(gx)[~owned] == 0x5A5A).all() and (raw(gz)[~owned] == 0x5A5A).all()
    assert torch.isfinite(gx[owned].float()).all()


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
@pytest.mark.parametrize("counts,H,F", [([3, 0, 17], 528, 256), ([70, 31], 400, 128)])
def test_block_rows_by_their_definition(counts, H, F, fmt):
    """Every row of the second product, within the bound of fp8_reference.product."""
    c = case(counts, H, F, fmt, gap=2)
    rows = dict(expert_start_loc=c["at"], num_tokens_per_expert=c["n"], expected_rows=sum(counts))
    y = epl.gated_block_fp8(*c["x"], *c["w"], **rows, scale_format=fmt).cpu().double()
    w1, w1s, _, _ = c["w"]
    h, hc, hs = epl.expert_product_fp8(*c["x"], w1, w1s, **rows, activation="swiglu",
                                       out_dtype=torch.float32, quantized=fmt)
    xc, xs, w1, w2, starts = c["cpu"]
    s2 = ref.weight_scales(w2[1], H, F)
    for e, (s, m) in enumerate(zip(starts, counts)):
        if m == 0:
            continue
        _, scale = ref.cast_rows(h[s:s + m].cpu(), fmt)
        z, tol = ref.product(hc[s:s + m].cpu(), ref.numbers(scale), w2[0][e], s2[e][:, ::128])
        assert ((y[s:s + m] - z).abs() <= tol + 2.0 ** -8 * (z.abs() + tol)).all()


def test_layer_hands_every_row_on():
    """Cast, dispatch, block, combine and back: each token's rows, sums and gradients, by
    themselves."""
    T, H, F, E, K = 150, 256, 128, 8, 2
    w = [t.to(DEV) for t in (*ref.cast_weight(randn(E, 2 * F, H, seed=1, std=H ** -0.5), "f32"),
                             *ref.cast_weight(randn(E, H, F, seed=2, std=F ** -0.5), "f32"))]
    dy = randn(T, H, seed=3).to(DEV)
    idx, wt = epl.route(randn(T, E, seed=4).to(DEV), K, renormalize=True)
    codes, scale = epl.quantize(randn(T, H, seed=0).to(DEV))
    p = epl.Problem.make(T, K, E, 1, H, H // 128)
    cap = epl.epl_capacity_rows(p)
    e32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    cnt, per_rank, at, oi, m = e32(E), e32(1), e32(E), e32(T, K), e32(cap)
    rows, rows_scale = filled((cap, H), torch.uint8), filled((cap, H // 128), torch.float32)
    epl.epl_dispatch_fp8(p, idx, codes, scale, epl.EPL_SCALE_F32, cap, cnt, per_rank, None,
                         torch.empty(T, 1, dtype=torch.uint8, device=DEV), at, None, rows,
                         rows_scale, m, oi,
                         torch.empty(epl.epl_workspace_bytes(p), dtype=torch.uint8, device=DEV))
    slots = oi.long()
    assert slots.min() >= 0 and slots.unique().numel() == T * K
    assert torch.equal(rows[slots], codes[:, None].expand(T, K, H))
    assert torch.equal(rows_scale[slots], scale[:, None].expand(T, K, H // 128))
    z = torch.zeros(cap, 2 * F, dtype=torch.bfloat16, device=DEV)
    o = epl.gated_block_fp8(rows, rows_scale, *w, at, cnt, pre=z, expected_rows=T * K)
    y = epl.combine(o, oi, wt)
    each = wt.double()[:, :, None] * o.double()[slots]
    # two rounded products and their sum
    assert ((y.double() - each.sum(1)).abs() <= 4 * U * each.abs().sum(1)).all()
    # a token's row of an expert is that of a call with this row alone, but for the kernel
    xv = epl.dequantize(codes, scale, out_dtype=torch.float32).double()
    v1 = ref.decode(w[0].cpu()) * ref.weight_scales(w[1].cpu(), 2 * F, H)
    zz = torch.einsum("th,tkfh->tkf", xv.cpu(), v1[idx.cpu()])
    mag = torch.einsum("th,tkfh->tkf", xv.cpu().abs(), v1[idx.cpu()].abs())
    # 7 2^-10 of the magnitudes inside a block, binary32 sums, bf16
    assert ((z.cpu().double()[slots.cpu()] - zz).abs() <=
            7 * 2.0 ** -10 * 1.01 * mag + 2.0 ** -8 * zz.abs()).all()

    do, dwt = epl.combine_backward(dy, o, oi, wt)
    assert torch.equal(do[slots], (wt[:, :, None] * dy[:, None]).bfloat16())
    dots = dy.double()[:, None] * o.double()[slots]
    assert ((dwt.double() - dots.sum(2)).abs() <= (H + 1) * 2 * U * dots.abs().sum(2)).all()
    drows, dz = epl.gated_block_fp8_backward(do, z, *w, at, cnt, expected_rows=T * K)
    dx = epl.dispatch_backward(drows, oi)
    each = drows.double()[slots]
    assert ((dx.double() - each.sum(1)).abs() <= 4 * U * each.abs().sum(1)).all()


def silu(z):
    return z * torch.sigmoid(z)


def silu_slope(z):
    p = torch.sigmoid(z)
    return p + z * p * torch.sigmoid(-z)


def in_64_bits(w):
    return ref.decode(w[0]) * ref.weight_scales(w[1], *w[0].shape[1:])


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
@pytest.mark.parametrize("counts", [[3, 0, 2], [90, 50]])       # few rows, tiles
def test_block_gradient_against_differences_of_the_block(counts, fmt):
    """gated_block_fp8_backward against central differences of the block in 64 bits. Rows, weights
    and dy are positive, so that nothing cancels and relative errors pass through sums as they
    are; dy is its own cast."""
    H = F = 128
    E, total = len(counts), sum(counts)
    starts = [sum(counts[:e]) for e in range(E)]
    owner = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    w_fmt = "ue8m0" if fmt == "ue8m0" else "f32"
    xc, xs = ref.cast_rows(randn(total, H, seed=0, std=0.25).abs(), fmt)
    w1 = ref.cast_weight(randn(E, 2 * F, H, seed=1, std=0.1).abs(), w_fmt)
    w2 = ref.cast_weight(randn(E, H, F, seed=2, std=0.1).abs(), w_fmt)
    dyc = torch.randint(0x30, 0x7F, (total, H), generator=torch.Generator().manual_seed(3),
                        dtype=torch.uint8)
    dyc[:, 7] = 0x7E                                           # 448: the scale is 1
    dy = ref.decode(dyc)
    w = [t.to(DEV) for t in (*w1, *w2)]
    at, n = i32(starts), i32(counts)
    pre = torch.empty(total, 2 * F, dtype=torch.bfloat16, device=DEV)
    epl.gated_block_fp8(xc.to(DEV), ref.lay(xs, fmt).to(DEV), *w, at, n, pre=pre, scale_format=fmt)
    gx, gz = epl.gated_block_fp8_backward(dy.bfloat16().to(DEV), pre, *w, at, n, scale_format=fmt)

    v1, v2 = in_64_bits(w1)[owner], in_64_bits(w2)[owner]      # a row's own weights
    x = ref.decode(xc) * ref.numbers(xs)

    def value(z):
        g, u = z.chunk(2, 1)
        return ((v2 * (silu(g) * u)[:, None]).sum(2) * dy).sum(1)          # of each row

    def project(rows):
        return (v1 * rows[:, None]).sum(2)

    step = 1e-5
    v = randn(total, H, seed=4).abs().double() + 0.1
    slope = (value(project(x + step * v)) - value(project(x - step * v))) / (2 * step)
    z = project(x)
    vz = randn(total, 2 * F, seed=5).abs().double() + 0.1
    slope_z = (value(z + step * vz) - value(z - step * vz)) / (2 * step)

    # dz = [dh u silu'(g), dh silu(g)]: dh and z within 7 2^-10 each (bits inside a block; all
    # terms are positive), z rounded to bf16 (2^-8); silu(g) passes a relative error of g on at most
    # 2 times and silu'(g) at most half (g > 0); binary32 below 2^-16; dz in bf16 2^-8.
    # The differences: 1e-6.
    assert (z > 0).all()
    bits, half = 7 * 2.0 ** -10, 2.0 ** -8
    of_z = (1 + bits) * (1 + half) - 1
    of_dz = (1 + bits) * (1 + 2 * of_z) * (1 + 2.0 ** -16) - 1
    slope_of = lambda g, d: (g.cpu().double() * d).sum(1)  # noqa: E731
    err_z = (slope_of(gz, vz) - slope_z).abs()
    assert (err_z <= ((1 + of_dz) * (1 + half) - 1 + 1e-6) * slope_z).all()
    # dx: dz cast (2^-4, and 2^-10 of its scale near zero), its product and bf16 again
    g, u = z.chunk(2, 1)
    dh = (v2 * dy[:, :, None]).sum(1)
    dz = torch.cat([dh * u * silu_slope(g), dh * silu(g)], 1)
    scale = dz.view(total, 2, 128).amax(2) * (1 + of_dz) / 448 * (2 if fmt == "ue8m0" else 1)
    low = (v1 * (2.0 ** -10 * scale).repeat_interleave(128, 1)[:, :, None]).sum(1)
    rel = (1 + of_dz) * (1 + 2.0 ** -4) * (1 + bits) * (1 + half) - 1
    err = (slope_of(gx, v) - slope).abs()
    assert (err <= (rel + 1e-6) * slope + 1.02 * (low * v).sum(1)).all()


def test_both_weight_gradients():
    """dw2 and dw1 of the block, by expert_weight_grad: of w2 with the block's h cast and made
    bf16 again from the kept z, of w1 with dz and x made bf16 again. Each element within the sum
    of its terms' errors."""
    counts, H, F, total = [40, 0, 7, 90], 400, 256, 150
    starts = [2, 43, 43, 55]
    E = len(counts)
    owned = torch.zeros(total, dtype=torch.bool)
    for s, m in zip(starts, counts):
        owned[s:s + m] = True
    xc, xs = ref.cast_rows(randn(total, H, seed=0), "f32")
    xc[~owned] = 0x7F
    w1 = ref.cast_weight(randn(E, 2 * F, H, seed=1, std=H ** -0.5), "f32")
    w2 = ref.cast_weight(randn(E, H, F, seed=2, std=F ** -0.5), "f32")
    dy = randn(total, H, seed=3).bfloat16()
    dy[~owned] = float("nan")
    rows = dict(expert_start_loc=i32(starts), num_tokens_per_expert=i32(counts))
    w = [t.to(DEV) for t in (*w1, *w2)]
    x = [xc.to(DEV), xs.to(DEV)]
    pre = filled((total, 2 * F), torch.bfloat16)
    epl.gated_block_fp8(*x, *w, **rows, pre=pre)
    _, dz = epl.gated_block_fp8_backward(dy.to(DEV), pre, *w, **rows)
    h = epl.dequantize(*epl.quantize(pre, activation="swiglu", **rows), **rows)
    dw2 = epl.expert_weight_grad(dy.to(DEV), h, **rows, out_dtype=torch.float32)
    dw1 = epl.expert_weight_grad(dz, epl.dequantize(*x, **rows), **rows, out_dtype=torch.float32)
    assert dw2.shape == (E, H, F) and dw1.shape == (E, 2 * F, H)
    dw2, dw1, dz = dw2.cpu().double(), dw1.cpu().double(), dz.cpu().double()
    wide = ref.numbers(xs).repeat_interleave(128, 1)[:, :H]
    for e, (s, m) in enumerate(zip(starts, counts)):
        at = slice(s, s + m)
        if m == 0:
            assert not dw2[e].any() and not dw1[e].any()
            continue
        s1 = ref.weight_scales(w1[1], 2 * F, H)[e][:, ::128]
        z, tol = ref.product(xc[at], ref.numbers(xs)[at], w1[0][e], s1)
        tol = tol + 2.0 ** -8 * (z.abs() + tol)                # kept in bf16
        g, u = z.chunk(2, 1)
        tg, tu = tol.chunk(2, 1)
        v = silu(g) * u
        tv = 1.13 * tg * (u.abs() + tu) + silu(g).abs() * tu + 32 * U * (1 + v.abs())
        # its cast: half a step, 2^-4 of the value, or 2^-10 of its scale; then bf16
        most = ((v.abs() + tv).view(m, -1, 128).amax(2) / 448).repeat_interleave(128, 1)
        cast = tv + 2.0 ** -4 * (v.abs() + tv) + 2.0 ** -10 * most
        cast = cast + 2.0 ** -8 * (v.abs() + cast)
        d = dy[at].double()
        sums = (m + 1) * 2.0 ** -23
        lim = d.abs().t() @ cast + sums * (d.abs().t() @ (v.abs() + cast))
        assert ((dw2[e] - d.t() @ v).abs() <= lim).all()
        xv = ref.decode(xc[at]) * wide[at]
        mag = dz[at].abs().t() @ xv.abs()
        assert ((dw1[e] - dz[at].t() @ xv).abs() <= (2.0 ** -8 + sums) * 1.01 * mag).all()


@pytest.mark.parametrize("cap", [16, 48])
def test_layer_in_a_rectangle(cap):
    """The low-latency dispatch's rectangle through the block and back, as it lies: rows, results
    and weight gradients are those of the same rows packed, kernels chosen by the routed rows."""
    T, H, F, E, K = 40, 256, 128, 8, 2
    idx = torch.stack([(torch.arange(T) * 3) % E, (torch.arange(T) * 3 + 1) % E], 1).to(DEV)
    x = randn(T, H, seed=0).bfloat16().to(DEV)
    p = epl.Problem.make(T, K, E, 1, H, H // 128)
    e32 = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    out, scale, oi, cnt = filled((E, cap, H), torch.uint8), filled((E, H // 128, cap), torch.float32), \
        e32(T, K), e32(E)
    epl.epl_ll_dispatch(p, T, cap, idx, x, out, scale, cnt, e32(E, cap), e32(E, 1, 2), oi,
                        torch.empty(epl.epl_ll_workspace_bytes(p, T), dtype=torch.uint8, device=DEV))
    codes, routed = out.view(-1, H), idx.numel()
    rows = dict(expert_start_loc=cap * torch.arange(E, dtype=torch.int32, device=DEV),
                num_tokens_per_expert=cnt)
    w = [t.to(DEV) for t in (*ref.cast_weight(randn(E, 2 * F, H, seed=1, std=H ** -0.5), "f32"),
                             *ref.cast_weight(randn(E, H, F, seed=2, std=F ** -0.5), "f32"))]
    wt = torch.rand(T, K, generator=torch.Generator().manual_seed(3)).to(DEV)
    dy = randn(T, H, seed=4).to(DEV)

    def layer(codes, scale, rows, oi):
        """Forwards and back, as the documentation writes it."""
        pre = torch.empty(codes.shape[0], 2 * F, dtype=torch.bfloat16, device=DEV)
        o = epl.gated_block_fp8(codes, scale, *w, **rows, pre=pre, expected_rows=routed)
        do, dweights = epl.combine_backward(dy, o, oi, wt)
        dx, dz = epl.gated_block_fp8_backward(do, pre, *w, **rows, expected_rows=routed)
        dw1 = epl.expert_weight_grad(dz, epl.dequantize(codes, scale, **rows), **rows,
                                     out_dtype=torch.float32, expected_rows=routed)
        h = epl.dequantize(*epl.quantize(pre, activation="swiglu", **rows), **rows)
        dw2 = epl.expert_weight_grad(do, h, **rows, out_dtype=torch.float32, expected_rows=routed)
        return epl.combine(o, oi, wt), dweights, epl.dispatch_backward(dx, oi), dw1, dw2

    got = layer(codes, scale, rows, oi)
    n = cnt.cpu()
    starts = (torch.cumsum(n, 0) - n).to(DEV)
    e = (oi // cap).long()
    packed_oi = (starts[e] + oi % cap).int()
    packed, packed_scale = (torch.cat([v[i, :m] for i, m in enumerate(n.tolist())])
                            for v in (out, scale.transpose(1, 2)))
    want = layer(packed.contiguous(), packed_scale.contiguous(),
                 dict(expert_start_loc=starts.int(), num_tokens_per_expert=cnt), packed_oi)
    for a, b in zip(got, want):
        assert torch.isfinite(a.float()).all() and torch.equal(raw(a), raw(b))
