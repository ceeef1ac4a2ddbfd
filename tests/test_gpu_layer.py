"""A whole layer: router, dispatch, two expert products, combine, and back,
against the same layer in 64 bits under autograd; captured and replayed."""
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


def inputs(T, H, F, E, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    return dict(x=n(T, H).bfloat16().to(DEV), gate=n(E, H, std=H ** -0.5).to(DEV),
                bias=n(E, std=0.02).to(DEV), w1=n(E, 2 * F, H, std=H ** -0.5).bfloat16().to(DEV),
                b1=n(E, 2 * F, std=0.1).to(DEV), w2=n(E, H, F, std=F ** -0.5).bfloat16().to(DEV),
                dy=n(T, H).to(DEV), mask=(torch.arange(T) % 9 != 4).to(torch.uint8).to(DEV))


RULES = dict(score="sigmoid", num_groups=4, topk_groups=2, group_top=2, renormalize=True, scale=2.5)


def forward(s, K, ranks=4, alignment=0):
    E = s["w1"].shape[0]
    logits = s["x"].float() @ s["gate"].t()
    idx, w = epl.route(logits, K, bias=s["bias"], token_mask=s["mask"], **RULES)
    r = epl.dispatch(s["x"], idx, E, ranks, expert_alignment=alignment)
    at, n = r.expert_start_loc, r.num_tokens_per_expert
    slots = idx.numel()
    z = torch.empty(r.out.shape[0], s["w1"].shape[1], dtype=torch.bfloat16, device=DEV)
    h = epl.expert_product(r.out, s["w1"], at, n, bias=s["b1"], activation="swiglu", pre=z,
                           expected_rows=slots)
    v = epl.expert_product(h, s["w2"], at, n, expected_rows=slots)
    y = epl.combine(v, r.output_index, w)
    return dict(logits=logits, idx=idx, w=w, r=r, z=z, h=h, v=v, y=y)


def backward(s, f):
    r, at, n = f["r"], f["r"].expert_start_loc, f["r"].num_tokens_per_expert
    slots = f["idx"].numel()
    dv, dw = epl.combine_backward(s["dy"], f["v"], r.output_index, f["w"])
    dz = epl.expert_product(dv, s["w2"], at, n, activation="swiglu_grad", pre=f["z"],
                            transposed=True, expected_rows=slots)
    db1 = torch.empty(s["b1"].shape, device=DEV)
    dw2 = epl.expert_weight_grad(dv, f["h"], at, n, out_dtype=torch.float32)
    dw1 = epl.expert_weight_grad(dz, r.out, at, n, out_dtype=torch.float32, bias_grad=db1)
    drows = epl.expert_product(dz, s["w1"], at, n, transposed=True, expected_rows=slots)
    dx = epl.dispatch_backward(drows, r.output_index)
    dl = epl.route_backward(f["logits"], f["idx"], dw, score="sigmoid", renormalize=True, scale=2.5)
    return dict(dw1=dw1, db1=db1, dw2=dw2, dx=dx, dl=dl)


def reference(s, f, K):
    """The layer in 64 bits with the choice that the router made."""
    leaf = {k: s[k].double().requires_grad_(True) for k in ("x", "w1", "b1", "w2")}
    logits = f["logits"].double().requires_grad_(True)
    p = torch.sigmoid(logits)
    idx = f["idx"]
    chosen = torch.where(idx >= 0, p.gather(1, idx.clamp(min=0)), 0.0)
    total = chosen.sum(1, keepdim=True)
    w = 2.5 * chosen / torch.where(total > 0, total, 1.0)
    y = torch.zeros_like(leaf["x"])
    for k in range(K):
        t = torch.nonzero(idx[:, k] >= 0)[:, 0]
        e = idx[t, k]
        z = (leaf["x"][t][:, None, :] * leaf["w1"][e]).sum(2) + leaf["b1"][e]
        g, u = z.chunk(2, 1)
        v = ((g * torch.sigmoid(g) * u)[:, None, :] * leaf["w2"][e]).sum(2)
        y = y.index_add(0, t, w[t, k][:, None] * v)
    y.backward(s["dy"].double())
    return dict(y=y.detach(), dw1=leaf["w1"].grad, db1=leaf["b1"].grad, dw2=leaf["w2"].grad,
                dx=leaf["x"].grad, dl=logits.grad)


# The 2-norm of the error over the result's. Each of the roundings to bf16 on
# the way (h, v forwards; dv, dz, drows, z backwards) is off by at most 2^-8 of
# the value it rounds, so a chain of n of them and sums of such values are off
# by at most n 2^-8 of the norm with all signs against it; the layer's longest
# chain has 5 roundings, and cancellation between experts is allowed a factor
# of 2.
TOL = 2 * 5 * 2.0 ** -8


def far(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("T,K,alignment", [(1, 4, 0), (7, 4, 0), (150, 4, 16), (1500, 6, 0)])
def test_layer_forwards_and_back(T, K, alignment):
    s = inputs(T, 128, 48, 16, seed=T)
    f = forward(s, K, alignment=alignment)
    g = backward(s, f)
    ref = reference(s, f, K)
    assert far(f["y"], ref["y"]) < TOL
    for name in ("dw1", "db1", "dw2", "dx", "dl"):
        assert far(g[name], ref[name]) < TOL, name
    off = s["mask"] == 0
    assert (f["idx"][off] == -1).all() and (f["y"][off] == 0).all()
    assert (g["dx"][off] == 0).all() and (g["dl"][off] == 0).all()


def test_captured_layer_replays_like_eager():
    s = inputs(300, 128, 48, 16, seed=3)
    K, E, H, F = 4, 16, 128, 48
    T = 300
    p = epl.Problem.make(T, K, E, 4, H)
    cap = epl.epl_capacity_rows(p)
    e32 = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device=DEV)  # noqa: E731
    b16 = lambda *sh: torch.zeros(*sh, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    f32 = lambda *sh: torch.zeros(*sh, device=DEV)  # noqa: E731
    ws = torch.zeros(epl.epl_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    logits, idx, w = f32(T, E), torch.zeros(T, K, dtype=torch.int64, device=DEV), f32(T, K)
    cnt, per_rank, start, oi = e32(E), e32(4), e32(E), e32(T, K)
    in_rank = torch.zeros(T, 4, dtype=torch.uint8, device=DEV)
    rows, m, z, h, v = b16(cap, H), e32(cap), b16(cap, 2 * F), b16(cap, F), b16(cap, H)
    y, dv, dw, dz, drows = f32(T, H), b16(cap, H), f32(T, K), b16(cap, 2 * F), b16(cap, H)
    dw1, dw2, db1, dx = f32(E, 2 * F, H), f32(E, H, F), f32(E, 2 * F), f32(T, H)
    dl, ones = f32(T, E), torch.ones(T, K, device=DEV)
    router = epl.Router(T, K, E, 1, 4, 2, 2, 1, 0, 2.5, 0)
    desc = lambda i, o, layout, act, typ: epl.Product(cap, 0, E, i, o, layout, act, typ, 0)  # noqa: E731

    def step():
        epl.epl_route(router, logits, s["bias"], s["mask"], idx, w)
        epl.epl_dispatch(p, idx, s["x"], None, cap, cnt, per_rank, None, in_rank, start, None,
                         rows, None, m, oi, ws)
        epl.epl_expert_product(desc(H, 2 * F, 0, 3, 1), rows, s["w1"], s["b1"], None, start, cnt,
                               z, h)
        epl.epl_expert_product(desc(F, H, 0, 0, 1), h, s["w2"], None, None, start, cnt, None, v)
        epl.epl_combine(p, v, cap, oi, w, epl.EPL_OUT_F32, y, ws)
        epl.epl_combine_backward(p, s["dy"], v, cap, oi, w, dv, dw, ws)
        epl.epl_expert_product(desc(H, F, 1, 6, 1), dv, s["w2"], None, None, start, cnt, z, dz)
        epl.epl_expert_weight_grad(desc(F, H, 0, 0, 0), dv, h, start, cnt, False, dw2)
        epl.epl_expert_weight_grad(desc(H, 2 * F, 0, 0, 0), dz, rows, start, cnt, False, dw1, db1)
        epl.epl_expert_product(desc(2 * F, H, 1, 0, 1), dz, s["w1"], None, None, start, cnt, None,
                               drows)
        epl.epl_combine(p, drows, cap, oi, ones, epl.EPL_OUT_F32, dx, ws)
        epl.epl_route_backward(router, logits, idx, dw, dl)

    outs = (idx, w, y, dw1, dw2, db1, dx, dl)
    made = []
    for seed in (11, 12, 13):
        logits.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(seed)))
        step()
        made.append([o.clone() for o in outs])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(6):
        for o in outs:
            o.zero_()
        logits.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(11 + n % 3)))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, made[n % 3]):
            assert torch.equal(got, want)
        _ = (s["x"].float() @ s["gate"].t()).sum()          # the program's own work between
