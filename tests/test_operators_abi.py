"""Refusals of the router's, the products' and the combine gradient's C entry
points and Python wrappers, on the host only: every bad description, pointer
or tensor is rejected before anything is enqueued."""
import ctypes

import pytest

import permute_ep_layout_amd as epl

torch = pytest.importorskip("torch")

PTR = ctypes.c_void_p(1 << 20)     # aligned, never dereferenced: the calls refuse first
ODD = ctypes.c_void_p((1 << 20) + 2)
NUL = None


@pytest.fixture(scope="module")
def lib():
    epl.ensure_built()
    return epl.load()


def router(**kw):
    base = dict(num_tokens=64, num_topk=8, num_experts=256, score=0, num_groups=1, topk_groups=1,
                group_top=1, renormalize=0, logits_type=0, scale=1.0, reserved=0)
    base.update(kw)
    return epl.Router(**base)


def product(**kw):
    base = dict(num_rows=128, expected_rows=0, num_experts=8, in_cols=64, out_cols=32,
                weight_layout=0, activation=0, out_type=1, reserved=0)
    base.update(kw)
    return epl.Product(**base)


def test_struct_layouts():
    assert ctypes.sizeof(epl.Router) == 48 and epl.Router.scale.offset == 40
    assert ctypes.sizeof(epl.Product) == 48 and epl.Product.num_experts.offset == 16


@pytest.mark.parametrize("kw", [
    {}, dict(num_tokens=0), dict(num_experts=2048, num_topk=64), dict(num_experts=1, num_topk=1),
    dict(num_groups=8, topk_groups=4, group_top=2), dict(num_groups=64, topk_groups=2),
    dict(score=1, renormalize=1, logits_type=1, scale=-2.5),
])
def test_router_accepts(lib, kw):
    assert epl.epl_router_validate(router(**kw)) == epl.EPL_OK


@pytest.mark.parametrize("kw", [
    dict(num_tokens=-1), dict(num_topk=0), dict(num_topk=65), dict(num_topk=9, num_experts=8),
    dict(num_experts=0), dict(num_experts=2049), dict(score=2), dict(score=-1),
    dict(num_groups=0), dict(num_groups=7), dict(num_groups=128), dict(topk_groups=0),
    dict(num_groups=4, topk_groups=5), dict(num_groups=64, topk_groups=1), dict(group_top=0),
    dict(group_top=3), dict(renormalize=2), dict(logits_type=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(reserved=1), dict(num_tokens=1 << 31),
])
def test_router_refuses(lib, kw):
    p = router(**kw)
    assert epl.epl_router_validate(p) == epl.EPL_EINVAL
    assert lib.epl_route(ctypes.byref(p), PTR, NUL, NUL, PTR, PTR, NUL) == epl.EPL_EINVAL
    assert lib.epl_route_backward(ctypes.byref(p), PTR, PTR, PTR, PTR, NUL) == epl.EPL_EINVAL


def test_route_pointers(lib):
    p = ctypes.byref(router())
    good = [PTR, NUL, NUL, PTR, PTR]
    for i, bad in ((0, NUL), (0, ODD), (1, ODD), (3, NUL), (3, ODD), (4, NUL), (4, ODD)):
        args = list(good)
        args[i] = bad
        assert lib.epl_route(p, *args, NUL) == epl.EPL_EINVAL, i
    for i in range(4):
        for bad in (NUL, ODD):
            args = [PTR] * 4
            args[i] = bad
            assert lib.epl_route_backward(p, *args, NUL) == epl.EPL_EINVAL, i
    assert lib.epl_route(NUL, *good, NUL) == epl.EPL_EINVAL
    none = ctypes.byref(router(num_tokens=0))
    assert lib.epl_route(none, NUL, NUL, NUL, NUL, NUL, NUL) == epl.EPL_OK
    assert lib.epl_route_backward(none, NUL, NUL, NUL, NUL, NUL) == epl.EPL_OK


@pytest.mark.parametrize("kw", [
    {}, dict(num_rows=0), dict(activation=3), dict(activation=6, out_cols=24),
    dict(weight_layout=1, out_type=0), dict(in_cols=1 << 20, out_cols=512),
    dict(num_experts=2048, expected_rows=1 << 40),
])
def test_product_accepts(lib, kw):
    assert epl.epl_product_validate(product(**kw)) == epl.EPL_OK


@pytest.mark.parametrize("kw", [
    dict(num_rows=-1), dict(num_rows=1 << 31), dict(expected_rows=-1), dict(num_experts=0),
    dict(num_experts=2049), dict(in_cols=0), dict(in_cols=12), dict(in_cols=(1 << 20) + 8),
    dict(out_cols=0), dict(out_cols=20), dict(out_cols=(1 << 20) + 8),
    dict(in_cols=1 << 20, out_cols=520), dict(weight_layout=2), dict(weight_layout=-1),
    dict(activation=7), dict(activation=-1), dict(activation=3, out_cols=24), dict(out_type=2),
    dict(reserved=1),
])
def test_product_refuses(lib, kw):
    p = product(**kw)
    assert epl.epl_product_validate(p) == epl.EPL_EINVAL
    assert lib.epl_expert_product(ctypes.byref(p), *[PTR] * 9, NUL) == epl.EPL_EINVAL
    assert lib.epl_expert_weight_grad(ctypes.byref(p), PTR, PTR, PTR, PTR, 0, PTR, NUL,
                                      NUL, NUL) == epl.EPL_EINVAL


def test_product_pointers(lib):
    p = ctypes.byref(product())
    # x, weight, bias, residual, start, count, pre, y, workspace
    good = [PTR, PTR, NUL, NUL, PTR, PTR, NUL, PTR, NUL]
    bads = [(i, NUL) for i in (0, 1, 4, 5, 7)] + [(i, ODD) for i in range(9)]
    for i, bad in bads:
        args = list(good)
        args[i] = bad
        assert lib.epl_expert_product(p, *args, NUL) == epl.EPL_EINVAL, (i, bad)
    for act in (epl.EPL_ACT_SILU_GRAD, epl.EPL_ACT_GELU_GRAD, epl.EPL_ACT_SWIGLU_GRAD):
        g = ctypes.byref(product(activation=act))
        for args in ([PTR, PTR, NUL, NUL, PTR, PTR, NUL, PTR, NUL],      # no pre
                     [PTR, PTR, PTR, NUL, PTR, PTR, PTR, PTR, NUL],      # a bias
                     [PTR, PTR, NUL, PTR, PTR, PTR, PTR, PTR, NUL]):     # a residual
            assert lib.epl_expert_product(g, *args, NUL) == epl.EPL_EINVAL
    empty = ctypes.byref(product(num_rows=0))
    assert lib.epl_expert_product(empty, NUL, PTR, NUL, NUL, PTR, PTR, NUL, NUL, NUL,
                                  NUL) == epl.EPL_OK
    # grad, x, start, count, accumulate, grad_weight, grad_bias, workspace
    good = [PTR, PTR, PTR, PTR, 0, PTR, NUL, NUL]
    for i, bad in [(i, NUL) for i in (0, 1, 2, 3, 5)] + [(i, ODD) for i in (0, 1, 2, 3, 5, 6, 7)] + \
            [(4, 2), (4, -1)]:
        args = list(good)
        args[i] = bad
        assert lib.epl_expert_weight_grad(p, *args, NUL) == epl.EPL_EINVAL, (i, bad)
    for kw in (dict(activation=1), dict(weight_layout=1)):
        assert lib.epl_expert_weight_grad(ctypes.byref(product(**kw)), *good,
                                          NUL) == epl.EPL_EINVAL


def test_product_workspace_sizes(lib):
    """Partial tiles: none for few rows or a short contraction, else a header
    and at most 256 of 256 KB."""
    head = 256
    size = epl.epl_product_workspace_bytes
    assert size(product()) == 0 and size(product(in_cols=12)) == 0
    big = dict(num_rows=32768, in_cols=7168, out_cols=4096)
    assert size(product(**big)) == head + 256 * 256 * 256 * 4
    assert size(product(expected_rows=8, **big)) == 0
    parts = (800 // 128 + 8) * 2 * 2
    assert size(product(num_rows=800, in_cols=512, out_cols=256)) == head + parts * 64 * 1024
    grad = epl.epl_weight_grad_workspace_bytes
    assert grad(product(**big)) == head + 256 * 256 * 256 * 4
    assert grad(product(num_rows=800, in_cols=512, out_cols=256)) == 0
    assert grad(product(num_rows=8 * 512, in_cols=64, out_cols=512)) == head + 8 * 2 * 2 * 128 * 1024


def test_combine_backward_arguments(lib):
    p = epl.Problem.make(64, 2, 16, 8, 128)
    b = ctypes.byref(p)
    good = [0, PTR, PTR, 128, PTR, PTR, PTR, PTR, NUL]
    for i, bad in [(0, 2), (3, -1), (8, ODD)] + [(i, v) for i in (1, 2, 4, 5, 6, 7)
                                                 for v in (NUL, ODD)]:
        args = list(good)
        args[i] = bad
        assert lib.epl_combine_backward(b, *args, NUL) == epl.EPL_EINVAL, (i, bad)
    bad = epl.Problem.make(64, 2, 16, 8, 132)
    assert lib.epl_combine_backward(ctypes.byref(bad), *good, NUL) == epl.EPL_EINVAL
    none = epl.Problem.make(0, 2, 16, 8, 128)
    assert lib.epl_combine_backward(ctypes.byref(none), 0, NUL, NUL, 0, NUL, NUL, NUL, NUL, NUL,
                                    NUL) == epl.EPL_OK


def test_python_wrappers_refuse_before_the_gpu(lib):
    cpu = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        epl.route(cpu, 2)
    with pytest.raises(ValueError, match="unknown score"):
        epl.route(cpu, 2, score="relu")
    with pytest.raises(TypeError, match="float32 or"):
        epl.route(cpu.double(), 2)
    with pytest.raises(ValueError, match="2 dimensions"):
        epl.route(cpu[0], 2)
    with pytest.raises(epl.EplError):
        epl.route(cpu, 17)
    with pytest.raises(epl.EplError):
        epl.route(cpu, 2, num_groups=4, topk_groups=0)
    i32 = torch.zeros(2, dtype=torch.int32)
    x, w = torch.zeros(4, 16).bfloat16(), torch.zeros(2, 32, 16).bfloat16()
    with pytest.raises(ValueError, match="unknown activation"):
        epl.expert_product(x, w, i32, i32, activation="tanh")
    with pytest.raises(ValueError, match="3 dimensions"):
        epl.expert_product(x, w[0], i32, i32)
    with pytest.raises(TypeError, match="x must be"):
        epl.expert_product(x.float(), w, i32, i32, out=torch.zeros(4, 32))
    with pytest.raises(ValueError, match="GPU tensor"):
        epl.expert_product(x, w, i32, i32)
    with pytest.raises(ValueError, match="out is"):
        epl.expert_product(x, w, i32, i32, out=torch.zeros(4, 32), out_dtype=torch.bfloat16)
    with pytest.raises(epl.EplError):
        epl.expert_product(x, torch.zeros(2, 40, 16).bfloat16()[:, :24].contiguous(), i32, i32,
                           activation="swiglu")
    with pytest.raises(ValueError, match="accumulate needs out"):
        epl.expert_weight_grad(x, x, i32, i32, accumulate=True)
    with pytest.raises(ValueError, match="GPU tensor"):
        epl.combine_backward(torch.zeros(4, 16), x, torch.zeros(4, 1, dtype=torch.int32),
                             torch.zeros(4, 1))
