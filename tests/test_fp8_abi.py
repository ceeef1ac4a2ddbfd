"""Refusals of the 8-bit operators' C entry points and Python wrappers, on the
host only: every bad description, pointer or tensor is rejected before
anything is enqueued."""
import ctypes

import pytest

import permute_ep_layout_amd as epl

torch = pytest.importorskip("torch")

PTR = ctypes.c_void_p(1 << 20)     # aligned, never dereferenced: the calls refuse first
ODD = ctypes.c_void_p((1 << 20) + 2)
ONE = ctypes.c_void_p((1 << 20) + 1)
NUL = None


@pytest.fixture(scope="module")
def lib():
    epl.ensure_built()
    return epl.load()


def cast(**kw):
    base = dict(num_rows=64, num_experts=0, cols=256, value_type=1, activation=0, scale_format=1,
                rows_per_expert=0, reserved=0, reserved2=0)
    base.update(kw)
    return epl.Cast(**base)


def weight(**kw):
    base = dict(num_experts=2, out_cols=300, in_cols=256, value_type=1, scale_format=1, reserved=0)
    base.update(kw)
    return epl.WeightCast(**base)


def product(**kw):
    base = dict(num_rows=128, expected_rows=0, num_experts=8, in_cols=64, out_cols=32,
                weight_layout=0, activation=0, out_type=1, scale_format=1, rows_per_expert=0,
                weight_scale_format=1, codes_scale_format=0, reserved=0, reserved2=0)
    base.update(kw)
    return epl.ProductFp8(**base)


def test_struct_layouts():
    assert ctypes.sizeof(epl.Cast) == 40 and epl.Cast.num_experts.offset == 8
    assert ctypes.sizeof(epl.WeightCast) == 24
    assert ctypes.sizeof(epl.ProductFp8) == 64 and epl.ProductFp8.scale_format.offset == 40


@pytest.mark.parametrize("kw", [
    {}, dict(num_rows=0), dict(num_experts=2048), dict(cols=16), dict(cols=1 << 20),
    dict(value_type=0), dict(activation=3), dict(scale_format=2),
    dict(scale_format=3, rows_per_expert=16), dict(num_rows=0x7FFFFFFF - 1023),
])
def test_cast_accepts(lib, kw):
    assert epl.epl_cast_validate(cast(**kw)) == epl.EPL_OK


@pytest.mark.parametrize("kw", [
    dict(num_rows=-1), dict(num_rows=0x7FFFFFFF - 1022), dict(num_experts=-1),
    dict(num_experts=2049), dict(cols=0), dict(cols=8), dict(cols=24), dict(cols=(1 << 20) + 16),
    dict(value_type=2), dict(activation=1), dict(activation=6), dict(scale_format=0),
    dict(scale_format=4), dict(scale_format=3), dict(scale_format=3, rows_per_expert=60),
    dict(rows_per_expert=16), dict(scale_format=2, rows_per_expert=16), dict(reserved=1),
    dict(reserved2=1),
])
def test_cast_refuses(lib, kw):
    p = cast(**kw)
    assert epl.epl_cast_validate(p) == epl.EPL_EINVAL
    assert lib.epl_quantize(ctypes.byref(p), *[PTR] * 5, NUL) == epl.EPL_EINVAL
    assert lib.epl_dequantize(ctypes.byref(p), *[PTR] * 5, NUL) == epl.EPL_EINVAL


def test_cast_pointers(lib):
    p, e = ctypes.byref(cast()), ctypes.byref(cast(num_experts=4))
    # x, start, count, codes, scale
    for i in (0, 3, 4):
        for bad in (NUL, ODD):
            args = [PTR] * 5
            args[i] = bad
            assert lib.epl_quantize(p, *args, NUL) == epl.EPL_EINVAL, i
    for i in range(5):
        for bad in (NUL, ODD):
            args = [PTR] * 5
            args[i] = bad
            assert lib.epl_quantize(e, *args, NUL) == epl.EPL_EINVAL, i
            assert lib.epl_dequantize(e, *args, NUL) == epl.EPL_EINVAL, i
    gated = ctypes.byref(cast(activation=3))
    assert lib.epl_dequantize(gated, *[PTR] * 5, NUL) == epl.EPL_EINVAL
    none = ctypes.byref(cast(num_rows=0))
    assert lib.epl_quantize(none, *[NUL] * 5, NUL) == epl.EPL_OK
    assert lib.epl_dequantize(none, *[NUL] * 5, NUL) == epl.EPL_OK


@pytest.mark.parametrize("kw", [{}, dict(out_cols=1), dict(in_cols=16), dict(scale_format=2),
                                dict(num_experts=2048, out_cols=1 << 20, in_cols=16)])
def test_weight_accepts(lib, kw):
    assert epl.epl_weight_cast_validate(weight(**kw)) == epl.EPL_OK


@pytest.mark.parametrize("kw", [
    dict(num_experts=0), dict(num_experts=2049), dict(out_cols=0), dict(out_cols=(1 << 20) + 1),
    dict(in_cols=0), dict(in_cols=24), dict(in_cols=(1 << 20) + 16), dict(value_type=3),
    dict(scale_format=0), dict(scale_format=3), dict(reserved=1),
    dict(num_experts=2048, out_cols=1 << 20, in_cols=1 << 20),
])
def test_weight_refuses(lib, kw):
    p = weight(**kw)
    assert epl.epl_weight_cast_validate(p) == epl.EPL_EINVAL
    assert lib.epl_quantize_weight(ctypes.byref(p), PTR, PTR, PTR, NUL) == epl.EPL_EINVAL


def test_weight_pointers(lib):
    p = ctypes.byref(weight())
    for i in range(3):
        for bad in (NUL, ODD):
            args = [PTR] * 3
            args[i] = bad
            assert lib.epl_quantize_weight(p, *args, NUL) == epl.EPL_EINVAL, i


@pytest.mark.parametrize("kw", [
    {}, dict(num_rows=0), dict(activation=3), dict(activation=6), dict(weight_layout=1),
    dict(out_type=0), dict(in_cols=1 << 20, out_cols=1024), dict(num_experts=2048),
    dict(scale_format=2, weight_scale_format=2), dict(scale_format=3, rows_per_expert=16),
    dict(out_cols=128, codes_scale_format=1), dict(out_cols=256, activation=3, codes_scale_format=2),
    dict(out_cols=128, activation=6, codes_scale_format=1), dict(in_cols=16, out_cols=16),
])
def test_product_accepts(lib, kw):
    assert epl.epl_product_fp8_validate(product(**kw)) == epl.EPL_OK


@pytest.mark.parametrize("kw", [
    dict(num_rows=-1), dict(num_rows=0x7FFFFFFF - 1022), dict(expected_rows=-1),
    dict(num_experts=0), dict(num_experts=2049), dict(in_cols=0), dict(in_cols=24),
    dict(in_cols=(1 << 20) + 16), dict(out_cols=0), dict(out_cols=24),
    dict(out_cols=(1 << 20) + 16), dict(in_cols=1 << 20, out_cols=1040), dict(weight_layout=2),
    dict(activation=7), dict(activation=-1), dict(out_type=2), dict(scale_format=0),
    dict(scale_format=3), dict(scale_format=3, rows_per_expert=100), dict(rows_per_expert=16),
    dict(weight_scale_format=0), dict(weight_scale_format=3), dict(codes_scale_format=1),
    dict(codes_scale_format=3, out_cols=128), dict(out_cols=128, activation=3, codes_scale_format=1),
    dict(out_cols=64, activation=6, codes_scale_format=1), dict(reserved=1), dict(reserved2=1),
])
def test_product_refuses(lib, kw):
    p = product(**kw)
    assert epl.epl_product_fp8_validate(p) == epl.EPL_EINVAL
    assert epl.epl_product_fp8_workspace_bytes(p) == 0
    assert lib.epl_expert_product_fp8(ctypes.byref(p), *[PTR] * 13, NUL) == epl.EPL_EINVAL


def test_product_pointers(lib):
    # x, x_scale, weight, weight_scale, bias, residual, start, count, pre, y, codes, codes_scale, ws
    plain = [PTR, PTR, PTR, PTR, NUL, NUL, PTR, PTR, NUL, PTR, NUL, NUL, NUL]
    p = ctypes.byref(product())
    bads = [(i, NUL) for i in (0, 1, 2, 3, 6, 7, 9)] + [(i, ODD) for i in range(13)] + \
        [(10, PTR), (11, PTR)]
    for i, bad in bads:
        args = list(plain)
        args[i] = bad
        assert lib.epl_expert_product_fp8(p, *args, NUL) == epl.EPL_EINVAL, (i, bad)
    both = [PTR, PTR, PTR, PTR, NUL, NUL, PTR, PTR, NUL, NUL, PTR, PTR, NUL]
    q = ctypes.byref(product(out_cols=128, codes_scale_format=1))
    for i in (10, 11):
        for bad in (NUL, ODD):
            args = list(both)
            args[i] = bad
            assert lib.epl_expert_product_fp8(q, *args, NUL) == epl.EPL_EINVAL, (i, bad)
    for act in (epl.EPL_ACT_SILU_GRAD, epl.EPL_ACT_GELU_GRAD, epl.EPL_ACT_SWIGLU_GRAD):
        g = ctypes.byref(product(activation=act))
        for i, v, kept in ((8, NUL, NUL), (4, PTR, PTR), (5, PTR, PTR)):  # no pre, bias, residual
            args = list(plain)
            args[8] = kept
            args[i] = v
            assert lib.epl_expert_product_fp8(g, *args, NUL) == epl.EPL_EINVAL
    empty = ctypes.byref(product(num_rows=0))
    args = list(plain)
    args[0] = args[1] = args[9] = NUL
    assert lib.epl_expert_product_fp8(empty, *args, NUL) == epl.EPL_OK


def test_python_wrappers_refuse_before_the_gpu(lib):
    x = torch.zeros(4, 256)
    u8 = torch.zeros(4, 256, dtype=torch.uint8)
    i32 = torch.zeros(2, dtype=torch.int32)
    w, ws = torch.zeros(2, 256, 256, dtype=torch.uint8), torch.zeros(2, 2, 2)
    xs = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        epl.quantize(x)
    with pytest.raises(ValueError, match="unknown activation"):
        epl.quantize(x, activation="silu")
    with pytest.raises(ValueError, match="unknown scale format"):
        epl.quantize(x, scale_format="e8m0")
    with pytest.raises(TypeError, match="float32 or"):
        epl.quantize(x.half())
    with pytest.raises(ValueError, match="2 dimensions"):
        epl.quantize(x[0])
    with pytest.raises(ValueError, match="even number"):
        epl.quantize(x[:, :255], activation="swiglu")
    with pytest.raises(epl.EplError):
        epl.quantize(x[:, :40].contiguous())
    with pytest.raises(TypeError, match="expert_start_loc"):
        epl.quantize(x, num_tokens_per_expert=i32)
    with pytest.raises(ValueError, match="empty"):
        epl.quantize(x, expert_start_loc=i32[:0], num_tokens_per_expert=i32[:0])
    with pytest.raises(TypeError, match="out_scale must be"):
        epl.quantize(x, out_scale=xs.double())
    with pytest.raises(ValueError, match="GPU tensor"):
        epl.dequantize(u8, xs)
    with pytest.raises(epl.EplError):                      # 4 rows are no rectangles of 3
        epl.dequantize(u8, torch.zeros(1, 2, 3))
    with pytest.raises(ValueError, match="out is"):
        epl.dequantize(u8, xs, out=x, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        epl.quantize_weight(torch.zeros(2, 8, 16))
    with pytest.raises(ValueError, match="3 dimensions"):
        epl.quantize_weight(x)
    with pytest.raises(ValueError, match="GPU tensor"):
        epl.expert_product_fp8(u8, xs, w, ws, i32, i32)
    with pytest.raises(TypeError, match="x must be"):
        epl.expert_product_fp8(x, xs, w, ws, i32, i32)
    with pytest.raises(ValueError, match="unknown scale format"):
        epl.expert_product_fp8(u8, xs, w, ws, i32, i32, quantized="bf16")
    with pytest.raises(epl.EplError):                      # half a group of columns
        epl.expert_product_fp8(u8, xs, w[:, :64].contiguous(), ws[:, :1], i32, i32, quantized="f32")
    with pytest.raises(ValueError, match="quantized scales"):
        epl.expert_product_fp8(u8, xs, w, ws, i32, i32, quantized=(u8, torch.zeros(2, 2, 2)))
    with pytest.raises(ValueError, match="3 dimensions"):
        epl.gated_block_fp8(u8, xs, w[0], ws, w, ws, i32, i32)
    with pytest.raises(ValueError, match="2 dimensions"):
        epl.gated_block_fp8_backward(x[0], None, w, ws, w, ws, i32, i32)
