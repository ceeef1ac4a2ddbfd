"""Plain definitions of the 8-bit rows and weights, for the tests: on the CPU,
casts in the binary32 steps of their definition, products in 64 bits.
"""
import torch

GROUP = 128
TOP = 448.0


def groups(n):
    return (n + GROUP - 1) // GROUP


def two_to(byte):
    """The value of UE8M0 exponent bytes, in 64 bits."""
    v = torch.exp2(byte.double() - 127)
    return torch.where(byte == 255, torch.full_like(v, float("nan")), v)


def cast(x, fmt):
    """Codes (uint8) and scales (fp32, or uint8 exponents) of fp32 x [..., n]: one scale."""
    assert x.dtype == torch.float32
    amax = torch.nan_to_num(x.abs(), nan=0.0, posinf=float("inf")).amax(-1)
    if fmt == "ue8m0":
        bits = amax.view(torch.int32)
        b = (bits >> 23) + ((bits & 0x7FFFFF) > 0x600000).int()
        scale = torch.where(bits >= 0x7F800000, 255, (b - 8).clamp(min=1)).to(torch.uint8)
        inv = torch.where(scale == 255, 0.0, torch.exp2(127.0 - scale.double())).float()
        v = x * inv[..., None]
    else:
        scale = amax / TOP
        # 448 / amax as if binary32 had no smallest number
        up = torch.where(amax < 2.0 ** -64, 2.0 ** 64, 1.0).float()
        # (a number over a tensor is its reciprocal times the number: two roundings)
        inv = torch.where(amax > 0, torch.full_like(amax, TOP) / (amax * up), 0.0)
        v = (x * up[..., None]) * inv[..., None]
    return v.to(torch.float8_e4m3fn).view(torch.uint8), scale


def cast_rows(x, fmt):
    """Codes [rows, cols] and scales [rows, groups]."""
    rows, cols = x.shape
    s = groups(cols)
    pad = torch.nn.functional.pad(x, (0, s * GROUP - cols)).view(rows, s, GROUP)
    codes, scale = cast(pad, fmt)
    return codes.view(rows, s * GROUP)[:, :cols].contiguous(), scale


def cast_weight(w, fmt):
    e, n, k = w.shape
    nb, kb = groups(n), groups(k)
    pad = torch.nn.functional.pad(w, (0, kb * GROUP - k, 0, nb * GROUP - n))
    pad = pad.view(e, nb, GROUP, kb, GROUP).transpose(2, 3).reshape(e, nb, kb, GROUP * GROUP)
    codes, scale = cast(pad, fmt)
    codes = codes.view(e, nb, kb, GROUP, GROUP).transpose(2, 3).reshape(e, nb * GROUP, kb * GROUP)
    return codes[:, :n, :k].contiguous(), scale


def pack(scale):
    """uint8 exponents [rows, groups] -> int32 [ceil(groups / 4), rows]."""
    rows, s = scale.shape
    b = torch.nn.functional.pad(scale, (0, -s % 4)).contiguous()
    return b.view(torch.int32).t().contiguous()


def lay(scale, fmt, cap=0):
    """Row scales [rows, groups] as the operators take them."""
    if fmt == "ue8m0":
        return pack(scale)
    if fmt == "rect":
        return scale.view(-1, cap, scale.shape[1]).transpose(1, 2).contiguous()
    return scale


def decode(codes):
    return codes.view(torch.float8_e4m3fn).double()


def numbers(scale):
    return two_to(scale) if scale.dtype == torch.uint8 else scale.double()


def weight_scales(scale, n, k):
    """[E, n, k] of a weight's block scales, in 64 bits."""
    return numbers(scale).repeat_interleave(GROUP, 1)[:, :n].repeat_interleave(GROUP, 2)[:, :, :k]


def product(xc, xs, wc, ws):
    """(z, bound) of codes xc [m, k] with scales xs [m, groups], and wc [n, k]
    with full scales ws [n, groups of k], both in 64 bits: z the exact sum, and how far the
    instruction's may be.

    The instruction adds the products of 8 neighbouring k and drops of each the
    bits below 2^(E - 13), E the largest sum of two exponents in the group (a
    code's exponent is at least -6, zero's too). A product has 8 significant
    bits, so that one of at least 2^(E - 6) loses nothing and another less than
    2^(E - 13), and never more than itself. The rest are binary32 sums: 16
    groups to a block of 128, the blocks, the product of the scales and one
    fused step each: (16 + blocks + 2) full steps of 2^-23 of the magnitudes."""
    m, k = xc.shape
    n = wc.shape[0]
    pad = -k % GROUP
    xv = torch.nn.functional.pad(decode(xc), (0, pad))
    wv = torch.nn.functional.pad(decode(wc), (0, pad))
    blocks = xv.shape[1] // GROUP
    z, bound = torch.zeros(m, n).double(), torch.zeros(m, n).double()
    for b in range(blocks):
        at = slice(b * GROUP, (b + 1) * GROUP)
        x, w = xv[:, at], wv[:, at]
        s = xs[:, b][:, None] * ws[:, b][None]
        p = (x[:, None, :] * w[None]).view(m, n, 16, 8)
        low = 2.0 ** -6
        e = torch.floor(torch.log2(x.abs().clamp(min=low)))[:, None] + \
            torch.floor(torch.log2(w.abs().clamp(min=low)))[None]
        last = torch.exp2(e.view(m, n, 16, 8).amax(3, keepdim=True) - 13)
        lost = torch.where(p.abs() >= last * 128, torch.zeros_like(p), torch.minimum(p.abs(), last))
        z += p.sum((2, 3)) * s
        bound += (lost.sum((2, 3)) + (16 + blocks + 2) * 2.0 ** -23 * p.abs().sum((2, 3))) * s
    return z, bound
