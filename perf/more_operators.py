"""Cases of the MoE layer's operators on 8-bit rows: the cast of rows and of
weights to e4m3 with a scale for each block of 128, the way back, the experts'
matrix products on such rows and weights, and the experts' gated feed-forward
block on them, forwards and backwards. Each can run in a plain form (elementary
torch operations in 32 bits) or through the package.

A case is one call of one operator, ``case["op"]``:

    quantize         rows [, gate] -> e4m3 codes, a scale for each 128 columns
    dequantize       codes, scales -> rows
    quantize_weight  weights -> e4m3 codes, a scale for each 128 x 128 block
    product          8-bit rows @ 8-bit weight of their expert, with bias, activation, residual
    block            8-bit rows -> gate and up projection, gated activation, its cast to 8 bits,
                     down projection
    block_grad       gradient of a block's result -> of its projections and of its rows

Codes are returned as float8_e4m3fn numbers next to their scales. Scales are
fp32 ("f32") or powers of two as exponents ("ue8m0"): of rows packed four to
an int32, column-major; of weights one byte each. "rect" is the rectangle of
the low-latency dispatch, with its own order of scales.
"""
import math

import torch

own = False

BLOCK = 128          # columns (and rows of a weight) that share a scale
TOP = 448.0          # largest e4m3 number


def listed():
    return [
        # decode: one token's hidden state before the dispatch; latency only
        dict(name="quantize, one token", op="quantize", rows=1, cols=7168, act="none",
             dtype="bf16", fmt="f32", experts=0, spare=0),
        # gated activation and cast between two products where the backward pass keeps the
        # first product's result in bf16
        dict(name="quantize, gated, 32768 rows", op="quantize", rows=32768, cols=2048,
             act="swiglu", dtype="bf16", fmt="f32", experts=8, spare=1024),
        # one low-latency batch looked at in bf16
        dict(name="dequantize, rectangle", op="dequantize", rows=64, cols=7168, dtype="bf16",
             fmt="rect", experts=8, spare=0),
        # received rows made bf16 again for the weight gradient
        dict(name="dequantize, 29765 rows", op="dequantize", rows=29765, cols=7168, dtype="bf16",
             fmt="ue8m0", experts=8, spare=0),
        # one small expert from fp32 master weights, odd sizes
        dict(name="quantize_weight, one expert", op="quantize_weight", experts=1, n=1000, k=1040,
             dtype="f32", fmt="ue8m0"),
        # a rank's gate and up projections after the optimizer's step
        dict(name="quantize_weight, 8 experts", op="quantize_weight", experts=8, n=4096, k=7168,
             dtype="bf16", fmt="f32"),
        # 2048 tokens, top-6 of 64 experts: bytes and operations in balance, whole epilogue
        dict(name="product, 64 experts", op="product", experts=64, rows=12288, k=4096, n=2048,
             act="gelu", bias=True, residual=True, pre=False, transposed=False, fmt="f32",
             spread="uniform", spare=0),
        # data gradient of a small layer's first product, a few rows behind the last expert
        dict(name="product, small", op="product", experts=16, rows=500, k=640, n=512,
             act="none", bias=False, residual=False, pre=False, transposed=True, fmt="f32",
             spread="uniform", spare=12),
        # decode: 64 routed rows over the 8 experts of a rank, in the low-latency rectangle; the
        # weights' bytes are the cost
        dict(name="block, decode", op="block", experts=8, rows=64, k=7168, f=2048, pre=False,
             fmt="rect", spread="uniform", spare=0),
        # receive side, training: 32768 rows over a rank's 8 experts; the projections are kept
        # for the way back
        dict(name="block, 32768 rows", op="block", experts=8, rows=32768, k=7168, f=2048,
             pre=True, fmt="f32", spread="uniform", spare=0),
        # a small step of fine-tuning, scales that are powers of two
        dict(name="block_grad, small", op="block_grad", experts=16, rows=500, k=640, f=256,
             fmt="ue8m0", spread="uniform", spare=0),
        # the way back through a rank's experts, unevenly filled, in a buffer with room to spare
        dict(name="block_grad, 12289 rows", op="block_grad", experts=8, rows=12289, k=7168,
             f=2048, fmt="f32", spread="skew", spare=511),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "quantize_weight", "product", "product", "block",
                     "block", "block_grad"])
    if op == "quantize":
        act = rng.choice(["none", "swiglu"])
        while True:
            rows, cols = _spread(rng, 1, 32768), 16 * _spread(rng, 1, 448)
            if rows * cols <= 32768 * 2048:
                break
        # the exponent of a result that the activation's last bit decides is no measure
        return dict(op=op, rows=rows, cols=cols, act=act, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    fmt="f32" if act == "swiglu" else rng.choice(["f32", "ue8m0"]),
                    experts=rng.choice([0, 0, 8, 64]), spare=rng.choice([0, 0, 37]))
    if op == "dequantize":
        while True:
            rows, cols = _spread(rng, 1, 32768), 16 * _spread(rng, 1, 448)
            if rows * cols <= 29765 * 7168:
                break
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f32"]),
                    fmt=rng.choice(["f32", "ue8m0", "rect"]), experts=rng.choice([8, 16, 64]),
                    spare=rng.choice([0, 37]))
    if op == "quantize_weight":
        while True:
            experts, n, k = rng.choice([1, 2, 8, 64]), 8 * _spread(rng, 1, 896), \
                16 * _spread(rng, 1, 448)
            if experts * n * k <= 8 * 4096 * 7168:
                break
        return dict(op=op, experts=experts, n=n, k=k, dtype=rng.choice(["bf16", "f32"]),
                    fmt=rng.choice(["f32", "ue8m0"]))
    experts = rng.choice([1, 2, 8, 16, 64])
    common = dict(op=op, experts=experts, spread=rng.choice(["uniform", "skew"]),
                  spare=rng.choice([0, 0, 37]))
    if op != "product":
        while True:
            rows, k, f = _spread(rng, 1, 16384), 128 * _spread(rng, 1, 56), \
                128 * _spread(rng, 1, 32)
            if experts * k * f <= 64 * 2048 * 1024 and rows * k * f <= 12289 * 7168 * 2048:
                break
        return dict(common, rows=rows, k=k, f=f,
                    fmt=rng.choice(["f32", "ue8m0"] if op == "block_grad" else
                                   ["f32", "ue8m0", "rect"]),
                    **(dict(pre=rng.random() < 0.5) if op == "block" else {}))
    while True:
        rows, k, n = _spread(rng, 1, 16384), 16 * _spread(rng, 4, 448), 16 * _spread(rng, 4, 256)
        if experts * k * n <= 64 * 4096 * 2048 and rows * k * n <= 16384 * 7168 * 2048:
            break
    act = rng.choice(["none", "silu", "gelu", "swiglu", "swiglu", "silu_grad", "gelu_grad",
                      "swiglu_grad"])
    grad = act.endswith("_grad")
    return dict(common, rows=rows, k=k, n=n, act=act, bias=not grad and rng.random() < 0.4,
                residual=not grad and rng.random() < 0.3,
                pre=grad or (act != "none" and rng.random() < 0.4),
                transposed=rng.random() < (0.7 if grad else 0.2),
                fmt=rng.choice(["f32", "ue8m0", "rect"]))


_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _blocks_of(n):
    return (n + BLOCK - 1) // BLOCK


# ------------------------------------------------- the cast, in plain steps --

def _power(amax):
    """The exponent byte of the least power of two that amax / 448 does not pass."""
    mantissa, exponent = torch.frexp(amax)                 # amax = mantissa 2^exponent
    byte = (exponent - 9 + (mantissa > 0.875).int() + 127).clamp(1, 254)
    return torch.where(amax > 0, byte, 1).int()


def _two_to(byte):
    return torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte - 127)


def _cast(x, fmt):
    """Codes (float8_e4m3fn) and one scale (a number, or an exponent byte) for each group of
    the last dimension of x [..., groups, BLOCK]."""
    amax = x.abs().amax(-1)
    if fmt == "ue8m0":
        scale = _power(amax)
        inv = 1.0 / _two_to(scale)
    else:
        scale = amax / TOP
        # (a number over a tensor is its reciprocal times the number: two roundings)
        inv = torch.where(amax > 0, torch.full_like(amax, TOP) / amax, 0.0)
    return (x * inv[..., None]).to(torch.float8_e4m3fn), scale


def _cast_rows(x, fmt):
    """Codes [rows, cols] and scales [rows, groups] of x [rows, cols]."""
    rows, cols = x.shape
    groups = _blocks_of(cols)
    pad = torch.nn.functional.pad(x, (0, groups * BLOCK - cols)).view(rows, groups, BLOCK)
    codes, scale = _cast(pad, fmt)
    return codes.view(rows, groups * BLOCK)[:, :cols].contiguous(), scale


def _pack(bytes_, words):
    """Exponent bytes [rows, groups] -> int32 [words, rows], unused bytes zero."""
    rows, groups = bytes_.shape
    b = torch.nn.functional.pad(bytes_, (0, 4 * words - groups)).view(rows, words, 4).long()
    v = b[:, :, 0] + (b[:, :, 1] << 8) + (b[:, :, 2] << 16) + (b[:, :, 3] << 24)
    return v.to(torch.int32).t().contiguous()


def _row_scales(c, scale):
    """Scales [rows, groups] as numbers, from any layout."""
    if c["fmt"] == "ue8m0":
        words, rows = scale.shape
        b = scale.t().reshape(-1).view(torch.uint8).view(rows, 4 * words)
        return _two_to(b.int())
    if c["fmt"] == "rect":
        return scale.transpose(1, 2).reshape(-1, scale.shape[1])
    return scale


def _lay(c, scale, groups):
    """Scales [rows, groups] in the layout of c["fmt"]."""
    if c["fmt"] == "ue8m0":
        return _pack(scale, (groups + 3) // 4)
    if c["fmt"] == "rect":
        return scale.view(c["experts"], -1, groups).transpose(1, 2).contiguous()
    return scale


def _decode(codes, scale):
    """Rows in fp32 from codes [rows, cols] and scales [rows, groups]."""
    cols = codes.shape[1]
    wide = scale.repeat_interleave(BLOCK, 1)[:, :cols]
    return codes.view(torch.float8_e4m3fn).float() * wide


def _cast_weight(w, fmt):
    """Codes [E, n, k] and scales [E, n / 128, k / 128] of w [E, n, k]."""
    e, n, k = w.shape
    nb, kb = _blocks_of(n), _blocks_of(k)
    pad = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - k, 0, nb * BLOCK - n))
    pad = pad.view(e, nb, BLOCK, kb, BLOCK).transpose(2, 3).reshape(e, nb, kb, BLOCK * BLOCK)
    codes, scale = _cast(pad, fmt)
    codes = codes.view(e, nb, kb, BLOCK, BLOCK).view(torch.uint8).transpose(2, 3)
    codes = codes.reshape(e, nb * BLOCK, kb * BLOCK)[:, :n, :k].contiguous()
    return codes, scale.to(torch.uint8) if fmt == "ue8m0" else scale


def _decode_weight(codes, scale):
    n, k = codes.shape[1:]
    if scale.dtype == torch.uint8:
        scale = _two_to(scale.int())
    wide = scale.repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)[:, :, :k]
    return codes.view(torch.float8_e4m3fn).float() * wide


# ----------------------------------------------------------------- inputs --

def _share(c, gen, dev):
    """How many rows each expert has, where its block starts (int32), and how many rows the
    buffers have."""
    e = c["experts"]
    odds = torch.ones(e, device=dev)
    if c.get("spread") == "skew":
        # a few experts get most rows
        odds = 1.0 / torch.arange(1, e + 1, device=dev, dtype=torch.float32).sqrt()
        odds = odds[torch.randperm(e, generator=gen, device=dev)]
    edges = torch.cumsum(odds / odds.sum(), 0)[:-1].contiguous()
    ids = torch.bucketize(torch.rand(c["rows"], generator=gen, device=dev), edges)
    counts = torch.bincount(ids, minlength=e)
    if c["fmt"] == "rect":
        # room for the largest share and eight standard deviations; a program drops the rest
        parts = sum((i + 1) ** -0.5 for i in range(e)) if c.get("spread") == "skew" else e
        most = c["rows"] / parts
        cap = min(c["rows"], int(most + 8 * math.sqrt(most)) + 8) + c["spare"]
        counts = counts.clamp(max=cap)
        starts = torch.arange(e, device=dev) * cap
        return counts.int(), starts.int(), e * cap
    starts = torch.cumsum(counts, 0) - counts
    return counts.int(), starts.int(), c["rows"] + c["spare"]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype).mul_(std)

    def rows_of(rows, cols):
        """Rows whose columns differ in size, as hidden states do."""
        x = normal(rows, cols)
        return x.mul_(torch.exp(normal(cols, std=0.5)))

    s = {"case": dict(case)}
    op, fmt = case["op"], case["fmt"]
    if op == "quantize_weight":
        s["w"] = normal(case["experts"], case["n"], case["k"], std=0.02).to(_DTYPE[case["dtype"]])
        return s
    s["counts"] = s["starts"] = None
    if case["experts"]:
        s["counts"], s["starts"], total = _share(case, gen, dev)
        s["longest"] = int(s["counts"].max())      # a program that pads knows how far
    else:
        total = case["rows"] + case["spare"]
    if op == "quantize":
        cols, groups = case["cols"], _blocks_of(case["cols"])
        wide = 2 * cols if case["act"] == "swiglu" else cols
        s["x"] = rows_of(total, wide).to(_DTYPE[case["dtype"]])
        s["codes"] = torch.zeros(total, cols, dtype=torch.uint8, device=dev)
        s["scale"] = torch.zeros((groups + 3) // 4, total, dtype=torch.int32, device=dev) \
            if fmt == "ue8m0" else torch.zeros(total, groups, device=dev)
        return s
    e = case["experts"]
    weight_fmt = "ue8m0" if fmt == "ue8m0" else "f32"

    def weight(n, k):
        return _cast_weight(normal(e, n, k, std=1.0 / math.sqrt(k)), weight_fmt)

    if op in ("block", "block_grad"):
        s["w1"], s["w1_scale"] = weight(2 * case["f"], case["k"])
        s["w2"], s["w2_scale"] = weight(case["k"], case["f"])
        s["y"] = torch.zeros(total, case["k"], dtype=torch.bfloat16, device=dev)
        s["pre"] = None
        if op == "block_grad":
            s["pre"] = normal(total, 2 * case["f"], dtype=torch.bfloat16)
            s["dy"] = rows_of(total, case["k"]).to(torch.bfloat16)
            s["dz"] = torch.zeros_like(s["pre"])
            return s
        if case["pre"]:
            s["pre"] = torch.zeros(total, 2 * case["f"], dtype=torch.bfloat16, device=dev)
    k = case["cols"] if op == "dequantize" else case["k"]
    codes, scale = _cast_rows(rows_of(total, k), fmt)
    s["x"] = codes.view(torch.uint8)
    s["x_scale"] = _lay(case, scale, _blocks_of(k))
    if op == "dequantize":
        s["y"] = torch.zeros(total, k, dtype=_DTYPE[case["dtype"]], device=dev)
    if op != "product":
        return s
    n, act = case["n"], case["act"]
    s["w"], s["w_scale"] = weight(k, n) if case["transposed"] else weight(n, k)
    s["b"] = normal(e, n, std=0.5) if case["bias"] else None
    cols = n // 2 if act == "swiglu" else 2 * n if act == "swiglu_grad" else n
    s["res"] = normal(total, cols, dtype=torch.bfloat16) if case["residual"] else None
    s["y"] = torch.zeros(total, cols, dtype=torch.bfloat16, device=dev)
    s["pre"] = None
    if act.endswith("_grad"):
        s["pre"] = normal(total, cols, dtype=torch.bfloat16)
    elif case["pre"]:
        s["pre"] = torch.zeros(total, n, dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------ plain forms --

def _used(s, total):
    """Which rows belong to an expert, their expert, and their place in its block."""
    row = torch.arange(total, device=s["starts"].device)
    expert = torch.searchsorted(s["starts"].long(), row, right=True) - 1
    # of experts that start at one place only the last can have rows
    place = row - s["starts"].long()[expert]
    return place < s["counts"].long()[expert], expert, place


def _silu_gelu(act, z):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _slope(act, z):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + \
        z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _plain_quantize(c, s):
    x = s["x"].float()
    if c["act"] == "swiglu":
        f = c["cols"]
        x = _silu_gelu("silu", x[:, :f]) * x[:, f:]
    codes, scale = _cast_rows(x, c["fmt"])
    codes = codes.view(torch.uint8)
    if s["starts"] is not None:
        used = _used(s, x.shape[0])[0][:, None]
        codes = torch.where(used, codes, s["codes"])
        scale = torch.where(used, scale, 0)
    return codes.view(torch.float8_e4m3fn), _lay(c, scale, scale.shape[1])


def _plain_dequantize(c, s):
    y = _decode(s["x"], _row_scales(c, s["x_scale"])[:, :_blocks_of(c["cols"])])
    used = _used(s, y.shape[0])[0][:, None]
    return torch.where(used, y.to(s["y"].dtype), s["y"])


def _plain_quantize_weight(c, s):
    codes, scale = _cast_weight(s["w"], c["fmt"])
    return codes.view(torch.float8_e4m3fn), scale


def _plain_rows(s, x, w, transposed):
    """z [rows, n] of fp32 rows x and fp32 weights w: each row with its expert's."""
    total = x.shape[0]
    _, expert, place = _used(s, total)
    longest = max(s["longest"], 1)
    at = torch.arange(longest, device=x.device)
    live = at < s["counts"][:, None]
    rows = (s["starts"][:, None] + at).clamp(max=total - 1).long()
    z = torch.bmm(torch.where(live[:, :, None], x[rows], 0.0),
                  w if transposed else w.transpose(1, 2))
    return z[expert, place.clamp(max=longest - 1)]


def _gate_grad(z, pre):
    """Gradient of silu(a) u with respect to pre = [a, u]."""
    half = z.shape[1]
    gate, up = pre[:, :half].float(), pre[:, half:].float()
    return torch.cat([z * up * _slope("silu", gate), z * _silu_gelu("silu", gate)], 1)


def _plain_product(c, s):
    act = c["act"]
    used, expert, _ = _used(s, s["x"].shape[0])
    x = _decode(s["x"], _row_scales(c, s["x_scale"])[:, :_blocks_of(c["k"])])
    z = _plain_rows(s, x, _decode_weight(s["w"], s["w_scale"]), c["transposed"])
    if s["b"] is not None:
        z = z + s["b"][expert]
    if act == "none":
        y = z
    elif act == "swiglu":
        half = z.shape[1] // 2
        y = _silu_gelu("silu", z[:, :half]) * z[:, half:]
    elif act == "swiglu_grad":
        y = _gate_grad(z, s["pre"])
    elif act.endswith("_grad"):
        y = z * _slope(act[:4], s["pre"].float())
    else:
        y = _silu_gelu(act, z)
    if s["res"] is not None:
        y = y + s["res"].float()
    used = used[:, None]
    y = torch.where(used, y.to(torch.bfloat16), s["y"])
    if s["pre"] is None or act.endswith("_grad"):
        return y
    return y, torch.where(used, z.to(torch.bfloat16), s["pre"])


def _again(x, fmt):
    """fp32 rows through 8 bits and back, with the scales that a block uses inside."""
    codes, scale = _cast_rows(x, fmt)
    return _decode(codes.view(torch.uint8), _two_to(scale) if fmt == "ue8m0" else scale)


def _plain_block(c, s):
    x = _decode(s["x"], _row_scales(c, s["x_scale"])[:, :_blocks_of(c["k"])])
    z = _plain_rows(s, x, _decode_weight(s["w1"], s["w1_scale"]), False)
    h = _silu_gelu("silu", z[:, :c["f"]]) * z[:, c["f"]:]
    y = _plain_rows(s, _again(h, "f32"), _decode_weight(s["w2"], s["w2_scale"]), False)
    used = _used(s, x.shape[0])[0][:, None]
    y = torch.where(used, y.to(torch.bfloat16), s["y"])
    return y if s["pre"] is None else (y, torch.where(used, z.to(torch.bfloat16), s["pre"]))


def _plain_block_grad(c, s):
    used = _used(s, s["dy"].shape[0])[0][:, None]
    dh = _plain_rows(s, _again(s["dy"].float(), "f32"), _decode_weight(s["w2"], s["w2_scale"]),
                     True)
    dz = _gate_grad(dh, s["pre"])
    dx = _plain_rows(s, _again(dz, "f32"), _decode_weight(s["w1"], s["w1_scale"]), True)
    return (torch.where(used, dx.to(torch.bfloat16), s["y"]),
            torch.where(used, dz.to(torch.bfloat16), s["dz"]))


_PLAIN = {"quantize": _plain_quantize, "dequantize": _plain_dequantize,
          "quantize_weight": _plain_quantize_weight, "product": _plain_product,
          "block": _plain_block, "block_grad": _plain_block_grad}


# -------------------------------------------------- the package's operators --

def _own_quantize(epl, c, s):
    codes, scale = epl.quantize(s["x"], activation=c["act"], scale_format=c["fmt"],
                                expert_start_loc=s["starts"], num_tokens_per_expert=s["counts"],
                                out=s["codes"], out_scale=s["scale"])
    return codes.view(torch.float8_e4m3fn), scale


def _own_dequantize(epl, c, s):
    return epl.dequantize(s["x"], s["x_scale"], expert_start_loc=s["starts"],
                          num_tokens_per_expert=s["counts"], out=s["y"])


def _own_quantize_weight(epl, c, s):
    codes, scale = epl.quantize_weight(s["w"], scale_format=c["fmt"])
    return codes.view(torch.float8_e4m3fn), scale


def _own_product(epl, c, s):
    y = epl.expert_product_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["starts"],
                               s["counts"], bias=s["b"], activation=c["act"], residual=s["res"],
                               pre=s["pre"], out=s["y"], transposed=c["transposed"],
                               expected_rows=c["rows"])
    return y if s["pre"] is None or c["act"].endswith("_grad") else (y, s["pre"])


def _own_block(epl, c, s):
    y = epl.gated_block_fp8(s["x"], s["x_scale"], s["w1"], s["w1_scale"], s["w2"], s["w2_scale"],
                            s["starts"], s["counts"], pre=s["pre"], out=s["y"],
                            expected_rows=c["rows"])
    return y if s["pre"] is None else (y, s["pre"])


def _own_block_grad(epl, c, s):
    return epl.gated_block_fp8_backward(s["dy"], s["pre"], s["w1"], s["w1_scale"], s["w2"],
                                        s["w2_scale"], s["starts"], s["counts"],
                                        grad_x=s["y"], grad_pre=s["dz"],
                                        expected_rows=c["rows"])


_OWN = {"quantize": _own_quantize, "dequantize": _own_dequantize,
        "quantize_weight": _own_quantize_weight, "product": _own_product, "block": _own_block,
        "block_grad": _own_block_grad}


def run(state):
    c = state["case"]
    if own:
        import permute_ep_layout_amd as epl
        return _OWN[c["op"]](epl, c, state)
    return _PLAIN[c["op"]](c, state)


def work(case):
    op, fmt = case["op"], case["fmt"]
    per = 1 if fmt == "ue8m0" else 4                  # bytes of a scale
    if op == "quantize_weight":
        e, n, k = case["experts"], case["n"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": e * (n * k * (size + 1) + _blocks_of(n) * _blocks_of(k) * per),
                "flops": 3 * e * n * k}
    rows = case["rows"]
    if op in ("quantize", "dequantize"):
        cols = case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        gated = case.get("act") == "swiglu"
        return {"bytes": rows * (cols * (size * (2 if gated else 1) + 1) + _blocks_of(cols) * per),
                "flops": rows * cols * (8 if gated else 3)}
    e, k = case["experts"], case["k"]
    used = e * (1.0 - (1.0 - 1.0 / e) ** rows)        # experts with at least one row
    if op in ("block", "block_grad"):
        f = case["f"]
        weights = used * 3 * (f * k + _blocks_of(f) * _blocks_of(k) * per)
        if op == "block":                             # x, y and, where it is kept, z
            return {"bytes": weights + rows * (k + _blocks_of(k) * per + 2 * k +
                                               (4 * f if case["pre"] else 0)),
                    "flops": 6.0 * rows * k * f + 20 * rows * f}
        return {"bytes": weights + rows * (4 * k + 8 * f),           # dy, dx, z, dz
                "flops": 6.0 * rows * k * f + 30 * rows * f}
    n, act = case["n"], case["act"]
    cols = n / 2 if act == "swiglu" else 2 * n if act == "swiglu_grad" else n
    return {"bytes": rows * (k + _blocks_of(k) * per) +
            used * (n * k + _blocks_of(n) * _blocks_of(k) * per) + 2 * rows * cols +
            (4 * used * n if case["bias"] else 0) + (2 * rows * cols if case["residual"] else 0) +
            (2 * rows * (cols if act.endswith("_grad") else n) if case["pre"] else 0),
            "flops": 2.0 * rows * k * n + 10 * rows * n}


# ------------------------------------------- definitions, in 64 bits --
#
# A code that is returned is held to the number that it rounds, x / scale; one that a block
# casts inside is rounded as the definition says.

def _exact_cast(x, fmt):
    """(x / scale, scale or exponent byte) by groups of 128 columns, in 64 bits."""
    rows, cols = x.shape
    out, scales = torch.empty_like(x), []
    for g in range(0, cols, BLOCK):
        part = x[:, g:g + BLOCK]
        amax = part.abs().max(dim=1, keepdim=True).values
        if fmt == "ue8m0":
            byte = torch.ceil(torch.log2(amax / TOP)).clamp(-126, 127)
            scales.append(byte + 127)
            scale = torch.exp2(byte)
        else:
            scale = amax / TOP
            scales.append(scale)
        out[:, g:g + BLOCK] = torch.where(scale > 0, part / scale, torch.zeros_like(part))
    return out, torch.cat(scales, 1)


def _each(s):
    """(expert, first row, last row + 1) of the experts that have rows."""
    for e, (n, at) in enumerate(zip(s["counts"].tolist(), s["starts"].tolist())):
        if n:
            yield e, at, at + n


def _exact_words(scales, words):
    rows, groups = scales.shape
    v = torch.zeros(words, rows, dtype=torch.int64, device=scales.device)
    for g in range(groups):
        v[g // 4] += scales[:, g].long() << (8 * (g % 4))
    return v.to(torch.int32)


def _exact_quantize(c, s):
    f, x = c["cols"], s["x"].double()
    if c["act"] == "swiglu":
        x = x[:, :f] * torch.sigmoid(x[:, :f]) * x[:, f:]
    codes, scale = _exact_cast(x, c["fmt"])
    if s["starts"] is not None:
        keep = torch.zeros(x.shape[0], 1, dtype=torch.float64, device=x.device)
        for _, a, b in _each(s):
            keep[a:b] = 1
        codes, scale = codes * keep, scale * keep
    return codes, _exact_words(scale, s["scale"].shape[0]) if c["fmt"] == "ue8m0" else scale


def _exact_rows(c, s, a, b, cols):
    """Rows a .. b - 1 of the 8-bit input, in 64 bits."""
    y = s["x"][a:b].view(torch.float8_e4m3fn).double()
    sc = s["x_scale"]
    for g in range(_blocks_of(cols)):
        if c["fmt"] == "ue8m0":
            one = torch.exp2((((sc[g // 4, a:b].long() >> (8 * (g % 4))) & 255) - 127).double())
        elif c["fmt"] == "rect":
            cap = sc.shape[2]
            one = sc[a // cap, g, a % cap:a % cap + b - a].double()
        else:
            one = sc[a:b, g].double()
        y[:, g * BLOCK:(g + 1) * BLOCK] *= one[:, None]
    return y


def _exact_dequantize(c, s):
    y = s["y"].double()
    for _, a, b in _each(s):
        y[a:b] = _exact_rows(c, s, a, b, c["cols"])
    return y


def _exact_quantize_weight(c, s):
    e, n, k = c["experts"], c["n"], c["k"]
    codes = torch.empty(e, n, k, dtype=torch.float64, device=s["w"].device)
    scale = torch.empty(e, _blocks_of(n), _blocks_of(k), dtype=torch.float64,
                        device=s["w"].device)
    for i in range(e):
        for j in range(scale.shape[1]):
            band = s["w"][i, j * BLOCK:(j + 1) * BLOCK].double()
            flat = torch.zeros(band.shape[0], scale.shape[2] * BLOCK, dtype=torch.float64,
                               device=band.device)
            flat[:, :k] = band
            amax = flat.abs().view(band.shape[0], -1, BLOCK).amax((0, 2))
            if c["fmt"] == "ue8m0":
                power = torch.ceil(torch.log2(amax / TOP)).clamp(-126, 127)
                scale[i, j], one = power + 127, torch.exp2(power)
            else:
                scale[i, j] = one = amax / TOP
            one = one.repeat_interleave(BLOCK)[:k]
            codes[i, j * BLOCK:(j + 1) * BLOCK] = torch.where(one > 0, band / one, 0.0)
    return codes, scale.to(torch.uint8) if c["fmt"] == "ue8m0" else scale


def _exact_weight(s, e, name):
    w = s[name][e].view(torch.float8_e4m3fn).double()
    sc = s[name + "_scale"][e]
    sc = torch.exp2(sc.double() - 127) if sc.dtype == torch.uint8 else sc.double()
    for i in range(sc.shape[0]):
        w[i * BLOCK:(i + 1) * BLOCK] *= sc[i].repeat_interleave(BLOCK)[:w.shape[1]]
    return w


def _exact_gate_grad(z, kept):
    gate, up = kept.double().chunk(2, 1)
    p = torch.sigmoid(gate)
    return torch.cat([z * up * (p + gate * p * torch.sigmoid(-gate)), z * gate * p], 1)


def _exact_again(x):
    """Rows through 8 bits and back: to the nearest of the 127 magnitudes, ties to even codes.
    The cast is defined in binary32 steps (x times the rounded 448 / amax): in exact numbers
    many bf16 values would lie right between two codes."""
    x = x.float()
    v, wide = torch.empty_like(x), torch.empty_like(x)
    for g in range(0, x.shape[1], BLOCK):
        part = x[:, g:g + BLOCK]
        amax = part.abs().max(dim=1, keepdim=True).values
        inv = torch.full_like(amax, TOP) / amax
        v[:, g:g + BLOCK] = torch.where(amax > 0, part * inv, torch.zeros_like(part))
        wide[:, g:g + BLOCK] = amax / TOP
    v = v.double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP) * wide.double()


def _exact_product(c, s):
    act = c["act"]
    grad = act.endswith("_grad")
    keeps = s["pre"] is not None and not grad
    y = s["y"].double()
    pre = s["pre"].double() if keeps else None
    for e, a, b in _each(s):
        w = _exact_weight(s, e, "w")
        z = _exact_rows(c, s, a, b, c["k"]) @ (w if c["transposed"] else w.t())
        if s["b"] is not None:
            z += s["b"][e].double()
        if keeps:
            pre[a:b] = z
        kept = s["pre"][a:b].double() if grad else None
        if act == "none":
            v = z
        elif act == "silu":
            v = z * torch.sigmoid(z)
        elif act == "gelu":
            v = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        elif act == "swiglu":
            gate, up = z.chunk(2, 1)
            v = gate * torch.sigmoid(gate) * up
        elif act == "silu_grad":
            p = torch.sigmoid(kept)
            v = z * (p + kept * p * torch.sigmoid(-kept))
        elif act == "gelu_grad":
            v = z * (0.5 * torch.erfc(-kept / math.sqrt(2.0)) +
                     kept * torch.exp(-kept.square() / 2) * 0.3989422804014327)
        else:
            v = _exact_gate_grad(z, kept)
        if s["res"] is not None:
            v = v + s["res"][a:b].double()
        y[a:b] = v
    return (y, pre) if keeps else y


def _exact_block(c, s):
    y = s["y"].double()
    pre = None if s["pre"] is None else s["pre"].double()
    for e, a, b in _each(s):
        z = _exact_rows(c, s, a, b, c["k"]) @ _exact_weight(s, e, "w1").t()
        if pre is not None:
            pre[a:b] = z
        gate, up = z.chunk(2, 1)
        y[a:b] = _exact_again(gate * torch.sigmoid(gate) * up) @ _exact_weight(s, e, "w2").t()
    return y if pre is None else (y, pre)


def _exact_block_grad(c, s):
    dx, dz = s["y"].double(), s["dz"].double()
    for e, a, b in _each(s):
        dh = _exact_again(s["dy"][a:b].double()) @ _exact_weight(s, e, "w2")
        dz[a:b] = _exact_gate_grad(dh, s["pre"][a:b])
        dx[a:b] = _exact_again(dz[a:b]) @ _exact_weight(s, e, "w1")
    return dx, dz


_EXACT = {"quantize": _exact_quantize, "dequantize": _exact_dequantize,
          "quantize_weight": _exact_quantize_weight, "product": _exact_product,
          "block": _exact_block, "block_grad": _exact_block_grad}


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))
