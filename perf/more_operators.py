"""Cases of the MoE layer's operators on 8-bit rows: the cast of rows and of
weights to e4m3 with a scale for each block of 128, the way back, and the
experts' matrix products on such rows and weights, with the gated activation
and the cast of its result in the epilogue, forwards and backwards. Each can
run in a plain form (elementary torch operations in 32 bits) or through the
package.

A case is one call of one operator, ``case["op"]``:

    quantize         rows [, gate] -> e4m3 codes, a scale for each 128 columns
    dequantize       codes, scales -> rows
    quantize_weight  weights -> e4m3 codes, a scale for each 128 x 128 block
    product          8-bit rows @ 8-bit weight of their expert, with bias, activation and
                     residual; result in bf16 or fp32, as codes and scales, or both

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
        # decode: gate and up projection, activation and cast in one call; weights' bytes cost
        dict(name="product, decode", op="product", experts=8, rows=64, k=7168, n=4096,
             act="swiglu", bias=False, residual=False, pre=False, transposed=False, out="none",
             codes=True, fmt="f32", spread="uniform", spare=0),
        # 2048 tokens, top-6 of 64 experts: bytes and operations in balance, whole epilogue
        dict(name="product, 64 experts", op="product", experts=64, rows=12288, k=4096, n=2048,
             act="gelu", bias=True, residual=True, pre=False, transposed=False, out="bf16",
             codes=False, fmt="f32", spread="uniform", spare=0),
        # receive side, training: gated block whose first product is kept for the way back
        dict(name="product, 32768 rows", op="product", experts=8, rows=32768, k=7168, n=4096,
             act="swiglu", bias=False, residual=False, pre=True, transposed=False, out="none",
             codes=True, fmt="f32", spread="uniform", spare=0),
        # its second product, scales that are powers of two
        dict(name="product, second, ue8m0", op="product", experts=8, rows=32768, k=2048, n=7168,
             act="none", bias=False, residual=False, pre=False, transposed=False, out="bf16",
             codes=False, fmt="ue8m0", spread="uniform", spare=0),
        # data gradient of the second product through the gated activation: bf16 for the weight
        # gradient and codes for the next product at once; uneven experts
        dict(name="product, data gradient", op="product", experts=8, rows=12289, k=7168, n=2048,
             act="swiglu_grad", bias=False, residual=False, pre=True, transposed=True,
             out="bf16", codes=True, fmt="f32", spread="skew", spare=511),
        # data gradient of the first product, decoder-sized batch of a small layer
        dict(name="product, small", op="product", experts=16, rows=500, k=640, n=512,
             act="none", bias=False, residual=False, pre=False, transposed=True, out="f32",
             codes=False, fmt="f32", spread="uniform", spare=12),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "quantize_weight", "product", "product", "product"])
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
    while True:
        experts = rng.choice([1, 2, 8, 16, 64])
        rows = _spread(rng, 1, 16384)
        k = 16 * _spread(rng, 4, 448)
        n = 16 * _spread(rng, 4, 256)
        if experts * k * n <= 64 * 4096 * 2048 and rows * k * n <= 16384 * 7168 * 2048:
            break
    act = rng.choice(["none", "silu", "gelu", "swiglu", "swiglu", "silu_grad", "gelu_grad",
                      "swiglu_grad"])
    grad = act.endswith("_grad")
    codes = rng.random() < 0.5
    if codes:                            # whole blocks of the result
        n = 256 * max(1, round(n / 256))
    return dict(op=op, experts=experts, rows=rows, k=k, n=n, act=act,
                bias=not grad and rng.random() < 0.4, residual=not grad and rng.random() < 0.3,
                pre=grad or (act != "none" and rng.random() < 0.4),
                transposed=rng.random() < (0.7 if grad else 0.2),
                out=rng.choice(["bf16", "none"]) if codes else rng.choice(["bf16", "bf16", "f32"]),
                codes=codes, fmt=rng.choice(["f32", "ue8m0", "rect"]),
                spread=rng.choice(["uniform", "skew"]), spare=rng.choice([0, 0, 37]))


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
        inv = torch.where(amax > 0, TOP / amax, 0.0)
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
        b = scale.t().contiguous().view(torch.uint8).view(rows, 4 * words)
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
    k = case["cols"] if op == "dequantize" else case["k"]
    codes, scale = _cast_rows(rows_of(total, k), fmt)
    s["x"] = codes.view(torch.uint8)
    s["x_scale"] = _lay(case, scale, _blocks_of(k))
    if op == "dequantize":
        s["y"] = torch.zeros(total, k, dtype=_DTYPE[case["dtype"]], device=dev)
        return s
    e, n, act = case["experts"], case["n"], case["act"]
    w = normal(*((e, k, n) if case["transposed"] else (e, n, k)), std=1.0 / math.sqrt(k))
    s["w"], s["w_scale"] = _cast_weight(w, "ue8m0" if fmt == "ue8m0" else "f32")
    del w
    s["b"] = normal(e, n, std=0.5) if case["bias"] else None
    cols = n // 2 if act == "swiglu" else 2 * n if act == "swiglu_grad" else n
    s["res"] = normal(total, cols, dtype=torch.bfloat16) if case["residual"] else None
    s["y"] = None if case["out"] == "none" else torch.zeros(total, cols, dtype=_DTYPE[case["out"]],
                                                            device=dev)
    s["codes"] = s["scale"] = None
    if case["codes"]:
        s["codes"] = torch.zeros(total, cols, dtype=torch.uint8, device=dev)
        s["scale"] = torch.zeros(total, cols // BLOCK, device=dev)
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


def _outputs(y, codes, scale, z):
    return [v for v in (y, None if codes is None else codes.view(torch.float8_e4m3fn), scale, z)
            if v is not None]


def _plain_product(c, s):
    act, total = c["act"], s["x"].shape[0]
    used, expert, place = _used(s, total)
    x = _decode(s["x"], _row_scales(c, s["x_scale"])[:, :_blocks_of(c["k"])])
    w = _decode_weight(s["w"], s["w_scale"])
    longest = max(s["longest"], 1)
    at = torch.arange(longest, device=x.device)
    live = at < s["counts"][:, None]
    rows = (s["starts"][:, None] + at).clamp(max=total - 1).long()
    z = torch.bmm(torch.where(live[:, :, None], x[rows], 0.0),
                  w if c["transposed"] else w.transpose(1, 2))
    z = z[expert, place.clamp(max=longest - 1)]
    if s["b"] is not None:
        z = z + s["b"][expert]
    if act == "none":
        y = z
    elif act == "swiglu":
        half = z.shape[1] // 2
        y = _silu_gelu("silu", z[:, :half]) * z[:, half:]
    elif act == "swiglu_grad":
        half = z.shape[1]
        gate, up = s["pre"][:, :half].float(), s["pre"][:, half:].float()
        y = torch.cat([z * up * _slope("silu", gate), z * _silu_gelu("silu", gate)], 1)
    elif act.endswith("_grad"):
        y = z * _slope(act[:4], s["pre"].float())
    else:
        y = _silu_gelu(act, z)
    if s["res"] is not None:
        y = y + s["res"].float()
    used = used[:, None]
    codes = scale = None
    if c["codes"]:
        codes, scale = _cast_rows(y, "f32")
        codes = torch.where(used, codes.view(torch.uint8), s["codes"])
        scale = torch.where(used, scale, s["scale"])
    kept = None
    if s["pre"] is not None and not act.endswith("_grad"):
        kept = torch.where(used, z.to(torch.bfloat16), s["pre"])
    y = None if s["y"] is None else torch.where(used, y.to(s["y"].dtype), s["y"])
    return _outputs(y, codes, scale, kept)


_PLAIN = {"quantize": _plain_quantize, "dequantize": _plain_dequantize,
          "quantize_weight": _plain_quantize_weight, "product": _plain_product}


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
    epl.expert_product_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["starts"], s["counts"],
                           bias=s["b"], activation=c["act"], residual=s["res"], pre=s["pre"],
                           out=s["y"], quantized=(s["codes"], s["scale"]) if c["codes"] else None,
                           transposed=c["transposed"], expected_rows=c["rows"])
    return _outputs(s["y"], s["codes"], s["scale"],
                    None if c["act"].endswith("_grad") else s["pre"])


_OWN = {"quantize": _own_quantize, "dequantize": _own_dequantize,
        "quantize_weight": _own_quantize_weight, "product": _own_product}


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
    e, k, n = case["experts"], case["k"], case["n"]
    used = e * (1.0 - (1.0 - 1.0 / e) ** rows)        # experts with at least one row
    act = case["act"]
    cols = n / 2 if act == "swiglu" else 2 * n if act == "swiglu_grad" else n
    out = {"none": 0, "bf16": 2, "f32": 4}[case["out"]] * cols
    if case["codes"]:
        out += cols + 4 * cols / BLOCK
    return {"bytes": rows * (k + _blocks_of(k) * per) +
            used * (n * k + _blocks_of(n) * _blocks_of(k) * per) + rows * out +
            (4 * used * n if case["bias"] else 0) + (2 * rows * cols if case["residual"] else 0) +
            (2 * rows * (cols if act.endswith("_grad") else n) if case["pre"] else 0),
            "flops": 2.0 * rows * k * n + 10 * rows * n}


# ------------------------------------------- definitions, in 64 bits --
#
# A code is held to the number that it rounds, x / scale.

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


def _exact_weight(s, e):
    w = s["w"][e].view(torch.float8_e4m3fn).double()
    sc = s["w_scale"][e]
    sc = torch.exp2(sc.double() - 127) if sc.dtype == torch.uint8 else sc.double()
    for i in range(sc.shape[0]):
        w[i * BLOCK:(i + 1) * BLOCK] *= sc[i].repeat_interleave(BLOCK)[:w.shape[1]]
    return w


def _exact_product(c, s):
    act = c["act"]
    grad = act.endswith("_grad")
    keeps = s["pre"] is not None and not grad
    total = s["x"].shape[0]
    cols = c["n"] // 2 if act == "swiglu" else 2 * c["n"] if act == "swiglu_grad" else c["n"]
    y = torch.zeros(total, cols, dtype=torch.float64, device=s["x"].device)
    pre = s["pre"].double() if keeps else None
    for e, a, b in _each(s):
        w = _exact_weight(s, e)
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
            gate, up = kept.chunk(2, 1)
            p = torch.sigmoid(gate)
            v = torch.cat([z * up * (p + gate * p * torch.sigmoid(-gate)), z * gate * p], 1)
        if s["res"] is not None:
            v = v + s["res"][a:b].double()
        y[a:b] = v
    codes = scale = None
    if c["codes"]:
        codes, scale = _exact_cast(y, "f32")
    return [v for v in (None if s["y"] is None else y, codes, scale, pre) if v is not None]


_EXACT = {"quantize": _exact_quantize, "dequantize": _exact_dequantize,
          "quantize_weight": _exact_quantize_weight, "product": _exact_product}


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))
