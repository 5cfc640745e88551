"""Cases of the microscaled 4-bit operators: quantisation, the product of quantised matrices, and
the products grouped by expert, each in its plain torch form and through the framework's calls.

The format: blocks of 32 neighbouring values along the contracted axis share one power of two,
2^(s - 127) with s the block's 8-bit scale code, and every value is a 4-bit float (sign, two bits of
exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6).  s is the biased binary32 exponent of the
block's largest magnitude minus 2, at least 0; 255 stands for a block that holds a NaN or an
infinity.  A value is rounded to the nearest (ties to the even code) and magnitudes above 6 give 6.

A quantised matrix of R rows and K columns is held as `codes`, uint8 [R, P / 2] (the even column in
the low four bits), and `scales`, uint8 [R, P / 32], with P = K rounded up to 128 and zeros behind K.
"""
import math

import torch

own = False

BLOCK, PAD = 32, 128
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def listed():
    return [
        # the 4-bit form of an adapter-sized matrix with odd sides: what a call costs at least
        {"name": "quantize rows, small odd", "op": "quantize", "both": False, "rows": 33, "cols": 1000, "dtype": "fp32"},
        # an embedding of 32000 x 1024 in 16-bit floats, as a serving program lays its weights out
        {"name": "quantize rows, embedding", "op": "quantize", "both": False, "rows": 32000, "cols": 1024, "dtype": "bf16"},
        # a large activation along both axes, as a training step needs it
        {"name": "quantize both axes, large", "op": "quantize", "both": True, "rows": 16384, "cols": 8192, "dtype": "bf16"},
        # serving one token through a square projection
        {"name": "product, one token", "op": "product", "m": 1, "k": 4096, "n": 4096, "dtype": "bf16"},
        # a batch of 13 sequences, one token each, through the output head, logits in 32 bits
        {"name": "product, 13 tokens, head", "op": "product", "m": 13, "k": 1024, "n": 32000, "dtype": "fp32"},
        # a short ragged prompt, sides that are no multiple of any tile
        {"name": "product, odd prompt", "op": "product", "m": 777, "k": 4104, "n": 2063, "dtype": "fp16"},
        # a long prompt or a large batch of them
        {"name": "product, long prompt", "op": "product", "m": 8192, "k": 8192, "n": 8192, "dtype": "bf16"},
        # a layer's training step: forward, the input's gradient and the weight's
        {"name": "layer step, fp32", "op": "layer", "m": 500, "k": 1024, "n": 4096, "dtype": "fp32"},
        {"name": "layer step, large", "op": "layer", "m": 8192, "k": 4096, "n": 8192, "dtype": "bf16"},
        # serving eight tokens, each sent to two of 16 experts
        {"name": "experts, eight tokens", "op": "experts", "m": 16, "k": 1024, "n": 4096, "experts": 16, "skew": 1.0, "dtype": "bf16"},
        # a prompt's tokens over 32 experts, some of them with very many and some with none
        {"name": "experts, long prompt", "op": "experts", "m": 16000, "k": 2048, "n": 4096, "experts": 32, "skew": 1.5, "dtype": "bf16"},
        # a training step of an expert layer
        {"name": "expert layer step", "op": "expert layer", "m": 8190, "k": 2048, "n": 4096, "experts": 16, "skew": 0.7, "dtype": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number, its logarithm even over the range."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "layer", "experts", "expert layer"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "quantize":
        rows, cols = _spread(rng, 1, 16384), _spread(rng, 16, 8192)
        return {"op": op, "both": rng.random() < 0.5, "rows": rows, "cols": cols, "dtype": dtype}
    if op == "product":
        m, k, n = _spread(rng, 1, 8192), _spread(rng, 32, 8192), _spread(rng, 32, 8192)
        return {"op": op, "m": m, "k": k, "n": n, "dtype": dtype}
    if op == "layer":
        m, k, n = _spread(rng, 16, 8192), _spread(rng, 64, 4096), _spread(rng, 64, 8192)
        return {"op": op, "m": m, "k": k, "n": n, "dtype": dtype}
    experts = _spread(rng, 2, 64)
    m, k, n = _spread(rng, 1, 8192), _spread(rng, 64, 2048), _spread(rng, 64, 4096)
    return {"op": op, "m": m, "k": k, "n": n, "experts": experts, "skew": round(rng.uniform(0.0, 2.0), 2), "dtype": dtype}


# ------------------------------------------------------------------ the plain form

def _padded(k):
    return -(-k // PAD) * PAD


def _power(biased):
    """2^(biased - 127) in 32 bits from its exponent field, 2^-127 (a subnormal number) for 0."""
    return torch.where(biased == 0, 1 << 22, biased << 23).to(torch.int32).view(torch.float32)


def _quantize(x):
    """[..., K] to the 4-bit values in units of their block's scale [..., B, 32] and the scale codes [..., B]."""
    x = x.float()
    x = torch.nn.functional.pad(x, (0, _padded(x.shape[-1]) - x.shape[-1])).unflatten(-1, (-1, BLOCK))
    top = x.abs().amax(-1).view(torch.int32) >> 23
    scale = torch.where(top == 255, top, (top - 2).clamp(min=0))
    m = (x * _power((254 - scale).clamp(min=1)).unsqueeze(-1)).abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).to(torch.uint8)
    return code | (torch.signbit(x).to(torch.uint8) << 3), scale.to(torch.uint8)


def _value(code, scale):
    """The 32-bit values of codes [..., B, 32] with scale codes [..., B], flattened to [..., P]."""
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=code.device)
    s = torch.where(scale == 255, math.nan, _power(scale.int()))
    return (levels[code.long()] * s.unsqueeze(-1)).flatten(-2)


def _rounded(x):
    """x [..., K] with every value replaced by the one that its 4-bit form stands for."""
    return _value(*_quantize(x))[..., : x.shape[-1]]


def _pack(x):
    code, scale = _quantize(x)
    code = code.flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), scale.contiguous()


def _unpack(codes, scales, k):
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, BLOCK))
    return _value(code, scales)[..., :k]


def _by_expert(rows, offsets, capacity):
    """Rows [T, C] laid out by expert, [E, capacity, C], zeros behind each; and each row's place there."""
    t, e = rows.shape[0], offsets.shape[0] - 1
    at = torch.arange(t, device=rows.device)
    expert = torch.searchsorted(offsets[1:].contiguous(), at, right=True)
    place = expert * capacity + (at - offsets[expert])
    out = torch.zeros(e * capacity, rows.shape[1], device=rows.device)
    out[place] = rows
    return out.view(e, capacity, -1), place


def _run_plain(s):
    dtype = s["dtype"]
    if s["op"] == "quantize":
        x = s["x"]
        outs = [_rounded(x).to(dtype)]
        if s["both"]:
            outs.append(_rounded(x.t()).to(dtype))
        return outs
    if s["op"] == "product":
        return [(_rounded(s["x"]) @ _unpack(*s["w"], s["k"]).t()).to(dtype)]
    if s["op"] == "layer":
        x, w, dy = s["x"].detach(), s["w"].detach(), s["dy"]
        y = _rounded(x) @ _rounded(w).t()
        dx = _rounded(dy) @ _rounded(w.t()).t()
        dw = _rounded(dy.t()) @ _rounded(x.t()).t()
        return [y.to(dtype), dx.to(dtype), dw.to(dtype)]
    offsets, capacity = s["offsets"].long(), s["capacity"]
    if s["op"] == "experts":
        x, place = _by_expert(_rounded(s["x"]), offsets, capacity)
        y = torch.bmm(x, _unpack(*s["w"], s["k"]).transpose(1, 2).contiguous())
        return [y.flatten(0, 1)[place].to(dtype)]
    x, w, dy = s["x"].detach(), s["w"].detach(), s["dy"]
    xe, place = _by_expert(_rounded(x), offsets, capacity)
    de, _ = _by_expert(_rounded(dy), offsets, capacity)
    y = torch.bmm(xe, _rounded(w).transpose(1, 2).contiguous())
    dx = torch.bmm(de, _rounded(w.transpose(1, 2)).transpose(1, 2).contiguous())
    xt, _ = _by_expert(x.float(), offsets, capacity)
    dt, _ = _by_expert(dy.float(), offsets, capacity)
    dw = torch.bmm(_rounded(dt.transpose(1, 2)), _rounded(xt.transpose(1, 2)).transpose(1, 2).contiguous())
    return [y.flatten(0, 1)[place].to(dtype), dx.flatten(0, 1)[place].to(dtype), dw.to(dtype)]


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    import optimizer_update_amd as ou

    if s["op"] == "quantize":
        if s["both"]:
            q, qt = ou.mx4_quantize_both(s["x"])
            return [ou.mx4_dequantize(q, s["dtype"]), ou.mx4_dequantize(qt, s["dtype"])]
        return [ou.mx4_dequantize(ou.mx4_quantize(s["x"]), s["dtype"])]
    if s["op"] == "product":
        return [ou.mx4_matmul(s["x"], ou.Mx4(*s["w"], s["k"]))]
    if s["op"] == "layer":
        y = ou.mx4_linear(s["x"], s["w"])
        return [y.detach(), *torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])]
    if s["op"] == "experts":
        return [ou.mx4_grouped_matmul(s["x"], ou.Mx4(*s["w"], s["k"]), s["offsets"])]
    y = ou.mx4_grouped_linear(s["x"], s["w"], s["offsets"])
    return [y.detach(), *torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ inputs

def _activation(shape, gen, dtype):
    """Rows of unit scale; a few columns that are 20 times as large, some rows a thousandth, one row of zeros."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.where(torch.rand(shape[-1], generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    x *= torch.where(torch.rand(shape[0], 1, generator=gen, device="cuda") < 0.05, 1e-3, 1.0)
    if shape[0] > 2:
        x[shape[0] // 2] = 0
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "dtype": dtype}
    if op == "quantize":
        s.update(both=case["both"], x=_activation((case["rows"], case["cols"]), gen, dtype))
        return s
    m, k, n = case["m"], case["k"], case["n"]
    experts = case.get("experts")
    wide = (n, k) if experts is None else (experts, n, k)
    s.update(k=k, x=_activation((m, k), gen, dtype))
    w = (torch.randn(wide, generator=gen, device="cuda") / math.sqrt(k)).to(dtype)
    if experts is not None:
        share = (torch.arange(1, experts + 1, device="cuda", dtype=torch.float32) ** -case["skew"])[torch.randperm(experts, generator=gen, device="cuda")]
        chosen = torch.multinomial(share, m, replacement=True, generator=gen)
        counts = torch.bincount(chosen, minlength=experts)
        offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = counts.cumsum(0)
        s.update(offsets=offsets, capacity=int(counts.max()))
    if op in ("product", "experts"):
        s["w"] = _pack(w)
        return s
    s["x"].requires_grad_(True)
    s.update(w=w.requires_grad_(True), dy=(torch.randn((m, n), generator=gen, device="cuda") * 1e-3).to(dtype))
    return s


def work(case):
    size = SIZE[case["dtype"]]
    held = lambda r, c: r * c * (1 / 2 + 1 / BLOCK)  # noqa: E731
    if case["op"] == "quantize":  # values in, the 4-bit form out and in again, its values out
        one = case["rows"] * case["cols"]
        axes = 2 if case["both"] else 1
        return {"bytes": one * size + axes * (2 * held(1, one) + one * size), "flops": 0}
    m, k, n, e = case["m"], case["k"], case["n"], case.get("experts", 1)
    reached = min(e, m)  # experts that have rows, at most
    if case["op"] in ("product", "experts"):
        return {"bytes": m * k * size + held(reached * n, k) + m * n * size, "flops": 2 * m * n * k}
    # values of x, w and dy in, y and both gradients out; the products themselves
    return {"bytes": size * (2 * m * k + 2 * m * n + reached * n * k + e * n * k), "flops": 6 * m * n * k}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_power(e):
    """2^e in 64 bits, e a whole number from -1022 to 1023, from the number's own exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rounded(x):
    """x [..., K] in 64 bits, each block of 32 along the last axis rounded by the definition."""
    k = x.shape[-1]
    v = x.double()
    v = torch.cat((v, v.new_zeros(*v.shape[:-1], -k % BLOCK)), -1)
    v = v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    biggest = v.abs().max(-1, keepdim=True).values
    exponent = torch.frexp(biggest).exponent - 1  # floor(log2), of a number that is not zero
    unit = _exact_power(torch.where(biggest == 0, -127, (exponent - 2).clamp(min=-127)))
    m = v.abs() / unit
    # half steps of the four binades of the format: spacing 0.5 below 2, 1 below 4, 2 above
    spacing = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    m = (torch.round(m / spacing) * spacing).clamp(max=6.0)  # round() takes ties to even
    return (torch.copysign(m, v) * unit).flatten(-2)[..., :k]


def _exact_held(codes, scales, k):
    low, high = (codes % 16).long(), (codes // 16).long()
    c = torch.stack((low, high), dim=-1).reshape(*codes.shape[:-1], -1)
    e, f = (c // 2) % 4, (c % 2).double()
    m = torch.where(e == 0, f * 0.5, (1 + f / 2) * _exact_power(e - 1))
    m = torch.where(c >= 8, -m, m)
    return (m * _exact_power(scales.long() - 127).repeat_interleave(BLOCK, dim=-1))[..., :k]


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].detach()
    if s["op"] == "quantize":
        return [_exact_rounded(x)] + ([_exact_rounded(x.t())] if s["both"] else [])
    if s["op"] == "product":
        return [torch.mm(_exact_rounded(x), _exact_held(*s["w"], s["k"]).t())]
    if s["op"] == "layer":
        w, dy = s["w"].detach(), s["dy"]
        return [
            torch.mm(_exact_rounded(x), _exact_rounded(w).t()),
            torch.mm(_exact_rounded(dy), _exact_rounded(w.t()).t()),
            torch.mm(_exact_rounded(dy.t()), _exact_rounded(x.t()).t()),
        ]
    bounds = s["offsets"].tolist()
    spans = list(zip(bounds[:-1], bounds[1:]))
    if s["op"] == "experts":
        codes, scales = s["w"]
        return [torch.cat([_exact_rounded(x[a:b]) @ _exact_held(codes[i], scales[i], s["k"]).t() for i, (a, b) in enumerate(spans)])]
    w, dy = s["w"].detach(), s["dy"]
    return [
        torch.cat([_exact_rounded(x[a:b]) @ _exact_rounded(w[i]).t() for i, (a, b) in enumerate(spans)]),
        torch.cat([_exact_rounded(dy[a:b]) @ _exact_rounded(w[i].t()).t() for i, (a, b) in enumerate(spans)]),
        torch.stack([_exact_rounded(dy[a:b].t()) @ _exact_rounded(x[a:b].t()).t() if b > a else torch.zeros_like(w[i], dtype=torch.float64) for i, (a, b) in enumerate(spans)]),
    ]
