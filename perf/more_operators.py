"""What is measured of a layer's norms and projections in microscaled form, and their plain forms.

Three operators around a grouped-query attention, as its server calls them, and two of them in turn:

  norm    the residual's addition and the layer's RMS norm in one pass, to bf16 or to a microscaled
          tensor, whose values are then read back
  quant   a bf16 tensor to a microscaled one (an attention's output, a projection's weights), and read back
  linear  the product of two microscaled tensors of one kind, activations [tokens][in] and weights [out][in]
  proj    norm, then the q, k and v projections of its output

A microscaled tensor holds groups of 32 consecutive values of a row as value = code * 2^e.  Kind mx8:
codes are e4m3 (a byte each), mx4: e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives: two a byte, the
even column in the low half).  e is the least whole number from -127 on with which no value of the group is
beyond the largest code (448 or 6), held as a byte e + 127; codes are rounded to nearest, ties to the
even code.  Scale bytes lie in tiles of 128 rows by 4 groups: tile (row // 128, group // 4) of 512 bytes,
byte 16 (row % 32) + 4 (row % 128 // 32) + group % 4 of it.
"""
import math
import random

import torch

own = False

EPS = 1.0e-6
TOP = {"mx8": 448.0, "mx4": 6.0}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a user's decode step: latency
        {"name": "norm_1x4096_mx8", "op": "norm", "tokens": 1, "hidden": 4096, "kind": "mx8", "add": True, "strided": False},
        # the ordinary serving batch, for projections in 16 bits
        {"name": "norm_64x4096_bf16", "op": "norm", "tokens": 64, "hidden": 4096, "kind": "bf16", "add": True, "strided": False},
        # a prompt chunk's first norm (nothing to add), rows inside a wider buffer, a width that no power of two divides
        {"name": "norm_1001x5120_mx4", "op": "norm", "tokens": 1001, "hidden": 5120, "kind": "mx4", "add": False, "strided": True},
        # a prompt batch
        {"name": "norm_8192x4096_mx8", "op": "norm", "tokens": 8192, "hidden": 4096, "kind": "mx8", "add": True, "strided": False},
        # the attention's output of the serving batch, before o_proj
        {"name": "quant_64x4096_mx4", "op": "quant", "rows": 64, "cols": 4096, "kind": "mx4", "strided": False},
        # the same of a prompt batch; or a layer's weights at load
        {"name": "quant_8192x4096_mx8", "op": "quant", "rows": 8192, "cols": 4096, "kind": "mx8", "strided": False},
        # q, k and v of one token
        {"name": "linear_1x4096x6144_mx4", "op": "linear", "tokens": 1, "in": 4096, "out": 6144, "kind": "mx4"},
        # o_proj of the serving batch
        {"name": "linear_64x4096x4096_mx8", "op": "linear", "tokens": 64, "in": 4096, "out": 4096, "kind": "mx8"},
        # a short prompt beside the batch, k or v alone
        {"name": "linear_333x4096x1024_mx4", "op": "linear", "tokens": 333, "in": 4096, "out": 1024, "kind": "mx4"},
        # the step workload's prompt chunk
        {"name": "linear_2048x4096x6144_mx8", "op": "linear", "tokens": 2048, "in": 4096, "out": 6144, "kind": "mx8"},
        # a prompt batch
        {"name": "linear_8192x4096x6144_mx4", "op": "linear", "tokens": 8192, "in": 4096, "out": 6144, "kind": "mx4"},
        # a layer's start in the serving batch's decode step
        {"name": "proj_64x4096_mx4", "op": "proj", "tokens": 64, "hidden": 4096, "kv_heads": 8, "kind": "mx4"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "linear", "linear", "linear", "proj"])
    kind = rng.choice(["mx8", "mx4"])
    wide = lambda lo, hi: 128 * _spread(rng, lo, hi)  # noqa: E731
    if op == "norm":
        kind = rng.choice(["bf16", "mx8", "mx4"])
        hidden = 8 * _spread(rng, 16, 1024) if kind == "bf16" else wide(1, 64)
        return {"op": op, "tokens": _spread(rng, 1, 8192 * 4096 // max(hidden, 4096)), "hidden": hidden, "kind": kind,
                "add": rng.random() < 0.7, "strided": rng.random() < 0.3}
    if op == "quant":
        cols = wide(1, 64)
        return {"op": op, "rows": _spread(rng, 1, 8192 * 4096 // max(cols, 4096)), "cols": cols, "kind": kind,
                "strided": rng.random() < 0.3}
    if op == "linear":
        i, o = wide(1, 64), wide(1, 64)
        return {"op": op, "tokens": _spread(rng, 1, min(8192, 8192 * 4096 * 6144 // (i * o))), "in": i, "out": o, "kind": kind}
    return {"op": op, "tokens": _spread(rng, 1, 4096), "hidden": wide(4, 32), "kv_heads": rng.choice([1, 2, 4, 8]), "kind": kind}


def _held(kind, rows, cols):
    """Bytes of a tensor of that kind."""
    return rows * cols * 2 if kind == "bf16" else rows * cols // (1 if kind == "mx8" else 2) + rows * cols // 32


def work(case):
    op, kind = case["op"], case["kind"]
    if op == "norm":
        t, h = case["tokens"], case["hidden"]
        # x (and the residual in and out), the weights, the output, and a microscaled one read back
        n = t * h * (6 if case["add"] else 2) + 2 * h + _held(kind, t, h)
        return {"bytes": n + (0 if kind == "bf16" else _held(kind, t, h) + t * h * 2), "flops": 8 * t * h}
    if op == "quant":
        r, c = case["rows"], case["cols"]
        return {"bytes": 4 * r * c + 2 * _held(kind, r, c), "flops": 4 * r * c}
    if op == "linear":
        t, i, o = case["tokens"], case["in"], case["out"]
        return {"bytes": _held(kind, t, i) + _held(kind, o, i) + t * o * 2, "flops": 2 * t * i * o}
    t, h, o = case["tokens"], case["hidden"], case["kv_heads"] * 6 * 128
    return {"bytes": t * h * 6 + 2 * h + 2 * _held(kind, t, h) + _held(kind, o, h) + t * o * 2, "flops": 2 * t * h * o}


# ------------------------------------------------------------------ the format

def _quantise(x, kind):
    """(codes as values, e) of x [rows][cols], in x's type (32 or 64 bits)."""
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    part, e = torch.frexp(top)                       # top = part * 2^e, part in [0.5, 1)
    bits, least, limit = (3, -6, 0.875) if kind == "mx8" else (1, 0, 0.75)
    e = torch.where(top > 0, e - (9 if kind == "mx8" else 3) + (part > limit).int(), -127).clamp(min=-127)
    y = torch.ldexp(g, -e[..., None])
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=least) - bits)
    return torch.round(y / step) * step, e


def _values(code, e):
    return torch.ldexp(code, e[..., None].to(code.dtype)).flatten(-2)


def _tiles(e, cols):
    """Scale bytes [rows][groups] as they lie in memory."""
    rows, groups = e.shape
    out = torch.full((-(-rows // 128) * 128, groups), 127, dtype=torch.uint8, device=e.device)
    out[:rows] = (e + 127).to(torch.uint8)
    return out.view(-1, 4, 32, groups // 4, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()


def _pack(code, e, kind):
    """The bytes of codes and scales."""
    code = code.flatten(-2)
    if kind == "mx8":
        return code.float().to(torch.float8_e4m3fn).view(torch.uint8), _tiles(e, code.shape[-1])
    levels = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], device=code.device, dtype=code.dtype)
    n = torch.searchsorted(levels, code.abs().contiguous()).to(torch.uint8) + 8 * torch.signbit(code).to(torch.uint8)
    return n[..., 0::2] + 16 * n[..., 1::2], _tiles(e, code.shape[-1])


def _unpack(codes, scales, kind, rows, cols):
    """The values of a microscaled tensor, in 32 bits."""
    if kind == "mx8":
        code = codes.view(torch.float8_e4m3fn).float()
    else:
        level = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        code = level[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    e = scales.view(-1, cols // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, cols // 32)[:rows].int() - 127
    return _values(code.unflatten(-1, (-1, 32)), e)


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)


def _stream(gen, rows, cols, strided=False):
    """A layer's activations: order 1, and some channels far larger, as a residual stream has them."""
    x = _randn(gen, rows, cols)
    loud = torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device=gen.device)
    x[:, loud] *= 24.0
    if not strided:
        return x.to(torch.bfloat16)
    wide = torch.zeros(rows, cols + 264, dtype=torch.bfloat16, device=gen.device)
    wide[:, 256:256 + cols] = x.to(torch.bfloat16)
    return wide[:, 256:256 + cols]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, kind = case["op"], case["kind"]
    s = {"op": op, "kind": kind}
    bf = dict(dtype=torch.bfloat16, device=dev)
    if op in ("norm", "proj"):
        t, h = case["tokens"], case["hidden"]
        add = case.get("add", True)
        s["x"] = _stream(gen, t, h, case.get("strided", False))
        s["residual"] = _stream(gen, t, h) if add else None
        s["w"] = (torch.rand(h, generator=gen, device=dev) + 0.5).to(torch.bfloat16)
        s["h"] = torch.empty(t, h, **bf) if add else None
        s["y"] = torch.empty(t, h, **bf)
        rows, cols = t, h
    elif op == "quant":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _stream(gen, rows, cols, case["strided"])
        s["y"] = torch.empty(rows, cols, **bf)
    else:
        rows, cols = case["tokens"], case["in"]
        s["shape"] = (rows, cols, case["out"])
        s["xm"] = _pack(*_quantise(_stream(gen, rows, cols).float(), kind), kind)
        s["wm"] = _pack(*_quantise((_randn(gen, case["out"], cols) * 0.02).to(torch.bfloat16).float(), kind), kind)
        s["y"] = torch.empty(rows, case["out"], **bf)
    g = case.get("kv_heads", 8)
    if op == "proj":
        s["shape"] = (rows, cols, 6 * g * 128)
        s["wm"] = _pack(*_quantise((_randn(gen, 6 * g * 128, cols) * 0.02).to(torch.bfloat16).float(), kind), kind)
        s["q"], s["k"], s["v"] = (torch.empty(rows, x, 128, **bf) for x in (4 * g, g, g))
    if own:
        import paged_kv_gqa_qk_gb300 as pkv
        blank = torch.zeros(2, g, 64, 128, **bf)
        s["pool"] = pkv.PagedKVPool(blank[0], blank[1], cfg=dict(heads=4 * g, kv_heads=g, max_seq=64))
        s["out"] = s["y"] if kind == "bf16" else pkv.MxTensor.empty(kind, rows, cols, device=dev)
        for name, shape in (("xm", (rows, cols)), ("wm", s.get("shape", (0, 0, 0))[2:0:-1])):
            if name in s:
                s[name] = pkv.MxTensor(kind, *shape, *s[name])
    return s


# ------------------------------------------------------------------ the operators

def _norm(s, wide):
    """The residual's sum, rounded to bf16, and its norm (unrounded, in 64 bits if `wide`)."""
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    z = h.to(torch.float64 if wide else torch.float32)
    return h, z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s["w"].to(z.dtype)


def run(s):
    """One pass.  norm: the new residual (where one is added) and the output's values; quant: the values; linear: the
    product; proj: the new residual, q, k and v."""
    op, kind = s["op"], s["kind"]
    if op == "norm":
        if own:
            s["pool"].add_norm(s["x"], s["residual"], s["w"], out=s["out"], residual_out=s["h"])
            if kind != "bf16":
                s["pool"].mx_read(s["out"], out=s["y"])
            return (s["y"],) if s["h"] is None else (s["h"], s["y"])
        h, y = _norm(s, kind != "bf16")      # (values next to a border between two codes: in 64 bits)
        if kind != "bf16":
            y = _values(*_quantise(y, kind))
        return (y.to(torch.bfloat16),) if s["residual"] is None else (h, y.to(torch.bfloat16))
    if op == "quant":
        if own:
            s["pool"].mx_quantize(s["x"], kind, out=s["out"])
            return s["pool"].mx_read(s["out"], out=s["y"])
        return _values(*_quantise(s["x"].float(), kind)).to(torch.bfloat16)
    if op == "linear":
        if own:
            return s["pool"].mx_linear(s["xm"], s["wm"], y=s["y"])
        t, i, o = s["shape"]
        x, w = _unpack(*s["xm"], kind, t, i), _unpack(*s["wm"], kind, o, i)
        return torch.matmul(x, w.T).to(torch.bfloat16)
    if own:
        s["pool"].add_norm(s["x"], s["residual"], s["w"], out=s["out"], residual_out=s["h"])
        s["pool"].mx_qkv_proj(s["out"], s["wm"], s["q"], s["k"], s["v"])
        return s["h"], s["q"], s["k"], s["v"]
    t, i, o = s["shape"]
    h, y = _norm(s, True)
    x, w = _values(*_quantise(y, kind)).float(), _unpack(*s["wm"], kind, o, i)
    y = torch.matmul(x, w.T).to(torch.bfloat16)
    q, k, v = torch.split(y, [s[n].shape[1] * 128 for n in "qkv"], 1)
    return h, q.view_as(s["q"]).contiguous(), k.view_as(s["k"]).contiguous(), v.view_as(s["v"]).contiguous()


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    dev = s["y"].device
    top = TOP.get(kind)
    two = torch.tensor([2.0 ** n for n in range(-300, 301)], dtype=torch.float64, device=dev)
    positive = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6] if kind == "mx4" else
                            [m * 2.0 ** -9 for m in range(8)] +
                            [(1 + m / 8) * 2.0 ** n for n in range(-6, 9) for m in range(8)][:-1],
                            dtype=torch.float64, device=dev)
    half = (positive[1:] + positive[:-1]) / 2

    def held(x):
        """Each value of x [rows][cols] as its group's code and scale hold it: of the codes below and above the nearer,
        between two the one with an even number."""
        out = torch.empty_like(x)
        for b in range(0, x.shape[0], 1024):
            g = x[b:b + 1024].reshape(-1, 32)
            most = g.abs().max(1, keepdim=True).values
            e = torch.ceil(torch.log2((most / top).clamp(min=2.0 ** -127))).long()
            e = torch.where(top * two[e - 1 + 300] >= most, e - 1, e)
            e = torch.where(top * two[e + 300] < most, e + 1, e).clamp(min=-127)
            y = g.abs() / two[e + 300]
            n = torch.bucketize(y, half)                       # borders below y
            tie = y == half[n.clamp(max=len(half) - 1)]
            n = torch.where(tie & (n % 2 == 1), n + 1, n)
            out[b:b + 1024] = (torch.sign(g) * positive[n] * two[e + 300]).view(-1, x.shape[1])
        return out

    def stored(m, rows, cols):
        """The values of a microscaled tensor's bytes."""
        codes, scales = (m.codes, m.scales) if own else m
        r, g = torch.arange(rows, device=dev)[:, None], torch.arange(cols // 32, device=dev)[None]
        at = (r // 128 * (cols // 128) + g // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + g % 4
        unit = two[scales.flatten().long()[at] - 127 + 300].repeat_interleave(32, 1)
        n = codes.view(rows, -1).long()
        if kind == "mx4":
            n = torch.stack([n % 16, n // 16], -1).view(rows, cols)
        size, sign = (8, 8) if kind == "mx4" else (128, 128)
        return positive[(n % size).clamp(max=len(positive) - 1)] * unit * torch.where(n >= sign, -1.0, 1.0)

    if case["op"] == "linear":
        t, i, o = s["shape"]
        return torch.mm(stored(s["xm"], t, i), stored(s["wm"], o, i).t())
    if case["op"] == "quant":
        return held(s["x"].double())
    h = s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(torch.bfloat16).double()   # (a sum of two bf16 is exact in 64 bits, or far from a border)
    y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / h.shape[1] + EPS) * s["w"].double()
    if case["op"] == "norm":
        y = y if kind == "bf16" else held(y)
        return (y,) if s["residual"] is None else (h, y)
    t, i, o = s["shape"]
    y = torch.mm(held(y), stored(s["wm"], o, i).t())
    n = [s[x].shape[1] * 128 for x in "qkv"]
    return (h, *(x.reshape(t, -1, 128) for x in torch.split(y, n, 1)))
