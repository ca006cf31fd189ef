"""What is measured of the operators around a 4-bit key/value cache, and their plain forms.

Four operators of a grouped-query attention layer, as its server calls them:

  decode     one new token per row over a paged cache held in 4 bits: QK-norm and RoPE of q and k,
             the new k and v quantised into the cache, attention over the row's cached positions
  append     quantising a prompt's k and v into the cache as they are written, and reading the
             written positions back
  read       reading whole rows of the cache back into the page layout of a 16-bit cache
  norm_rope  QK-norm of every head and the position rotation in one pass, with half and
             interleaved pairs, a rotation of part of the head, and frequencies scaled for long
             contexts

The 4-bit cache: each head vector of 128 values is 8 groups of 16; a value is code * scale * s
with code one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives (sign, two exponent bits, one
mantissa bit), scale its group's, in 8 bits (e4m3), and s a power of two of the whole cache.
scale is max|x| / (6 s) rounded to e4m3, code x / (scale s) rounded, ties to even; x are the bf16
values that a 16-bit cache would hold.  A page of one kv head is 4 blocks of 16 positions, each of
2304 bytes: K codes [16][64], V codes [16][64], K scales [128], V scales [128]; see _maps for
where each lies.
"""
import math
import random

import torch

own = False

HEAD, PAGE, BLOCK, BLOCK_BYTES, GROUP = 128, 64, 16, 2304, 4
THETA, EPS = 1.0e6, 1.0e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a chat turn of one user: latency
        {"name": "decode_1x700", "op": "decode", "rows": 1, "lo": 700, "hi": 700, "kv_heads": 8, "idle": 0, "share": 0},
        # a small batch of short conversations on a card that holds a quarter of the heads
        {"name": "decode_24x1to640", "op": "decode", "rows": 24, "lo": 1, "hi": 640, "kv_heads": 2, "idle": 3, "share": 0},
        # the ordinary serving batch of the benchmark's sweep
        {"name": "decode_64x512to4096", "op": "decode", "rows": 64, "lo": 512, "hi": 4096, "kv_heads": 8, "idle": 0, "share": 0},
        # few rows with long contexts: the long axis is split
        {"name": "decode_8x32768to40960", "op": "decode", "rows": 8, "lo": 32768, "hi": 40960, "kv_heads": 8, "idle": 0, "share": 0},
        # the benchmark's default batch: rows of one group share the pages of a prompt prefix
        {"name": "decode_256x1024to8192", "op": "decode", "rows": 256, "lo": 1024, "hi": 8192, "kv_heads": 8, "idle": 0, "share": 16},
        # one short prompt
        {"name": "append_1x77", "op": "append", "tokens": 77, "prompts": 1, "start": 0, "kv_heads": 8, "sk": 0, "sv": 0},
        # prompt chunks of four users, continuing inside their rows
        {"name": "append_4x2048", "op": "append", "tokens": 2048, "prompts": 4, "start": 4096, "kv_heads": 8, "sk": 1, "sv": -3},
        # a throughput batch of long prompts
        {"name": "append_8x16384", "op": "append", "tokens": 16384, "prompts": 8, "start": 0, "kv_heads": 8, "sk": 0, "sv": 0},
        # a prefix brought back for the next prompt chunk
        {"name": "read_1x1000", "op": "read", "rows": 1, "lo": 1000, "hi": 1000, "kv_heads": 8},
        # many rows moved back to 16 bits
        {"name": "read_16x512to4096", "op": "read", "rows": 16, "lo": 512, "hi": 4096, "kv_heads": 8},
        # one token of a decode step whose q and k lie in one projection row
        {"name": "norm_rope_1", "op": "norm_rope", "tokens": 1, "kv_heads": 8, "packed": True, "layout": "half", "rot": 128,
         "scaling": "none", "factor": 1.0, "max_seq": 40960, "norm": True, "f32": False},
        # a prompt batch of a model with interleaved pairs, half of the head rotated, at 4 times the trained context
        {"name": "norm_rope_8192", "op": "norm_rope", "tokens": 8192, "kv_heads": 8, "packed": True, "layout": "interleaved",
         "rot": 64, "scaling": "ramp", "factor": 4.0, "max_seq": 131072, "norm": True, "f32": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "append", "read", "norm_rope"])
    g = rng.choice([1, 2, 4, 8, 8])
    if op == "decode":
        rows = _spread(rng, 1, 256)
        most = min(40960, 880000 // rows)
        hi = _spread(rng, 1, most)
        return {"op": op, "rows": rows, "lo": _spread(rng, 1, hi), "hi": hi, "kv_heads": g,
                "idle": rng.choice([0, 0, rng.randint(0, rows - 1)]), "share": rng.choice([0, 0, 4, 16])}
    if op == "append":
        tokens = _spread(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "prompts": rng.randint(1, min(tokens, 8)), "start": _spread(rng, 1, 4096) - 1,
                "kv_heads": g, "sk": rng.randint(-2, 2), "sv": rng.randint(-8, 2)}
    if op == "read":
        rows = _spread(rng, 1, 32)
        hi = _spread(rng, 1, 32768 // rows)
        return {"op": op, "rows": rows, "lo": _spread(rng, 1, hi), "hi": hi, "kv_heads": g}
    scaling = rng.choice(["none", "none", "linear", "base", "ramp"])
    return {"op": op, "tokens": _spread(rng, 1, 8192), "kv_heads": g, "packed": rng.random() < 0.5,
            "layout": rng.choice(["half", "interleaved"]), "rot": rng.choice([32, 64, 96, 128, 128]), "scaling": scaling,
            "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 2.5]), "max_seq": rng.choice([4096, 40960]),
            "norm": rng.random() < 0.8, "f32": rng.random() < 0.5}


def _lengths(case):
    """The rows' lengths (0: the row takes no step), the same for every seed."""
    r = random.Random("lengths %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["rows"])]
    for b in r.sample(range(case["rows"]), case.get("idle", 0)):
        n[b] = 0
    return n


def _shared(case, lengths):
    """Per row, the first pages that it shares with its group of `share` rows (8 to 32, before any write page)."""
    n = case.get("share", 0)
    if not n:
        return [0] * len(lengths)
    r = random.Random("shared %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    got = []
    for g0 in range(0, len(lengths), n):
        group = lengths[g0:g0 + n]
        most = min([(x - 1) // PAGE for x in group if x] or [0])
        got += [min(most, r.randint(8, 32))] * len(group)
    return got


def _chunks(case):
    """The prompts' (start, length), packed end to end."""
    r = random.Random("chunks %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    cuts = sorted(r.sample(range(1, case["tokens"]), case["prompts"] - 1))
    ends = cuts + [case["tokens"]]
    return [(r.randint(0, case["start"]), e - b) for b, e in zip([0] + cuts, ends)]


def work(case):
    g, h = case["kv_heads"], case["kv_heads"] * GROUP
    cached = 2 * g * (HEAD // 2 + HEAD // 16)          # bytes of one position's k and v in the cache
    raw = 2 * g * HEAD * 2                              # and as bf16
    if case["op"] == "decode":
        n, shared = _lengths(case), _shared(case, _lengths(case))
        steps = sum(x > 0 for x in n)
        once = sum(n)
        if case["share"]:
            for g0 in range(0, len(n), case["share"]):
                live = [s for x, s in zip(n[g0:g0 + case["share"]], shared[g0:]) if x]
                once -= PAGE * sum(live[1:])
        pages = sum(-(-x // PAGE) for x in n)
        # the cache, each row's q, k, v and table in, its outputs out, its new cache entry out and read back
        return {"bytes": once * cached + 4 * pages + steps * (2 * h * HEAD * 2 + raw + 2 * cached + raw) + 4 * len(n),
                "flops": 4 * h * HEAD * sum(n)}
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": t * (raw + cached + cached + raw + 8), "flops": 10 * t * g * HEAD}
    if case["op"] == "read":
        n = sum(_lengths(case))
        return {"bytes": n * (cached + raw + 8), "flops": 4 * n * g * HEAD}
    t = case["tokens"]
    return {"bytes": t * ((h + g) * HEAD * (2 + (4 if case["f32"] else 2)) + 4), "flops": 10 * t * (h + g) * HEAD}


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)


def _cache(gen, pages, g):
    """A cache's bytes: every code, and scales near those of values of order 1."""
    data = torch.randint(0, 256, (pages, g, PAGE // BLOCK, BLOCK_BYTES), generator=gen, device=gen.device, dtype=torch.uint8)
    data[..., 2048:] = data[..., 2048:] % 16 + 32
    return data


def _maps(dev):
    """Where a block of 16 positions keeps position i's codes (byte j of its 64: dims 2j and 2j + 1, low half first)
    and group g's scales of K and of V."""
    i, j, g = torch.arange(16, device=dev)[:, None], torch.arange(64, device=dev)[None], torch.arange(8, device=dev)[None]
    b = i // 4 % 2
    c = (i % 4) ^ b
    code = i * 64 + (j ^ (32 * (i // 2 % 2)))
    k_scale = 16 * (2 * c + b) + 4 * (g // 2) + g % 2 + 2 * (i // 8)
    v_scale = 16 * g + 4 * c + b + 2 * (i // 8)
    return {"k_code": code, "v_code": 1024 + code, "k_scale": 2048 + k_scale, "v_scale": 2176 + v_scale,
            "value": torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=dev)}


def _table(gen, lengths, shared, group, extra=0):
    """A page table over shuffled pages (page 0 is no row's), and the number of pages."""
    need = [-(-(x + extra) // PAGE) for x in lengths]
    width, used = max(1, max(need)), 0
    owner = {}
    rows = []
    for b, n in enumerate(need):
        s = min(shared[b], n)
        key = b // group if group else None
        if s and key not in owner:
            owner[key] = list(range(used, used + s))
            used += s
        rows.append((owner[key] if s else []) + list(range(used, used + n - s)))
        used += n - s
    place = torch.randperm(used, generator=torch.Generator().manual_seed(int(gen.initial_seed() % (1 << 31)))) + 1
    flat = torch.zeros(len(lengths), width, dtype=torch.int32)
    for b, r in enumerate(rows):
        if r:
            flat[b, :len(r)] = place[r].to(torch.int32)
    return flat.to(gen.device), used + 1


def _weights(gen):
    return (torch.rand(HEAD, generator=gen, device=gen.device) + 0.5).to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    g, h = case["kv_heads"], case["kv_heads"] * GROUP
    s = {"op": case["op"], "g": g, "maps": _maps(dev)}
    if case["op"] == "decode":
        n = _lengths(case)
        s["table"], pages = _table(gen, n, _shared(case, n), case["share"])
        s["data"] = _cache(gen, pages, g)
        s["positions"] = torch.tensor([x - 1 for x in n], dtype=torch.int32, device=dev)
        r = len(n)
        s["q"], s["k"], s["v"] = (_randn(gen, r, x, HEAD).to(torch.bfloat16) for x in (h, g, g))
        s["qw"], s["kw"] = _weights(gen), _weights(gen)
        s["out"] = torch.empty_like(s["q"])
        s["k_new"], s["v_new"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        s["ks"] = s["vs"] = 1.0
    elif case["op"] == "append":
        chunks = _chunks(case)
        ends = [b + n for b, n in chunks]
        s["table"], pages = _table(gen, ends, [0] * len(ends), 0)
        s["data"] = _cache(gen, pages, g)
        s["positions"] = torch.cat([torch.arange(b, b + n, dtype=torch.int32) for b, n in chunks]).to(dev)
        s["prow"] = torch.cat([torch.full((n,), r, dtype=torch.int32) for r, (b, n) in enumerate(chunks)]).to(dev)
        t = case["tokens"]
        s["ks"], s["vs"] = 2.0 ** case["sk"], 2.0 ** case["sv"]
        s["k"], s["v"] = _randn(gen, t, g, HEAD).to(torch.bfloat16), (_randn(gen, t, g, HEAD) * s["vs"]).to(torch.bfloat16)
        s["kw"] = _weights(gen)
        s["k_new"], s["v_new"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    elif case["op"] == "read":
        n = _lengths(case)
        s["table"], pages = _table(gen, n, [0] * len(n), 0)
        s["data"] = _cache(gen, pages, g)
        s["ks"], s["vs"] = 1.0, 0.125
        s["positions"] = torch.cat([torch.arange(x, dtype=torch.int32) for x in n]).to(dev)
        s["prow"] = torch.cat([torch.full((x,), b, dtype=torch.int32) for b, x in enumerate(n)]).to(dev)
        s["K"], s["V"] = (torch.empty(g, sum(n), HEAD, dtype=torch.bfloat16, device=dev) for _ in range(2))
    else:
        t = case["tokens"]
        if case["packed"]:  # a row of the projection: q, k and v of one token
            row = _randn(gen, t, (h + 2 * g) * HEAD).to(torch.bfloat16)
            s["q"], s["k"] = row[:, :h * HEAD].view(t, h, HEAD), row[:, h * HEAD:(h + g) * HEAD].view(t, g, HEAD)
        else:
            s["q"], s["k"] = _randn(gen, t, h, HEAD).to(torch.bfloat16), _randn(gen, t, g, HEAD).to(torch.bfloat16)
        s["qw"], s["kw"] = (_weights(gen), _weights(gen)) if case["norm"] else (None, None)
        start = int(torch.randint(0, case["max_seq"] - min(t, case["max_seq"]) + 1, (1,), generator=gen, device=dev))
        s["positions"] = ((start + torch.arange(t, device=dev)) % case["max_seq"]).to(torch.int32)
        s["layout"], s["rot"] = case["layout"], case["rot"]
        s["scaling"], s["factor"], s["trained"] = case["scaling"], case["factor"], case["max_seq"] / case["factor"]
        kind = torch.float32 if case["f32"] else torch.bfloat16
        s["q_out"], s["k_out"] = (torch.empty(t, x, HEAD, dtype=kind, device=dev) for x in (h, g))
    if own:
        import paged_kv_gqa_qk_gb300 as pkv
        if case["op"] == "norm_rope":
            blank = torch.zeros(2, g, PAGE, HEAD, dtype=torch.bfloat16, device=dev)
            s["pool"] = pkv.PagedKVPool(blank[0], blank[1], cfg=dict(heads=h, kv_heads=g, max_seq=case["max_seq"], rotary_dim=case["rot"]))
            if case["scaling"] != "none":
                s["pool"].set_rope(*pkv.pkv_rope_frequencies(s["pool"].cfg, case["scaling"], case["factor"], int(s["trained"])))
        else:
            s["pool"] = pkv.Q4KVPool(s["data"], cfg=dict(heads=h, kv_heads=g, max_seq=PAGE * s["table"].shape[1]),
                                     k_scale=s["ks"], v_scale=s["vs"])
    return s


# ------------------------------------------------------------------ plain forms

def _angles(s, pos, rot):
    """cos and sin of each rotated pair, in 64 bits, and the factor on both."""
    i = torch.arange(rot // 2, device=pos.device, dtype=torch.float64)
    base, factor = THETA, s.get("factor", 1.0)
    kind = s.get("scaling", "none")
    if kind == "base":
        base = THETA * factor ** (rot / (rot - 2.0))
    freq = base ** (-2.0 * i / rot)
    more = 1.0
    if kind == "linear":
        freq = freq / factor
    if kind == "ramp":
        trained = float(int(s["trained"]))
        at = [rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(THETA)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        freq = freq / factor * ramp + freq * (1 - ramp)
        more = 0.1 * math.log(factor) + 1
    a = pos.to(torch.float64)[:, None] * freq
    return torch.cos(a) * more, torch.sin(a) * more


def _norm_rope(x, w, cos, sin, rot, layout="half"):
    """x [tokens][heads][128], in its type: normed over the head (w not None) and its first `rot` dims rotated."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    c, n = cos.to(x.dtype)[:, None], sin.to(x.dtype)[:, None]
    r = x[..., :rot]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _codes(x, s):
    """x [..., 128] bf16 values: (bytes of codes [..., 64], scale bytes [..., 8]) of a cache whose power of two is s."""
    y = x.double().unflatten(-1, (8, 16))
    top = y.abs().amax(-1)
    # (torch divides by a number by multiplying with its rounded inverse, which moves ties)
    scale = (top / torch.full_like(top, 6 * s)).clamp(max=448).float().to(torch.float8_e4m3fn)
    step = scale.double() * s
    y = torch.where(step[..., None] > 0, y / torch.where(step > 0, step, 1.0)[..., None], y * 0)
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).to(torch.uint8)
    code = code + torch.signbit(y).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] + code[..., 1::2] * 16, scale.view(torch.uint8)


def _values(block, m, which, s):
    """The values [..., 16, 128] of the K or V of blocks [..., 2304], in 32 bits."""
    code = block[..., m[which + "_code"]]
    code = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    scale = block[..., m[which + "_scale"]].view(torch.float8_e4m3fn).float() * s
    return (m["value"][code.int()].unflatten(-1, (8, 16)) * scale[..., None]).flatten(-2)


def _write(s, page, pos, which, x):
    """Quantises x [tokens][g][128] (bf16) into the cache at (page, pos % 64) of each token."""
    code, scale = _codes(x, s[which + "s"])
    block, i = pos % PAGE // BLOCK, pos % BLOCK
    m, head = s["maps"], torch.arange(s["g"], device=pos.device)
    at = (page[:, None, None], head[None, :, None], block[:, None, None])
    s["data"][(*at, m[which + "_code"][i][:, None])] = code
    s["data"][(*at, m[which + "_scale"][i][:, None])] = scale


def _read(s, page, pos):
    """The cached k and v of each token, bf16 [tokens][g][128]."""
    block, i = s["data"][page, :, pos % PAGE // BLOCK], pos % BLOCK
    m, got = s["maps"], []
    for which in ("k", "v"):
        code = torch.gather(block, 2, m[which + "_code"][i][:, None].expand(-1, s["g"], -1))
        code = torch.stack([code & 15, code >> 4], -1).flatten(-2)
        scale = torch.gather(block, 2, m[which + "_scale"][i][:, None].expand(-1, s["g"], -1)).view(torch.float8_e4m3fn).float()
        v = m["value"][code.int()].unflatten(-1, (8, 16)) * scale[..., None] * s[which + "s"]
        got.append(v.flatten(-2).to(torch.bfloat16))
    return got


def _decode(s):
    pos, g = s["positions"].long(), s["g"]
    live = pos >= 0
    at = pos.clamp(min=0)
    rows = torch.arange(len(pos), device=pos.device)
    cos, sin = _angles(s, at, HEAD)
    q = _norm_rope(s["q"].float(), s["qw"], cos, sin, HEAD)
    k = _norm_rope(s["k"].double(), s["kw"], cos, sin, HEAD).to(torch.bfloat16)
    page = s["table"].long()[rows, at // PAGE]  # a row without a step has page 0, which is no row's
    _write(s, page, at, "k", k)
    _write(s, page, at, "v", s["v"])
    block = s["data"][s["table"].long()]        # [rows][pages][g][4][2304]
    r, w = block.shape[:2]
    key = _values(block, s["maps"], "k", s["ks"]).permute(0, 2, 1, 3, 4, 5).reshape(r, g, w * PAGE, HEAD)
    score = torch.matmul(q.view(r, g, GROUP, HEAD), key.transpose(2, 3)) / math.sqrt(HEAD)
    del key
    seen = torch.arange(w * PAGE, device=pos.device)[None] <= pos[:, None]
    score = torch.where(seen[:, None, None], score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    value = _values(block, s["maps"], "v", s["vs"]).permute(0, 2, 1, 3, 4, 5).reshape(r, g, w * PAGE, HEAD)
    out = torch.matmul(p, value) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    k_new, v_new = _read(s, page, at)
    return (out.view(r, g * GROUP, HEAD).to(torch.bfloat16),
            torch.where(live[:, None, None], k_new, 0), torch.where(live[:, None, None], v_new, 0))


def run(s):
    """One pass.  decode: the outputs and the rows' new cache entries, read back; append: the written entries, read
    back; read: the rows' k and v, packed end to end, [kv_heads][positions][128]; norm_rope: q and k."""
    if s["op"] == "decode":
        if own:
            s["pool"].decode(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["positions"], s["table"], out=s["out"])
            s["pool"].read(s["positions"], None, s["table"], s["k_new"], s["v_new"])
            return s["out"], s["k_new"], s["v_new"]
        return _decode(s)
    if s["op"] == "append":
        if own:
            s["pool"].append(s["k"], s["v"], s["kw"], s["positions"], s["prow"], s["table"])
            s["pool"].read(s["positions"], s["prow"], s["table"], s["k_new"], s["v_new"])
            return s["k_new"], s["v_new"]
        pos = s["positions"].long()
        page = s["table"].long()[s["prow"].long(), pos // PAGE]
        cos, sin = _angles(s, pos, HEAD)
        _write(s, page, pos, "k", _norm_rope(s["k"].double(), s["kw"], cos, sin, HEAD).to(torch.bfloat16))
        _write(s, page, pos, "v", s["v"])
        return _read(s, page, pos)
    if s["op"] == "read":
        if own:
            s["pool"].read(s["positions"], s["prow"], s["table"], s["K"].transpose(0, 1), s["V"].transpose(0, 1))
            return s["K"], s["V"]
        pos = s["positions"].long()
        page = s["table"].long()[s["prow"].long(), pos // PAGE]
        return [x.transpose(0, 1).contiguous() for x in _read(s, page, pos)]
    if own:
        s["pool"].norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["positions"], layout=s["layout"], q_out=s["q_out"], k_out=s["k_out"])
        return s["q_out"], s["k_out"]
    cos, sin = _angles(s, s["positions"], s["rot"])
    return (_norm_rope(s["q"].float(), s["qw"], cos, sin, s["rot"], s["layout"]).to(s["q_out"].dtype),
            _norm_rope(s["k"].float(), s["kw"], cos, sin, s["rot"], s["layout"]).to(s["k_out"].dtype))


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    dev, g = s["positions"].device, s["g"]
    levels = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], device=dev, dtype=torch.float64)
    powers = torch.tensor([2.0 ** e for e in range(-32, 32)], device=dev, dtype=torch.float64)

    def two_to(e):
        return powers[e.long() + 32]

    def turned(x, w, pos, rot=HEAD, layout="half", freq=None, more=1.0):
        """RMS norm over the head, then the rotation of each pair as a complex product."""
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / HEAD + EPS) * w.double()
        if freq is None:
            freq = torch.exp(torch.arange(rot // 2, device=dev, dtype=torch.float64) * (-2.0 / rot * math.log(THETA)))
        a = torch.outer(pos.double(), freq)
        turn = torch.polar(torch.full_like(a, more), a)[:, None]
        lo, hi = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
        z = torch.complex(lo.contiguous(), hi.contiguous()) * turn
        y = x.clone()
        if layout == "half":
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        return y

    def to_e4m3(x):
        """x >= 0 rounded to a value of 1 + 3 mantissa bits, exponents from 2^-6 (below it steps of 2^-9), at most 448."""
        e = torch.floor(torch.log2(x.clamp(min=2.0 ** -6)))
        x = x.clamp(max=448.0)
        e = torch.where(two_to(e.clamp(max=9)) > x.clamp(min=2.0 ** -6), e - 1, e).clamp(max=8)
        step = two_to(e - 3)
        return (torch.round(x / step) * step).clamp(max=448.0)

    def held(x, unit):
        """The values that the cache holds for x [..., 128]: of the 8 levels the nearest, of two the one with an even number."""
        y = x.to(torch.bfloat16).double().reshape(*x.shape[:-1], 8, 16)
        top = y.abs().amax(-1, keepdim=True)
        scale = to_e4m3(torch.div(top, torch.full_like(top, 6.0)) / unit)
        z = torch.where(scale > 0, y.abs() / (scale * unit).clamp(min=1e-300), torch.zeros_like(y))
        far = (z.clamp(max=6)[..., None] - levels).abs()
        odd = torch.arange(8, device=dev) % 2
        near = torch.argmin(far * 4 + odd * 1e-9, -1)
        return (torch.sign(y) * levels[near] * scale * unit).reshape(x.shape)

    def block_values(block, i, which, unit):
        """Position i of each block [n][2304], from the bits: [n][128]."""
        m = s["maps"]
        byte = torch.gather(block, 1, m[which + "_code"][i]).long()
        nib = torch.stack([byte % 16, byte // 16], -1).reshape(len(block), HEAD)
        mag = torch.where(nib % 8 < 2, (nib % 8) * 0.5, (1.0 + (nib % 2) * 0.5) * two_to(nib % 8 // 2 - 1))
        sb = torch.gather(block, 1, m[which + "_scale"][i]).long()
        sc = torch.where(sb < 8, sb * 2.0 ** -9, (1.0 + (sb % 8) / 8.0) * two_to(sb // 8 - 7)) * unit
        return torch.where(nib >= 8, -mag, mag) * sc.repeat_interleave(16, -1)

    if case["op"] == "norm_rope":
        rot, i = case["rot"], torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64)
        wave = 2 * math.pi * THETA ** (2 * i / rot)       # the wavelength of each pair, in positions
        factor, more = case["factor"], 1.0
        if case["scaling"] == "linear":
            wave = wave * factor
        elif case["scaling"] == "base":
            wave = 2 * math.pi * (THETA * factor ** (rot / (rot - 2))) ** (2 * i / rot)
        elif case["scaling"] == "ramp":
            trained = int(case["max_seq"] / factor)
            pair = lambda turns: rot / 2 * math.log(trained / (2 * math.pi * turns), THETA)  # noqa: E731
            first, last = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
            kept = 1 - ((i - first) / max(last - first, 0.001)).clamp(0, 1)
            wave = 1 / (kept / wave + (1 - kept) / (wave * factor))
            more = 1 + math.log(factor) / 10
        go = lambda x, w: turned(x, w, s["positions"], rot, case["layout"], 2 * math.pi / wave, more)  # noqa: E731
        return go(s["q"], s["qw"]), go(s["k"], s["kw"])

    pos, table = s["positions"].long(), s["table"].long()
    if case["op"] == "append":
        return [held(turned(s["k"], s["kw"], pos), s["ks"]), held(s["v"], s["vs"])]
    if case["op"] == "read":
        page = table[s["prow"].long(), pos // PAGE]
        got = []
        for which in ("k", "v"):
            out = torch.empty(g, len(pos), HEAD, dtype=torch.float64, device=dev)
            for x in range(g):
                out[x] = block_values(s["data"][page, x, pos % PAGE // BLOCK], pos % BLOCK, which, s[which + "s"])
            got.append(out)
        return got
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    live = pos >= 0
    q = turned(s["q"], s["qw"], pos)
    k_new, v_new = held(turned(s["k"], s["kw"], pos), s["ks"]), held(s["v"], s["vs"])
    for b, last in enumerate(pos.tolist()):
        t = torch.arange(max(last, 0), device=dev)
        for x in range(g if last >= 0 else 0):
            block = s["data"][table[b, t // PAGE], x, t % PAGE // BLOCK]
            k = torch.cat([block_values(block, t % BLOCK, "k", 1.0), k_new[b, x][None]])
            v = torch.cat([block_values(block, t % BLOCK, "v", 1.0), v_new[b, x][None]])
            p = torch.softmax(q[b, GROUP * x:GROUP * (x + 1)] @ k.T / HEAD ** 0.5, -1)
            out[b, GROUP * x:GROUP * (x + 1)] = p @ v
    return out, k_new * live[:, None, None], v_new * live[:, None, None]
