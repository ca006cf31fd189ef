"""Microscaled tensors and the layer norm in 64 bits (numpy), from their definitions in include/pkv.h."""
import numpy as np
import torch

TOP = {"mx8": 448.0, "mx4": 6.0}
LEVELS = {"mx4": np.array([0.0, 0.5, 1, 1.5, 2, 3, 4, 6]),
          "mx8": np.array([m * 2.0 ** -9 for m in range(8)] +
                          [(1 + m / 8) * 2.0 ** n for n in range(-6, 9) for m in range(8)][:-1])}


def f64(t):
    return t.detach().cpu().double().numpy()


def bf16(x):
    """x rounded to bf16, ties to even (values in bf16's normal range; a double's 53 bits rounded once)."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 256), e - 8)


def quantise(x, kind):
    """(numbers of the codes' magnitudes, scale bytes) of x [rows][cols]."""
    g = np.abs(x).reshape(x.shape[0], -1, 32)
    top = g.max(-1)                              # (a NaN stays one)
    bad = ~np.isfinite(top)
    top = np.where(bad, 0, top)
    m, e = np.frexp(top / TOP[kind])             # exact but for 448 = 7 * 64: checked below
    e = np.where(m == 0.5, e - 1, e)
    e = np.where(top > TOP[kind] * np.exp2(e.astype(float)), e + 1, e)
    e = np.where(top <= TOP[kind] * np.exp2(e - 1.0), e - 1, e)
    e = np.where(top == 0, -127, np.maximum(e, -127)).astype(int)
    y = np.where(bad[..., None], 0, g) / np.exp2(e.astype(float))[..., None]
    lev = LEVELS[kind]
    half = (lev[1:] + lev[:-1]) / 2
    n = np.searchsorted(half, y)                 # half[n - 1] < y <= half[n]
    tie = (n < len(half)) & (y == half[np.minimum(n, len(half) - 1)])
    n = np.where(tie & (n % 2 == 1), n + 1, n)
    return n.reshape(x.shape), np.where(bad, 255, e + 127)


def values(n, byte, sign, kind):
    """The values of magnitudes n, scale bytes and signs (True: negative)."""
    unit = np.where(byte == 255, np.nan, np.exp2(byte - 127.0))
    return np.where(sign, -1.0, 1.0) * LEVELS[kind][n] * np.repeat(unit, 32, -1)


def held(x, kind):
    n, byte = quantise(x, kind)
    return values(n, byte, np.signbit(x), kind)


def unpack(t):
    """(magnitudes, scale bytes, signs) of an MxTensor's bytes."""
    codes, raw = t.codes.cpu().numpy(), t.scales.cpu().numpy()
    if t.kind == "mx4":
        codes = np.stack([codes & 15, codes >> 4], -1)
    codes = codes.reshape(t.rows, t.cols).astype(int)
    size = len(LEVELS[t.kind]) + (t.kind == "mx8")
    r, g = np.arange(t.rows)[:, None], np.arange(t.cols // 32)[None]
    at = (r // 128 * (t.cols // 128) + g // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + g % 4
    return codes % size, raw[at].astype(int), codes >= size


def stored(t):
    return values(*(lambda n, b, s: (n, b, s))(*unpack(t)), t.kind)


def norm(h, w, eps=1e-6):
    h = h.astype(np.longdouble)
    return (h / np.sqrt((h * h).mean(-1, keepdims=True) + np.longdouble(eps)) * w.astype(np.longdouble)).astype(np.float64)


def activations(rows, cols, seed, scale=1.0, loud=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen) * scale
    if loud:
        x[:, torch.randint(0, cols, (max(1, cols // 128),), generator=gen)] *= 24.0
    return x.to(torch.bfloat16)
