"""The 4-bit page format and the decode over it in plain numpy, in 64 bits, for the tests: the layout of
include/pkv.h written out position by position, the quantiser from its definition, norm and rotation,
and the attention of one row at a time."""
import numpy as np
import torch

BLOCK, PAGE, D = 16, 64, 128
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16(x) -> np.ndarray:
    """float64 values rounded to fp32 and then to bf16 (ties to even), as float64."""
    return torch.from_numpy(np.asarray(x, np.float64).astype(np.float32)).to(torch.bfloat16).double().numpy()


def e4m3(x) -> np.ndarray:
    """Nearest of the e4m3 values, ties to even, of x >= 0, at most 448."""
    x = np.minimum(np.asarray(x, np.float64), 448.0)
    e = np.maximum(np.frexp(x)[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.minimum(np.round(x / step) * step, 448.0)


def e4m3_byte(v) -> np.ndarray:
    v = np.asarray(v, np.float64)
    e = np.frexp(v)[1] - 1
    normal = v >= 2.0 ** -6
    mant = np.where(normal, np.round((v / np.ldexp(1.0, e) - 1) * 8), np.round(v * 512))
    return np.where(normal, (e + 7) * 8 + mant, mant).astype(np.uint8)


def e4m3_value(b) -> np.ndarray:
    b = np.asarray(b).astype(np.int64)
    m = b & 0x7f
    v = np.where(m < 8, m * 2.0 ** -9, np.ldexp(1.0 + (m & 7) / 8.0, (m >> 3) - 7))
    v = np.where(m == 0x7f, np.nan, v)
    return np.where(b & 0x80, -v, v)


def quantise(x, s):
    """bf16 values [..., 128] -> (codes [..., 128] in 0..15, scale bytes [..., 8])."""
    y = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], 8, 16)
    bad = ~np.isfinite(y).all(-1)
    y = np.where(bad[..., None], 0.0, y)
    scale = e4m3(np.abs(y).max(-1) / (6.0 * s))
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(scale[..., None] > 0, np.abs(y) / (scale[..., None] * s), 0.0)
    far = np.abs(np.minimum(z, 6.0)[..., None] - LEVELS)
    best = far.min(-1, keepdims=True)
    tied = far == best
    even = tied & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), tied.argmax(-1)).astype(np.uint8)
    code |= (np.signbit(y).astype(np.uint8) << 3)
    byte = np.where(bad, 0x7f, e4m3_byte(scale)).astype(np.uint8)
    return code.reshape(*np.shape(x)), byte


def values(code, byte, s):
    v = np.where(code & 8, -1.0, 1.0) * LEVELS[code & 7]
    return (v.reshape(*code.shape[:-1], 8, 16) * e4m3_value(byte)[..., None] * s).reshape(code.shape)


def _maps():
    code = np.zeros((16, 64), np.int64)
    ks, vs = np.zeros((16, 8), np.int64), np.zeros((16, 8), np.int64)
    for i in range(16):
        b = (i >> 2) & 1
        c = (i & 3) ^ b
        for j in range(64):
            code[i, j] = 64 * i + (j ^ (32 * ((i >> 1) & 1)))
        for g in range(8):
            ks[i, g] = 16 * (2 * c + b) + 4 * (g >> 1) + (g & 1) + 2 * (i >> 3)
            vs[i, g] = 16 * g + 4 * c + b + 2 * (i >> 3)
    return code, ks, vs


CODE, KS, VS = _maps()


class Cache:
    """A pool's bytes [pages][kv_heads][4][2304] and the values they stand for."""

    def __init__(self, data, ks=1.0, vs=1.0):
        self.data, self.ks, self.vs = data, ks, vs

    @classmethod
    def of(cls, K, V, ks=1.0, vs=1.0):
        """From bf16 values K, V [kv_heads][pages * 64][128]."""
        G, n, _ = K.shape
        data = np.zeros((n // PAGE, G, 4, 2304), np.uint8)
        c = cls(data, ks, vs)
        blocks = lambda x: x.reshape(G, n // PAGE, 4, BLOCK, D).transpose(1, 0, 2, 3, 4)  # noqa: E731
        for x, s, off, at, so in ((K, ks, 0, KS, 2048), (V, vs, 1024, VS, 2176)):
            code, byte = quantise(blocks(np.asarray(x, np.float64)), s)
            data[..., off + CODE] = code[..., 0::2] | (code[..., 1::2] << 4)
            data[..., so + at] = byte
        return c

    def put(self, page, pos, k, v):
        """k, v [kv_heads][128] (bf16 values) at position pos % 64 of a page."""
        blk, i = self.data[page, :, pos % PAGE // BLOCK], pos % BLOCK
        for x, s, off, at, so in ((k, self.ks, 0, KS, 2048), (v, self.vs, 1024, VS, 2176)):
            code, byte = quantise(x, s)
            blk[:, off + CODE[i]] = code[:, 0::2] | (code[:, 1::2] << 4)
            blk[:, so + at[i]] = byte

    def get(self, pages, n):
        """The values of the first n positions of a row's pages: K, V [n][kv_heads][128]."""
        blk = self.data[np.asarray(pages[:-(-n // PAGE)], np.int64)]      # [P][G][4][2304]
        out = []
        for s, off, at, so in ((self.ks, 0, KS, 2048), (self.vs, 1024, VS, 2176)):
            b = blk[..., off + CODE]
            code = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], D)
            x = values(code, blk[..., so + at], s)                        # [P][G][4][16][128]
            out.append(x.transpose(0, 2, 3, 1, 4).reshape(-1, blk.shape[1], D)[:n])
        return out


def norm_rope(x, w, pos, rot=D, theta=1e6, eps=1e-6, layout="half", freq=None, mscale=1.0):
    """x [tokens][heads][128] -> float64; w None: no norm."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    freq = theta ** (-2.0 * np.arange(rot // 2) / rot) if freq is None else np.asarray(freq)
    a = np.asarray(pos, np.float64)[:, None, None] * freq
    c, s, y = np.cos(a) * mscale, np.sin(a) * mscale, x.copy()
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def attend(q, K, V):
    """q [4 G][128] (float64), K, V [n][G][128]: (out, bound on |kernel - out| before bf16's rounding of out).

    The kernel rounds q to fp16 (2^-11 of each element; its products with the cached values and their sums are
    fp32), so a score is off by at most ds = 2^-11 sum |q k| / sqrt(128) (+ 2^-16 of it for the sums), a weight by
    a factor within exp(+-2 ds); the weights enter the second product as fp16: 2^-11 of each, or 2^-25 of the
    largest where they are below fp16's normal range."""
    G = K.shape[1]
    out, bound = np.zeros_like(q), np.zeros_like(q)
    for h in range(q.shape[0]):
        k, v = K[:, h // 4], V[:, h // 4]
        s = k @ q[h] / np.sqrt(D)
        ds = (2.0 ** -11 + 2.0 ** -16) * (np.abs(k) @ np.abs(q[h])).max() / np.sqrt(D)
        p = np.exp(s - s.max())
        total = p.sum()
        out[h] = p @ v / total
        bound[h] = (np.expm1(2 * ds) + 2.0 ** -11 + 2.0 ** -18) * (p @ np.abs(v)) / total \
            + 2.0 ** -25 * np.abs(v).sum(0) / total
    return out, bound
