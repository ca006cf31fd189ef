"""Microscaled tensors on the GPU (pkv_mx_quantize, pkv_mx_read, pkv_add_norm, pkv_mx_linear, pkv_mx_qkv_proj)
against the 64-bit forms of tests/_mx.py."""
import numpy as np
import pytest
import torch

import _mx
import paged_kv_gqa_qk_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = ["mx8", "mx4"]


@pytest.fixture(scope="module")
def pool():
    z = torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=8, kv_heads=2, max_seq=64))
    yield p
    p.close()


def same(t, x):
    """The tensor's bytes are those of the 64-bit values x: magnitudes, scales, and signs (also of what rounds to 0; 0 itself
    has either: -0 == 0)."""
    n, byte, sign = _mx.unpack(t)
    want_n, want_byte = _mx.quantise(x, t.kind)
    assert np.array_equal(byte, want_byte), np.argwhere(byte != want_byte)[:4]
    assert np.array_equal(n, want_n), np.argwhere(n != want_n)[:4]
    fine = np.repeat(byte != 255, 32, -1) & (x != 0)
    assert np.array_equal(sign[fine], np.signbit(x)[fine])


# ------------------------------------------------------------------ quantise, read

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (127, 384), (128, 128), (129, 640), (300, 1152), (2500, 4096)])
def test_quantise(pool, kind, rows, cols):
    x = _mx.activations(rows, cols, seed=rows + cols)
    t = pool.mx_quantize(x.to(DEV), kind)
    same(t, _mx.f64(x))
    assert np.array_equal(_mx.f64(pool.mx_read(t)), _mx.held(_mx.f64(x), kind))
    assert pool.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_every_bf16_value(pool, kind):
    """All finite bf16 values, each as the largest of its group beside smaller ones, and ties between codes."""
    bits = torch.arange(0x7f80, dtype=torch.int32)
    pos = (bits << 16).view(torch.float32)
    gen = torch.Generator().manual_seed(3)
    part = torch.randint(0, 33, (len(pos), 32), generator=gen) / 32.0 * torch.sign(torch.randn(len(pos), 32, generator=gen))
    part[:, 7] = torch.where(torch.arange(len(pos)) % 2 == 0, 1.0, -1.0)
    x = (pos[:, None].double() * part).to(torch.bfloat16)
    x = torch.cat([x, torch.zeros(-len(x) % 4, 32, dtype=torch.bfloat16)]).view(-1, 128)
    t = pool.mx_quantize(x.to(DEV), kind)
    same(t, _mx.f64(x))
    got, want = _mx.f64(pool.mx_read(t)), _mx.held(_mx.f64(x), kind)
    # the tensor holds 2^128 for values from 2^127 * (2 - 1/16) on (codes have 4 bits), which in bf16 is infinite:
    # its largest value is 2^127 * (2 - 2^-7), the next step would be 2^128
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    small = np.abs(want) < 2.0 ** -126   # bf16's steps there are 2^-133
    assert np.array_equal(got[~small], want[~small]) and (np.abs(got[small] - want[small]) <= 2.0 ** -134).all()


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan_take_their_group(pool, kind):
    x = _mx.activations(40, 256, seed=1)
    x[3, 5], x[3, 200], x[17, 64], x[39, 255] = float("inf"), float("nan"), -float("inf"), float("nan")
    t = pool.mx_quantize(x.to(DEV), kind)
    n, byte, _ = _mx.unpack(t)
    bad = {(3, 0), (3, 6), (17, 2), (39, 7)}
    assert {tuple(i) for i in np.argwhere(byte == 255)} == bad
    got = _mx.f64(pool.mx_read(t))
    clean = torch.where(torch.isfinite(x), x, 0)
    want = _mx.held(_mx.f64(clean), kind)
    for r, g in bad:
        assert (n[r, 32 * g:32 * g + 32] == 0).all()
        want[r, 32 * g:32 * g + 32] = np.nan
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("kind", KINDS)
def test_strides_and_untouched_bytes(pool, kind):
    rows, cols = 70, 384
    wide = _mx.activations(rows, cols + 72, seed=5).to(DEV)
    x = wide[:, 40:40 + cols]
    ref = pool.mx_quantize(x.contiguous(), kind)
    t = pkv.MxTensor.empty(kind, rows, cols)
    t.scales.fill_(77)
    pool.mx_quantize(x, kind, out=t)
    assert torch.equal(t.codes, ref.codes)
    n, byte, _ = _mx.unpack(t)
    assert np.array_equal(byte, _mx.unpack(ref)[1])
    tiles = t.scales.view(1, cols // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128, cols // 32)
    assert (tiles[rows:] == 77).all()                       # rows behind the last one stay as they were
    out = torch.full((rows, cols + 24), 5.0, dtype=torch.bfloat16, device=DEV)
    pool.mx_read(t, out=out[:, 8:8 + cols])
    assert torch.equal(out[:, 8:8 + cols], pool.mx_read(ref)) and (out[:, :8] == 5).all() and (out[:, 8 + cols:] == 5).all()


# ------------------------------------------------------------------ the residual's addition and the norm

def check_norm(pool, x, res, w, kind, eps=1e-6):
    h = _mx.f64(x) if res is None else _mx.bf16(_mx.f64(x) + _mx.f64(res))
    out, res_out = pool.add_norm(x, res, w, out=kind)
    if res is None:
        assert res_out is None
    else:
        assert np.array_equal(_mx.f64(res_out), h)
    y = _mx.norm(h, _mx.f64(w), eps)
    if kind == "bf16":
        assert np.array_equal(_mx.f64(out), _mx.bf16(y))    # one rounding, of the exact value
    else:
        same(out, y)
    assert pool.check_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", *KINDS])
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("tokens,hidden", [(1, 128), (2, 384), (1, 4096), (37, 1024), (150, 5120), (5, 8192), (3, 12288),
                                           (2, 32768)])
def test_add_norm(pool, kind, add, tokens, hidden):
    x = _mx.activations(tokens, hidden, seed=hidden + tokens).to(DEV)
    res = _mx.activations(tokens, hidden, seed=hidden + tokens + 1, scale=3.0).to(DEV) if add else None
    w = (torch.rand(hidden, generator=torch.Generator().manual_seed(9)) + 0.5).to(torch.bfloat16).to(DEV)
    check_norm(pool, x, res, w, kind)


@pytest.mark.parametrize("hidden", [8, 24, 136, 1000, 2056, 9992])
def test_add_norm_odd_widths(pool, hidden):
    x, res = (_mx.activations(11, hidden, seed=s).to(DEV) for s in (1, 2))
    w = torch.randn(hidden, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)   # (negative ones too)
    check_norm(pool, x, res, w, "bf16")
    check_norm(pool, x, None, w, "bf16")


@pytest.mark.parametrize("kind", ["bf16", *KINDS])
def test_add_norm_sizes_of_values(pool, kind):
    """Rows of zeros, tiny and large values, one dominant value, cancelling residuals."""
    x = _mx.activations(8, 512, seed=3, loud=False)
    res = _mx.activations(8, 512, seed=4, loud=False)
    x[0], res[0] = 0, 0
    x[1], res[1] = x[1] * 2.0 ** -60, res[1] * 2.0 ** -60
    x[2], res[2] = x[2] * 2.0 ** 40, res[2] * 2.0 ** 40
    x[3, 77] = 3e4
    x[4] = -res[4]
    x[5] = -res[5] * 1.0078125
    w = torch.ones(512, dtype=torch.bfloat16)
    w[::7] = 0
    check_norm(pool, x.to(DEV), res.to(DEV), w.to(DEV), kind)


@pytest.mark.parametrize("kind", ["bf16", *KINDS])
@pytest.mark.parametrize("hidden", [128, 2048, 4096, 16384])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_add_norm_uneven_rows(kind, hidden, eps):
    """Squares that span fp32's range within a thread's columns, a warp's and a row's: the sum is theirs, whatever the order."""
    gen = torch.Generator().manual_seed(hidden)
    x = torch.randn(9, hidden, generator=gen)
    size = torch.randint(-55, 55, (9, hidden), generator=gen).float()
    x[0] *= 2.0 ** size[0]
    x[1] *= 2.0 ** (size[1] / 8)
    x[2, :] = 1.0 + 2.0 ** -7                              # equal ones, whose sum is none of fp32's
    x[3] *= 2.0 ** -12
    x[3, hidden - 1] = 2.0 ** 50                           # one that dominates, in the last column
    x[4] *= 2.0 ** (torch.arange(hidden) % 8 * 6 - 20.0)   # by column of a thread
    x[5] *= 2.0 ** (torch.arange(hidden) // 8 % 32 - 16.0)  # by lane
    x[6] *= 2.0 ** (torch.arange(hidden) * 60.0 / hidden - 30)  # by warp
    x[7] = 0
    x[7, hidden // 2] = 3.0                                # one alone
    x = x.to(torch.bfloat16)
    w = torch.randn(hidden, generator=gen).to(torch.bfloat16)
    z = torch.zeros(2, 1, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=4, kv_heads=1, max_seq=64, eps=eps))
    out, _ = p.add_norm(x.to(DEV), None, w.to(DEV), out=kind)
    # Rows of equal values and of one that dominates have y on the very borders between two outputs, where the side is open
    # within 2^-40 of y.  That is what the pairs keep: a lane adds 16 squares to each of two sums; each addition loses 2^-24 of
    # the sum at most, which is kept, and the up to 16 * 2^-24 of the sum kept are themselves rounded 16 times, by 2^-24: 2^-40
    # of the sum.  A sum over a warp is off by one unit of 2^-24 a lane, of 2^24 units at least (2^-43), and a rounding of the
    # 2^7 units behind its first 24 bits (2^-42), twice.  The root halves these, 0.75 * 2^-40; its own error is 2^-45 and the
    # product's 2^-48.
    y, d = _mx.norm(_mx.f64(x), _mx.f64(w), eps), 2.0 ** -40
    form = _mx.bf16 if kind == "bf16" else lambda v: _mx.held(v, kind)
    got = _mx.f64(out) if kind == "bf16" else _mx.stored(out)
    assert ((got == form(y * (1 - d))) | (got == form(y * (1 + d)))).all() and p.check_errors() == 0
    p.close()


@pytest.mark.parametrize("kind", ["bf16", *KINDS])
def test_add_norm_rows_without_a_norm(pool, kind):
    """An Inf, a NaN and squares beyond fp32's range make their row NaN, and no other."""
    x = _mx.activations(5, 256, seed=3)
    x[1, 8], x[2, 100], x[3, 250] = float("inf"), float("nan"), 2.0 ** 70
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    out, _ = pool.add_norm(x.to(DEV), None, w, out=kind)
    got = _mx.f64(out if kind == "bf16" else pool.mx_read(out))
    assert np.isnan(got[1:4]).all() and np.isfinite(got[[0, 4]]).all()


def test_add_norm_in_place_and_strided(pool):
    wide = _mx.activations(33, 704, seed=6).to(DEV)         # (a row stride of 700 is refused: 16-byte loads)
    x = wide[:, 16:16 + 640]
    res = _mx.activations(33, 640, seed=7).to(DEV)
    w = torch.rand(640, device=DEV).to(torch.bfloat16)
    ref, ref_res = pool.add_norm(x.contiguous(), res, w, out="bf16")
    got, got_res = pool.add_norm(x, res, w, out="bf16")
    assert torch.equal(got, ref) and torch.equal(got_res, ref_res)
    own = res.clone()
    got, same_res = pool.add_norm(x, own, w, out="bf16", residual_out=own)      # the residual updated in place
    assert same_res is own and torch.equal(own, ref_res) and torch.equal(got, ref)
    dense, own = x.contiguous(), res.clone()
    pool.add_norm(dense, own, w, out=own, residual_out=dense)                   # outputs over both inputs
    assert torch.equal(own, ref) and torch.equal(dense, ref_res)


def test_add_norm_takes_the_pools_eps():
    z = torch.zeros(2, 1, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=4, kv_heads=1, max_seq=64, eps=0.25))
    check_norm(p, _mx.activations(3, 256, seed=1).to(DEV), None, torch.ones(256, dtype=torch.bfloat16, device=DEV), "mx8", 0.25)
    p.close()


# ------------------------------------------------------------------ the product

def operands(tokens, n_in, n_out, kind, seed):
    x = _mx.activations(tokens, n_in, seed=seed)
    w = _mx.activations(n_out, n_in, seed=seed + 1, scale=0.02, loud=False)
    return x.to(DEV), w.to(DEV)


def check_product(y, x, w):
    """Products are exact, the tensor cores add at most `in` of them in fp32, each sum off by at most 2^-23 of the running
    size, and the output is rounded once (2^-8)."""
    ref, size = x @ w.T, np.abs(x) @ np.abs(w).T
    off = np.abs(_mx.f64(y) - ref)
    bound = 2.0 ** -8 * np.abs(ref) + x.shape[1] * 2.0 ** -23 * size
    assert (off <= bound).all(), ((off / np.maximum(bound, 1e-300)).max(), np.argwhere(off > bound)[:4])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,n_in,n_out", [
    (1, 128, 128),          # one stage, half of it in 4 bits
    (1, 4096, 384),         # one token, split over a cluster
    (5, 384, 256),          # a 4-bit row of a stage and a half
    (16, 640, 128),
    (17, 1024, 640),
    (64, 4096, 1024),
    (65, 512, 384),
    (128, 1152, 256),
    (129, 256, 128),
    (200, 4096, 512),
    (333, 896, 1280),
    (700, 2048, 1536),      # more tiles than one a SM
    (257, 128, 128),        # one token beyond a tile, half a tile of features, less than a stage in 4 bits
    (1025, 1152, 640),      # a 4-bit row of a stage and a half, features of two tiles and a half
    (5000, 256, 1280),      # many tiles of few stages
    (384, 8192, 256),       # a long row
])
def test_linear(pool, kind, tokens, n_in, n_out):
    x, w = operands(tokens, n_in, n_out, kind, seed=tokens + n_in + n_out)
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    y = pool.mx_linear(xm, wm)
    assert pool.check_errors() == 0
    check_product(y, _mx.stored(xm), _mx.stored(wm))
    assert torch.equal(pool.mx_linear(x, wm), y)        # bf16 x: quantised to the weights' kind first
    assert torch.equal(pool.mx_linear(xm, wm), y)       # the same from run to run


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kv_heads", [1, 2, 3])
@pytest.mark.parametrize("tokens", [1, 70, 300])
def test_qkv_proj(kind, kv_heads, tokens):
    """q, k and v are the columns of the one product (tiles that span them included)."""
    z = torch.zeros(2, kv_heads, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=4 * kv_heads, kv_heads=kv_heads, max_seq=64))
    x, w = operands(tokens, 640, 6 * kv_heads * 128, kind, seed=tokens)
    xm, wm = p.mx_quantize(x, kind), p.mx_quantize(w, kind)
    q, k, v = p.mx_qkv_proj(xm, wm)
    assert q.shape == (tokens, 4 * kv_heads, 128) and k.shape == v.shape == (tokens, kv_heads, 128)
    y = p.mx_linear(xm, wm)
    check_product(y, _mx.stored(xm), _mx.stored(wm))
    assert torch.equal(torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1), y)
    for got, ref in zip(p.mx_qkv_proj(x, wm), (q, k, v)):
        assert torch.equal(got, ref)
    assert p.check_errors() == 0
    p.close()
