"""Products of microscaled tensors by kernel: every shape names the form it is for (tests/_mx_kernels.py) and runs there by the
library's rule."""
import pytest
import torch

import paged_kv_gqa_qk_gb300 as pkv
from _mx_kernels import FEW, MANY, PAIRS, route
from test_gpu_mx import DEV, KINDS, operands

pytestmark = pytest.mark.gpu
CASES = FEW + MANY
IDS = ["x".join(map(str, shape)) for shape, _ in CASES]


@pytest.fixture(scope="module")
def pool():
    z = torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=8, kv_heads=2, max_seq=64))
    yield p
    p.close()


def runs_in(kind, shape, where):
    assert route(kind, *shape, sms=torch.cuda.get_device_properties(0).multi_processor_count) == where


def check(y, x, w):
    """Products are exact; at most `in` of them are added in fp32, each sum off by at most 2^-23 of the running size; the
    output is rounded once.  x and w: the values that the tensors hold (exact in bf16)."""
    x, w = x.double(), w.double()
    ref, size = x @ w.T, x.abs() @ w.abs().T
    assert ((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + x.shape[1] * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,where", CASES, ids=IDS)
def test_product(pool, kind, shape, where):
    runs_in(kind, shape, where)
    x, w = operands(*shape, kind, seed=sum(shape))
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    y = pool.mx_linear(xm, wm)
    assert pool.check_errors() == 0
    check(y, pool.mx_read(xm), pool.mx_read(wm))
    assert torch.equal(pool.mx_linear(xm, wm), y)
    assert torch.equal(pool.mx_linear(x, wm), y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,where", CASES, ids=IDS)
def test_sums_of_whole_numbers_are_exact(pool, kind, shape, where):
    """Every partial sum is a whole number below 2^24, in whatever order, so fp32 sums are exact and y is the exact sum rounded
    once.  Products of 2^22 that cancel stand far apart along the row (or, in 8 bits, 2^16 within one instruction's 32 values), so
    a sum of fewer bits anywhere loses the ones between them."""
    runs_in(kind, shape, where)
    tokens, n_in, n_out = shape
    gen = torch.Generator(device=DEV).manual_seed(n_in)
    x, w = (torch.randint(-1, 2, s, generator=gen, device=DEV).to(torch.bfloat16) for s in ((tokens, n_in), (n_out, n_in)))
    last = n_in // 32 - 1
    for group, sign in {0: 1, last // 3: 1, last // 2: -1, last: -1}.items() if last >= 8 else {0: 1, last: -1}.items():
        x[:, 32 * group:32 * group + 32], w[:, 32 * group:32 * group + 32] = 0, 0
        x[:, 32 * group + 5], w[:, 32 * group + 5] = 2 ** 11, sign * 2 ** 11
    if kind == "mx8":
        for column, sign in ((32, 1), (60, -1)):
            x[:, column], w[:, column] = 2 ** 8, sign * 2 ** 8
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    assert torch.equal(pool.mx_read(xm), x) and torch.equal(pool.mx_read(wm), w)
    assert n_in + 2 ** 17 + 2 ** 23 < 2 ** 24
    assert torch.equal(pool.mx_linear(xm, wm), (x.double() @ w.double().T).to(torch.bfloat16))
    assert pool.check_errors() == 0


# ------------------------------------------------------------------ over pairs: outputs, NaN, padding, order of calls

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kv_heads,tokens", [(8, 200), (8, 500), (3, 700), (1, 3000)])
def test_qkv_proj(kind, kv_heads, tokens):
    """Three outputs, whose borders lie inside tiles."""
    runs_in(kind, (tokens, 640, 6 * kv_heads * 128), PAIRS)
    z = torch.zeros(2, kv_heads, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=4 * kv_heads, kv_heads=kv_heads, max_seq=64))
    x, w = operands(tokens, 640, 6 * kv_heads * 128, kind, seed=tokens)
    xm, wm = p.mx_quantize(x, kind), p.mx_quantize(w, kind)
    q, k, v = (torch.full((tokens + 1, n, 128), 7.0, dtype=torch.bfloat16, device=DEV) for n in (4 * kv_heads, kv_heads, kv_heads))
    p.mx_qkv_proj(xm, wm, q[:tokens], k[:tokens], v[:tokens])
    for t in (q, k, v):
        assert (t[tokens] == 7).all()                       # what lies behind the last token is left as it was
    got = torch.cat([t[:tokens].flatten(1) for t in (q, k, v)], 1)
    check(got, p.mx_read(xm), p.mx_read(wm))
    assert torch.equal(got, p.mx_linear(xm, wm))
    assert p.check_errors() == 0
    p.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(200, 640, 6656), (1000, 1152, 1280)])
def test_nan_stays_in_its_row_and_feature(pool, kind, shape):
    runs_in(kind, shape, PAIRS)
    x, w = operands(*shape, kind, seed=1)
    clean = pool.mx_linear(x, pool.mx_quantize(w, kind))
    rows, features = [0, 77, shape[0] - 1], [5, 777, shape[2] - 1]
    x[rows[0], 600], x[rows[1], 0], x[rows[2], 639] = float("nan"), float("inf"), -float("inf")
    w[features[0], 130], w[features[1], 0], w[features[2], 639] = float("inf"), float("nan"), float("nan")
    y = pool.mx_linear(x, pool.mx_quantize(w, kind))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[rows], bad[:, features] = True, True
    assert y[bad].isnan().all() and torch.equal(y[~bad], clean[~bad])
    assert pool.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [60, 130, 300])
def test_padding_of_the_scales_is_not_used(pool, kind, tokens):
    shape = (tokens, 384, 19712)
    runs_in(kind, shape, PAIRS)
    x, w = operands(*shape, kind, seed=tokens)
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    blocks = -(-tokens // 128)
    tiles = xm.scales.view(blocks, 3, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128 * blocks, 12)
    ref = None
    for fill in (127, 255, 0, 254):
        tiles[tokens:] = fill
        other = pkv.MxTensor(kind, tokens, 384, xm.codes, tiles.view(blocks, 4, 32, 3, 4).permute(0, 3, 2, 1, 4).contiguous().flatten())
        y = pool.mx_linear(other, wm)
        assert ref is None or torch.equal(y, ref)
        ref = y
    check(ref, pool.mx_read(xm), pool.mx_read(wm))
    assert pool.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_each_call_waits_for_the_one_before(pool, kind):
    """Operands, weights among them, that the call just before wrote; and the call after reads what this one wrote."""
    shape = (2560, 512, 512)
    runs_in(kind, shape, PAIRS)
    ones = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    few = operands(3, 512, 128, kind, seed=8)[0]
    sets = []
    for seed in range(4):
        x, w = operands(*shape, kind, seed=seed)
        y = pool.mx_linear(pool.mx_quantize(x, kind), pool.mx_quantize(w, kind))
        torch.cuda.synchronize()
        sets.append((x, w, y, pool.linear(few, y)))
        torch.cuda.synchronize()
    xm, wm = pkv.MxTensor.empty(kind, 2560, 512), pkv.MxTensor.empty(kind, 512, 512)
    y, z = torch.empty(2560, 512, dtype=torch.bfloat16, device=DEV), torch.empty(3, 2560, dtype=torch.bfloat16, device=DEV)
    wrong = torch.zeros(2, device=DEV)
    for i in range(200):
        x, w, ref, ref_z = sets[i * 7 % 4]
        if i % 2:
            pool.mx_quantize(x, out=xm)
            pool.mx_quantize(w, out=wm)
        else:
            pool.mx_quantize(w, out=wm)
            pool.add_norm(x, None, ones, out=xm)             # (lets the next call start early)
            pool.mx_quantize(x, out=xm)
        pool.mx_linear(xm, wm, y=y)
        pool.linear(few, y, y=z)                             # its weights: what the product just wrote
        wrong[0] += (y != ref).any()
        wrong[1] += (z != ref_z).any()
    assert wrong.tolist() == [0, 0] and pool.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_replayed_on_two_streams(pool, kind):
    shape = (700, 1152, 2048)
    runs_in(kind, shape, PAIRS)
    sets, graphs = [], []
    for seed in range(2):
        x, w = operands(*shape, kind, seed=seed)
        xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
        y, ref = torch.empty(700, 2048, dtype=torch.bfloat16, device=DEV), pool.mx_linear(xm, wm)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                pool.mx_linear(xm, wm, y=y)
        sets.append((xm, wm, y, ref))
        graphs.append((g, torch.cuda.Stream()))
    for _ in range(10):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, y, ref in sets:
        assert torch.equal(y, ref)
    assert pool.check_errors() == 0
