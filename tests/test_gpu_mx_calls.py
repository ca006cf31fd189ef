"""Microscaled tensors' calls as a server makes them: a layer's step with either pool, both ways of the binding, refusals,
streams, threads, captured graphs, memory beyond 2^31 elements."""
import threading

import numpy as np
import pytest
import torch

import _mx
import paged_kv_gqa_qk_gb300 as pkv
from test_gpu_mx import DEV, KINDS, check_product, operands

pytestmark = pytest.mark.gpu


def pool_of(kv_heads=2, **cfg):
    z = torch.zeros(2, kv_heads, 64, 128, dtype=torch.bfloat16, device=DEV)
    return pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=4 * kv_heads, kv_heads=kv_heads, max_seq=64, **cfg))


@pytest.fixture(scope="module")
def pool():
    p = pool_of()
    yield p
    p.close()


@pytest.fixture(params=["module", "ctypes"])
def way(request, monkeypatch):
    """The binding with csrc/pkv_torch.cpp's module, and without it."""
    pkv.load_library()
    assert pkv._fast is not None, "the module of csrc/pkv_torch.cpp was not built"
    if request.param == "ctypes":
        monkeypatch.setattr(pkv, "_fast", None)
    return request.param


# ------------------------------------------------------------------ a layer

class Layer:
    """One attention layer's step over a 4-bit pool with its norms and projections microscaled, and the second norm."""

    def __init__(self, kind, rows, hidden=512, kv_heads=2):
        gen = torch.Generator().manual_seed(7)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen) * scale).to(torch.bfloat16).to(DEV)  # noqa: E731
        self.kind, self.rows, self.kv_heads = kind, rows, kv_heads
        self.pool = pkv.Q4KVPool.empty(rows * 2 + 1, dict(heads=4 * kv_heads, kv_heads=kv_heads, max_seq=128))
        self.table = (torch.arange(rows * 2, dtype=torch.int32).view(rows, 2) + 1).to(DEV)
        self.w1, self.w2, self.qw, self.kw = r(hidden), r(hidden), r(128), r(128)
        self.wqkv = self.pool.mx_quantize(r(6 * kv_heads * 128, hidden, scale=0.05), kind)
        self.wo = self.pool.mx_quantize(r(hidden, 4 * kv_heads * 128, scale=0.05), kind)
        self.x, self.residual = r(rows, hidden), r(rows, hidden)
        self.positions = torch.arange(rows, dtype=torch.int32, device=DEV) * 7 % 100

    def step(self):
        p = self.pool
        a, h = p.add_norm(self.x, self.residual, self.w1, out=self.kind)
        q, k, v = p.mx_qkv_proj(a, self.wqkv)
        o = p.decode(q, k, v, self.qw, self.kw, self.positions, self.table)
        y = p.mx_linear(o.flatten(1), self.wo)
        b, h2 = p.add_norm(y, h, self.w2, out=self.kind)
        return a, h, q, k, v, o, y, b, h2


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 5, 70])
def test_layer(kind, rows):
    """Each step of the layer against the 64-bit forms on what the step before it gave."""
    layer = Layer(kind, rows)
    a, h, q, k, v, o, y, b, h2 = layer.step()
    f = _mx.f64
    assert np.array_equal(f(h), _mx.bf16(f(layer.x) + f(layer.residual)))
    assert np.array_equal(_mx.stored(a), _mx.held(_mx.norm(f(h), f(layer.w1)), kind))
    qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
    check_product(qkv, _mx.stored(a), _mx.stored(layer.wqkv))
    check_product(y, _mx.held(f(o.flatten(1)), kind), _mx.stored(layer.wo))
    assert np.array_equal(f(h2), _mx.bf16(f(y) + f(h)))
    assert np.array_equal(_mx.stored(b), _mx.held(_mx.norm(f(h2), f(layer.w2)), kind))
    assert layer.pool.check_errors() == 0
    # the same values through the bf16 projection: q, k and v differ by the sums' order alone
    ref = layer.pool.mx_read(a).float() @ layer.pool.mx_read(layer.wqkv).float().T
    assert ((qkv.float() - ref).abs() <= 2.0 ** -7 * ref.abs() + 1e-3).all()


@pytest.mark.parametrize("kind", KINDS)
def test_layer_captured_and_replayed(kind):
    """A captured layer follows its inputs' new values; two graphs of it and calls between them do not disturb each other."""
    one, two = Layer(kind, 6), Layer(kind, 6)
    graphs = []
    for layer in (one, two):
        layer.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = layer.step()
        graphs.append((g, outs))
    for seed in (1, 2, 3):
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn(6, 512, generator=gen).to(torch.bfloat16).to(DEV)
        for layer in (one, two):
            layer.x.copy_(x)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        first = [o.codes if isinstance(o, pkv.MxTensor) else o for o in graphs[0][1]]
        for a, b in zip(first, graphs[1][1]):
            assert torch.equal(a, b.codes if isinstance(b, pkv.MxTensor) else b)
        eager = one.step()
        for a, b in zip(first, eager):
            assert torch.equal(a, b.codes if isinstance(b, pkv.MxTensor) else b)


# ------------------------------------------------------------------ both ways, refusals

def _calls(pool):
    """One of each call; every result on the host."""
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, res, w, wide = r(5, 256), r(5, 256), r(256), r(5, 320)
    got = []
    for kind in ("mx8", "mx4"):
        m = pool.mx_quantize(x, kind)
        n, h = pool.add_norm(x, res, w, out=kind)
        got += [m.codes, pool.mx_read(m), n.codes, pool.mx_read(n), h]
        got.append(pool.mx_quantize(wide[:, 32:288], kind, stream=torch.cuda.current_stream()).codes)
        n, none = pool.add_norm(wide[:, 32:288], None, w, out=kind)
        assert none is None
        got.append(n.codes)
        ws = pool.mx_quantize(r(6 * 2 * 128, 256), kind)
        got += [pool.mx_linear(m, ws), *pool.mx_qkv_proj(m, ws)]
        out = torch.zeros(5, 272, dtype=torch.bfloat16, device=DEV)
        pool.mx_read(m, out=out[:, :256])
        got.append(out)
    got += pool.add_norm(x, res, w, out="bf16")
    return [g.cpu() for g in got]


def test_both_ways_agree(pool, monkeypatch):
    """The module's calls and the ctypes functions' give the same bytes, and the module took every one of them."""
    counts = {}

    class Counting:
        def __getattr__(self, name):
            def call(*args):
                rc = getattr(real, name)(*args)
                counts[name, rc] = counts.get((name, rc), 0) + 1
                return rc
            return call
    real = pkv._fast
    assert real is not None
    monkeypatch.setattr(pkv, "_fast", Counting())
    mine = _calls(pool)
    assert counts == {("mx_quantize", 0): 6, ("mx_read", 0): 6, ("add_norm", 0): 5, ("mx_linear", 0): 2, ("mx_qkv_proj", 0): 2}
    monkeypatch.setattr(pkv, "_fast", None)
    for a, b in zip(mine, _calls(pool)):
        assert torch.equal(a, b)


def test_wrong_arguments_are_refused(pool, way):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    x, w, m8, m4 = bf(4, 256), bf(256), pkv.MxTensor.empty("mx8", 4, 256), pkv.MxTensor.empty("mx4", 4, 256)
    w8 = pkv.MxTensor.empty("mx8", 128, 256)
    host = torch.zeros(4, 256, dtype=torch.bfloat16)
    refused = [
        (TypeError, lambda: pool.mx_quantize(x.float(), "mx8")),
        (TypeError, lambda: pool.mx_quantize(x.half(), out=m8)),
        ((TypeError, ValueError), lambda: pool.mx_quantize(host, out=m8)),
        (ValueError, lambda: pool.mx_quantize(x, "mx4", out=m8)),
        (ValueError, lambda: pool.mx_quantize(x, "int8")),
        (ValueError, lambda: pool.mx_quantize(bf(5, 256), out=m8)),
        (ValueError, lambda: pool.mx_quantize(bf(256, 4).t(), out=m8)),          # rows that are not contiguous
        (pkv.PkvError, lambda: pool.mx_quantize(bf(4, 260)[:, :256], out=m8)),   # a row stride of 520 bytes
        (pkv.PkvError, lambda: pool.mx_quantize(bf(4, 264)[:, 4:260], out=m8)),  # rows on an 8-byte border
        (pkv.PkvError, lambda: pool.mx_quantize(bf(4, 200), "mx8")),
        (pkv.PkvError, lambda: pool.mx_quantize(bf(0, 256), "mx8")),
        (ValueError, lambda: pool.mx_read(m8, out=bf(4, 128))),
        ((TypeError, ValueError), lambda: pool.mx_read(m8, out=host)),
        (ValueError, lambda: pool.add_norm(x, None, w, out=m8, residual_out=x)),
        (ValueError, lambda: pool.add_norm(x, bf(4, 128), w, out=m8)),
        (ValueError, lambda: pool.add_norm(x, None, bf(128), out=m8)),
        (ValueError, lambda: pool.add_norm(x, None, w, out=pkv.MxTensor.empty("mx8", 5, 256))),
        (ValueError, lambda: pool.add_norm(x, None, w, out=bf(4, 264))),
        (TypeError, lambda: pool.add_norm(x, None, w, out=x.float())),
        (TypeError, lambda: pool.add_norm(x.float(), None, w, out=m8)),
        (TypeError, lambda: pool.add_norm(x, x.float(), w, out=m8, residual_out=x)),
        (ValueError, lambda: pool.add_norm(x, bf(4, 264)[:, :256], w, out=m8, residual_out=x)),
        (pkv.PkvError, lambda: pool.add_norm(bf(4, 200), None, bf(200), out="mx8")),
        (pkv.PkvError, lambda: pool.add_norm(bf(4, 20), None, bf(20), out="bf16")),
        (pkv.PkvError, lambda: pool.add_norm(bf(0, 256), None, w, out="bf16")),
        (pkv.PkvError, lambda: pool.add_norm(bf(1, 32776), None, bf(32776), out="bf16")),
        (ValueError, lambda: pool.mx_linear(m4, w8)),                            # kinds differ
        (ValueError, lambda: pool.mx_linear(pkv.MxTensor.empty("mx8", 4, 128), w8)),
        (ValueError, lambda: pool.mx_linear(m8, w8, y=bf(4, 256))),
        (TypeError, lambda: pool.mx_linear(m8, w8, y=torch.zeros(4, 128, device=DEV))),
        (pkv.PkvError, lambda: pool.mx_linear(m8, pkv.MxTensor.empty("mx8", 100, 256))),
        ((TypeError, AttributeError), lambda: pool.mx_linear(m8, x)),
        (ValueError, lambda: pool.mx_qkv_proj(m8, w8)),
        (ValueError, lambda: pool.mx_qkv_proj(m8, pkv.MxTensor.empty("mx8", 1536, 256), q=bf(4, 8, 64))),
    ]
    for what, call in refused:
        with pytest.raises(what):
            call()
    assert pool.check_errors() == 0


def test_tensors_of_another_device_are_refused(pool, way, monkeypatch):
    monkeypatch.setattr(pool, "_spec", (1, *pool._spec[1:]))
    monkeypatch.setattr(pkv, "_raw_stream", lambda device: 0)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    m = pkv.MxTensor.empty("mx8", 4, 256)
    w = pkv.MxTensor.empty("mx8", 1536, 256)
    for call in (lambda: pool.mx_quantize(x, out=m), lambda: pool.mx_read(m, out=x), lambda: pool.add_norm(x, None, x[0], out=m),
                 lambda: pool.mx_linear(m, w), lambda: pool.mx_qkv_proj(m, w)):
        with pytest.raises(ValueError, match="the pool on cuda:1"):
            call()


# ------------------------------------------------------------------ order of work

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [3, 400])
def test_each_call_waits_for_the_one_before(pool, kind, tokens):
    """Operands, weights among them, written by the call just before: products of what is there, never of what was."""
    sets = []
    for seed in range(4):
        x, w = operands(tokens, 512, 384, kind, seed=seed)
        sets.append((x, w, pool.mx_linear(pool.mx_quantize(x, kind), pool.mx_quantize(w, kind))))
    torch.cuda.synchronize()
    xm, wm = pkv.MxTensor.empty(kind, tokens, 512), pkv.MxTensor.empty(kind, 384, 512)
    y = torch.empty(tokens, 384, dtype=torch.bfloat16, device=DEV)
    ones = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    wrong = torch.zeros((), device=DEV)
    for i in range(200):
        x, w, ref = sets[i * 7 % 4]
        if i % 2:
            pool.mx_quantize(x, out=xm)
            pool.mx_quantize(w, out=wm)          # the weights last: the product's predecessor writes them
        else:
            pool.mx_quantize(w, out=wm)
            pool.add_norm(x, None, ones, out=xm)  # (a kernel that lets the next one start early)
            pool.mx_quantize(x, out=xm)
        pool.mx_linear(xm, wm, y=y)
        wrong += (y != ref).any()
    assert float(wrong) == 0 and pool.check_errors() == 0


@pytest.mark.parametrize("tokens", [1, 400])
def test_output_of_a_call_as_the_next_products_weights(pool, tokens):
    """A product of bf16 brings its weights' first boxes to L2 before the call before it has ended, and reads them after:
    weights that a product, a norm or a read wrote just before are the ones multiplied."""
    ones = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    kind, sets = "mx8", []
    for seed in range(4):
        a, b = operands(384, 640, 512, kind, seed=seed)
        am, bm = pool.mx_quantize(a, kind), pool.mx_quantize(b, kind)
        x = operands(tokens, 512, 128, kind, seed=9)[0]
        y = pool.mx_linear(am, bm)
        norm, read = pool.add_norm(y, None, ones, out="bf16")[0], torch.empty_like(y)
        ym = pool.mx_quantize(y, kind)
        pool.mx_read(ym, out=read)
        torch.cuda.synchronize()
        refs = []
        for w in (y, norm, read):
            refs.append(pool.linear(x, w))
            torch.cuda.synchronize()
        sets.append((x, am, bm, ym, y, refs))
    w, z = torch.empty(384, 512, dtype=torch.bfloat16, device=DEV), torch.empty(tokens, 384, dtype=torch.bfloat16, device=DEV)
    wrong = torch.zeros(3, device=DEV)
    for i in range(210):
        x, am, bm, ym, y, refs = sets[i * 7 % 4]
        if i % 3 == 0:
            pool.mx_linear(am, bm, y=w)
        elif i % 3 == 1:
            pool.add_norm(y, None, ones, out=w)
        else:
            pool.mx_read(ym, out=w)
        pool.linear(x, w, y=z)
        wrong[i % 3] += (z != refs[i % 3]).any()
    assert wrong.tolist() == [0, 0, 0] and pool.check_errors() == 0


def test_another_stream(pool):
    s = torch.cuda.Stream()
    x, w = operands(300, 1024, 640, "mx8", seed=2)
    wm = pool.mx_quantize(w, "mx8")
    ref = pool.mx_linear(x, wm)
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        busy = torch.cuda._sleep
        with torch.cuda.stream(s):
            busy(2_000_000)
            late = x.clone()                       # ordered on s alone
        y = pool.mx_linear(late, wm, stream=handle)
        n, h = pool.add_norm(late, late, torch.ones(1024, dtype=torch.bfloat16, device=DEV), out="mx4", stream=handle)
        s.synchronize()
        assert torch.equal(y, ref) and torch.equal(h, x + x)
    assert pool.check_errors() == 0


def test_host_threads(pool):
    """Calls of several threads on their own streams over one pool."""
    x, w = operands(65, 512, 256, "mx4", seed=5)
    wm = pool.mx_quantize(w, "mx4")
    ref = pool.mx_linear(x, wm)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                if not torch.equal(pool.mx_linear(x, wm), ref):
                    bad.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and pool.check_errors() == 0


# ------------------------------------------------------------------ what rows and padding may hold

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [1, 20, 40, 130, 300])
def test_padding_of_the_scales_is_not_used(pool, kind, tokens):
    x, w = operands(tokens, 384, 1280, kind, seed=tokens)
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    ref = pool.mx_linear(xm, wm)
    rows = -(-tokens // 128) * 128
    tiles = xm.scales.view(rows // 128, 3, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows, 12)
    for fill in (255, 0, 254):
        tiles[tokens:] = fill
        other = pkv.MxTensor(kind, tokens, 384, xm.codes,
                             tiles.view(rows // 128, 4, 32, 3, 4).permute(0, 3, 2, 1, 4).contiguous().flatten())
        assert torch.equal(pool.mx_linear(other, wm), ref)
    assert pool.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [4, 40, 700])
def test_nan_stays_in_its_row_and_feature(pool, kind, tokens):
    x, w = operands(tokens, 512, 1280, kind, seed=tokens)
    clean = pool.mx_linear(x, pool.mx_quantize(w, kind))
    x[tokens // 2, 300], w[777, 13] = float("nan"), float("inf")
    y = pool.mx_linear(x, pool.mx_quantize(w, kind))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[tokens // 2], bad[:, 777] = True, True
    assert y[bad].isnan().all() and torch.equal(y[~bad], clean[~bad])
    assert pool.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_scales_of_any_size(pool, kind):
    """Groups from 2^-30 to 2^30 in one row, zero rows, and the ends of the scales' range."""
    gen = torch.Generator().manual_seed(2)
    x, w = operands(70, 1024, 128, kind, seed=9)
    for t in (x, w):
        e = torch.randint(-30, 31, (t.shape[0], 32), generator=gen).to(DEV)
        t.copy_((t.float().view(-1, 32, 32) * torch.exp2(e.float())[..., None]).view(t.shape).to(torch.bfloat16))
    x[3], w[5] = 0, 0
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    y = pool.mx_linear(xm, wm)
    check_product(y, _mx.stored(xm), _mx.stored(wm))
    assert (y[3] == 0).all() and (y[:, 5] == 0).all()
    x.fill_(2.0 ** 60)
    w.fill_(2.0 ** -120)
    assert torch.equal(pool.mx_linear(x, pool.mx_quantize(w, kind)), torch.full_like(y, 1024 * 2.0 ** -60))


def test_shared_rows_do_not_affect_each_other(pool):
    """A token's outputs are the same alone, in a small batch and in a large one (to the sums' order)."""
    x, w = operands(600, 2048, 1024, "mx8", seed=4)
    wm = pool.mx_quantize(w, "mx8")
    xm = pool.mx_quantize(x, "mx8")
    ref = pool.mx_linear(xm, wm)
    size = np.abs(_mx.stored(xm)[:1]) @ np.abs(_mx.stored(wm)).T
    for n in (1, 17, 64, 100, 300):
        y = pool.mx_linear(x[:n].contiguous(), wm)
        off = np.abs(_mx.f64(y[0]) - _mx.f64(ref[0]))
        assert (off <= 2.0 ** -7 * np.abs(_mx.f64(ref[0])) + 2048 * 2.0 ** -22 * size[0]).all()


# ------------------------------------------------------------------ large tensors

def test_more_than_2_31_elements():
    p = pool_of(1)
    rows, cols = 68000, 32768                      # 2.2e9 elements, 4.5 GB
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = _mx.activations(300, cols, seed=1).to(DEV)
    x[:300].copy_(tail.flip(0))
    x[-300:].copy_(tail)
    for kind in KINDS:
        t = p.mx_quantize(x, kind)
        some = p.mx_quantize(tail, kind)
        assert torch.equal(t.codes[-300:], some.codes)
        y = p.mx_read(t)
        assert torch.equal(y[-300:], p.mx_read(some)) and torch.equal(y[:300].flip(0), p.mx_read(some))
        del y, t
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    n, h = p.add_norm(x, x, w, out="mx4")
    some, h_some = p.add_norm(tail, tail, w, out="mx4")
    assert torch.equal(n.codes[-300:], some.codes) and torch.equal(h[-300:], h_some)
    back = p.mx_read(n)
    assert torch.equal(back[-300:], p.mx_read(some))
    assert p.check_errors() == 0
    p.close()


def test_product_of_more_than_2_31_elements():
    p = pool_of(1)
    tokens, n_in, n_out = 140000, 128, 16384       # y: 2.3e9 elements
    x = torch.zeros(tokens, n_in, dtype=torch.bfloat16, device=DEV)
    x[-500:].copy_(_mx.activations(500, n_in, seed=1).to(DEV))
    w = _mx.activations(n_out, n_in, seed=2, loud=False).to(DEV)
    wm = p.mx_quantize(w, "mx8")
    y = p.mx_linear(x, wm)
    assert torch.equal(y[-500:], p.mx_linear(x[-500:].contiguous(), wm)) and (y[:1000] == 0).all() and (y[70000:70500] == 0).all()
    assert p.check_errors() == 0
    p.close()
