"""Calls over a 4-bit pool and of norm + rotation: both ways of the binding, what they refuse, the split attention
in graphs and behind 32-bit offsets, and the entries of the other pool format."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import paged_kv_gqa_qk_gb300 as pkv
from test_gpu_q4 import DEV, check, f64, inputs, make, pool_of, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["module", "ctypes"])
def way(request, monkeypatch):
    """The binding with csrc/pkv_torch.cpp's module, and without it."""
    pkv.load_library()
    assert pkv._fast is not None, "the module of csrc/pkv_torch.cpp was not built"
    if request.param == "ctypes":
        monkeypatch.setattr(pkv, "_fast", None)
    return request.param


# ------------------------------------------------------------------ both ways

def _steps(wl, cache):
    """One of each call; every result on the host."""
    pool = pool_of(wl, cache)
    q, k, v, qw, kw, pos, table = inputs(wl)
    res = [pool.decode(q, k, v, qw, kw, pos, table)]
    res.append(pool.decode(q, k, v, qw, kw, pos, table, out=torch.empty_like(q), stream=torch.cuda.current_stream()))
    pool.append(v, k, kw, pos, None, table)
    rows = torch.arange(len(pos), dtype=torch.int32, device=DEV)
    pool.append(k[1:], v[1:], kw, pos[1:], rows[1:], table)
    res += pool.read(pos, rows, table)
    wide = torch.zeros(2, k.shape[1], len(pos) + 3, 128, dtype=torch.bfloat16, device=DEV)
    slots = wide[:, :, 1:1 + len(pos)].transpose(1, 2)
    pool.read(pos, None, table, slots[0], slots[1])
    res.append(wide)
    for layout in ("half", "interleaved"):
        res += pool.norm_rope(q, k, qw, kw, pos, layout)
    res += [pool.norm_rope(q, None, qw, None, pos, dtype=torch.float32)[0], pool.norm_rope(None, k, None, None, pos)[1]]
    both = torch.cat([q, k], 1)
    pool.norm_rope(both[:, :q.shape[1]], both[:, q.shape[1]:], qw, kw, pos, q_out=both[:, :q.shape[1]],
                   k_out=both[:, q.shape[1]:])
    res.append(both)
    assert pool.check_errors() == 0
    res = [r.cpu() for r in (*res, pool.data)]
    pool.close()
    return res


def test_both_ways_agree(monkeypatch):
    """The module's calls and the ctypes functions' give the same bytes, and the module took every one of them."""
    pkv.load_library()
    wl, cache = make([200, 1, 65], 2)
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
    mine = _steps(wl, cache)
    assert counts == {("decode", 0): 1, ("append", 0): 2, ("read", 0): 2, ("norm_rope", 0): 5}
    monkeypatch.setattr(pkv, "_fast", None)
    for a, b in zip(mine, _steps(wl, cache)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ refusals

def test_wrong_arguments_are_refused(way):
    """Types, shapes, strides and devices; the pool stays as it was and the next call is right."""
    wl, cache = make([100, 30], 2)
    pool = pool_of(wl, cache)
    q, k, v, qw, kw, pos, table = inputs(wl)
    good = dict(q=q, k=k, v=v, q_norm_w=qw, k_norm_w=kw, positions=pos, table=table)
    after = reference(wl, cache)[2]
    pool.decode(**good)                        # (the stream has its workspace: the calls below reach the checks)
    before = pool.data.clone()
    spaced = torch.empty(2, 16, 128, dtype=torch.bfloat16, device=DEV)[:, ::2]
    for name, bad in [("q", q.float()), ("q", q[:1]), ("q", q[:, :4]), ("q", spaced), ("q", q.cpu()), ("k", k[:, :1]),
                      ("k", k.half()), ("v", v[:1]), ("v", None), ("q_norm_w", qw[:64]), ("k_norm_w", kw[::2]),
                      ("k_norm_w", torch.cat([kw, kw])), ("k_norm_w", kw.cpu()), ("positions", pos.long()),
                      ("positions", pos[:1]), ("positions", pos.cpu()), ("table", table[:1]), ("table", table.long()),
                      ("table", table.t()), ("table", None), ("out", torch.empty_like(q).float()),
                      ("out", torch.empty_like(q[:1]))]:
        with pytest.raises((ValueError, TypeError, AttributeError)):
            pool.decode(**{**good, name: bad})
    for name, bad in [("k", k[:1]), ("v", v.float()), ("v", v[..., :64]), ("k_norm_w", kw[:8]), ("positions", pos[:1]),
                      ("prow", pos[:1]), ("prow", pos.long()), ("table", table.float()), ("table", None)]:
        args = dict(k=k, v=v, k_norm_w=kw, positions=pos, prow=None, table=table)
        with pytest.raises((ValueError, TypeError)):
            pool.append(**{**args, name: bad})
    to = [torch.zeros_like(k) for _ in range(2)]
    for kk, vv in [(to[0][:1], to[1]), (to[0].float(), to[1]), (to[0], to[1].transpose(1, 2).contiguous().transpose(1, 2)),
                   (to[0][..., ::2], to[1][..., ::2]), (to[0].cpu(), to[1].cpu())]:
        with pytest.raises((ValueError, TypeError)):
            pool.read(pos, None, table, kk, vv)
    with pytest.raises((ValueError, TypeError)):
        pool.read(pos, pos[:1], table, *to)
    with pytest.raises(pkv.PkvError) as e:     # more tokens than table rows
        pool.read(pos, None, table[:1], *to)
    assert e.value.code == pkv.PKV_EINVAL
    off = torch.empty(2 * 2 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 2, 128)
    with pytest.raises(pkv.PkvError) as e:     # not on a 16-byte border
        pool.append(off, v, kw, pos, None, table)
    assert e.value.code == pkv.PKV_EINVAL
    assert torch.equal(pool.data, before) and not to[0].any() and not to[1].any() and pool.check_errors() == 0
    assert np.array_equal(before.cpu().numpy().reshape(after.data.shape), after.data)
    got = pool.decode(**good)
    check(got, *reference(wl, cache)[:2])
    pool.close()
    with pytest.raises((pkv.PkvError, AttributeError, TypeError)):
        pool.decode(**good)                    # closed


def test_norm_rope_refusals(way):
    z = torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16, device=DEV)
    pool = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=8, kv_heads=2, max_seq=4096))
    gen = torch.Generator().manual_seed(0)
    q, k = (torch.randn(3, h, 128, generator=gen).to(torch.bfloat16).to(DEV) for h in (8, 2))
    w, pos = torch.ones(128, dtype=torch.bfloat16, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)
    ref = pool.norm_rope(q, k, w, w, pos)
    good = dict(q=q, k=k, q_norm_w=w, k_norm_w=w, positions=pos)
    for name, bad in [("q", q.float()), ("q", q[:2]), ("q", q[:, :7]), ("q", q.cpu()), ("q", q.transpose(0, 1)),
                      ("q", q[..., ::2]), ("k", k[:, ::2]), ("q_norm_w", w[:64]), ("k_norm_w", w.float()),
                      ("positions", pos.long()), ("positions", pos[:2]), ("dtype", torch.float16),
                      ("q_out", torch.empty(3, 8, 128, device=DEV)), ("k_out", torch.empty_like(k[:1])),
                      ("q_out", torch.empty(3, 8, 256, dtype=torch.bfloat16, device=DEV)[..., ::2])]:
        with pytest.raises((ValueError, TypeError)):
            pool.norm_rope(**{**good, name: bad})
    with pytest.raises((KeyError, ValueError)):
        pool.norm_rope(**good, layout="other")
    with pytest.raises(ValueError):
        pkv.pkv_norm_rope(pool.handle, q, k, w, w, pos, None, torch.empty_like(k))
    with pytest.raises((pkv.PkvError, ValueError)):
        pool.norm_rope(None, None, w, w, pos, q_out=None, k_out=None)
    off = torch.empty(3 * 2 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(3, 2, 128)
    with pytest.raises(pkv.PkvError) as e:
        pool.norm_rope(q, off, w, w, pos)
    assert e.value.code == pkv.PKV_EINVAL
    assert all(torch.equal(a, b) for a, b in zip(pool.norm_rope(**good), ref))
    pool.close()


@pytest.mark.parametrize("ctas", [0, 152])
def test_weights_on_an_8_byte_border(ctas):
    """Norm weights inside a larger tensor: 8 bytes off a 16-byte border as any others, 4 off refused."""
    wl, cache = make([100, 30, 70], 8)
    pool = pool_of(wl, cache, ctas)
    q, k, v, qw, kw, pos, table = inputs(wl)
    both = torch.zeros(2, 132, dtype=torch.bfloat16, device=DEV)
    both[0, 4:], both[1, :128] = qw, kw
    qw8, kw8 = both[0, 4:], both[1, :128]
    assert qw8.data_ptr() % 16 == 8 and kw8.data_ptr() % 16 == 8
    ref, bound, after = reference(wl, cache)
    check(pool.decode(q, k, v, qw8, kw8, pos, table), ref, bound)
    pool.append(k, v, kw8, pos, None, table)
    assert pool.check_errors() == 0
    assert np.array_equal(pool.data.cpu().numpy().reshape(after.data.shape), after.data)
    odd = torch.zeros(130, dtype=torch.bfloat16, device=DEV)[2:]
    for call in (lambda: pool.decode(q, k, v, odd, kw, pos, table), lambda: pool.decode(q, k, v, qw, odd, pos, table),
                 lambda: pool.append(k, v, odd, pos, None, table), lambda: pool.norm_rope(q, k, odd, kw, pos)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.code == pkv.PKV_EINVAL
    pool.close()


def test_set_rope_refusals():
    wl, cache = make([20], 1)
    pool = pool_of(wl, cache)
    freq, _ = pkv.pkv_rope_frequencies(wl.cfg)
    with pytest.raises(ValueError):
        pool.set_rope(freq[:-1])
    for bad, m in [([float("nan")] + freq[1:], 1.0), ([-1.0] + freq[1:], 1.0), (freq, 0.0), (freq, float("nan")),
                   (freq, 2048.0)]:
        with pytest.raises(pkv.PkvError) as e:
            pool.set_rope(bad, m)
        assert e.value.code == pkv.PKV_EINVAL
    check(pool.decode(*inputs(wl)), *reference(wl, cache)[:2])
    pool.close()


def test_captured_calls_take_the_rotation_that_is_set_later():
    """A graph captured before set_rope replays with the new tables at the same accuracy: 4 million bytes, of which
    a k held in 24 bits instead of pairs of floats would move some."""
    n, cfg = 4096, dict(heads=32, kv_heads=8, max_seq=4096)
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(n, 8, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    kw = (torch.rand(128, generator=gen) + 0.5).to(torch.bfloat16).to(DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.arange(n // 64, dtype=torch.int32, device=DEV)[None]
    row = pos * 0
    pool, twin = (pkv.Q4KVPool.empty(n // 64, cfg) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pool.append(k, v, kw, pos, row, table)
    freq, _ = pkv.pkv_rope_frequencies(cfg, "linear", 2.0)
    for p in (pool, twin):
        p.set_rope(freq, 1000.0)
    graph.replay()
    twin.append(k, v, kw, pos, row, table)
    torch.cuda.synchronize()
    assert twin.data.any() and (pool.data != twin.data).sum() == 0
    assert pool.check_errors() == 0 and twin.check_errors() == 0
    pool.close()
    twin.close()


def test_each_format_refuses_the_others_entries():
    """Nothing is launched: the codes come back before any pointer is used."""
    wl, cache = make([20], 1)
    q4 = pool_of(wl, cache)
    z = torch.zeros(2, 1, 64, 128, dtype=torch.bfloat16, device=DEV)
    bf16 = pkv.PagedKVPool(z[0], z[1], cfg=wl.cfg)
    lib, n = pkv.load_library(), ctypes.c_size_t()
    x = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    p, s, e = x.data_ptr(), None, pkv.PKV_EINVAL
    assert lib.pkv_q4_append(bf16.handle, p, p, p, p, None, p, 1, 1, 1, s) == e
    assert lib.pkv_q4_read(bf16.handle, p, None, p, 1, 1, 1, p, p, 128, 128, s) == e
    assert lib.pkv_q4_decode(bf16.handle, p, p, p, p, p, p, p, 1, 1, p, p, 1 << 16, s) == e
    assert lib.pkv_q4_pool_data(bf16.handle, None, ctypes.byref(n)) == e
    assert lib.pkv_decode(q4.handle, p, p, p, p, p, p, p, 1, 1, p, p, 1 << 16, s) == e
    assert lib.pkv_decode_static(q4.handle, p, p, p, p, p, p, p, 1, 1, p, s) == e
    assert lib.pkv_step(q4.handle, p, p, p, p, p, p, p, p, p, p, 1, 1, 1, p, p, 1 << 16, s) == e
    assert lib.pkv_prefill(q4.handle, p, p, p, p, p, p, p, p, p, 1, 1, 1, p, p, 1 << 16, s) == e
    assert lib.pkv_decode_appended(q4.handle, p, p, p, 1, 1, p, p, 1 << 16, s) == e
    assert lib.pkv_qkv_proj_append(q4.handle, p, p, 1, 128, p, p, p, p, 1, p, s) == e
    assert pkv.pkv_pool_kv(q4.handle)[:2] == (None, None)
    torch.cuda.synchronize()
    assert not x.any() and q4.check_errors() == 0 and bf16.check_errors() == 0
    check(q4.decode(*inputs(wl)), *reference(wl, cache)[:2])
    q4.close()
    bf16.close()


def test_a_workspace_that_is_too_small():
    wl, cache = make([3000] * 8, 2)
    for ctas in (0, 152):
        pool = pool_of(wl, cache, ctas)
        args = inputs(wl)
        n = pkv.pkv_workspace_bytes(pool.handle, 8, wl.pages)
        out = torch.zeros_like(args[0])
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_q4_decode(pool.handle, *args, out, torch.empty(n - 1, dtype=torch.uint8, device=DEV))
        assert e.value.code == pkv.PKV_EWORKSPACE
        torch.cuda.synchronize()
        assert not out.any() and np.array_equal(pool.data.cpu().numpy().reshape(cache.data.shape), cache.data)
        ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        pkv.pkv_q4_decode(pool.handle, *args, out, ws[:n])
        check(out, *reference(wl, cache)[:2])
        assert (ws[n:] == 0xA5).all()          # nothing behind the size that was asked for
        pool.close()


# ------------------------------------------------------------------ the split attention

def test_split_attention_replays_from_graphs_beside_eager_calls():
    """As the small calls: two captured steps and eager ones on other streams, each with its own workspace."""
    wl, cache = make([300 + 77 * i for i in range(12)], 2)
    pool = pool_of(wl, cache, 152)
    q, k, v, qw, kw, pos, table = inputs(wl)
    ref = pool.decode(q, k, v, qw, kw, pos, table)
    check(ref, *reference(wl, cache)[:2])
    small = [x[:3].contiguous() for x in (q, k, v, pos, table)]
    outs = [torch.zeros_like(q), torch.zeros_like(small[0])]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0]):
        pool.decode(q, k, v, qw, kw, pos, table, out=outs[0])
    with torch.cuda.graph(graphs[1]):
        pool.decode(*small[:3], qw, kw, *small[3:], out=outs[1])
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        eager = pool.decode(q, k, v, qw, kw, pos, table)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref) and torch.equal(eager, ref)
        check(outs[1], *[x[:3] for x in reference(wl, cache)[:2]])
    assert pool.check_errors() == 0
    pool.close()


@pytest.mark.parametrize("rows,length,kv_heads,ctas", [
    (1, 4096, 8, 0), (1, 4033, 1, 0), (2, 2500, 2, 0), (3, 900, 3, 0),     # clusters of 16, 16, 16 and 4 CTAs a unit
    (1, 4096, 1, 152), (1, 3500, 8, 152), (5, 1500, 4, 152),               # 16, 16 and 8 warps for a head's pieces
    (40, 400, 4, 152), (80, 600, 4, 152)])                                 # 4, and one
def test_few_rows_many_pieces(rows, length, kv_heads, ctas):
    """Long rows cut among many warps, in either form of the call."""
    wl, cache = make([length - 7 * b for b in range(rows)], kv_heads, max_seq=4096)
    pool = pool_of(wl, cache, ctas)
    ref, bound, after = reference(wl, cache)
    check(pool.decode(*inputs(wl)), ref, bound)
    assert pool.check_errors() == 0
    assert np.array_equal(pool.data.cpu().numpy().reshape(after.data.shape), after.data)
    pool.close()


def test_split_attention_beyond_32_bit_offsets():
    """Rows whose pages lie behind byte 2^32 of a pool, read by many CTAs."""
    n, cfg = 60000, dict(heads=32, kv_heads=8, max_seq=4096)
    data = torch.zeros(n, 8, 4, 2304, dtype=torch.uint8, device=DEV)
    assert data.numel() > 2 ** 32
    wl, cache = make([1300, 64, 700], 8)
    P = cache.data.shape[0]
    data[n - P:] = torch.from_numpy(cache.data).to(DEV)
    pool = pkv.Q4KVPool(data, cfg)
    pkv.pkv_set_ctas(pool.handle, 152)
    q, k, v, qw, kw, pos, table = inputs(wl)
    out = pool.decode(q, k, v, qw, kw, pos, table + (n - P))
    assert pool.check_errors() == 0
    ref, bound, after = reference(wl, cache)
    check(out, ref, bound)
    assert np.array_equal(data[n - P:].cpu().numpy(), after.data) and not data[:8].any()
    pool.close()


@pytest.mark.parametrize("ctas", [0, 152])
def test_host_threads_on_their_own_streams(ctas):
    """Four threads of the host, a stream each, over one pool: every call of each gives the same bits."""
    wl, cache = make([400, 90, 1, 777], 2)
    pool = pool_of(wl, cache, ctas)
    args = inputs(wl)
    ref = pool.decode(*args)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                outs = [pool.decode(*args) for _ in range(25)]
                kv = [pool.read(args[5], None, args[6])[0] for _ in range(5)]
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(o, ref) for o in outs) or not all(torch.equal(x, kv[0]) for x in kv):
                    bad.append("different")
        except Exception as e:
            bad.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and pool.check_errors() == 0
    pool.close()


def test_steps_follow_one_another():
    """Many steps in a row without a wait between them: each attends over what the ones before it appended."""
    wl, cache = make([60, 5, 130], 2)
    q, k, v, qw, kw, pos, table = inputs(wl)
    step = torch.tensor([1, 0, 1], dtype=torch.int32, device=DEV)   # (row 1 rewrites its last position)
    for ctas in (0, 152):
        pool, twin = pool_of(wl, cache, ctas), pool_of(wl, cache, ctas)
        seen, want = [], []
        where = [pos + i * step for i in range(4)]
        torch.cuda.synchronize()
        for i, p in enumerate(where):
            seen.append(pool.decode(q.roll(i, 1), k.roll(i, 2), v, qw, kw, p, table))
        for i, p in enumerate(where):
            want.append(twin.decode(q.roll(i, 1), k.roll(i, 2), v, qw, kw, p, table).cpu())
            torch.cuda.synchronize()
        assert all(np.array_equal(f64(a), f64(b)) for a, b in zip(seen, want))
        assert torch.equal(pool.data, twin.data)
        pool.close()
        twin.close()
