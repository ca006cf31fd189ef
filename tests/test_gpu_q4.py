"""The 4-bit pool on the GPU against the 64-bit form of tests/_q4.py: appended bytes and read-back values
exactly, the decode attention within the bound that its roundings give."""
import numpy as np
import pytest
import torch

import _q4
import paged_kv_gqa_qk_gb300 as pkv
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().cpu().double().numpy()


def make(lengths, kv_heads=8, ks=1.0, vs=1.0, seed=0, rot=128, **kw):
    """A decode workload, its 4-bit cache (numpy) and the same bytes on the GPU in a pool."""
    cfg = dict(heads=4 * kv_heads, kv_heads=kv_heads, rotary_dim=rot, max_seq=kw.pop("max_seq", 4096))
    live = [max(n, 1) for n in lengths]
    wl = W.make_decode("q4", live, seed=seed, cfg=cfg, **kw)
    wl.step_positions = torch.tensor([n - 1 for n in lengths], dtype=torch.int32)
    cache = _q4.Cache.of(f64(wl.K0), f64(wl.V0) * vs, ks, vs)
    return wl, cache


def pool_of(wl, cache, ctas=0):
    pool = pkv.Q4KVPool(torch.from_numpy(cache.data.copy()).to(DEV), cfg=wl.cfg, k_scale=cache.ks, v_scale=cache.vs)
    if ctas:
        pkv.pkv_set_ctas(pool.handle, ctas)
    return pool


def inputs(wl, vs=1.0):
    return [t.to(DEV) for t in (wl.q, wl.k, (wl.v.float() * vs).to(torch.bfloat16), wl.q_norm_w, wl.k_norm_w,
                                wl.step_positions, wl.table)]


def reference(wl, cache, vs=1.0, skip=()):
    """(out, bound, cache after the step)."""
    after = _q4.Cache(cache.data.copy(), cache.ks, cache.vs)
    pos, table, rot = wl.step_positions.numpy(), wl.table.numpy(), wl.cfg["rotary_dim"]
    at = np.maximum(pos, 0)
    q = _q4.norm_rope(f64(wl.q), f64(wl.q_norm_w), at, rot)
    k = _q4.bf16(_q4.norm_rope(f64(wl.k), f64(wl.k_norm_w), at, rot))
    v = f64((wl.v.float() * vs).to(torch.bfloat16))
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(pos):
        if n >= 0 and b not in skip:
            after.put(table[b, n // 64], n, k[b], v[b])
    for b, n in enumerate(pos):
        if n >= 0 and b not in skip:
            out[b], bound[b] = _q4.attend(q[b], *after.get(table[b], n + 1))
    return out, bound, after


def check(out, ref, bound):
    got = f64(out)
    tol = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    off = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (off <= tol).all(), f"{(off > tol).sum()} of {off.size} outside; worst {(off - tol).max():.3e} over, " \
                               f"at {np.unravel_index(np.argmax(off - tol), off.shape)}"


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("kv_heads,ks,vs,rot", [(8, 1.0, 1.0, 128), (1, 0.5, 2.0 ** -6, 128), (2, 4.0, 16.0, 32), (3, 1.0, 1.0, 96)])
def test_append_bytes(kv_heads, ks, vs, rot):
    """Ragged prompt chunks, one from inside a block: the pool's bytes are the definition's, all of them."""
    cfg = dict(heads=4 * kv_heads, kv_heads=kv_heads, max_seq=4096, rotary_dim=rot)
    wl = W.make_prefill("q4 append", [70, 1, 130, 33], [61, 0, 1000, 15], seed=5, cfg=cfg)
    cache = _q4.Cache.of(f64(wl.K0), f64(wl.V0), ks, vs)
    pool = pool_of(wl, cache)
    P = wl.P
    pos, prow, table = wl.positions.numpy(), wl.prow.numpy(), wl.table.numpy()
    v = (wl.v[:P].float() * vs).to(torch.bfloat16)
    pool.append(wl.k[:P].to(DEV), v.to(DEV), wl.k_norm_w.to(DEV), wl.positions.to(DEV), wl.prow.to(DEV), wl.table.to(DEV))
    assert pool.check_errors() == 0
    k = _q4.bf16(_q4.norm_rope(f64(wl.k[:P]), f64(wl.k_norm_w), pos, rot))
    for t in range(P):
        cache.put(table[prow[t], pos[t] // 64], pos[t], k[t], f64(v[t]))
    got = pool.data.cpu().numpy().reshape(cache.data.shape)
    assert np.array_equal(got, cache.data), f"{(got != cache.data).sum()} bytes differ"
    kk, vv = pool.read(wl.positions.to(DEV), wl.prow.to(DEV), wl.table.to(DEV))
    for r in range(4):
        at = np.nonzero(prow == r)[0]
        K, V = cache.get(table[r], pos[at[-1]] + 1)
        assert np.array_equal(f64(kk)[at], K[pos[at]]) and np.array_equal(f64(vv)[at], V[pos[at]])
    pool.close()


def test_quantiser_borders():
    """v as given: every bf16 of a binade around each tie, groups of zeros, the smallest and largest values,
    and groups with Inf and NaN, which read back as NaN while their neighbours do not change."""
    rng = np.random.RandomState(1)
    n = 64
    top = np.repeat(np.linspace(1.0, 8.0, n), 8).reshape(n, 8, 1)
    z = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0, 6.0], size=(n, 8, 16)) * rng.choice([-1, 1], (n, 8, 16))
    v = z * _q4.e4m3(_q4.bf16(top) / 6)       # values on the ties of a scale near top / 6
    v[..., :1] = _q4.bf16(top)
    v = v.reshape(n, 1, 128)
    v[0] = 0.0
    v[1] = 2.0 ** -133                          # bf16's smallest
    v[2] = 3.0e38
    v[3, 0, 16:32] *= 2.0 ** -11                # a scale among the subnormals
    v[4, 0, 5] = np.inf
    v[5, 0, 40] = np.nan
    v = torch.from_numpy(v).to(torch.bfloat16)
    cfg = dict(heads=4, kv_heads=1, max_seq=64)
    pool = pkv.Q4KVPool.empty(1, cfg)
    k = torch.randn(n, 1, 128).to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    row = torch.zeros(n, dtype=torch.int32, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    pool.append(k.to(DEV), v.to(DEV), w, pos.to(DEV), row, table)
    _, got = pool.read(pos.to(DEV), row, table)
    assert pool.check_errors() == 0
    ref = _q4.values(*_q4.quantise(f64(v), 1.0), 1.0)
    nan = np.isnan(ref)
    assert nan.sum() == 32 and np.array_equal(np.isnan(f64(got)), nan)
    assert np.array_equal(f64(got)[~nan], ref[~nan])
    pool.close()


def test_untouched_positions_and_skipped_tokens():
    """Only written positions change; -1 and bad rows, positions and pages write nothing and read as zeros."""
    cfg = dict(heads=8, kv_heads=2, max_seq=256)
    data = torch.randint(0, 256, (5, 2, 4, 2304), dtype=torch.uint8, device=DEV)
    pool = pkv.Q4KVPool(data.clone(), cfg)
    table = torch.tensor([[1, 2, 99], [3, -1, 4]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([-1, 192, 3, 300, 64, 130, 17], dtype=torch.int32, device=DEV)
    row = torch.tensor([0, 0, 7, 0, 1, 0, 0], dtype=torch.int32, device=DEV)
    x = torch.randn(7, 2, 128, device=DEV).to(torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    pool.append(x, x, w, pos, row, table)
    assert pool.check_errors() == pkv.PKV_DEVERR_POSITION | pkv.PKV_DEVERR_ROW | pkv.PKV_DEVERR_PAGE
    k, v = (torch.full((7, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pool.read(pos, row, table, k, v)
    assert pool.check_errors() == pkv.PKV_DEVERR_POSITION | pkv.PKV_DEVERR_ROW | pkv.PKV_DEVERR_PAGE
    assert (k[:6] == 0).all() and (v[:6] == 0).all() and (v[6] != 0).any()
    same = pool.data == data
    blk = same.view(5, 2, 4, 2304)
    changed = (~blk).cpu().numpy()
    i = 17 % 16
    allowed = np.zeros(2304, bool)
    allowed[np.concatenate([_q4.CODE[i], 1024 + _q4.CODE[i], 2048 + _q4.KS[i], 2176 + _q4.VS[i]])] = True
    assert changed[1, :, 1].any() and not changed[1, :, 1][:, ~allowed].any()
    changed[1, :, 1] = False
    assert not changed.any()
    pool.close()


def test_read_into_a_bf16_pools_slots():
    wl, cache = make([200, 77], kv_heads=2)
    pool = pool_of(wl, cache)
    K = torch.full((2, 6 * 64, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    V = K.clone()
    pos = torch.arange(200, dtype=torch.int32, device=DEV)
    row = torch.zeros(200, dtype=torch.int32, device=DEV)
    pool.read(pos, row, wl.table.to(DEV), K[:, 64:264].transpose(0, 1), V[:, 64:264].transpose(0, 1))
    rk, rv = cache.get(wl.table[0].numpy(), 200)
    assert np.array_equal(f64(K[:, 64:264]), rk.transpose(1, 0, 2)) and np.array_equal(f64(V[:, 64:264]), rv.transpose(1, 0, 2))
    for x in (K, V):
        assert (x[:, :64] == 3).all() and (x[:, 264:] == 3).all()
    pool.close()


# ------------------------------------------------------------------ decode

LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 0, 127, 128, 129, 700, 1025]


@pytest.mark.parametrize("kv_heads,ks,vs", [(8, 1.0, 1.0), (1, 0.25, 2.0 ** -8), (3, 2.0, 64.0)])
@pytest.mark.parametrize("ctas", [0, 1, 7, 152])
def test_decode(kv_heads, ks, vs, ctas):
    """ctas 0: one launch for a call of this size; a set grid: the split attention."""
    wl, cache = make(LENGTHS, kv_heads, ks, vs, seed=kv_heads)
    pool = pool_of(wl, cache, ctas)
    out = pool.decode(*inputs(wl, vs))
    assert pool.check_errors() == 0
    ref, bound, after = reference(wl, cache, vs)
    check(out, ref, bound)
    assert (f64(out)[LENGTHS.index(0)] == 0).all()
    assert np.array_equal(pool.data.cpu().numpy().reshape(after.data.shape), after.data)
    again = pool.decode(*inputs(wl, vs))      # the same step again: the same bits
    assert torch.equal(out, again)
    pool.close()


@pytest.mark.parametrize("lengths,kw", [
    ([1 + (37 * i) % 90 for i in range(600)], dict(kv_heads=2)),             # many short rows
    ([512 + (997 * i) % 3000 for i in range(16)], dict(kv_heads=2, share_groups=8)),   # shared prefixes
    ([700], {}), ([3], dict(kv_heads=1)), ([4096, 4001], dict(kv_heads=2)),  # few units, 8, 1 and 4
    ([1, 64, 65, 0, 300, 256, 257], dict(kv_heads=6)),                       # one CTA a unit, more units than that
    ([5, 100], dict(kv_heads=2, table_pages=700)),                           # a table far wider than the rows
    ([2500, 40, 0, 2000], dict(kv_heads=1, table_pages=700)),
])
@pytest.mark.parametrize("ctas", [0, 152])
def test_decode_batches(lengths, kw, ctas):
    wl, cache = make(lengths, seed=len(lengths), **dict(kw))
    pool = pool_of(wl, cache, ctas)
    out = pool.decode(*inputs(wl))
    assert pool.check_errors() == 0
    ref, bound, after = reference(wl, cache)
    check(out, ref, bound)
    assert np.array_equal(pool.data.cpu().numpy().reshape(after.data.shape), after.data)
    pool.close()


@pytest.mark.parametrize("rot", [32, 64, 96])
@pytest.mark.parametrize("ctas", [0, 152])
def test_decode_partial_rotation(rot, ctas):
    wl, cache = make([5, 100, 333], 2, rot=rot)
    pool = pool_of(wl, cache, ctas)
    out = pool.decode(*inputs(wl))
    check(out, *reference(wl, cache)[:2])
    pool.close()


def test_decode_contiguous_rows():
    wl, cache = make([640, 1, 64, 200], 2, table_pages=10, contiguous=True)
    pool = pool_of(wl, cache)
    q, k, v, qw, kw, pos, _ = inputs(wl)
    out = pool.decode(q, k, v, qw, kw, pos, None, pages=10)
    assert pool.check_errors() == 0
    check(out, *reference(wl, cache)[:2])
    with pytest.raises(pkv.PkvError) as e:
        pool.decode(q, k, v, qw, kw, pos, None, pages=11)
    assert e.value.code == pkv.PKV_ERANGE
    pool.close()


@pytest.mark.parametrize("ctas", [0, 152])
def test_what_lies_behind_a_row_is_not_seen(ctas):
    """Every byte of the pool that no row's positions own is 0xff: codes of -6 and scales of NaN."""
    wl, cache = make([1, 17, 40, 64, 90], 2)
    own = np.zeros(cache.data.shape, bool)
    for b, n in enumerate(wl.step_positions.tolist()):
        for s in range(n):
            i = s % 16
            at = np.concatenate([_q4.CODE[i], 1024 + _q4.CODE[i], 2048 + _q4.KS[i], 2176 + _q4.VS[i]])
            own[wl.table[b, s // 64], :, s % 64 // 16][:, at] = True
    cache.data[~own] = 0xff
    pool = pool_of(wl, cache, ctas)
    out = pool.decode(*inputs(wl))
    assert pool.check_errors() == 0
    check(out, *reference(wl, cache)[:2])
    pool.close()


def test_precheck(monkeypatch):
    """PKV_CHECK=1: a row that reads another row's new slot, and two rows that write one slot, are refused."""
    monkeypatch.setenv("PKV_CHECK", "1")
    wl, cache = make([40, 41, 90], 2)
    pool = pool_of(wl, cache)
    q, k, v, qw, kw, pos, table = inputs(wl)
    check(pool.decode(q, k, v, qw, kw, pos, table), *reference(wl, cache)[:2])
    same = table.clone()
    same[1, 0] = same[0, 0]               # row 1 attends past the position that row 0 writes
    for p, tab in ((pos, same), (torch.tensor([39, 39, 89], dtype=torch.int32, device=DEV), same)):
        with pytest.raises(pkv.PkvError) as e:
            pool.decode(q, k, v, qw, kw, p, tab)
        assert e.value.code == pkv.PKV_EINVAL
    pool.append(k, v, kw, pos, None, same)    # distinct slots, and nothing is read
    row = torch.zeros(3, dtype=torch.int32, device=DEV)
    with pytest.raises(pkv.PkvError) as e:
        pool.append(k, v, kw, row + 7, row, table)
    assert e.value.code == pkv.PKV_EINVAL and pool.check_errors() == 0
    pool.close()


@pytest.mark.parametrize("ctas", [0, 152])
def test_bad_rows_give_zeros_and_leave_the_others(ctas):
    wl, cache = make([100, 100, 70, 200, 9], 2, max_seq=300)
    wl.table[1, 0] = -5              # a page before the written one
    wl.table[2, 1] = wl.num_pages    # the written page
    wl.step_positions[3] = 256       # beyond the table
    wl.step_positions[4] = -7
    before = cache.data.copy()
    pool = pool_of(wl, cache, ctas)
    out = pool.decode(*inputs(wl))
    assert pool.check_errors() == pkv.PKV_DEVERR_PAGE | pkv.PKV_DEVERR_POSITION
    wl.step_positions[3:] = -1
    ref, bound, after = reference(wl, _q4.Cache(before), skip=(1, 2))
    check(out, ref, bound)
    assert (f64(out)[1:] == 0).all()
    assert np.array_equal(pool.data.cpu().numpy().reshape(after.data.shape), after.data)
    pool.close()


@pytest.mark.parametrize("ctas", [0, 152])
def test_nan_stays_in_its_row(ctas):
    wl, cache = make([80, 80, 80], 2)
    v = wl.v.clone()
    v[1, 0, 3] = float("nan")
    wl.v = v
    pool = pool_of(wl, cache, ctas)
    out = f64(pool.decode(*inputs(wl)))
    assert np.isnan(out[1, :4, :16]).all() and np.isfinite(out[1, 4:]).all() and np.isfinite(out[1, :4, 16:]).all()
    assert np.isfinite(out[[0, 2]]).all()
    pool.close()


@pytest.mark.parametrize("ctas", [0, 152])
def test_sizes_of_q(ctas):
    """Queries of any size: weights of 2^-40 and 2^40 (scores near 0, and a one-hot softmax)."""
    wl, cache = make([300, 33], 2)
    small, big = wl.q_norm_w.clone() * 2.0 ** -40, wl.q_norm_w.clone() * 2.0 ** 6
    for w in (small, big):
        wl.q_norm_w = w
        pool = pool_of(wl, cache, ctas)
        out = pool.decode(*inputs(wl))
        check(out, *reference(wl, cache)[:2])
        pool.close()


def test_pages_beyond_32_bit_offsets():
    """A pool of over 2^32 bytes: rows whose pages lie at its end."""
    n, cfg = 60000, dict(heads=32, kv_heads=8, max_seq=4096)
    data = torch.zeros(n, 8, 4, 2304, dtype=torch.uint8, device=DEV)
    assert data.numel() > 2 ** 32
    wl, cache = make([130, 64], 8)
    P = cache.data.shape[0]
    data[n - P:] = torch.from_numpy(cache.data).to(DEV)
    pool = pkv.Q4KVPool(data, cfg)
    q, k, v, qw, kw, pos, table = inputs(wl)
    out = pool.decode(q, k, v, qw, kw, pos, table + (n - P))
    assert pool.check_errors() == 0
    ref, bound, after = reference(wl, cache)
    check(out, ref, bound)
    assert np.array_equal(data[n - P:].cpu().numpy(), after.data) and not data[:8].any()
    t = torch.tensor([129], dtype=torch.int32, device=DEV)
    kk, _ = pool.read(t, t * 0, table + (n - P))
    assert np.array_equal(f64(kk)[0], after.get(wl.table[0].numpy(), 130)[0][129])
    pool.close()


# ------------------------------------------------------------------ streams, graphs, waits

def test_decode_replays_from_graphs_beside_eager_calls():
    """Two captured steps of different sizes and eager calls of one pool: each keeps its own workspace."""
    wl, cache = make([300 + 50 * i for i in range(12)], 2)
    pool = pool_of(wl, cache)
    q, k, v, qw, kw, pos, table = inputs(wl)
    ref = pool.decode(q, k, v, qw, kw, pos, table)
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


def test_other_streams():
    wl, cache = make([200, 1000], 2)
    pool = pool_of(wl, cache)
    args = inputs(wl)
    ref = pool.decode(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [pool.decode(*args, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    pool.close()


def test_a_wait_that_runs_out_is_reported():
    """A limit of 0 gives up at the first copy that is not there yet (the cache is pushed out of L2 first)."""
    wl, cache = make([3000] * 40, 2)
    pool = pool_of(wl, cache)
    args = inputs(wl)
    ref = pool.decode(*args)
    assert pool.check_errors() == 0
    pkv.pkv_set_wait_limit(pool.handle, 0)
    torch.empty(1 << 28, dtype=torch.float32, device=DEV).fill_(1.0)
    pool.decode(*args)
    assert pool.check_errors() == pkv.PKV_DEVERR_TIMEOUT
    pkv.pkv_set_wait_limit(pool.handle, 10 ** 9)
    assert torch.equal(pool.decode(*args), ref) and pool.check_errors() == 0
    pool.close()


def test_timer_counts_the_attention():
    wl, cache = make([500, 20], 2)
    pool = pool_of(wl, cache)
    pkv.pkv_timer_enable(pool.handle, 1)
    for _ in range(3):
        out = pool.decode(*inputs(wl))
    ms, n = pkv.pkv_timer_read(pool.handle)
    assert n == 3 and 0 < ms < 1000
    pkv.pkv_timer_enable(pool.handle, 0)
    check(out, *reference(wl, cache)[:2])
    pool.close()


# ------------------------------------------------------------------ together

def test_prompt_decode_and_next_chunk():
    """A prompt through pkv_prefill on scratch pages and appended in 4 bits, decode steps over the 4-bit pool, then
    the row's prefix read back to the scratch pages and a second chunk over it."""
    import oracle
    cfg = dict(W.DEFAULT_CONFIG, heads=8, kv_heads=2, max_seq=512)
    gen = torch.Generator().manual_seed(3)
    n1, steps, n2, pages = 150, 5, 40, 4
    total = n1 + steps + n2
    q, k, v, qw, kw = W._tokens(gen, cfg, total)
    scratch = [torch.zeros(2, pages * 64, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    bf = pkv.PagedKVPool(*scratch, cfg=cfg)
    q4 = pkv.Q4KVPool.empty(pages + 1, cfg)
    table = torch.tensor([[4, 2, 1, 3]], dtype=torch.int32, device=DEV)
    g = [x.to(DEV) for x in (q, k, v, qw, kw)]
    zeros = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    pos = torch.arange(total, dtype=torch.int32, device=DEV)
    first = slice(0, n1)
    bf.prefill(g[0][first], g[1][first], g[2][first], g[3], g[4], pos[first], zeros(n1), None, None, rows=1, pages=pages)
    q4.append(g[1][first], g[2][first], g[4], pos[first], zeros(n1), table)
    cache = _q4.Cache(np.zeros((pages + 1, 2, 4, 2304), np.uint8))
    qh = _q4.norm_rope(f64(q), f64(qw), np.arange(total))
    kh = _q4.bf16(_q4.norm_rope(f64(k), f64(kw), np.arange(total)))
    tab = table.cpu().numpy()[0]
    for s in range(n1):
        cache.put(tab[s // 64], s, kh[s], f64(v[s]))
    for s in range(n1, n1 + steps):
        one = slice(s, s + 1)
        out = q4.decode(g[0][one], g[1][one], g[2][one], g[3], g[4], pos[one], table)
        cache.put(tab[s // 64], s, kh[s], f64(v[s]))
        ref, bound = _q4.attend(qh[s], *cache.get(tab, s + 1))
        check(out, ref[None], bound[None])
    assert np.array_equal(q4.data.cpu().numpy().reshape(cache.data.shape), cache.data)
    # the second chunk: the prefix back in 16 bits, then the bf16 pool's own prompt attention
    n = n1 + steps
    q4.read(pos[:n], zeros(n), table, scratch[0][:, :n].transpose(0, 1), scratch[1][:, :n].transpose(0, 1))
    K0, V0 = cache.get(tab, n)
    assert np.array_equal(f64(scratch[0][:, :n]), K0.transpose(1, 0, 2))
    last = slice(n, total)
    out = bf.prefill(g[0][last], g[1][last], g[2][last], g[3], g[4], pos[last], zeros(n2), None, None, rows=1, pages=pages)
    Kb, Vb = (W.bits(x.cpu()).copy() for x in scratch)
    ref, err = oracle.step(Kb, Vb, *(W.bits(torch.cat([x[last], x[:1]])) for x in (q, k, v)), W.bits(qw), W.bits(kw),
                           np.arange(n, total, dtype=np.int32), np.zeros(n2, np.int32), None,
                           np.array([-1], np.int32), np.arange(pages, dtype=np.int32)[None], cfg=cfg)
    assert err == 0
    off = np.abs(f64(out) - ref[:n2])
    assert off.max() <= 2e-2 and np.linalg.norm(off) <= 5e-3 * np.linalg.norm(ref[:n2])   # the prompt attention's own bar
    assert bf.check_errors() == 0 and q4.check_errors() == 0
    bf.close()
    q4.close()


def test_projection_and_gate_take_a_4_bit_pool():
    cfg = dict(heads=4, kv_heads=1, max_seq=128)
    q4 = pkv.Q4KVPool.empty(2, cfg)
    x, w = W.make_linear(3, 128, 768, seed=1)
    q, k, v = (torch.empty(3, h, 128, dtype=torch.bfloat16, device=DEV) for h in (4, 1, 1))
    pkv.pkv_qkv_proj(q4.handle, x.to(DEV), w.to(DEV), q, k, v)
    ref = f64(x) @ f64(w).T
    got = np.concatenate([f64(t).reshape(3, -1) for t in (q, k, v)], 1)
    assert np.abs(got - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4
    q4.close()
