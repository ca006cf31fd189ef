"""The forms that large calls take, against the definition: appends and reads of 8 heads a warp, norm + rotation with
several groups of heads a warp, clusters of 16 CTAs, half pages in several rounds, the largest grid; and what the
binding's module refuses of calls that are right but for one argument."""
import threading

import numpy as np
import pytest
import torch

import _q4
import paged_kv_gqa_qk_gb300 as pkv
from test_gpu_norm_rope import check as check_norm_rope
from test_gpu_norm_rope import draws
from test_gpu_norm_rope import pool_of as bf16_pool_of
from test_gpu_q4 import DEV, check, f64, inputs, make, pool_of, reference

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def put_all(data, page, pos, x, s, off, at, so):
    """Quantises x [tokens][G][128] into the bytes of a pool [pages][G][4][2304] at positions pos of pages page."""
    code, byte = _q4.quantise(x, s)
    i, blk = pos % 16, pos % 64 // 16
    where = page[:, None, None], np.arange(data.shape[1])[None, :, None], blk[:, None, None]
    data[(*where, off + _q4.CODE[i][:, None, :])] = code[..., 0::2] | (code[..., 1::2] << 4)
    data[(*where, so + at[i][:, None, :])] = byte


# 8 heads a warp from 32 quads of heads an SM on; 5 and 6 heads leave the second quad half empty, 9 and 11 the last pair
@pytest.mark.parametrize("kv_heads,rot,more", [(8, 128, 0), (8, 32, 77), (5, 128, 1), (6, 96, 0), (9, 128, 3), (11, 64, 1),
                                               (8, 128, -1)])
def test_append_and_read_of_many_tokens(kv_heads, rot, more):
    """Three prompts whose tokens come in any order, around the count from which a warp takes 8 heads: every byte of the
    pool is the definition's, the positions beside the written ones keep theirs, and all read back."""
    quads = (kv_heads + 3) // 4
    n = -(-32 * sms() // quads) + more
    rng = np.random.RandomState(kv_heads + rot)
    ends = [n // 5, n // 2, n]
    row = np.searchsorted(ends, np.arange(n), side="right").astype(np.int32)
    start = np.array([17, 0, 333])
    pos = (np.arange(n) - np.array([0] + ends[:2])[row] + start[row]).astype(np.int32)
    order = rng.permutation(n)
    row, pos = row[order], pos[order]
    pages = -(-(int(pos.max()) + 1) // 64)
    table = (rng.permutation(3 * pages) + 1).astype(np.int32).reshape(3, pages)
    cfg = dict(heads=4 * kv_heads, kv_heads=kv_heads, max_seq=64 * pages, rotary_dim=rot)
    data = rng.randint(0, 256, (3 * pages + 1, kv_heads, 4, 2304)).astype(np.uint8)
    ks, vs = 0.5, 2.0
    pool = pkv.Q4KVPool(torch.from_numpy(data.copy()).to(DEV), cfg, k_scale=ks, v_scale=vs)
    k, v = (torch.from_numpy(rng.randn(n, kv_heads, 128)).to(torch.bfloat16) for _ in range(2))
    kw = torch.from_numpy(rng.rand(128) + 0.5).to(torch.bfloat16)
    at = [torch.from_numpy(x).to(DEV) for x in (pos, row, table)]
    pool.append(k.to(DEV), v.to(DEV), kw.to(DEV), *at)
    assert pool.check_errors() == 0
    page = table[row, pos // 64].astype(np.int64)
    put_all(data, page, pos, _q4.bf16(_q4.norm_rope(f64(k), f64(kw), pos, rot)), ks, 0, _q4.KS, 2048)
    put_all(data, page, pos, f64(v), vs, 1024, _q4.VS, 2176)
    got = pool.data.cpu().numpy().reshape(data.shape)
    assert np.array_equal(got, data), f"{(got != data).sum()} bytes differ"
    kk, vv = (f64(x) for x in pool.read(*at))
    cache = _q4.Cache(data, ks, vs)
    for r in range(3):
        mine = row == r
        K, V = cache.get(table[r], int(pos[mine].max()) + 1)
        assert np.array_equal(kk[mine], K[pos[mine]]) and np.array_equal(vv[mine], V[pos[mine]])
    pool.close()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 96, 64, 32])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,kv_heads", [(200, 8), (700, 3), (3, 17)])
def test_norm_rope_with_several_groups_a_warp(layout, rot, kind, tokens, kv_heads):
    """More tokens than SMs, or more groups of 4 heads than 16 warps: a warp goes on from q's heads to k's."""
    pool = bf16_pool_of(kv_heads, rotary_dim=rot)
    q, k, qw, kw = draws(tokens, kv_heads, seed=tokens)
    pos = (np.arange(tokens) * 911 + 4095 - tokens) % 4096
    yq, yk = pool.norm_rope(q, k, qw, kw, torch.from_numpy(pos).int().to(DEV), layout=layout, dtype=kind)
    assert pool.check_errors() == 0
    check_norm_rope(yq, q, qw, pos, kind, rot=rot, layout=layout)
    check_norm_rope(yk, k, kw, pos, kind, rot=rot, layout=layout)
    pool.close()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_rope_of_many_tokens_in_place(layout):
    """5000 tokens (two warps a token), q and k in one row of a projection, onto themselves; what lies beside them and
    the tokens without a position; without a norm for one of the two."""
    n, g = 5000, 2
    pool = bf16_pool_of(g)
    gen = torch.Generator().manual_seed(1)
    row = torch.randn(n, 12 * 128, generator=gen).to(torch.bfloat16).to(DEV)
    q, k = row[:, :8 * 128].view(n, 8, 128), row[:, 8 * 128:10 * 128].view(n, 2, 128)
    before = row.clone()
    _, _, _, kw = draws(1, 2, seed=5)
    pos = np.arange(n) % 4096
    pos[[7, 4999]] = -1
    pool.norm_rope(q, k, None, kw, torch.from_numpy(pos).int().to(DEV), layout=layout, q_out=q, k_out=k)
    assert pool.check_errors() == 0 and torch.equal(row[:, 10 * 128:], before[:, 10 * 128:])
    assert (q[[7, 4999]] == 0).all() and (k[[7, 4999]] == 0).all()
    live = pos >= 0
    sel = torch.from_numpy(live).to(DEV)
    check_norm_rope(q[sel], before[:, :8 * 128].view(n, 8, 128)[sel], None, pos[live], torch.bfloat16, layout=layout)
    check_norm_rope(k[sel], before[:, 8 * 128:10 * 128].view(n, 2, 128)[sel], kw, pos[live], torch.bfloat16, layout=layout)
    pool.close()


@pytest.mark.parametrize("lengths,kv_heads", [
    ([6500], 1), ([5000, 4500], 1),            # more than 64 pages of few units: clusters of 16 CTAs, one round
    ([20000], 1), ([17000, 300], 1),           # more than 256: their rings are filled again
    ([1530, 1400] + [1 + (13 * b) % 64 for b in range(23)], 8),   # more units than SMs, 24 pages: half pages, 6 rounds
    ([700, 3, 650, 0, 500] + [1 + (13 * b) % 64 for b in range(70)], 8),   # units that take turns, 3 rounds
    ([0] * 20 + [900] + [64] * 9, 8)])
def test_one_launch_forms(lengths, kv_heads):
    wl, cache = make(lengths, kv_heads, max_seq=20480, seed=len(lengths))
    pool = pool_of(wl, cache)
    out = pool.decode(*inputs(wl))
    assert pool.check_errors() == 0
    ref, bound, after = reference(wl, cache)
    check(out, ref, bound)
    assert np.array_equal(pool.data.cpu().numpy().reshape(after.data.shape), after.data)
    assert torch.equal(out, pool.decode(*inputs(wl)))
    pool.close()


@pytest.mark.parametrize("ctas", [4096, 1 << 20])
def test_largest_grid(ctas):
    """4096 CTAs at most, of which 49152 warps share the chunks."""
    wl, cache = make([1 + (53 * i) % 900 for i in range(40)], 4)
    pool = pool_of(wl, cache, ctas)
    out = pool.decode(*inputs(wl))
    assert pool.check_errors() == 0
    check(out, *reference(wl, cache)[:2])
    pool.close()


@pytest.mark.parametrize("ctas", [0, 152])
@pytest.mark.parametrize("own_stream", [False, True])
def test_host_threads_on_one_stream(ctas, own_stream):
    """Four threads with queries of their own on the stream that they share: each gets its own outputs."""
    wl, cache = make([400, 90, 1, 777], 2)
    pool = pool_of(wl, cache, ctas)
    q, k, v, qw, kw, pos, table = inputs(wl)
    qs = [q.roll(i, 1) for i in range(4)]
    refs = [pool.decode(x, k, v, qw, kw, pos, table) for x in qs]
    torch.cuda.synchronize()
    shared = torch.cuda.Stream() if own_stream else torch.cuda.default_stream()
    bad = []

    def work(x, ref):
        try:
            with torch.cuda.stream(shared):
                outs = [pool.decode(x, k, v, qw, kw, pos, table) for _ in range(50)]
            shared.synchronize()
            bad.extend(1 for o in outs if not torch.equal(o, ref))
        except Exception as e:
            bad.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(qs, refs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and pool.check_errors() == 0
    pool.close()


def test_the_module_refuses_each_argument():
    """csrc/pkv_torch.cpp with tensors of the device: right calls reach the library (which refuses the null pool before
    anything is launched), and every one with a single wrong argument returns None before that."""
    fast = pkv._fast or (pkv.load_library(), pkv._fast)[1]
    assert fast is not None
    q, k, w, pos = (torch.zeros(3, 8, 128), torch.zeros(3, 2, 128), torch.zeros(128), torch.zeros(3, dtype=torch.int32))
    q, k, w, pos = q.to(torch.bfloat16).to(DEV), k.to(torch.bfloat16).to(DEV), w.to(torch.bfloat16).to(DEV), pos.to(DEV)
    table, f32 = torch.zeros(3, 5, dtype=torch.int32, device=DEV), torch.zeros(3, 8, 128, device=DEV)
    spec, e = (q.get_device(), 8, 2, 128), pkv.PKV_EINVAL
    junk = ["x", 1.5, (), (1, 2, 3), object(), [1]]

    def of(t):
        """Not t: other types, devices, shapes and strides."""
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=DEV)
        more = [] if t is w else [t[None]]     # (weights may have any shape of head_dim elements)
        return junk + more + [None, 7, t.cpu(), t.to(torch.float16), t.double(), torch.cat([t, t]), t[..., :-1],
                              t[:-1], t.flatten()[:-1], wide[..., ::2], wide]

    ints = junk + [None, 2 ** 70]

    def without(values, *drop):
        return [v for v in values if not any(v is d for d in drop)]
    handle = (0, ints)
    kv_specs = (spec, junk + [None, (9, 8, 2, 128), (spec[0], 8, 3, 128), (spec[0], 8, 2, 64), (spec[0], 8, 2, "x"),
                              (spec[0], 8, 2, 2 ** 70)])
    specs = (spec, kv_specs[1] + [(spec[0], 9, 2, 128)])
    tables = (table, [v for v in of(table) if v is not None and not (isinstance(v, torch.Tensor) and v.dim() == 2 and
              v.dtype == torch.int32 and v.is_cuda and v.is_contiguous() and v.shape[0] == 3)])
    any_table = (table, [v for v in tables[1] if not (isinstance(v, torch.Tensor) and v.dim() == 2 and v.is_cuda and
                 v.dtype == torch.int32 and v.is_contiguous())])
    skip = object()
    calls = {
        "decode": [handle, specs, (q, of(q)), (k, of(k)), (k, of(k)), (w, of(w)), (w, of(w)), (pos, of(pos)), tables,
                   (None, skip), (q, of(q)), (0, ints), (0, ints), (0, ints)],
        "append": [handle, kv_specs, (k, of(k)), (k, of(k)), (w, of(w)), (pos, of(pos)), (pos, without(of(pos), None)),
                   any_table, (None, skip), (None, skip), (0, ints)],
        "read": [handle, kv_specs, (pos, of(pos)), (pos, without(of(pos), None)), any_table, (k, of(k)), (k, of(k)),
                 (None, skip), (None, skip), (0, ints)],
        "norm_rope": [handle, specs, (q, of(q)), (k, of(k)), (w, without(of(w), None)), (w, without(of(w), None)),
                      (pos, of(pos)), (0, ints), (q, of(q) + [f32]), (k, of(k)), (0, ints)],
    }
    tried = 0
    for name, args in calls.items():
        good = [a for a, _ in args]
        f = getattr(fast, name)
        assert f(*good) == e, name
        assert f(*good[:-1]) is None and f(*good, 0) is None
        for i, (_, bad) in enumerate(args):
            for b in () if bad is skip else bad:
                assert f(*good[:i], b, *good[i + 1:]) is None, (name, i, b)
                tried += 1
    assert tried > 400
    # without a table the two numbers stand in for it
    for n in ints + [0, -1, 2 ** 31]:
        assert fast.decode(0, spec, q, k, k, w, w, pos, None, n, q, 0, 0, 0) is None
        assert fast.append(0, spec, k, k, w, pos, pos, None, n, 5, 0) is None
        assert fast.append(0, spec, k, k, w, pos, pos, None, 3, n, 0) is None
        assert fast.read(0, spec, pos, None, None, k, k, n, 5, 0) is None
    assert fast.decode(0, spec, q, k, k, w, w, pos, None, 5, q, 0, 0, 0) == e
    assert fast.append(0, spec, k, k, w, pos, None, None, 3, 5, 0) == e
    assert fast.read(0, spec, pos, None, None, k, k, 3, 5, 0) == e
    # k and v of different strides; q or k alone
    other = torch.zeros(3, 3, 128, dtype=torch.bfloat16, device=DEV)[:, :2]
    assert fast.read(0, spec, pos, None, table, other, other, 0, 0, 0) == e
    assert fast.read(0, spec, pos, None, table, k, other, 0, 0, 0) is None
    assert fast.norm_rope(0, spec, q, None, None, None, pos, 0, f32, None, 0) == e
    assert fast.norm_rope(0, spec, None, k, None, None, pos, 0, None, k, 0) == e
    assert fast.norm_rope(0, spec, q, None, None, None, pos, 0, f32, k, 0) is None
    assert fast.norm_rope(0, spec, None, None, None, None, pos, 0, None, None, 0) is None
    torch.cuda.synchronize()
