"""pkv_norm_rope and scaled rotations on the GPU against the 64-bit forms of tests/_q4.py and the oracle."""
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


def pool_of(kv_heads=2, **cfg):
    z = torch.zeros(2, kv_heads, 64, 128, dtype=torch.bfloat16, device=DEV)
    return pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=4 * kv_heads, kv_heads=kv_heads, **{"max_seq": 4096, **cfg}))


def draws(tokens, kv_heads, seed=0, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=gen) * scale).to(torch.bfloat16).to(DEV)  # noqa: E731
    w = lambda: (torch.rand(128, generator=gen) + 0.5).to(torch.bfloat16).to(DEV)  # noqa: E731
    return r(tokens, 4 * kv_heads, 128), r(tokens, kv_heads, 128), w(), w()


def check(got, x, w, pos, kind, **kw):
    """Roundings: cos and sin 2^-24, two products, their sum, the norm (9 sums under a square root, 2 ulp of rsqrt,
    one product, one by the inverse): under 2^-20 of the terms' sum of sizes; then one to the output's type."""
    ref = _q4.norm_rope(f64(x), None if w is None else f64(w), pos, **kw)
    m = kw.get("mscale", 1.0)
    size = np.abs(_q4.norm_rope(f64(x), None if w is None else f64(w), pos * 0, **{**kw, "mscale": 1.0}))
    rot, layout = kw.get("rot", 128), kw.get("layout", "half")
    both = size.copy()
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    both[..., lo] = both[..., hi] = (size[..., lo] + size[..., hi]) * m
    tol = 2.0 ** -20 * both
    if kind == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    off = np.abs(f64(got) - ref)
    assert got.dtype == kind and (off <= tol).all(), (off - tol).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 96, 64, 32])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope(layout, rot, kind, norm):
    for tokens, kv_heads in ((1, 8), (37, 2), (5, 1), (3, 3)):
        pool = pool_of(kv_heads, rotary_dim=rot)
        q, k, qw, kw = draws(tokens, kv_heads, seed=tokens)
        if not norm:
            qw = kw = None
        pos = (np.arange(tokens) * 911 + 4095 - tokens) % 4096
        yq, yk = pool.norm_rope(q, k, qw, kw, torch.from_numpy(pos).int().to(DEV), layout=layout, dtype=kind)
        assert pool.check_errors() == 0
        check(yq, q, qw, pos, kind, rot=rot, layout=layout)
        check(yk, k, kw, pos, kind, rot=rot, layout=layout)
        pool.close()


def test_strides_in_place_and_one_of_the_two():
    pool = pool_of(2)
    row = torch.randn(9, 2000, device=DEV).to(torch.bfloat16)[:, 4:]
    q, k = row[:, :1024].view(9, 8, 128), row[:, 1100:1356].view(9, 2, 128)
    _, _, qw, kw = draws(1, 2)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    before = row.clone()
    yq, yk = pool.norm_rope(q, k, qw, kw, pos)
    assert torch.equal(row, before)
    only_q, none = pool.norm_rope(q, None, qw, None, pos)
    assert none is None and torch.equal(only_q, yq)
    _, only_k = pool.norm_rope(None, k, None, kw, pos)
    assert torch.equal(only_k, yk)
    pool.norm_rope(q, k, qw, kw, pos, q_out=q, k_out=k)      # in place
    assert torch.equal(q, yq) and torch.equal(k, yk)
    rest = torch.ones(row.shape[1], dtype=torch.bool, device=DEV)
    rest[:1024] = rest[1100:1356] = False
    assert torch.equal(row[:, rest], before[:, rest])
    pool.close()


def test_positions_outside_the_table():
    pool = pool_of(2, max_seq=100)
    q, k, qw, kw = draws(4, 2)
    pos = torch.tensor([99, -1, 5, -1], dtype=torch.int32, device=DEV)
    yq, yk = pool.norm_rope(q, k, qw, kw, pos)
    assert pool.check_errors() == 0 and (yq[1] == 0).all() and (yk[3] == 0).all() and (yq[0] != 0).any()
    pos[3] = 100
    yq, yk = pool.norm_rope(q, k, qw, kw, pos)
    assert pool.check_errors() == pkv.PKV_DEVERR_POSITION and (yq[3] == 0).all()
    pool.close()


def test_interleaved_is_half_on_reordered_dims():
    pool = pool_of(2)
    q, k, _, _ = draws(6, 2)
    pos = torch.arange(6, dtype=torch.int32, device=DEV) * 600
    order = torch.cat([torch.arange(0, 128, 2), torch.arange(1, 128, 2)]).to(DEV)
    a, _ = pool.norm_rope(q, k, None, None, pos, layout="interleaved", dtype=torch.float32)
    b, _ = pool.norm_rope(q[..., order].contiguous(), k, None, None, pos, dtype=torch.float32)
    assert (a[..., order] - b).abs().max() <= 2.0 ** -20 * 16
    pool.close()


@pytest.mark.parametrize("scaling,factor,trained", [("linear", 4.0, 0), ("base", 2.5, 0), ("ramp", 4.0, 1024), ("ramp", 2.0, 64)])
def test_scaled_rotation_everywhere(scaling, factor, trained):
    """A pool's frequencies replaced: norm_rope, the 4-bit pool's append and the bf16 pool's decode all turn by them."""
    pool = pool_of(2)
    freq, m = pkv.pkv_rope_frequencies(pool.cfg, scaling, factor, trained)
    pool.set_rope(freq, m)
    q, k, qw, kw = draws(20, 2, seed=4)
    pos = np.arange(20) * 203
    dpos = torch.from_numpy(pos).int().to(DEV)
    for layout in ("half", "interleaved"):
        yq, yk = pool.norm_rope(q, k, qw, kw, dpos, layout=layout, dtype=torch.float32)
        check(yq, q, qw, pos, torch.float32, layout=layout, freq=freq, mscale=m)
        check(yk, k, kw, pos, torch.float32, layout=layout, freq=freq, mscale=m)
    pool.close()

    q4 = pkv.Q4KVPool.empty(64, dict(heads=8, kv_heads=2, max_seq=4096))
    q4.set_rope(freq, m)
    table = torch.arange(64, dtype=torch.int32, device=DEV)[None]
    row = torch.zeros(20, dtype=torch.int32, device=DEV)
    q4.append(k, k, kw, dpos, row, table)
    got, _ = q4.read(dpos, row, table)
    want = _q4.bf16(_q4.norm_rope(f64(k), f64(kw), pos, freq=freq, mscale=m))
    assert np.array_equal(f64(got), _q4.values(*_q4.quantise(want, 1.0), 1.0))
    q4.close()

    K = torch.zeros(2, 64 * 64, 128, dtype=torch.bfloat16, device=DEV)
    V = K.clone()
    bf = pkv.PagedKVPool(K, V, cfg=dict(heads=8, kv_heads=2, max_seq=4096))
    bf.set_rope(freq, m)
    one = torch.tensor([4000], dtype=torch.int32, device=DEV)
    bf.decode(q[:1].contiguous(), k[:1].contiguous(), k[:1].contiguous(), qw, kw, one, table)
    got = f64(K[:, 4000])
    want = _q4.norm_rope(f64(k[:1]), f64(kw), np.array([4000]), freq=freq, mscale=m)[0]
    assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -40).all()   # within one bf16 ulp
    assert bf.check_errors() == 0
    bf.close()


def test_feeds_the_attention_of_prepared_rows():
    """fp32 queries from norm_rope into pkv_decode_appended give what pkv_decode gives, to bf16's rounding."""
    wl = W.make_decode("prepared", [100, 300, 64], seed=9)
    args = [t.to(DEV) for t in (wl.q, wl.k, wl.v, wl.q_norm_w, wl.k_norm_w, wl.step_positions, wl.table)]
    pool = pkv.PagedKVPool(wl.K0.to(DEV), wl.V0.to(DEV), cfg=wl.cfg)
    ref = pool.decode(*args)
    q_hat, _ = pool.norm_rope(args[0], None, args[3], None, args[5], dtype=torch.float32)
    out = torch.empty_like(ref)
    pkv.pkv_decode_appended(pool.handle, q_hat, args[5], args[6], out, pool.workspace(3, wl.pages))
    assert pool.check_errors() == 0
    # queries differ by 2^-20 of a head's largest products: scores by under 2^-14, outputs by a bf16 ulp at most
    assert ((out.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 2.0 ** -12).all()
    pool.close()


def test_graph():
    pool = pool_of(2)
    q, k, qw, kw = draws(8, 2)
    pos = torch.arange(8, dtype=torch.int32, device=DEV)
    ref = pool.norm_rope(q, k, qw, kw, pos)
    out = [torch.zeros_like(x) for x in ref]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.norm_rope(q, k, qw, kw, pos, q_out=out[0], k_out=out[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    pool.close()
