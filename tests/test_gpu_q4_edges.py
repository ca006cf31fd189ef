"""The quantiser at the far ends of what a pool's scales and a cache's values may be."""
import numpy as np
import pytest
import torch

import _q4
import paged_kv_gqa_qk_gb300 as pkv
from test_gpu_q4 import DEV, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e", [-60, -52, -40, -34, -33, -20, 0, 30, 60])
def test_values_beyond_the_largest_scale(e):
    """Groups whose scale stays at 448, with values from the smallest bf16 to the largest beside the codes' ties at that
    scale: what is too large is 6 * 448 * s with its own sign, the rest the nearest code."""
    s = 2.0 ** e
    tops = [t for t in (6.5 * 448 * s, 1e5 * s, 2.0 ** 60, 2.0 ** 100, 2.0 ** 101.2, 2.0 ** 101.3, 2.0 ** 103, 2.0 ** 110,
                        2.0 ** 120, 2.0 ** 127, 2.0 ** 127.2, 2.0 ** 127.3, 3.0e38) if 6 * 448 * s < t < 3.3e38]
    rng = np.random.RandomState(0)
    n = 4 * len(tops)
    assert n > 0
    inner = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0, 6.0, 0.6, 4.4]) * 448 * s
    x = rng.choice(inner, size=(n, 8, 16))
    for i in range(n):
        x[i, :, :3] = tops[i // 4]
        x[i, :, 3:8] = rng.choice(tops + [2.0 ** -133], size=(8, 5))
    x *= rng.choice([-1.0, 1.0], x.shape)
    v = torch.from_numpy(x.reshape(n, 1, 128)).to(torch.bfloat16)
    pages = -(-n // 64)
    pool = pkv.Q4KVPool.empty(pages, dict(heads=4, kv_heads=1, max_seq=64 * pages), v_scale=s)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    k, w = torch.ones(n, 1, 128, dtype=torch.bfloat16, device=DEV), torch.ones(128, dtype=torch.bfloat16, device=DEV)
    pool.append(k, v.to(DEV), w, pos, pos * 0, table)
    _, got = pool.read(pos, pos * 0, table)
    assert pool.check_errors() == 0
    ref = _q4.values(*_q4.quantise(f64(v), s), s)
    assert np.array_equal(f64(got), ref), f"{(f64(got) != ref).sum()} of {ref.size} differ"
    pool.close()


@pytest.mark.parametrize("kv_heads", [2, 8])
def test_a_key_with_an_infinity_is_nan_as_a_whole(kv_heads):
    """k with an Inf or a NaN: that head's position is NaN in all its dims; the other heads, the other positions and all
    of v are as ever.  Large keys are normed like others."""
    n = 64
    rng = np.random.RandomState(2)
    x = rng.randn(n, kv_heads, 128) * 2.0 ** rng.randint(-20, 58, (n, kv_heads, 1))
    x[3, 1, 7], x[9, 0, 100], x[10, 1, 64] = np.inf, np.nan, -np.inf
    k = torch.from_numpy(x).to(torch.bfloat16)
    v = torch.from_numpy(rng.randn(n, kv_heads, 128)).to(torch.bfloat16)
    w = torch.from_numpy(rng.rand(128) + 0.5).to(torch.bfloat16)
    pool = pkv.Q4KVPool.empty(1, dict(heads=4 * kv_heads, kv_heads=kv_heads, max_seq=64))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    pool.append(k.to(DEV), v.to(DEV), w.to(DEV), pos, pos * 0, table)
    kk, vv = (f64(t) for t in pool.read(pos, pos * 0, table))
    assert pool.check_errors() == 0
    bad = np.zeros((n, kv_heads), bool)
    bad[3, 1] = bad[9, 0] = bad[10, 1] = True
    assert np.isnan(kk[bad]).all() and np.isfinite(kk[~bad]).all()
    with np.errstate(invalid="ignore"):
        want = _q4.bf16(np.where(bad[..., None], 0.0, _q4.norm_rope(f64(k), f64(w), np.arange(n))))
    assert np.array_equal(kk[~bad], _q4.values(*_q4.quantise(want, 1.0), 1.0)[~bad])
    assert np.array_equal(vv, _q4.values(*_q4.quantise(f64(v), 1.0), 1.0))
    pool.close()
