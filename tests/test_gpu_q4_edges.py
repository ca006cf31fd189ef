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
