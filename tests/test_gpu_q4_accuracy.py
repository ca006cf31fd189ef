"""The 4-bit decode where its roundings would show: scores of 40 and more that lie close together, weights far below the
largest, and sums that cancel.  The bounds count what the kernels may lose and were fixed before the first run."""
import numpy as np
import pytest
import torch

import _q4
import paged_kv_gqa_qk_gb300 as pkv
from test_gpu_q4 import DEV, f64

pytestmark = pytest.mark.gpu


def attend(q, K, V):
    """q [4 G][128], K, V [n][G][128] in 64 bits: (out, bound on |kernel - out| before bf16's rounding of out).

    Without a rotation (cos 1, sin 0) the kernel's q is off by under 2^-20 of itself (19 sums of squares under a root:
    10 2^-24, rsqrt 2^-22, two products).  Split into an fp16 and the fp16 of the rest it keeps 2^-22 of itself or
    2^-25 of the head's largest.  A score is 8 products of 16 in fp32, each within 2^-22 of its terms' sizes (2^-19 in
    all), times a multiplier (3 2^-24): 2^-18 of sum |q k| covers these.  The exponent's rounding (2^-20, arguments up
    to 32), ex2 (2^-22) and a weight's own split (2^-21) are under 2^-19 + 2^-22 of it, and the split loses 2^-32 of the
    largest where it ends in fp16's subnormals.  The
    weighted sums add 2^-22 of their sizes per 16 positions, and a few more where pieces are joined."""
    n, G = K.shape[0], K.shape[1]
    out, bound = np.zeros_like(q), np.zeros_like(q)
    for h in range(q.shape[0]):
        k, v = K[:, h // 4], V[:, h // 4]
        s = k @ q[h] / np.sqrt(128)
        ds = (2.0 ** -18 * (np.abs(k) @ np.abs(q[h])) + 2.0 ** -25 * np.abs(q[h]).max() * np.abs(k).sum(-1)) / np.sqrt(128)
        p = np.exp(s - s.max())
        total = p.sum()
        e = np.expm1(ds) + 2.0 ** -19 + 2.0 ** -22
        off = p * e + 2.0 ** -32                                # of each weight
        out[h] = p @ v / total
        bound[h] = (off @ np.abs(v) + np.abs(out[h]) * off.sum() + (n / 16 + 8) * 2.0 ** -22 * 2 * (p @ np.abs(v))) / total
    return out, bound


def run(K0, V0, x, w, ctas, vs=1.0):
    """One decode step of one row whose cached positions are K0, V0 [n][G][128], over a pool that does not rotate:
    (out, q, K, V) with the cache's values, the new position's included."""
    n, G, _ = K0.shape
    pages = -(-(n + 1) // 64)
    cfg = dict(heads=4 * G, kv_heads=G, max_seq=64 * pages)
    full = [np.zeros((G, 64 * pages, 128)) for _ in range(2)]
    for f, a in zip(full, (K0, V0)):
        f[:, :n] = _q4.bf16(a).transpose(1, 0, 2)
    cache = _q4.Cache.of(*full, 1.0, vs)
    pool = pkv.Q4KVPool(torch.from_numpy(cache.data.copy()).to(DEV), cfg, v_scale=vs)
    pool.set_rope([0.0] * 64)
    if ctas:
        pkv.pkv_set_ctas(pool.handle, ctas)
    k = torch.ones(1, G, 128, dtype=torch.bfloat16)
    kw = torch.full((128,), 2.0 ** -8, dtype=torch.bfloat16)    # the new position's own score is near 0
    v = torch.zeros(1, G, 128, dtype=torch.bfloat16)
    out = pool.decode(*[t.to(DEV) for t in (x, k, v, w, kw, torch.tensor([n], dtype=torch.int32),
                                            torch.arange(pages, dtype=torch.int32)[None])])
    assert pool.check_errors() == 0
    pool.close()
    cache.put(n // 64, n, _q4.bf16(_q4.norm_rope(f64(k), f64(kw), np.zeros(1)))[0], f64(v)[0])
    q = f64(x)[0] / np.sqrt((f64(x)[0] ** 2).mean(-1, keepdims=True) + 1e-6) * f64(w)
    return f64(out)[0], q, *cache.get(np.arange(pages), n + 1)


def within(got, q, K, V):
    ref, bound = attend(q, K, V)
    tol = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    off = np.abs(got - ref)
    assert (off <= tol).all(), f"{(off > tol).sum()} of {off.size} outside; worst {(off / tol).max():.1f} times the bound"


@pytest.mark.parametrize("ctas", [0, 1, 152])
@pytest.mark.parametrize("n,G", [(40, 2), (63, 1), (300, 1), (1000, 2)])
def test_large_scores_close_together(n, G, ctas):
    """Keys with one value that is not 0, so that a score is one product: an error of q's is that of the score, which
    40 makes large."""
    rng = np.random.RandomState(n + G)
    x = torch.from_numpy(rng.randn(1, 4 * G, 128)).to(torch.bfloat16)
    w = torch.from_numpy(16.0 * (rng.rand(128) + 0.5)).to(torch.bfloat16)
    q = f64(x)[0] / np.sqrt((f64(x)[0] ** 2).mean(-1, keepdims=True) + 1e-6) * f64(w)
    K0 = np.zeros((n, G, 128))
    for i in range(n):
        for g in range(G):
            h = 4 * g + i % 4
            d = rng.choice(np.nonzero(np.abs(q[h]) > 8)[0])
            K0[i, g, d] = 40.0 * np.sqrt(128) / q[h, d]
    V0 = rng.randn(n, G, 128)
    within(*run(K0, V0, x, w, ctas))


@pytest.mark.parametrize("ctas", [0, 1, 152])
def test_weights_that_cancel(ctas):
    """Every key twice, every value with both signs: what is left is the difference of two weights, near 0."""
    rng = np.random.RandomState(3)
    n, G = 60, 2
    x = torch.from_numpy(rng.randn(1, 4 * G, 128)).to(torch.bfloat16)
    w = torch.full((128,), 0.25, dtype=torch.bfloat16)
    K0 = rng.randn(n, G, 128)
    K0[1::2] = K0[0::2]
    K0[1::2, :, 3] *= 0.25
    V0 = rng.randn(n, G, 128)
    V0[1::2] = -V0[0::2]
    within(*run(K0, V0, x, w, ctas))


@pytest.mark.parametrize("ctas", [0, 1, 152])
@pytest.mark.parametrize("below", [12.0, 18.0, 20.0])
def test_weights_far_below_the_largest(below, ctas):
    """One position whose value is 0 holds nearly all the weight; the output is what the others' 62 add up to."""
    rng = np.random.RandomState(4)
    n, G = 63, 1
    x = torch.ones(1, 4, 128, dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    K0 = np.full((n, G, 128), 0.0)
    K0[:, :, 0] = -below * np.sqrt(128) * (1 + 0.01 * rng.rand(n, 1))
    K0[0] = 0.0
    V0 = 2000.0 * (1 + rng.rand(n, G, 128) * 0.2) * np.where(rng.rand(128) < 0.5, -1.0, 1.0)
    V0[0] = 0.0
    within(*run(K0, V0, x, w, ctas))
