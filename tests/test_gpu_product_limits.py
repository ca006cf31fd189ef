"""The products' bounded waits, run out on purpose.

With a limit of 0 each role of a product gives up at the first check that finds its copy not yet landed, as every real
call has one.  The call must return, report PKV_DEVERR_TIMEOUT and no CUDA error, and leave nothing behind: the next call at
the ordinary limit gives the bits of one before.  A role that gave up still waits for the same copies, so nothing here is
read or overwritten out of turn; the failure is only a wait that is told to give up early."""
import pytest
import torch

import paged_kv_gqa_qk_gb300 as pkv
from test_gpu_mx import DEV, KINDS, operands

pytestmark = pytest.mark.gpu


@pytest.fixture
def pool():
    z = torch.zeros(2, 8, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=32, kv_heads=8, max_seq=64))
    yield p
    p.close()


def runs_out_and_recovers(pool, call):
    ref = [t.clone() for t in call()]
    assert pool.check_errors() == 0
    for limit in (0, 0, 1):     # (a limit above 0 is looked at after some polls only, and may not be reached)
        pkv.pkv_set_wait_limit(pool.handle, limit)
        call()
        flags = pool.check_errors()
        assert flags == pkv.PKV_DEVERR_TIMEOUT or limit and not flags, (limit, flags)
    pkv.pkv_set_wait_limit(pool.handle, 10 ** 9)
    for _ in range(3):
        for a, b in zip(call(), ref):
            assert torch.equal(a, b)
    assert pool.check_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,n_in,n_out", [
    (1, 4096, 6144), (1, 8192, 1024), (20, 2048, 1024), (64, 4096, 4096), (128, 4096, 6144),  # split 1 to 8 times
    (40, 4096, 20480),          # a ring that is used again, every SM in turns
    (300, 4096, 20480),         # CTA pairs: several tiles each, rings used again
    (2048, 512, 6144),
])
def test_microscaled_products(pool, kind, tokens, n_in, n_out):
    x, w = operands(tokens, n_in, n_out, kind, seed=tokens)
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    runs_out_and_recovers(pool, lambda: [pool.mx_linear(xm, wm)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [3, 500])
def test_microscaled_qkv(pool, kind, tokens):
    x, w = operands(tokens, 1024, 48 * 128, kind, seed=tokens)
    xm, wm = pool.mx_quantize(x, kind), pool.mx_quantize(w, kind)
    runs_out_and_recovers(pool, lambda: list(pool.mx_qkv_proj(xm, wm)))


@pytest.mark.parametrize("tokens,n_in,n_out", [(1, 4096, 6144), (64, 4096, 4096), (100, 2048, 1024), (700, 4096, 3200)])
def test_products_of_bf16(pool, tokens, n_in, n_out):
    x, w = operands(tokens, n_in, n_out, "mx8", seed=tokens)
    runs_out_and_recovers(pool, lambda: [pool.linear(x, w)])


@pytest.mark.parametrize("tokens", [3, 500])
def test_qkv_of_bf16(pool, tokens):
    x, w = operands(tokens, 1024, 48 * 128, "mx8", seed=tokens)
    runs_out_and_recovers(pool, lambda: list(pool.qkv_proj(x, w)))


@pytest.mark.parametrize("tokens", [2, 200])
def test_projection_with_its_append(pool, tokens):
    """q and the pool's rows after a call that ran out and one that did not."""
    x, w = operands(tokens, 1024, 48 * 128, "mx8", seed=tokens)
    p = pkv.PagedKVPool(*torch.zeros(2, 8, 64 * (tokens + 1), 128, dtype=torch.bfloat16, device=DEV),
                        cfg=dict(heads=32, kv_heads=8, max_seq=64))
    ones = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    positions = (torch.arange(tokens, device=DEV) * 5 % 64).int()
    table = (torch.arange(tokens, device=DEV).int() + 1).view(-1, 1)
    q_hat = torch.empty(tokens, 32, 128, device=DEV)

    def call():
        pkv.pkv_qkv_proj_append(p.handle, x, w, ones, ones, positions, table, q_hat)
        return [q_hat, p.K, p.V]
    runs_out_and_recovers(p, call)
    p.close()
