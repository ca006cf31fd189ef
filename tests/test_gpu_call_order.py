"""A call reads its tokens' positions and pages after the call before it has written them, also where that one lets it start early."""
import pytest
import torch

import paged_kv_gqa_qk_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tokens", [8, 150])
def test_positions_written_just_before(tokens):
    """The projection with its append resolves positions beside its product.  They come here as the bits of a sum that
    pkv_add_norm writes (x + 0, 32768 tokens of work of which theirs is the last), a call that lets the next start early."""
    hidden, rows = 1024, 32768
    gen = torch.Generator().manual_seed(1)
    bf = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(DEV)  # noqa: E731
    pool = pkv.PagedKVPool(*torch.zeros(2, 8, 64 * (2 * tokens + 1), 128, dtype=torch.bfloat16, device=DEV),
                           cfg=dict(heads=32, kv_heads=8, max_seq=128))
    x, w, qw, kw = bf(tokens, hidden), bf(48 * 128, hidden), bf(128), bf(128)
    table = (torch.arange(2 * tokens, device=DEV).int() + 1).view(tokens, 2)
    ones, zeros = torch.ones(hidden, dtype=torch.bfloat16, device=DEV), torch.zeros(rows, hidden, dtype=torch.bfloat16, device=DEV)
    carrier, scratch = torch.zeros_like(zeros), torch.empty_like(zeros)
    positions = carrier[-1].view(torch.int32)[:tokens]
    q_hat = torch.empty(tokens, 32, 128, device=DEV)
    sets = []
    for s in range(3):
        given = (torch.arange(tokens) * 7 + 31 * s) % 128
        bits = torch.zeros(rows, hidden, dtype=torch.bfloat16, device=DEV)
        bits[-1].view(torch.int32)[:tokens] = given.int().to(DEV)
        pkv.pkv_qkv_proj_append(pool.handle, x, w, qw, kw, given.int().to(DEV), table, q_hat)
        sets.append((bits, given.int().to(DEV), q_hat.clone()))
        torch.cuda.synchronize()
    wrong = torch.zeros(2, device=DEV)
    for i in range(60):
        bits, given, ref = sets[i % 3]
        pool.add_norm(bits, zeros, ones, out=scratch, residual_out=carrier)
        pkv.pkv_qkv_proj_append(pool.handle, x, w, qw, kw, positions, table, q_hat)
        wrong[0] += (positions != given).any()
        wrong[1] += (q_hat != ref).any()
    assert wrong.tolist() == [0, 0] and pool.check_errors() == 0
    pool.close()
