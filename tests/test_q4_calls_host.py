"""Q4KVPool's way through its calls, on the CPU with the library's entries replaced."""
import ctypes
import threading
import time

import pytest
import torch

import __graft_entry__
import paged_kv_gqa_qk_gb300 as pkv


@pytest.fixture
def pool(monkeypatch):
    """A 4-bit pool of one page on the host; nothing of it reaches a GPU."""
    __graft_entry__.build()
    pkv.load_library()
    monkeypatch.setattr(pkv, "pkv_q4_pool_wrap", lambda *a: ctypes.c_void_p(64))
    monkeypatch.setattr(pkv, "pkv_pool_free", lambda handle: None)
    monkeypatch.setattr(pkv, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(pkv, "_dev", lambda t, *a, **kw: t.data_ptr())
    p = pkv.Q4KVPool(torch.zeros(9216, dtype=torch.uint8), dict(heads=4, kv_heads=1, max_seq=64))
    p._streams[0] = (256, 1 << 20, None)
    yield p
    p.close()


def arguments():
    q, k = torch.zeros(1, 4, 128, dtype=torch.bfloat16), torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    w, pos = torch.ones(128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    return dict(q=q, k=k, v=k, q_norm_w=w, k_norm_w=w, positions=pos, table=pos[None], out=torch.empty_like(q))


@pytest.mark.parametrize("module", [True, False])
def test_threads_on_one_stream_enqueue_one_call_at_a_time(pool, monkeypatch, module):
    """Threads that share a stream share its workspace: between a call's launches there may be no other call's."""
    inside, most = [], []

    def entry(*args):
        inside.append(1)
        most.append(len(inside))
        time.sleep(0.002)          # (without the interpreter's lock, as the library's calls)
        inside.pop()
        return 0

    class Entries:
        decode = staticmethod(entry)
        pkv_q4_decode = staticmethod(entry)
    monkeypatch.setattr(pkv, "_fast", Entries if module else None)
    pool._lib = Entries
    args = arguments()
    threads = [threading.Thread(target=lambda: [pool.decode(**args) for _ in range(5)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(most) == 20 and max(most) == 1
