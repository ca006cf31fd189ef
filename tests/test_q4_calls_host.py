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


@pytest.mark.parametrize("call", ["decode", "append", "read", "norm_rope"])
def test_a_code_of_the_library_is_raised_at_once(pool, monkeypatch, call):
    """What the library refused or could not enqueue is not tried a second time another way."""
    tried = []

    def entry(*args):
        tried.append(args)
        return pkv.PKV_ECUDA

    class Entries:
        def __getattr__(self, name):
            return entry
    monkeypatch.setattr(pkv, "_fast", Entries())
    pool._lib = Entries()
    monkeypatch.setattr(pkv, "pkv_norm_rope", lambda *a, **kw: pkv._check(entry(), "pkv_norm_rope"))
    a = arguments()
    calls = {
        "decode": lambda: pool.decode(**a),
        "append": lambda: pool.append(a["k"], a["v"], a["k_norm_w"], a["positions"], None, a["table"]),
        "read": lambda: pool.read(a["positions"], None, a["table"], a["k"], a["v"]),
        "norm_rope": lambda: pool.norm_rope(a["q"], a["k"], None, None, a["positions"]),
    }
    with pytest.raises(pkv.PkvError) as e:
        calls[call]()
    assert e.value.code == pkv.PKV_ECUDA and len(tried) == 1


def test_a_workspace_that_has_become_too_small_is_replaced(pool, monkeypatch):
    """PKV_EWORKSPACE is not an error of the call: it is made again with a larger one, which is kept."""
    seen = []

    class Entries:
        @staticmethod
        def decode(*args):
            return pkv.PKV_EWORKSPACE

        @staticmethod
        def pkv_q4_decode(*args):
            seen.append(args[-2])
            return pkv.PKV_OK if args[-2] >= 1 << 21 else pkv.PKV_EWORKSPACE
    monkeypatch.setattr(pkv, "_fast", Entries)
    monkeypatch.setattr(pkv, "pkv_workspace_bytes", lambda *a: 1 << 21)
    monkeypatch.setattr(pkv, "_capturing", lambda stream: False)
    pool._lib = Entries
    pool.decode(**arguments())
    assert seen == [1 << 20, 1 << 21] and pool._streams[0][1] == 1 << 21
