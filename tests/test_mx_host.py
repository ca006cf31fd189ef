"""Microscaled tensors on the host: sizes, the entries' refusals, the binding's checks (nothing reaches a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import _mx
import paged_kv_gqa_qk_gb300 as pkv


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return pkv.load_library()


def test_sizes(lib):
    assert pkv.pkv_mx_bytes("mx8", 1, 128) == (128, 512)
    assert pkv.pkv_mx_bytes("mx4", 1, 128) == (64, 512)
    assert pkv.pkv_mx_bytes("mx8", 129, 640) == (129 * 640, 2 * 5 * 512)
    assert pkv.pkv_mx_bytes("mx4", 1 << 24, 1 << 20) == (1 << 43, (1 << 17) * (1 << 13) * 512)
    assert lib.pkv_mx_bytes(2, 4, 256, None, None) == pkv.PKV_OK
    for args, code in [((0, 4, 256), pkv.PKV_EINVAL), ((1, 4, 256), pkv.PKV_EINVAL), ((4, 4, 256), pkv.PKV_EINVAL),
                       ((2, 0, 256), pkv.PKV_EINVAL), ((2, -1, 256), pkv.PKV_EINVAL), ((2, 4, 0), pkv.PKV_EINVAL),
                       ((2, 4, 96), pkv.PKV_ENOTIMPL), ((3, 4, 64), pkv.PKV_ENOTIMPL), ((2, (1 << 24) + 1, 128), pkv.PKV_ERANGE),
                       ((3, 1, (1 << 20) + 128), pkv.PKV_ERANGE)]:
        assert lib.pkv_mx_bytes(*args, None, None) == code, args


def test_null_and_wrong_arguments(lib):
    p = ctypes.c_void_p(4096)      # never followed: every call below is refused before
    n = None
    E = pkv.PKV_EINVAL
    assert lib.pkv_mx_quantize(n, p, 128, 4, 128, 2, p, p, n) == E
    assert lib.pkv_mx_read(n, 2, p, p, 4, 128, p, 128, n) == E
    assert lib.pkv_add_norm(n, p, 128, p, p, p, 4, 128, 2, p, p, n) == E
    assert lib.pkv_mx_linear(n, 2, p, p, p, p, p, 4, 128, 128, n) == E
    assert lib.pkv_mx_qkv_proj(n, 2, p, p, p, p, 4, 128, p, p, p, n) == E


class FakePool:
    """The fields of a pool that the entries look at before they refuse (no device is 12345)."""

    def __init__(self):
        self.cfg = pkv.pkv_config_default()
        self.raw = (ctypes.c_char * 4096)()
        ctypes.memmove(self.raw, ctypes.byref(self.cfg), ctypes.sizeof(self.cfg))
        ctypes.memmove(ctypes.addressof(self.raw) + ctypes.sizeof(self.cfg), ctypes.byref(ctypes.c_int(12345)), 4)
        self.handle = ctypes.c_void_p(ctypes.addressof(self.raw))


def test_codes_of_the_entries(lib):
    """Sizes, alignment and missing pointers are refused before the device is asked for; then PKV_EDEVICE."""
    fake = FakePool()
    f = fake.handle
    p, odd, n = ctypes.c_void_p(4096), ctypes.c_void_p(4104), None
    E, I, R, D = pkv.PKV_EINVAL, pkv.PKV_ENOTIMPL, pkv.PKV_ERANGE, pkv.PKV_EDEVICE
    q = lambda *a: lib.pkv_mx_quantize(f, *a, n)  # noqa: E731
    assert q(p, 256, 4, 256, 2, p, p) == D
    for a, code in [((n, 256, 4, 256, 2, p, p), E), ((p, 256, 4, 256, 2, n, p), E), ((p, 256, 4, 256, 2, p, n), E),
                    ((p, 248, 4, 256, 2, p, p), E), ((p, 260, 4, 256, 2, p, p), E), ((odd, 256, 4, 256, 2, p, p), E),
                    ((p, 256, 4, 256, 2, odd, p), E), ((p, 256, 4, 256, 2, p, odd), E), ((p, 256, 0, 256, 2, p, p), E),
                    ((p, 256, 4, 256, 1, p, p), E), ((p, 256, 4, 200, 2, p, p), I), ((p, 256, 1 << 25, 256, 2, p, p), R)]:
        assert q(*a) == code, a
    r = lambda *a: lib.pkv_mx_read(f, *a, n)  # noqa: E731
    assert r(3, p, p, 4, 256, p, 256) == D
    for a, code in [((3, n, p, 4, 256, p, 256), E), ((3, p, p, 4, 256, n, 256), E), ((3, p, p, 4, 256, p, 255), E),
                    ((3, p, p, 4, 256, odd, 256), E), ((0, p, p, 4, 256, p, 256), E), ((3, p, p, 4, 192, p, 256), I)]:
        assert r(*a) == code, a
    a_n = lambda *a: lib.pkv_add_norm(f, *a, n)  # noqa: E731
    assert a_n(p, 256, p, p, p, 4, 256, 2, p, p) == D and a_n(p, 24, n, n, p, 4, 24, 0, p, n) == D
    for a, code in [((n, 256, p, p, p, 4, 256, 2, p, p), E), ((p, 256, p, n, p, 4, 256, 2, p, p), E),
                    ((p, 256, n, p, p, 4, 256, 2, p, p), E), ((p, 256, p, p, n, 4, 256, 2, p, p), E),
                    ((p, 256, p, p, p, 4, 256, 2, n, p), E), ((p, 256, p, p, p, 4, 256, 2, p, n), E),
                    ((p, 256, p, p, p, 4, 256, 0, p, p), E), ((p, 256, p, p, p, 4, 256, 1, p, n), E),
                    ((p, 256, p, p, p, 0, 256, 2, p, p), E), ((p, 128, p, p, p, 4, 256, 2, p, p), E),
                    ((p, 260, p, p, p, 4, 256, 2, p, p), E), ((p, 256, odd, p, p, 4, 256, 2, p, p), E),
                    ((p, 256, p, odd, p, 4, 256, 2, p, p), E), ((p, 256, p, p, odd, 4, 256, 2, p, p), E),
                    ((p, 192, p, p, p, 4, 192, 3, p, p), I), ((p, 24, p, p, p, 4, 20, 0, p, n), I),
                    ((p, 32896, p, p, p, 4, 32896, 2, p, p), R), ((p, 256, p, p, p, 1 << 25, 256, 2, p, p), R)]:
        assert a_n(*a) == code, a
    l = lambda *a: lib.pkv_mx_linear(f, *a, n)  # noqa: E731,E741
    assert l(2, p, p, p, p, p, 4, 256, 384) == D
    for a, code in [((2, n, p, p, p, p, 4, 256, 384), E), ((2, p, n, p, p, p, 4, 256, 384), E),
                    ((2, p, p, n, p, p, 4, 256, 384), E), ((2, p, p, p, n, p, 4, 256, 384), E),
                    ((2, p, p, p, p, n, 4, 256, 384), E), ((2, p, p, p, p, odd, 4, 256, 384), E),
                    ((2, odd, p, p, p, p, 4, 256, 384), E), ((0, p, p, p, p, p, 4, 256, 384), E),
                    ((2, p, p, p, p, p, 0, 256, 384), E), ((2, p, p, p, p, p, 4, 256, 0), E),
                    ((2, p, p, p, p, p, 4, 200, 384), I), ((2, p, p, p, p, p, 4, 256, 200), I),
                    ((2, p, p, p, p, p, 1 << 25, 256, 384), R), ((2, p, p, p, p, p, 4, 256, (1 << 20) + 128), R)]:
        assert l(*a) == code, a
    w = lambda *a: lib.pkv_mx_qkv_proj(f, *a, n)  # noqa: E731
    assert w(3, p, p, p, p, 4, 256, p, p, p) == D
    for a, code in [((3, p, p, p, p, 4, 256, p, n, p), E), ((3, p, p, p, p, 4, 256, p, p, odd), E),
                    ((3, p, p, p, p, 4, 64, p, p, p), I), ((3, p, p, p, p, -1, 256, p, p, p), E)]:
        assert w(*a) == code, a


def test_tensor_checks(lib):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    t = pkv.MxTensor("mx4", 130, 256, u8(130, 128), u8(2048))
    assert t.shape == (130, 256) and t.device.type == "cpu"
    assert pkv.MxTensor.empty("mx8", 3, 128, device="cpu").codes.shape == (3, 128)
    for args, what in [(("fp8", 130, 256, u8(130, 128), u8(2048)), ValueError), (("mx8", 130, 256, u8(130, 128), u8(2048)), ValueError),
                       (("mx4", 130, 256, u8(130, 128), u8(1024)), ValueError), (("mx4", 130, 200, u8(130, 100), u8(2048)), pkv.PkvError),
                       (("mx4", 0, 256, u8(0, 128), u8(0)), pkv.PkvError),
                       (("mx4", 130, 256, u8(130, 256)[:, ::2], u8(2048)), ValueError),
                       (("mx4", 130, 256, torch.zeros(130, 128), u8(2048)), TypeError)]:
        with pytest.raises(what):
            pkv.MxTensor(*args)
    with pytest.raises(ValueError, match="kind must be one of"):
        pkv.MxTensor.empty("mx6", 3, 128, device="cpu")


def test_host_tensors_are_refused(lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    mx = pkv.MxTensor.empty("mx8", 4, 256, device="cpu")
    for call in (lambda: pkv.pkv_mx_quantize(None, x, mx), lambda: pkv.pkv_mx_read(None, mx, x), lambda: pkv.pkv_mx_linear(None, mx, mx, x)):
        with pytest.raises((TypeError, ValueError), match="CUDA"):
            call()
    with pytest.raises(ValueError, match="together"):
        pkv.pkv_add_norm(None, x, x, x[0], mx)


def test_the_short_way_leaves_what_it_does_not_like(lib):
    """csrc/pkv_torch.cpp's functions return None for wrong arguments of any kind and launch nothing."""
    if pkv._fast is None:
        pytest.skip("the module was not built")
    x, b, s = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(1024, dtype=torch.uint8), (0, 32, 8, 128)
    mx = (2, 4, 256)
    good = {"mx_quantize": (0, s, x, mx, b, b, 0), "mx_read": (0, s, mx, b, b, x, 0),
            "add_norm": (0, s, x, x, x[0], mx, b, b, x, 0), "mx_linear": (0, s, mx, b, b, mx, b, b, x, 0),
            "mx_qkv_proj": (0, s, mx, b, b, mx, b, b, x, x, x, 0)}
    for name, args in good.items():
        f = getattr(pkv._fast, name)
        assert f() is None and f(*args[:-1]) is None and f(*args, 1) is None
        assert f(*args) is None                     # tensors of the host
        for k in range(len(args)):
            for bad in ("x", None, 1.5, -1, 2 ** 70, (), (1, 2), (2, 2 ** 40, 2 ** 40), (9, 4, 256), (2, -4, 256), object()):
                assert f(*args[:k], bad, *args[k + 1:]) is None


def test_the_64_bit_forms_agree_with_the_bytes():
    """_mx.quantise against torch's own e4m3 and a list of hand-made groups."""
    x = np.zeros((6, 32))
    x[0, :3] = 448, 1, -1.0625          # e = 0; ties to even: 1.0625 -> 1
    x[1, :3] = 449, 2, 3                # beyond the largest code: e = 1
    x[2, 0] = 2.0 ** -140               # e = -127, code 2^-13 -> 0
    x[3, :2] = 256, 2.0 ** -10          # half of the smallest code: to 0
    x[4, :2] = np.inf, 1
    n, byte = _mx.quantise(x, "mx8")
    assert byte[:, 0].tolist() == [127, 128, 0, 127, 255, 0]
    got = _mx.values(n, byte, np.signbit(x), "mx8")
    assert got[0, :3].tolist() == [448, 1, -1] and got[1, :3].tolist() == [448, 2, 3]
    assert got[3, :2].tolist() == [256, 0] and np.isnan(got[4]).all()
    r = torch.randn(50, 64, dtype=torch.float64) * 100
    n, byte = _mx.quantise(r.numpy(), "mx8")
    unit = np.repeat(np.exp2(byte - 127.0), 32, -1)
    want = torch.from_numpy(r.numpy() / unit).float().to(torch.float8_e4m3fn).double().numpy() * unit
    assert np.array_equal(_mx.values(n, byte, np.signbit(r.numpy()), "mx8"), want)
    y = np.zeros((1, 32))
    y[0, :9] = 6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.2
    n, byte = _mx.quantise(y, "mx4")
    assert _mx.values(n, byte, np.signbit(y), "mx4")[0, :9].tolist() == [6, 4, 4, 2, 2, 1, 1, 0, 0] and byte[0, 0] == 127
