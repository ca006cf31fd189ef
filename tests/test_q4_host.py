"""The 4-bit pool's and the rotation's host side, without a GPU: refusals, sizes, frequencies, and the tests' own
64-bit form of the format against its definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
import _q4
import paged_kv_gqa_qk_gb300 as pkv

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return pkv.load_library()


def test_layout_is_a_permutation():
    for m, n in ((_q4.CODE, 1024), (_q4.KS, 128), (_q4.VS, 128)):
        assert sorted(m.ravel().tolist()) == list(range(n))


def test_e4m3_agrees_with_torch():
    b = torch.arange(0, 127, dtype=torch.uint8)
    v = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_q4.e4m3_value(b.numpy()), v) and np.array_equal(_q4.e4m3_byte(v), b.numpy())
    x = np.abs(np.random.RandomState(0).randn(5000)) * np.exp2(np.random.RandomState(1).randint(-12, 10, 5000))
    x = np.minimum(np.concatenate([x, (v[1:] + v[:-1]) / 2]), 448)     # with every tie
    assert np.array_equal(_q4.e4m3(x), torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())


def test_a_value_is_the_nearest_its_scale_allows():
    x = _q4.bf16(np.random.RandomState(2).randn(40, 128) * 3)
    code, byte = _q4.quantise(x, 0.5)
    v = _q4.values(code, byte, 0.5)
    step = np.repeat(_q4.e4m3_value(byte) * 0.5, 16, -1)
    assert (np.abs(v - x) <= step * 1.0 + 1e-12).all()                 # half of the widest gap, 4 to 6
    inside = np.abs(x) <= 6 * step
    near = np.abs(np.abs(x)[..., None] - _q4.LEVELS * step[..., None]).min(-1)
    assert np.allclose(np.abs(v - x)[inside], near[inside], atol=1e-12)


def test_page_bytes(lib):
    assert pkv.pkv_q4_pool_bytes(None, 1) == 8 * 9216
    assert pkv.pkv_q4_pool_bytes(dict(heads=4, kv_heads=1), 7) == 7 * 9216
    n = ctypes.c_size_t()
    cfg = pkv.pkv_config_default()
    assert lib.pkv_q4_pool_bytes(None, 1, ctypes.byref(n)) == pkv.PKV_EINVAL
    assert lib.pkv_q4_pool_bytes(ctypes.byref(cfg), 0, ctypes.byref(n)) == pkv.PKV_EINVAL
    assert lib.pkv_q4_pool_bytes(ctypes.byref(cfg), 1 << 26, ctypes.byref(n)) == pkv.PKV_ERANGE
    cfg.head_dim = 64
    assert lib.pkv_q4_pool_bytes(ctypes.byref(cfg), 1, ctypes.byref(n)) == pkv.PKV_ENOTIMPL


@pytest.mark.parametrize("bad", [0.0, -1.0, 3.0, 0.1, float("inf"), float("nan"), 2.0 ** 61, 2.0 ** -61])
def test_scales_must_be_powers_of_two(lib, bad):
    out, cfg = vp(), pkv.pkv_config_default()
    for ks, vs in ((bad, 1.0), (1.0, bad)):
        assert lib.pkv_q4_pool_alloc(ctypes.byref(cfg), 1, ks, vs, None, ctypes.byref(out)) == pkv.PKV_EINVAL
        assert lib.pkv_q4_pool_wrap(ctypes.byref(cfg), 1, vp(0x10000), ks, vs, None, ctypes.byref(out)) == pkv.PKV_EINVAL


def test_null_and_misaligned_arguments(lib):
    out, cfg, n = vp(), pkv.pkv_config_default(), ctypes.c_size_t()
    for data in (None, vp(0x10080)):
        assert lib.pkv_q4_pool_wrap(ctypes.byref(cfg), 1, data, 1.0, 1.0, None, ctypes.byref(out)) == pkv.PKV_EINVAL
    assert lib.pkv_q4_pool_alloc(None, 1, 1.0, 1.0, None, ctypes.byref(out)) == pkv.PKV_EINVAL
    assert lib.pkv_q4_pool_data(None, None, ctypes.byref(n)) == pkv.PKV_EINVAL
    x = vp(0x1000)
    assert lib.pkv_q4_append(None, x, x, x, x, None, x, 1, 1, 1, None) == pkv.PKV_EINVAL
    assert lib.pkv_q4_read(None, x, None, x, 1, 1, 1, x, x, 1024, 128, None) == pkv.PKV_EINVAL
    assert lib.pkv_q4_decode(None, x, x, x, x, x, x, x, 1, 1, x, x, 1, None) == pkv.PKV_EINVAL
    assert lib.pkv_norm_rope(None, x, x, x, x, x, 1, 0, 0, 4096, 1024, x, x, 4096, 1024, None) == pkv.PKV_EINVAL
    assert lib.pkv_pool_set_rope(None, None, 1.0, None) == pkv.PKV_EINVAL


def test_frequencies(lib):
    cfg = dict(rotary_dim=64)
    f, m = pkv.pkv_rope_frequencies(cfg)
    plain = [1e6 ** (-2 * i / 64) for i in range(32)]
    assert m == 1 and np.allclose(f, plain, rtol=1e-15)
    f, m = pkv.pkv_rope_frequencies(cfg, "linear", 4.0)
    assert m == 1 and np.allclose(f, np.array(plain) / 4, rtol=1e-15)
    f, m = pkv.pkv_rope_frequencies(cfg, "base", 3.0)
    assert m == 1 and f[0] == 1 and math.isclose(f[31], plain[31] / 3, rel_tol=1e-12)
    f, m = pkv.pkv_rope_frequencies(cfg, "ramp", 4.0, 32768)
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    turns = 32768 * np.array(plain) / (2 * math.pi)
    kept = np.isclose(f, plain, rtol=1e-15)
    cut = np.isclose(f, np.array(plain) / 4, rtol=1e-15)
    assert kept[turns > 64].all() and cut[turns < 0.5].all()
    assert not (kept | cut)[(turns < 20) & (turns > 2)].any() and (np.diff(f) < 0).all()
    assert pkv.pkv_rope_frequencies(cfg, "ramp", 1.0, 32768)[1] == 1


@pytest.mark.parametrize("args", [("linear", 0.5, 1), ("linear", float("nan"), 1), ("base", float("inf"), 1),
                                  ("ramp", 2.0, 0), ("ramp", 2.0, -5)])
def test_frequency_refusals(lib, args):
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_rope_frequencies(None, *args)
    assert e.value.code == pkv.PKV_EINVAL


def test_unknown_scaling(lib):
    cfg, f, m = pkv.pkv_config_default(), (ctypes.c_double * 64)(), ctypes.c_double()
    for kind in (-1, 4):
        assert lib.pkv_rope_frequencies(ctypes.byref(cfg), kind, 1.0, 1, f, ctypes.byref(m)) == pkv.PKV_EINVAL
    with pytest.raises(KeyError):
        pkv.pkv_rope_frequencies(None, "other")


def test_tensors_of_another_device_are_refused():
    t = torch.zeros(2)
    pkv._on_device(-1, a=t, b=None)
    with pytest.raises(ValueError, match="weights lies on cpu, the pool on cuda:1"):
        pkv._on_device(1, table=None, weights=t)


def test_the_short_way_leaves_what_it_does_not_like(lib):
    """csrc/pkv_torch.cpp's functions return None for wrong arguments of any kind and launch nothing."""
    if pkv._fast is None:
        pytest.skip("the module was not built")
    t, i = torch.zeros(1, 8, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    spec = (0, 32, 8, 128)
    good = {"decode": (0, spec, t, t, t, t, t, i, i, None, t, 0, 0, 0), "append": (0, spec, t, t, t, i, None, i, 1, 1, 0),
            "read": (0, spec, i, None, i, t, t, 1, 1, 0), "norm_rope": (0, spec, t, t, t, t, i, 0, t, t, 0)}
    for name, args in good.items():
        f = getattr(pkv._fast, name)
        assert f() is None and f(*args[:-1]) is None and f(*args, 1) is None
        assert f(*args) is None                     # tensors of the host
        for k in range(len(args)):
            for bad in ("x", None, 1.5, -1, 2 ** 70, (), (1, 2, 3, "x"), object()):
                assert f(*args[:k], bad, *args[k + 1:]) is None
    with pytest.raises(TypeError):
        pkv._fast.bind(1, 2)
