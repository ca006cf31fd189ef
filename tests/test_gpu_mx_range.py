"""pkv_add_norm at the ends of the ranges that include/pkv.h gives: sums of squares near fp32's largest and smallest numbers,
weights of any size."""
import numpy as np
import pytest
import torch

import _mx
import paged_kv_gqa_qk_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
OUTS = ["bf16", "mx8", "mx4"]


def norm_of(x, w, kind, eps):
    """The norm's values as the output holds them."""
    z = torch.zeros(2, 1, 64, 128, dtype=torch.bfloat16, device=DEV)
    p = pkv.PagedKVPool(z[0], z[1], cfg=dict(heads=4, kv_heads=1, max_seq=64, eps=eps))
    out, _ = p.add_norm(x.to(DEV), None, w.to(DEV), out=kind)
    assert p.check_errors() == 0
    p.close()
    return _mx.f64(out) if kind == "bf16" else _mx.stored(out)


def held(y, kind):
    """Values beyond fp32's (and bf16's) range are infinite; in microscaled form their group is NaN."""
    y = np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y)
    if kind != "bf16":
        return _mx.held(y, kind)
    with np.errstate(invalid="ignore"):
        b = np.where(np.isfinite(y), _mx.bf16(np.where(np.isfinite(y), y, 0)), y)
    return np.where(np.abs(b) >= 2.0 ** 128, np.copysign(np.inf, b), b)


def check(got, y, kind, d):
    """Each value is the rounding of y or of what lies within d of it."""
    ok = np.zeros(got.shape, bool)
    for e in (-d, d):
        want = held(y * (1 + e), kind)
        ok |= (got == want) | (np.isnan(got) & np.isnan(want))
    assert ok.all(), (np.argwhere(~ok)[:4], got[~ok][:4], y[~ok][:4])


def uneven(rows, cols, seed, size):
    """Values of size * [1, 2) with all of bf16's bits and both signs."""
    gen = torch.Generator().manual_seed(seed)
    m = 1.0 + torch.randint(0, 128, (rows, cols), generator=gen).double() / 128
    m *= torch.randint(0, 2, (rows, cols), generator=gen) * 2 - 1
    return (m * size).to(torch.bfloat16)


@pytest.mark.parametrize("kind", OUTS)
@pytest.mark.parametrize("hidden,size", [(128, 2.0 ** 59), (256, 2.0 ** 59), (4096, 2.0 ** 57), (8192, 2.0 ** 56),
                                         (256, 2.0 ** 51), (256, 2.0 ** 46), (1024, 2.0 ** -40), (1024, 2.0 ** -45)])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_sums_near_the_largest_number(kind, hidden, size, eps):
    """A mean square of up to 2^120 (the sum stays below 2^128), and of 2^-90: as exact as any other, to 2^-40."""
    x = uneven(4, hidden, hidden, size)
    x[1] = float(np.float32(size * 1.53125))         # equal values: the root of one square, on every border
    assert float(x.double().square().sum(-1).max()) < 2.0 ** 127.9
    w = uneven(1, hidden, 1, 0.75)[0]
    check(norm_of(x, w, kind, eps), _mx.norm(_mx.f64(x), _mx.f64(w), eps), kind, 2.0 ** -40)


@pytest.mark.parametrize("kind", OUTS)
@pytest.mark.parametrize("hidden", [128, 1024, 4096, 16384])
@pytest.mark.parametrize("size", [2.0 ** -66, 2.0 ** -60])
def test_rows_of_tiny_values_without_eps(kind, hidden, size):
    """Squares from 2^-132 on are whole multiples of 2^-146, which fp32's subnormals hold: the sum keeps them but for the
    roundings of a warp's parts, 16 units of 2^-149 twice, of at least 128 * 2^-132: 2^-19, which the root halves."""
    x = uneven(3, hidden, hidden, size)
    w = uneven(1, hidden, 2, 0.75)[0]
    check(norm_of(x, w, kind, 0.0), _mx.norm(_mx.f64(x), _mx.f64(w), 0.0), kind, 2.0 ** -19)


@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 52, 1.0, 2.0 ** -30])
def test_digits_of_the_root(size):
    """Rows whose root is off a whole one by 2^-35: 64 of 256 values are c, one is c / 2^14, so y = 2 w (1 - 2^-35), and in 4
    bits 3.5 (1 - 2^-35) is 3, where 3.5 itself would be 4.  All mantissas of c."""
    c = (1.0 + torch.arange(128).double() / 128) * size
    x = torch.zeros(128, 256, dtype=torch.float64)
    x[:, :64], x[:, 100] = c[:, None], c / 2 ** 14
    w = torch.full((256,), 1.75, dtype=torch.bfloat16)
    w[:64:4] = 3.0
    got = norm_of(x.to(torch.bfloat16), w, "mx4", 0.0)
    assert np.array_equal(got[:, :64], np.broadcast_to(np.where(np.arange(64) % 4 == 0, 6.0, 3.0), (128, 64)))


@pytest.mark.parametrize("kind", OUTS)
@pytest.mark.parametrize("hidden", [128, 4096, 16384])
@pytest.mark.parametrize("size", [2.0 ** 56, 1.0, 2.0 ** -50])
def test_weights_of_any_size(kind, hidden, size):
    """An h w of 2^128 or more makes its y NaN, in microscaled form the group; everything else is exact."""
    if hidden == 16384 and size > 1:
        size /= 16
    x = uneven(4, hidden, hidden, size)
    x[2, ::3] = 0
    x[3] = float(np.float32(size * 1.53125))
    w = uneven(1, hidden, 3, 1.0)[0]
    gen = torch.Generator().manual_seed(4)
    w *= 2.0 ** torch.randint(-20, 118, (hidden,), generator=gen).float()
    w[:64] = uneven(1, 64, 5, 1.0)[0]               # (two groups of ordinary ones)
    w[64:68] = torch.tensor([2.0 ** 68, -(2.0 ** 117), 2.0 ** 64, -(2.0 ** 65)])
    w = w.to(torch.bfloat16)
    y, hw = _mx.norm(_mx.f64(x), _mx.f64(w), 1e-6), _mx.f64(x) * _mx.f64(w)
    assert np.isfinite(y).all() and (np.abs(y) < 2.0 ** 128).all() and (np.abs(hw) < 2.0 ** 128).any(-1).all()
    y = np.where(np.abs(hw) >= 2.0 ** 128, np.nan, y)
    check(norm_of(x, w, kind, 1e-6), y, kind, 2.0 ** -40)


@pytest.mark.parametrize("kind", OUTS)
def test_infinite_and_nan_weights(kind):
    x = uneven(4, 256, 1, 1.0)
    x[1, 40] = 0
    x[3, 3] = 2.0 ** 70                              # (a row without a norm)
    w = uneven(1, 256, 2, 1.0)[0]
    w[40], w[200] = float("inf"), float("nan")
    clean = w.clone()
    clean[40], clean[200] = 1, 1
    y = _mx.norm(_mx.f64(x), _mx.f64(clean), 1e-6)
    y[:, [40, 200]], y[3] = np.nan, np.nan
    check(norm_of(x, w, kind, 1e-6), y, kind, 2.0 ** -40)


@pytest.mark.parametrize("kind", OUTS)
def test_where_squares_leave_the_range(kind):
    """A row's squares may add up to anything below 2^128; from there on it is NaN."""
    for hidden, value, finite in [(128, 2.0 ** 60, True), (128, 1.25 * 2.0 ** 60, True), (128, 1.5 * 2.0 ** 60, False),
                                  (4096, 1.9375 * 2.0 ** 57, True), (4096, 2.0 ** 58, False),
                                  (32768, 1.375 * 2.0 ** 56, True), (32768, 1.4375 * 2.0 ** 56, False)]:
        assert (hidden * value ** 2 < 2.0 ** 128) == finite
        x = torch.ones(2, hidden, dtype=torch.bfloat16)
        x[1] = value
        w = torch.ones(hidden, dtype=torch.bfloat16)
        w[::32] = 2.0                                # (a code without a border beside it)
        got = norm_of(x, w, kind, 1e-6)
        assert np.isfinite(got[0]).all()
        if finite:
            check(got[1:], _mx.norm(_mx.f64(x[1:]), _mx.f64(w), 1e-6), kind, 2.0 ** -40)
        else:
            assert np.isnan(got[1]).all()
