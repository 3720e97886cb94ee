"""Pins of the rotary-position oracle, and the prepared tables of the library
against it (host only)."""
import ctypes
import math

import numpy as np
import pytest

from confidence_gated_kv_logit_b200 import ConfKVError, Rope, binding, build
from oracle.rope import frequencies, rotate_row


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def rows(n, d, seed=0):
    return np.random.RandomState(seed).randn(n, d)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rd", [0, 2, 6, 16])
def test_position_zero_and_the_inverse(layout, rd):
    f, mag = frequencies(rd) if rd else (np.zeros(0), 1.0)
    for x in rows(4, 16):
        assert np.array_equal(rotate_row(x, 0, f, mag, layout), x)
        y = rotate_row(rotate_row(x, 1234, f, mag, layout), -1234, f, mag, layout)
        np.testing.assert_allclose(y, x, atol=1e-12)
        assert np.array_equal(rotate_row(x, 99, f, mag, layout)[rd:], x[rd:])


def test_lengths_and_relative_positions():
    f, mag = frequencies(32, theta=500.0)
    q, k = rows(2, 32, 3)
    for layout in ("half", "interleaved"):
        a = rotate_row(q, 17, f, mag, layout) @ rotate_row(k, 5, f, mag, layout)
        b = rotate_row(q, 1017, f, mag, layout) @ rotate_row(k, 1005, f, mag, layout)
        assert abs(a - b) < 1e-10
        y = rotate_row(q, 17, f, mag, layout)
        pairs = (y[:16], y[16:]) if layout == "half" else (y[0::2], y[1::2])
        orig = (q[:16], q[16:]) if layout == "half" else (q[0::2], q[1::2])
        np.testing.assert_allclose(np.hypot(*pairs), np.hypot(*orig), atol=1e-12)


def test_interleaved_is_complex_multiplication():
    f, mag = frequencies(8)
    x = rows(1, 8)[0]
    z = (x[0::2] + 1j * x[1::2]) * np.exp(1j * 77 * f)
    y = rotate_row(x, 77, f, mag, "interleaved")
    np.testing.assert_allclose(y[0::2] + 1j * y[1::2], z, atol=1e-12)


def test_norm_by_hand():
    x = np.array([3.0, 4.0, 0.0, 0.0])
    y = rotate_row(x, 0, *frequencies(4), "half", weight=[1, 2, 1, 1], eps=0.0)
    np.testing.assert_allclose(y, [3 / 2.5, 8 / 2.5, 0, 0])


def test_scalings_by_hand():
    f, m = frequencies(4, theta=100.0)
    np.testing.assert_allclose(f, [1.0, 0.1])
    assert m == 1.0
    np.testing.assert_allclose(frequencies(4, theta=100.0, scaling="linear", factor=2.0)[0], [0.5, 0.05])
    # theta * 4^2 = 1600, so the second pair turns by 1600^-1/2 = 1/40
    np.testing.assert_allclose(frequencies(4, theta=100.0, scaling="ntk", factor=4.0)[0], [1.0, 0.025])
    # turns within 100 positions: 100/2pi = 15.9 (kept), 1.59 (between 1 and 4 bands), 0.159 (divided)
    f = frequencies(6, theta=1000.0, scaling="banded", factor=8.0, low_band=1.0, high_band=4.0, original_length=100)[0]
    t = (10 / (2 * math.pi) - 1) / 3
    np.testing.assert_allclose(f, [1.0, 0.1 * ((1 - t) / 8 + t), 0.01 / 8])
    f, m = frequencies(64, theta=10000.0, scaling="yarn", factor=4.0, original_length=4096)
    assert m == pytest.approx(0.1 * math.log(4) + 1)
    plain = frequencies(64)[0]
    # pair 10: floor(64 ln(4096 / 64 pi) / (2 ln 1e4)) = 10; ceil of beta_slow's = 23
    np.testing.assert_allclose(f[:11], plain[:11])
    np.testing.assert_allclose(f[23:], plain[23:] / 4)
    np.testing.assert_allclose(f[16], plain[16] * (6 / 13 / 4 + 7 / 13))


CASES = [dict(), dict(theta=1e6, scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
         dict(theta=5e5, scaling="banded", factor=8.0, original_length=8192, low_band=1.0, high_band=4.0),
         dict(theta=1e6, scaling="yarn", factor=4.0, original_length=32768), dict(magnitude=1.5)]


@pytest.mark.parametrize("kw", CASES)
@pytest.mark.parametrize("rd", [2, 30, 96, 128])
def test_prepared_tables(kw, rd):
    r = Rope(128, rotary_dim=rd, **kw)
    f, mag = frequencies(rd, **kw)
    got = np.array([int(t) for t in r.table.turns[:rd // 2]], dtype=object)
    want = [v / (2 * math.pi) * 2.0 ** 64 for v in f]
    # the table holds 62 bits of a turn; fp64 frequencies agree to a few parts in 1e16
    for g, w in zip(got, want):
        assert abs(g - w) <= 4 + 4e-15 * w
    assert r.table.magnitude == np.float32(mag)
    assert (r.table.rotary_dim, r.table.head_dim) == (rd, 128)


@pytest.mark.parametrize("args,kw", [
    ((0,), {}), ((258,), {}), ((127,), {}), ((128, 130), {}), ((128, 3), {}), ((128, -2), {}),
    ((128,), dict(theta=1.0)), ((128,), dict(theta=float("nan"))), ((128,), dict(scaling="linear", factor=0.5)),
    ((128,), dict(scaling="linear", factor=float("inf"))), ((128,), dict(magnitude=-1.0)),
    ((128,), dict(scaling="banded", factor=2.0, low_band=4.0, high_band=4.0)),
    ((128,), dict(scaling="banded", factor=2.0, original_length=0)),
    ((128,), dict(scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0)),
])
def test_bad_parameters_are_refused(args, kw):
    with pytest.raises(ConfKVError) as e:
        Rope(*args, **kw)
    assert e.value.status == 1


def test_bad_names_are_refused():
    with pytest.raises(ValueError):
        Rope(128, layout="other")
    with pytest.raises(ValueError):
        Rope(128, scaling="other")
    with pytest.raises(TypeError):
        Rope(128, base=1.0)


def test_calls_are_checked_on_the_host():
    """Refused before anything is launched: no device is needed to see it."""
    lib = binding.load_library()
    t = Rope(128).table
    ok = dict(x=4096, y=1 << 20, weight=None, heads=2, x_batch=256, x_token=256, x_head=128, y_batch=256, y_token=256,
              y_head=128)

    def call(table=t, batch=1, tokens=1, pos=4096, xt=1, yt=1, eps=1e-6, **kw):
        r = binding.RopeRows(**dict(ok, **kw))
        return lib.confkv_rope(ctypes.byref(table) if table else None, batch, tokens, pos, xt, yt, eps,
                               ctypes.byref(r), None, None)

    assert call(batch=0) == 0 and call(tokens=0) == 0
    for bad in (dict(table=None), dict(batch=-1), dict(tokens=-1), dict(pos=None), dict(pos=4097), dict(xt=3),
                dict(yt=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(heads=0), dict(x=None), dict(y=None),
                dict(x=4097), dict(y=4097), dict(weight=4098), dict(x_head=-128), dict(y_head=64),
                dict(tokens=2, y_token=100), dict(batch=2, y_batch=1),
                dict(y=4096, yt=2), dict(y=4096, x_head=256)):
        assert call(**bad) == 1, bad
    broken = binding.RopeTable.from_buffer_copy(t)
    broken.rotary_dim = 300
    assert call(table=broken) == 1


@pytest.mark.parametrize("kw", [dict(magnitude=1e39), dict(magnitude=1e-60), dict(scaling="ntk", factor=1e300),
                                dict(scaling="ntk", factor=1e200, theta=1e200)])
def test_parameters_beyond_what_a_table_holds_are_refused(kw):
    """A factor that is inf or 0 in fp32, and a base beyond fp64, would turn every value into inf, 0 or itself."""
    with pytest.raises(binding.ConfKVError) as e:
        binding.Rope(128, **kw)
    assert e.value.status == 1
    binding.Rope(128, magnitude=1e38)
    binding.Rope(128, scaling="ntk", factor=1e100)
