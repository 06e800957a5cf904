"""Pins of the cache-side oracle, and the host side of the rotary frequencies (no GPU)."""

import math

import numpy as np
import pytest

import lossless_draft_verification_speculative_b200 as dv
from lossless_draft_verification_speculative_b200 import build_lib
from oracle import cache_ref as ref


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib.build()
    return dv.load_library()


def test_rotate_by_hand():
    """A quarter turn sends (1, 0) to (0, 1) and (0, 1) to (-1, 0); the rest is copied."""
    f = np.array([math.pi / 2, math.pi])
    x = np.array([[1.0, 2.0, 0.0, 3.0, 7.0]])
    y, _ = ref.rotate(x, 1, f)                       # pairs (0, 2), (1, 3)
    np.testing.assert_allclose(y, [[0.0, -2.0, 1.0, -3.0, 7.0]], atol=1e-15)
    y, _ = ref.rotate(x, 1, f, interleaved=True)     # pairs (0, 1), (2, 3)
    np.testing.assert_allclose(y, [[-2.0, 1.0, 0.0, -3.0, 7.0]], atol=1e-15)
    y, _ = ref.rotate(x, 3, f, magnitude=2.0)        # three quarter turns, doubled
    np.testing.assert_allclose(y, [[0.0, -4.0, -2.0, -6.0, 7.0]], atol=1e-14)


def test_rotation_keeps_relative_positions():
    """q . k after rotation depends on the distance alone."""
    rng = np.random.default_rng(1)
    f, _ = ref.frequencies(16, 100.0)
    q, k = rng.standard_normal((1, 16)), rng.standard_normal((1, 16))
    for il in (False, True):
        a = ref.rotate(q, 40, f, il)[0] @ ref.rotate(k, 33, f, il)[0].T
        b = ref.rotate(q, 1007, f, il)[0] @ ref.rotate(k, 1000, f, il)[0].T
        np.testing.assert_allclose(a, b, atol=1e-11)


def test_attend_by_hand():
    """Two equal scores average their values; a log(3) advantage weighs 3 to 1; a token before
    the cache's start sees nothing."""
    K = np.array([[[0.0]], [[0.0]], [[math.log(3.0)]]])
    V = np.array([[[1.0]], [[3.0]], [[10.0]]])
    r = ref.attend(np.ones((2, 1, 1)), K, V, 2, 1.0)
    np.testing.assert_allclose(r.out[:, 0, 0], [2.0, (1 + 3 + 3 * 10) / 5])
    np.testing.assert_allclose(r.lse[:, 0], [math.log(2), math.log(5)])
    r = ref.attend(np.ones((2, 1, 1)), K, V, 2, 1.0, causal=False, window=2)
    np.testing.assert_allclose(r.out[:, 0, 0], [(1 + 3 + 30) / 5, (3 + 30) / 4])
    r = ref.attend(np.ones((4, 1, 1)), K, V, 4, 1.0)
    assert r.out[0, 0, 0] == 0 and r.lse[0, 0] == -np.inf and r.seen.tolist() == [0, 1, 2, 3]


def test_unseen_places_do_not_matter():
    rng = np.random.default_rng(2)
    K, V, q = rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 2, 4)), \
        rng.standard_normal((2, 4, 4))
    a = ref.attend(q, K, V, 2, 0.5, window=3)
    K[:5], V[:5] = np.nan, np.inf
    b = ref.attend(q, K, V, 2, 0.5, window=3)
    assert np.array_equal(a.out, b.out) and np.isfinite(b.out).all()


def test_gather_follows_the_table():
    pages = np.arange(3 * 2).reshape(3, 2, 1, 1).astype(float)
    assert ref.gather(pages, [2, 0], 3)[:, 0, 0].tolist() == [4.0, 5.0, 0.0]
    assert np.isnan(ref.gather(pages, [2, 3], 3)[2]).all()


@pytest.mark.parametrize("R", [2, 4, 64, 96, 128])
@pytest.mark.parametrize("scaling,kw", [
    (None, {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
    ("yarn", dict(factor=16.0, trained=4096.0)),
    ("yarn", dict(factor=2.0, trained=40.0, low=2.0, high=3.0)),
    ("bands", dict(factor=8.0, trained=8192.0)),
])
def test_frequencies_match_the_formulas(R, scaling, kw):
    """Each frequency is the float64 formula's, rounded once to float32 (half a step, 2^-24),
    plus the float64 arithmetic's own few steps."""
    if scaling == "ntk" and R == 2:
        with pytest.raises(dv.DsparkError):
            dv.rotary_frequencies(R, 1e4, scaling=scaling, **kw)
        return
    f, mag = dv.rotary_frequencies(R, 500000.0, scaling=scaling, **kw)
    ends = dict(zip(("low", "high"), (1.0, 32.0) if scaling == "yarn" else (1.0, 4.0)))
    want, wmag = ref.frequencies(R, 500000.0, scaling, **{**ends, **kw})
    np.testing.assert_allclose(f.numpy().astype(np.float64), want, rtol=2.0 ** -24 + 1e-14)
    assert abs(mag - wmag) <= 2.0 ** -24 * wmag + 1e-15


def test_long_context_scalings_keep_and_stretch():
    """YARN and bands keep the fastest pair and divide the slowest by the factor."""
    plain, _ = dv.rotary_frequencies(128, 1e4)
    for s in ("yarn", "bands"):
        f, _ = dv.rotary_frequencies(128, 1e4, scaling=s, factor=8.0, trained=4096.0)
        assert f[0] == plain[0] and abs(f[-1] * 8 / plain[-1] - 1) < 1e-6
        assert (f[:-1] >= f[1:]).all()


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=2048), dict(theta=1.0),
    dict(theta=float("inf")), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=float("nan")), dict(scaling="yarn", factor=2.0, trained=0.0),
    dict(scaling="bands", factor=2.0, low=4.0, high=4.0),
    dict(scaling="bands", factor=2.0, low=0.0),
])
def test_frequencies_refuse(bad):
    a = {"rotary_dim": 64, "theta": 1e4, **bad}
    with pytest.raises(dv.DsparkError):
        dv.rotary_frequencies(a.pop("rotary_dim"), a.pop("theta"), **a)


def test_frequencies_refuse_an_unknown_scaling():
    with pytest.raises(ValueError):
        dv.rotary_frequencies(64, scaling="other")
