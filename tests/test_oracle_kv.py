"""Pins of the cache oracle (oracle/kv_oracle.py): rotation properties, the 4-bit grid and its
rounding, attention against a plain softmax; and the host-side frequency scalings."""
import math

import numpy as np
import pytest

from eagle_speculative_decoding_03_gb300 import binding as eb
from oracle import kv_oracle as K


def test_rotation_preserves_norms_and_relative_positions():
    rng = np.random.default_rng(0)
    w = 1e4 ** (-np.arange(8) / 8.0)
    for inter in (False, True):
        x = rng.standard_normal((2, 1, 24))
        a = K.rotary(np.repeat(x[:1], 5, 0), [0, 1, 7, 100, 100000], w, inter)
        b = K.rotary(np.repeat(x[1:], 5, 0), [3, 4, 10, 103, 100003], w, inter)
        assert np.allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x[0]), rtol=1e-12)
        assert np.allclose((a * b).sum(-1), (a[0] * b[0]).sum(-1), rtol=1e-9)   # only the distance counts
        assert (a[..., 16:] == x[0, :, 16:]).all() and np.allclose(a[0], x[0])


def test_interleaved_and_half_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(1)
    w = 1e4 ** (-np.arange(16) / 16.0)
    x = rng.standard_normal((3, 2, 32))
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    assert np.allclose(K.rotary(x, [1, 5, 9], w, True)[..., perm], K.rotary(x[..., perm], [1, 5, 9], w, False))


def test_four_bit_rounding_ties_and_saturation():
    # a group whose largest magnitude is 6 has scale 1: borders go to the even code
    x = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -5, .26, .24, 0, 5.1, -6.0])
    code, sc, val = K.quantise(x, 1.0)
    assert K.E4M3[sc[0]] == 1.0
    assert val.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4, .5, 0, 0, 6, -6]
    assert code[8] == 8 and code[9] == 10
    code, sc, val = K.quantise(np.full(16, 1e9), 1.0)
    assert K.E4M3[sc[0]] == 448 and (val == 2688).all()
    code, sc, val = K.quantise(np.full(16, 1e-6), 1.0)      # the scale rounds to 0: zeros
    assert sc[0] == 0 and (val == 0).all() and (code == 0).all()
    code, sc, val = K.quantise(np.r_[np.nan, np.full(15, 3.0)], 1.0)
    assert val[0] == 0 and np.allclose(val[1:], 3.0)


def test_four_bit_relative_error_bound():
    """|value - stored| <= half the widest code gap (1 of 6) plus the scale's own rounding (2^-4)."""
    rng = np.random.default_rng(2)
    x = K.bf16(rng.standard_normal((200, 64)))
    _, _, v = K.quantise(x, 1.0)
    top = np.abs(x.reshape(200, 4, 16)).max(-1).repeat(16, -1)
    assert (np.abs(v - x) <= top * (1 / 6 + 2.0 ** -4) + 1e-12).all()


def test_attention_matches_dense_softmax():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    see = rng.random((3, 7)) < 0.6
    see[1] = False
    o, l, mag, qk, vs = K.attention(q, k, v, see, 0.3)
    for i in range(3):
        for h in range(4):
            s = np.where(see[i], k[:, h // 2] @ q[i, h] * 0.3, -np.inf)
            if not see[i].any():
                assert (o[i, h] == 0).all() and l[i, h] == -np.inf
                continue
            p = np.exp(s - s[np.isfinite(s)].max())
            assert np.allclose(o[i, h], p @ v[:, h // 2] / p.sum()) and np.isclose(l[i, h], np.log(np.exp(s).sum()))


def test_rope_frequencies():
    w = eb.rope_frequencies(64, 1e4)
    assert len(w) == 32 and w[0] == 1.0 and math.isclose(w[31], 1e4 ** (-62 / 64))
    assert [a / b for a, b in zip(w, eb.rope_frequencies(64, 1e4, linear=4.0))] == pytest.approx([4.0] * 32)
    b = eb.rope_frequencies(64, 1e4, banded=(8.0, 1.0, 4.0, 8192))
    for a, x in zip(w, b):
        wave = 2 * math.pi / a
        if wave < 8192 / 4:
            assert x == pytest.approx(a)
        elif wave > 8192:
            assert x == pytest.approx(a / 8)
        else:
            assert a / 8 <= x <= a
    r = eb.rope_frequencies(64, 1e4, ramped=(4.0, 32, 1, 4096))
    assert r[0] == w[0] and r[-1] == pytest.approx(w[-1] / 4) and all(x >= y for x, y in zip(r, r[1:]))
    for bad in (dict(rot_dim=7), dict(rot_dim=64, theta=0.0), dict(rot_dim=64, linear=0.0),
                dict(rot_dim=64, banded=(8, 1, 4, 8192), ramped=(4, 32, 1, 4096)), dict(rot_dim=64, banded=(8, 4, 4, 8192)),
                dict(rot_dim=64, ramped=(0, 32, 1, 4096))):
        with pytest.raises(eb.EagleError):
            eb.rope_frequencies(**bad)


@pytest.mark.parametrize("rot,theta,factor,fast,slow,original", [
    (64, 1e4, 8.0, 32, 1, 131072),       # the ramp ends behind the last pair (index 34 of 0 .. 31)
    (64, 1e4, 4.0, 32, 1, 4096), (128, 5e5, 16.0, 32, 1, 8192), (16, 1e4, 2.0, 8, 2, 100000), (32, 1e4, 8.0, 64, 4, 10 ** 9),
    (64, 1e4, 8.0, 2, 1, 4), (2, 1e4, 8.0, 32, 1, 64)])
def test_ramped_frequencies_follow_the_correction_range(rot, theta, factor, fast, slow, original):
    """The published range: index of a pair that turns n times = rot ln(original / (2 pi n)) / (2 ln
    theta), ends rounded outwards and clamped to [0, rot - 1]; and what the rule promises of the
    pairs outside it."""
    w = np.array(eb.rope_frequencies(rot, theta))
    got = np.array(eb.rope_frequencies(rot, theta, ramped=(factor, fast, slow, original))) / w
    ends = [rot * np.log(original / (2 * np.pi * n)) / (2 * np.log(theta)) for n in (fast, slow)]
    lo, hi = max(np.floor(ends[0]), 0), min(np.ceil(ends[1]), rot - 1)
    if lo < hi:
        ramp = np.clip((np.arange(rot // 2) - lo) / (hi - lo), 0, 1)
        assert np.allclose(got, (1 - ramp) + ramp / factor, rtol=1e-12)
    turns = original * w / (2 * np.pi)
    assert np.allclose(got[turns > fast], 1.0) and (got[turns > slow] > 1.0 / factor).all()
    whole = np.arange(rot // 2) >= np.ceil(ends[1])
    assert np.allclose(got[whole], 1.0 / factor) and np.allclose(got[turns < slow], 1.0 / factor)


def test_a_ramp_needs_falling_frequencies():
    for theta in (1.0, 0.5):
        with pytest.raises(eb.EagleError):
            eb.rope_frequencies(64, theta, ramped=(4.0, 32, 1, 4096))
