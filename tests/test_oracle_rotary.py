"""Pins of the oracle's 4-bit rows and rotary positions."""

import math

import numpy as np
import pytest
import torch

from oracle import e2m1, model, rotary


def test_values_are_those_of_the_format():
    assert e2m1.MAGNITUDE.tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert e2m1.value(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_rounding_by_definition():
    v = e2m1.MAGNITUDE
    for c in range(8):
        assert e2m1.round_code(v[c]) == c and e2m1.round_code(-v[c]) == c | 8
    for c in range(7):                                     # ties to the even index, either side to its own
        mid = (v[c] + v[c + 1]) / 2
        assert e2m1.round_code(mid) == (c if c % 2 == 0 else c + 1)
        assert e2m1.round_code(mid * (1 - 1e-9)) == c and e2m1.round_code(mid * (1 + 1e-9)) == c + 1
    assert e2m1.round_code(1e30) == 7 and e2m1.round_code(-1e30) == 15
    assert e2m1.round_code(-0.1) == 8


def test_bf16_rounding_is_torchs():
    x = torch.randn(10000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-38, 37, 10000)
    want = x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert (e2m1.bf16_bits(x.numpy()) == want).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_records_hold_rows_to_half_a_step(hd):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, hd)) * np.exp(rng.standard_normal((50, 1)))).astype(np.float32)
    x[0] = 0
    r = e2m1.pack(x)
    assert r.shape == (50, hd * 5 // 8)
    back = e2m1.unpack(r)
    s = np.repeat(e2m1.scales(x), 16, -1)
    y = np.abs(x) / s
    step = np.select([y < 2, y < 4], [0.5, 1.0], 2.0)
    assert (np.abs(back - x) <= step / 2 * s * (1 + 2.0 ** -20) + np.maximum(y - 6, 0) * s).all()
    assert (y <= 6 * (1 + 2.0 ** -8)).all() and (back[0] == 0).all()


def test_what_is_not_finite_reads_back_as_nan():
    x = np.ones((1, 64), dtype=np.float32)
    x[0, 20] = np.inf
    back = e2m1.unpack(e2m1.pack(x))
    assert np.isnan(back[0, 16:32]).all() and np.isfinite(np.delete(back[0], np.s_[16:32])).all()


def test_frequencies_by_parts():
    plain = rotary.frequencies(64, 1e4)
    assert plain[0] == 1.0 and math.isclose(plain[-1], 1e4 ** (-62 / 64))
    slow = rotary.frequencies(64, 1e4, stretch=8.0)
    assert np.allclose(np.array(slow) * 8, plain)
    parts = np.array(rotary.frequencies(64, 1e4, stretch=8.0, trained=8192))
    turns = 8192 * np.array(plain) / (2 * math.pi)
    assert (parts[turns >= 4] == np.array(plain)[turns >= 4]).all()
    assert np.allclose(parts[turns <= 1] * 8, np.array(plain)[turns <= 1])
    between = (turns > 1) & (turns < 4)
    assert between.any() and (np.diff(parts) < 0).all()


def test_rotation_is_the_models():
    """Half layout over a whole head against the drafter's own oracle."""
    x = np.random.default_rng(0).standard_normal((5, 3, 64))
    pos = np.array([0, 1, 17, 4000, 99999])
    got = rotary.rotate(x, pos, rotary.frequencies(64, 1e4), 0)
    np.testing.assert_allclose(got, model.rope(x, pos, 1e4), atol=1e-9)
    # interleaved: the same pairs elsewhere
    order = np.arange(64).reshape(2, 32).T.reshape(-1)
    np.testing.assert_allclose(rotary.rotate(x[..., order], pos, rotary.frequencies(64, 1e4), 1), got[..., order], atol=1e-12)


def test_angles_of_far_positions():
    for p in (0, -5, 2 ** 31, 2 ** 40 + 3):
        t = rotary.angle(p, 1.0)
        # e^(i p) by squaring, with enough digits
        z, b, n = 1 + 0j, complex(math.cos(1.0), math.sin(1.0)), abs(p)
        while n:
            z, b, n = (z * b if n & 1 else z), b * b, n >> 1
        z = z.conjugate() if p < 0 else z
        assert abs(z / abs(z) - complex(math.cos(t), math.sin(t))) < 1e-9 * max(1.0, abs(p) * 2.0 ** -20)
