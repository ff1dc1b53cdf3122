"""The oracle of the target's side, held to closed forms and to torch's own
float64 softmax."""

import numpy as np
import pytest
import torch

from oracle import quant
from oracle import target as ot


def test_places_and_visible_ranges():
    table = [[4, 1, 7], [2, 0, 5]]
    got = ot.places([0, 2, 2 + 3], [18, 2], table, 16)
    assert got == [(0, 0, 16, 1, 0), (1, 0, 17, 1, 1), (3, 1, 0, 2, 0), (4, 1, 1, 2, 1)]
    assert ot.visible(5, 9, True, 0) == (0, 6)
    assert ot.visible(5, 9, False, 0) == (0, 9)
    assert ot.visible(5, 9, True, 2) == (4, 6)
    lo, hi = ot.visible(-1, 3, True, 0)
    assert hi <= lo


def test_quantize_is_the_weights_rule_per_row():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 64)).astype(np.float32)
    x[1, 0] = 0.0
    x[2, 1, 5] = np.nan
    codes, scale = ot.quantize(x)
    for r in range(3):
        for h in range(2):
            if (r, h) == (2, 1):
                assert np.isnan(scale[r, h])
                continue
            c, s = quant.quantize_rows(x[r, h][None])
            assert (c[0] == codes[r, h]).all() and s[0] == scale[r, h]
    assert scale[1, 0] == 1.0


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3), (False, 4)])
def test_attention_against_masked_softmax(causal, window):
    rng = np.random.default_rng(1)
    n, n_q, n_kv, hd, length = 5, 6, 2, 16, 11
    q, k, v = rng.normal(size=(n, n_q, hd)), rng.normal(size=(length, n_kv, hd)), rng.normal(size=(length, n_kv, hd))
    out, lse, mean, size = ot.attention(q, k, v, length, causal, window, 0.25)
    pos = torch.arange(length - n, length)[:, None]
    key = torch.arange(length)[None]
    ok = torch.ones(n, length, dtype=torch.bool)
    if causal:
        ok &= key <= pos
    if window:
        ok &= key > pos - window
    for h in range(n_q):
        z = torch.from_numpy(q[:, h] @ k[:, h // 3].T * 0.25).masked_fill(~ok, -np.inf)
        np.testing.assert_allclose(out[:, h], torch.softmax(z, 1).numpy() @ v[:, h // 3], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse[:, h], torch.logsumexp(z, 1).numpy(), rtol=1e-12)
    assert (np.abs(out) <= mean + 1e-12).all() and (size > 0).all()


def test_rows_that_see_nothing_are_zero():
    q = np.ones((2, 1, 4))
    out, lse, _, _ = ot.attention(q, np.ones((1, 1, 4)), np.ones((1, 1, 4)), 1, True, 0, 1.0)
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf and (out[1] == 1).all()


def test_adjust_counts_the_blocks_own_drafts():
    z = np.zeros((1, 3, 4))
    z[0, :, 1] = 2.0
    z[0, :, 2] = -2.0
    prompt = np.zeros((1, 4), dtype=bool)
    prompt[0, 2] = True
    out, _ = ot.adjust(z, counts=np.array([[0, 0, 0, 3]]), prompt=prompt, draft=np.array([[1, 1]]),
                       repetition=[2.0], frequency=[0.5], presence=[0.25], bias=[(0, 0, 1.0), (0, 0, 2.0)],
                       allow=np.array([[[1, 1, 1, 1], [1, 1, 1, 1], [1, 1, 0, 1]]], dtype=bool))
    np.testing.assert_allclose(out[0, 0], [3.0, 2.0, -4.0, -1.75])
    np.testing.assert_allclose(out[0, 1], [3.0, 1.0 - 0.75, -4.0, -1.75])
    np.testing.assert_allclose(out[0, 2], [3.0, 1.0 - 1.25, -np.inf, -1.75])
