"""Arguments of the rotary positions' host calls at the ends of their ranges."""

import ctypes
import math

import pytest

import block_speculative_decoding_ctx_gb300 as dfl
from block_speculative_decoding_ctx_gb300 import build as dbuild
from oracle import rotary


@pytest.fixture(scope="module")
def L():
    dbuild.build()
    return dfl.lib()


@pytest.mark.parametrize("kw", [
    dict(theta=1e-320), dict(theta=1e-320, trained=4096.0, stretch=4.0), dict(theta=1e4, stretch=1e-310),
    dict(theta=5e-324, trained=1.0, slow=-1e300, fast=1e300), dict(theta=1e4, stretch=5e-324, trained=4096.0),
])
def test_frequencies_that_are_not_finite_are_refused(L, kw):
    """Every argument is finite, some frequency is not: none is handed out."""
    with pytest.raises(dfl.DflashError, match="ARG"):
        dfl.dflash_rope_frequencies(128, **kw)
    out = (ctypes.c_double * 64)(*[7.0] * 64)
    a = dict(stretch=1.0, trained=0.0, slow=1.0, fast=4.0)
    a.update(kw)
    assert L.dflash_rope_frequencies(128, a["theta"], a["stretch"], a["trained"], a["slow"], a["fast"], out) == -1
    assert list(out) == [7.0] * 64


@pytest.mark.parametrize("kw", [dict(theta=1e-150), dict(theta=1e308), dict(theta=1e4, stretch=1e-300), dict(theta=1e4, stretch=1e308),
                                dict(theta=1.0, trained=1e308, slow=0.0, fast=1e-3, stretch=1e-300)])
def test_frequencies_at_the_ends_of_their_range(L, kw):
    got = dfl.dflash_rope_frequencies(128, **kw)
    assert all(math.isfinite(f) for f in got)
    want = rotary.frequencies(128, **kw)
    assert all(abs(g - w) <= 1e-13 * abs(w) for g, w in zip(got, want))
