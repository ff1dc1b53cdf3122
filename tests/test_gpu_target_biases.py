"""Logit adjustment with more biases of one request than are gathered at a
time (1,024): sums over several gatherings, masks over all of them."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import target as ot
from test_gpu_target import bits, words_of
from target_testutil import to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


@pytest.mark.parametrize("V", [1500, 2049, 9000])
@pytest.mark.parametrize("counts", [(1024, 1025), (1100, 0, 5000), (2600,), (3, 2048, 2049)])
def test_biases_past_the_first_gathering_obey_the_mask(V, counts):
    B, G = len(counts), 5
    rng = np.random.default_rng(V + sum(counts))
    z = torch.from_numpy(rng.normal(size=(B, G, V)).astype(np.float32) * 3).cuda()
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ids = rng.integers(0, V, size=start[-1]).astype(np.int32)
    vals = rng.normal(size=start[-1]).astype(np.float32)
    for b in range(B):       # one id in a row of entries, over the gatherings' borders
        ids[start[b] + 1000:start[b + 1]:13] = 7
    # ids banned and forced by infinite biases, early and late ones
    ids[(ids == 11) | (ids == 12)] = 13
    for b in range(B):
        for v, x in ((11, np.inf), (12, -np.inf)):
            at = [start[b] + i for i in (1, 1030, 2060) if start[b] + i + v < start[b + 1]]
            for e in at:
                ids[e + v], vals[e + v] = v, x
    words = (V + 31) // 32
    allow = rng.random((B, G, words * 32)) < 0.5
    draft = rng.integers(0, V, size=(B, G - 1)).astype(np.int32)
    draft[:, 1] = 7
    f = rng.random(B).astype(np.float32)
    ref = dict(draft=draft, frequency=f, allow=allow[:, :, :V],
               bias=[(b, int(ids[e]), float(vals[e])) for b in range(B) for e in range(start[b], start[b + 1])])
    want, size = ot.adjust(to64(z), **ref)
    assert not np.isnan(want).any() and (want == np.inf).any() == any(c > 20 for c in counts)
    kw = dict(draft=torch.from_numpy(draft).cuda(), frequency=torch.from_numpy(f).cuda(), allow=words_of(allow),
              bias_start=torch.from_numpy(start).cuda(), bias_ids=torch.from_numpy(ids).cuda(),
              bias_vals=torch.from_numpy(vals).cuda())
    out = torch.empty_like(z)
    ws = dfl.workspace(dfl.dflash_logits_adjust_workspace_bytes())
    dfl.dflash_logits_adjust(z, out, ws, **kw)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    got = to64(out)
    np.testing.assert_array_equal(np.where(np.isfinite(got), 0.0, got), np.where(np.isfinite(want), 0.0, want))
    fine = np.isfinite(want)
    # two products and sums, and a sum per bias of an id, half a step of float32
    # of what it adds up each
    most = 6 + np.unique([v for _, v, _ in ref["bias"]], return_counts=True)[1].max()
    with np.errstate(invalid="ignore"):
        assert (np.abs(got - want)[fine] <= (most * 2.0 ** -24 * size)[fine]).all()
    dfl.dflash_logits_adjust(z, z, ws, **kw)                # in place
    torch.cuda.synchronize()
    assert torch.equal(bits(z), bits(out))
