"""Appends and reads back of batches whose rows are not one full list: padding
behind the last request, rows before the first, requests that do not fit in
front of ones that do; attention of items of very different sizes."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import target as ot
from target_testutil import Paged, check_attention, rows_tensor, run_attention, to64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


BATCHES = [
    # row_start, rows of the tensors, requests that fit, new rows of each, status
    ([0, 3, 5, 9], 400, {0: (0, 3), 1: (3, 2), 2: (5, 4)}, 0),       # padded
    ([6, 8, 8, 12], 12, {0: (6, 2), 2: (8, 4)}, 0),                  # rows before the first
    ([0, 25, 5, 10], 12, {2: (5, 5)}, -2),                           # past the tensors, then decreasing
    ([5, 10, 0, 3], 12, {0: (5, 5), 2: (0, 3)}, -2),                 # decreasing in the middle
    ([0, 6, 4, 4], 12, {0: (0, 6)}, -2),                             # the last decreasing
    ([-2, 3, 7, 9], 12, {1: (3, 4), 2: (7, 2)}, -2),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("start,rows,fits,status", BATCHES)
def test_requests_that_fit_are_moved_whatever_stands_before_them(start, rows, fits, status, e4m3):
    lens, n_kv, hd, page = [40, 33, 50], 2, 64, 16
    p = Paged(lens, [0, 0, 0], n_kv, hd, page, BF, e4m3, garbage=False)
    row_start = torch.tensor(start, dtype=torch.int32, device="cuda")
    batch = (row_start, p.kv_len, p.table)
    x = [rows_tensor(rows, n_kv, hd, BF, 5 + i) for i in range(2)]
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    # read back what is there, then write other rows and look at the pages
    back = [torch.full_like(t, 7.0) for t in x]
    dfl.dflash_paged_gather(p.cache, back[0], back[1], *batch, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == status
    want = [t.copy() if t is not None else None for t in p.host()]
    for i in range(2):
        ref = np.full((rows, n_kv, hd), 7.0)
        codes, scale = ot.quantize(x[i].float().cpu().numpy())
        for b, (s0, n) in fits.items():
            for j in range(n):
                pos = lens[b] - n + j
                pid, at = p.table_np[b, pos // page], pos % page
                ref[s0 + j] = ot.read(p.host()[i], p.host()[2 + i], pid, at, e4m3)
                want[i][pid, :, at] = codes[s0 + j] if e4m3 else to64(x[i])[s0 + j]
                if e4m3:
                    want[2 + i][pid, :, at] = scale[s0 + j]
        ref = torch.from_numpy(ref.astype(np.float32)).to(BF).double().numpy()
        np.testing.assert_array_equal(to64(back[i]), ref)
    ws.zero_()
    dfl.dflash_paged_append(p.cache, x[0], x[1], *batch, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == status
    for got, w in zip(p.host(), want):
        if w is not None:
            np.testing.assert_array_equal(got, w)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_attention_of_small_and_large_items_in_turn_over_codes(dtype, hd):
    """Items of one and of two query tiles, of 1 to 8 key tiles, in one call and
    so many that a CTA meets several of either kind: every depth of the rings of
    slots, each left at an odd place by some item before."""
    rng = np.random.default_rng(7)
    lens, rows = [], []
    for i in range(110):
        n = int(rng.choice([0, 1, 3, 10, 17, 40, 90]))
        rows.append(n)
        lens.append(n + int(rng.choice([0, 1, 127, 128, 300, 900])))
    p = Paged(lens, rows, 3, hd, 32, dtype, True, seed=11)
    q = rows_tensor(p.n_rows, 12, hd, dtype, 3, extra=1, size=1.5)
    first = None
    for _ in range(3):
        out, lse, status = run_attention(p, q, window=500)
        assert status == 0
        if first is None:
            first = (out.clone(), lse.clone())
            check_attention(p, q, out, lse, window=500)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
