"""Attention over a paged cache in 4 bits where a request may have more than 128 packed
rows: pages that are none, requests that do not fit, rows and items that see nothing."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from paged4_testutil import BF, F16, Paged4, check, run
from target_testutil import rows_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


class WithPageOfZeros:
    """p with one more page, of zeros, in the places [(request, entry)] of its table: what
    pages that are none read as."""

    def __init__(self, p, places):
        self.__dict__.update(p.__dict__)
        self.table_np = p.table_np.copy()
        for b, e in places:
            self.table_np[b, e] = p.n_pages

    def host(self):
        pages = [t.cpu().numpy() for t in self.pages]
        return [np.concatenate([t, np.zeros_like(t[:1])]) for t in pages]


def attend(p, q, table, max_rows, **kw):
    ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(q.shape[1], p.n_kv, q.shape[2], max_rows))
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    dfl.dflash_paged_attention(p.cache, q, out, p.row_start, p.kv_len, table, max_rows, ws, lse=lse, **kw)
    return out, lse, dfl.dflash_read_status(ws)


@pytest.mark.parametrize("hd,page,rows,max_rows", [(64, 16, 40, 40), (128, 32, 90, 90), (64, 16, 4, 40), (128, 128, 40, 200)])
def test_pages_that_are_none_read_as_zeros(hd, page, rows, max_rows):
    """Bad ids inside a key tile, at its end, for a whole tile, and of the last page, which
    ends inside one; the other requests' results are what they are without."""
    lens = [600, 600, 590]
    p = Paged4(lens, [rows] * 3, 2, hd, page, BF, seed=5)
    q = rows_tensor(p.n_rows, 8, hd, BF, 4, extra=max_rows)
    clean, clean_l, status = attend(p, q, p.table, max_rows)
    assert status == 0
    check(p, q, clean, clean_l, max_rows=max_rows)
    per = 128 // page
    places = [(1, per // 2), (1, 2 * per - 1), (1, 599 // page)] + [(1, e) for e in range(3 * per, 4 * per)]
    table = p.table.clone()
    for i, (b, e) in enumerate(places):
        table[b, e] = (-1, p.n_pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    out, lse, status = attend(p, q, table, max_rows)
    assert status == -1
    for b in (0, 2):
        at = slice(p.start_np[b], p.start_np[b + 1])
        assert torch.equal(out[at], clean[at]) and torch.equal(lse[at], clean_l[at])
    check(WithPageOfZeros(p, places), q, out, lse, max_rows=max_rows)


@pytest.mark.parametrize("rows,max_rows", [(40, 40), (4, 40), (100, 100)])
def test_requests_that_do_not_fit_stay(rows, max_rows):
    p = Paged4([300, 300, 300, 300], [rows, rows + 1, rows, rows], 2, 64, 16, BF, seed=5)
    q = rows_tensor(p.n_rows, 8, 64, BF, 4, extra=max_rows)
    clean, clean_l, _ = attend(p, q, p.table, max_rows + 1)
    for how in ("long", "negative", "more rows"):
        bad = 1 if how == "more rows" else 2
        if how == "more rows" and rows < max_rows:
            continue
        lens = p.kv_len.clone()
        if how != "more rows":
            lens[2] = 16 * p.width + 1 if how == "long" else -1
        ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(8, 2, 64, max_rows + 1))
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        dfl.dflash_paged_attention(p.cache, q, out, p.row_start, lens, p.table, max_rows + (how != "more rows"), ws, lse=lse)
        assert dfl.dflash_read_status(ws) == -2, how
        for b in range(4):
            at = slice(p.start_np[b], p.start_np[b + 1])
            if b == bad:
                assert (out[at] == 7.0).all() and (lse[at] == 7.0).all(), how
        # a cut of the line that differs may round otherwise: against the oracle
        check(p, q, out, lse, only=[b for b in range(4) if b != bad], max_rows=max_rows + (how != "more rows"))


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("n_q,causal,window", [(8, True, 0), (8, False, 0), (2, True, 1), (2, True, 30), (8, False, 40), (2, False, 1)])
def test_rows_and_items_that_see_nothing(n_q, causal, window, dtype):
    """Lengths below the new rows, 0 and 1 among them, beside chunks: rows before position 0
    see nothing when causal, whole items of them have no key tile, an empty request none at
    all; small windows leave rows of an item whole jobs without a visible key."""
    lens = [3, 0, 1, 0, 700, 90, 128, 64]
    rows = [300, 4, 200, 0, 300, 290, 129, 64]
    p = Paged4(lens, rows, 2, 64, 16, dtype, seed=12)
    q = rows_tensor(p.n_rows, n_q, 64, dtype, 4, extra=5)
    out, lse, status = run(p, q, causal=causal, window=window)
    assert status == 0
    check(p, q, out, lse, causal, window)
    if causal:
        start = p.start_np
        for b in (0, 1, 2, 5):
            before = slice(start[b], start[b] + rows[b] - lens[b])
            assert (out[before] == 0).all() and (lse[before] == -np.inf).all()


def test_every_request_is_empty():
    """No item of the call has a key tile."""
    p = Paged4([0, 0], [200, 100], 2, 128, 64, BF)
    q = rows_tensor(p.n_rows, 8, 128, BF, 4)
    for causal in (True, False):
        out, lse, status = run(p, q, causal=causal)
        assert status == 0 and (out == 0).all() and (lse == -np.inf).all()
