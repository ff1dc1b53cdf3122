"""GPU parity of the target-side operators against the float64 oracle: paged
cache writes and reads (bit for bit), attention over the cache and logit
adjustment (within bounds derived from the arithmetic), what they leave alone,
and how they report what they refuse."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import target as ot
from target_testutil import (HALF_STEP, F8, Paged, attention_reference, check_attention, rows_tensor, run_attention,
                             to64)

pytestmark = pytest.mark.gpu
BF, FH = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


# ------------------------------------------------------------ append, gather

MOVES = [
    # lens, rows, n_kv, hd, page, dtype, e4m3, spread, order
    ([1], [1], 1, 64, 16, BF, False, 0, "rhd"),
    ([1], [1], 1, 128, 16, FH, True, 0, "rhd"),
    ([37, 5, 64, 200], [3, 5, 0, 130], 2, 64, 16, FH, False, 16, "hrd"),
    ([37, 5, 64, 200], [3, 5, 0, 130], 2, 64, 32, BF, True, 32, "wide"),
    ([300, 129, 128], [17, 1, 128], 8, 128, 128, BF, True, 0, "rhd"),
    ([300, 129, 128], [17, 1, 128], 3, 128, 64, BF, False, 0, "wide"),
    ([700] * 40, [8] * 40, 8, 128, 64, FH, True, 0, "rhd"),
    ([0, 9, 0], [0, 9, 0], 1, 128, 32, FH, True, 0, "hrd"),
]


@pytest.mark.parametrize("lens,rows,n_kv,hd,page,dtype,e4m3,spread,order", MOVES)
def test_append_writes_the_new_rows_and_nothing_else(lens, rows, n_kv, hd, page, dtype, e4m3, spread, order):
    p = Paged(lens, rows, n_kv, hd, page, dtype, e4m3, seed=len(lens), spread=spread)
    x = [rows_tensor(p.n_rows, n_kv, hd, dtype, 5 + i, extra=3, order=order, size=3.0) for i in range(2)]
    if p.n_rows > 2:
        x[0][1, 0] = 0                            # a row of zeros
        x[1][2, n_kv - 1, 3] = float("inf")       # rows that are not finite
        x[1][0, 0, 1] = float("nan")
    want = [t.copy() if t is not None else None for t in p.host()]
    for i in range(2):
        vals = x[i].float().cpu().numpy()
        codes, scale = ot.quantize(vals)
        for n, _, _, pid, at in ot.places(p.start_np, lens, p.table_np, page):
            want[i][pid, :, at] = codes[n] if e4m3 else vals[n]
            if e4m3:
                want[2 + i][pid, :, at] = scale[n]
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append(p.cache, x[0], x[1], *p.batch, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    got = p.host()
    for i in range(2):
        if e4m3:
            np.testing.assert_array_equal(np.isnan(got[2 + i]), np.isnan(want[2 + i]))
            ok = ~np.isnan(want[2 + i])
            np.testing.assert_array_equal(got[2 + i][ok], want[2 + i][ok])
            np.testing.assert_array_equal(got[i][ok], want[i][ok])
        else:
            np.testing.assert_array_equal(got[i], want[i])


@pytest.mark.parametrize("lens,rows,n_kv,hd,page,dtype,e4m3,spread,order", MOVES)
def test_gather_reads_back_and_leaves_other_rows(lens, rows, n_kv, hd, page, dtype, e4m3, spread, order):
    p = Paged(lens, rows, n_kv, hd, page, dtype, e4m3, seed=10 + len(lens), spread=spread)
    x = [torch.full_like(rows_tensor(p.n_rows, n_kv, hd, dtype, 5, extra=3, order=order), 7.0) for _ in range(2)]
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_gather(p.cache, x[0], x[1], *p.batch, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    host = p.host()
    for i in range(2):
        want = np.full(x[i].shape, 7.0)
        for n, _, _, pid, at in ot.places(p.start_np, lens, p.table_np, page):
            want[n] = ot.read(host[i], host[2 + i], pid, at, e4m3)
        # code * scale is rounded to float32 and then to the row's type
        want = torch.from_numpy(want.astype(np.float32)).to(dtype)
        assert torch.equal(bits(x[i].cpu()), bits(want))


def test_append_then_gather_returns_16_bit_rows_exactly_and_codes_within_half_a_step():
    lens, rows = [100, 3, 77], [50, 3, 77]
    for e4m3 in (False, True):
        p = Paged(lens, rows, 4, 128, 32, BF, e4m3, fill=False)
        k, v = (rows_tensor(p.n_rows, 4, 128, BF, s, size=0.3) for s in (1, 2))
        k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
        ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
        dfl.dflash_paged_append(p.cache, k, v, *p.batch, ws)
        dfl.dflash_paged_gather(p.cache, k2, v2, *p.batch, ws)
        torch.cuda.synchronize()
        for a, b in ((k, k2), (v, v2)):
            if not e4m3:
                assert torch.equal(a, b)
                continue
            # half a step of E4M3 is 2^-4 of the value, or 2^-10 of the scale
            # where it is subnormal; bf16 rounds once more
            a, b = a.double(), b.double()
            step = torch.maximum(a.abs() * 2.0 ** -4, a.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10)
            assert ((a - b).abs() <= step + b.abs() * 2.0 ** -7).all()


@pytest.mark.parametrize("dtype", [BF, FH])
def test_append_codes_of_ties_and_of_very_small_and_large_rows(dtype):
    """Bit for bit where quotients lie half way between codes (small integers
    over each other) and where the scale leaves the ordinary range."""
    n, hd = 512, 128
    rng = np.random.default_rng(4)
    x = rng.integers(-40, 41, size=(n, 1, hd)).astype(np.float64)
    lo, hi = (-132, 120) if dtype == BF else (-24, 9)
    x *= 2.0 ** rng.integers(lo, hi, size=(n, 1, 1))
    x[::7] *= 1.3
    k = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    p = Paged([n], [n], 1, hd, 64, dtype, True)
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append(p.cache, k, k, *p.batch, ws)
    torch.cuda.synchronize()
    codes, scale = ot.quantize(k.float().cpu().numpy())
    kp, vp, ks, vs = p.host()
    for r, _, _, pid, at in ot.places(p.start_np, p.lens, p.table_np, 64):
        np.testing.assert_array_equal(ks[pid, :, at], scale[r])
        np.testing.assert_array_equal(kp[pid, :, at], codes[r])
        np.testing.assert_array_equal(vp[pid, :, at], codes[r])


def test_pages_past_2_to_31_elements():
    """Page strides whose offsets need 64 bits, in 8 and in 16 bits."""
    for e4m3, stride in ((True, 3 << 29), (False, 3 << 28)):
        n_kv, hd, page, n_pages = 1, 64, 16, 4
        cell = torch.uint8 if e4m3 else BF
        big = [torch.empty((n_pages - 1) * stride + n_kv * page * hd, dtype=cell, device="cuda") for _ in range(2)]
        pages = [t.as_strided((n_pages, n_kv, page, hd), (stride, page * hd, hd, 1)) for t in big]
        scale = [torch.zeros(n_pages, n_kv, page, device="cuda") if e4m3 else None for _ in range(2)]
        cache = dfl.paged_cache(pages[0], pages[1], scale[0], scale[1])
        k, v = (rows_tensor(40, n_kv, hd, BF, s) for s in (3, 4))
        k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
        batch = (torch.tensor([0, 40], dtype=torch.int32, device="cuda"), torch.tensor([40], device="cuda"),
                 torch.tensor([[3, 0, 2]], dtype=torch.int32, device="cuda"))
        ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(2, 1, hd, 40))
        dfl.dflash_paged_append(cache, k, v, *batch, ws)
        dfl.dflash_paged_gather(cache, k2, v2, *batch, ws)
        q = rows_tensor(40, 2, hd, BF, 5)
        out = torch.zeros_like(q)
        dfl.dflash_paged_attention(cache, q, out, *batch, 40, ws)
        torch.cuda.synchronize()
        assert dfl.dflash_read_status(ws) == 0
        if not e4m3:
            assert torch.equal(k, k2) and torch.equal(v, v2)
        z = (q.double().transpose(0, 1) @ k2.double()[:, 0].T) / 8
        z = z.masked_fill(torch.ones(40, 40, device="cuda").triu(1).bool(), -float("inf"))
        want = (torch.softmax(z, -1) @ v2.double()[:, 0]).transpose(0, 1)
        # weights and output rounded to bf16, the read-back rows too
        # (2^-8 each): 2^-6 of the largest value covers them
        assert (out.double() - want).abs().max() <= 2.0 ** -6 * v2.abs().max()


def test_a_batch_without_new_rows():
    p = Paged([40, 7], [0, 0], 2, 64, 16)
    x = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    before = p.host()
    ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(4, 2, 64, 0))
    dfl.dflash_paged_append(p.cache, x, x, *p.batch, ws)
    dfl.dflash_paged_gather(p.cache, x, x.clone(), *p.batch, ws)
    q = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    dfl.dflash_paged_attention(p.cache, q, q.clone(), *p.batch, 0, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    for x0, x1 in zip(before[:2], p.host()[:2]):
        np.testing.assert_array_equal(x0, x1)


# --------------------------------------------------------------- attention

def rid(v):
    return str(v) if not isinstance(v, (list, tuple)) else "-".join(map(str, v))[:40]


ATT = [
    # lens, rows, n_q, n_kv, hd, page, dtype, e4m3, causal, window, order
    ([1], [1], 1, 1, 64, 16, BF, False, True, 0, "rhd"),
    ([1], [1], 8, 1, 128, 16, FH, True, True, 0, "rhd"),
    ([257], [1], 5, 1, 128, 64, BF, False, True, 0, "rhd"),
    ([128, 127, 129, 1], [1, 1, 1, 1], 8, 2, 64, 128, FH, False, True, 0, "rhd"),
    ([600, 31], [8, 8], 10, 2, 128, 64, BF, False, True, 0, "wide"),
    ([600, 31], [8, 8], 10, 2, 128, 64, BF, True, True, 0, "hrd"),
    ([333, 16], [16, 16], 14, 2, 64, 32, FH, True, False, 0, "rhd"),
    ([333, 16, 90], [16, 0, 33], 14, 2, 64, 16, FH, False, False, 40, "hrd"),
    ([500], [130], 7, 1, 128, 16, BF, False, True, 100, "rhd"),
    ([390, 140], [129, 40], 8, 2, 64, 64, BF, True, True, 1, "rhd"),
    ([300, 270], [300, 200], 4, 2, 128, 128, BF, False, True, 0, "wide"),
    ([300, 270], [300, 200], 4, 2, 128, 32, FH, True, True, 64, "rhd"),
    ([5, 0, 700, 2, 64], [9, 3, 70, 2, 64], 6, 3, 128, 64, BF, False, True, 0, "rhd"),   # rows before position 0
    ([5, 0, 700, 2, 64], [9, 3, 70, 2, 64], 6, 3, 64, 16, FH, True, True, 33, "rhd"),
    ([2100], [3], 20, 2, 128, 64, BF, True, True, 0, "rhd"),
    ([2100, 1999, 40], [3, 65, 1], 16, 1, 64, 128, FH, False, True, 1500, "rhd"),
]


@pytest.mark.parametrize("lens,rows,n_q,n_kv,hd,page,dtype,e4m3,causal,window,order", ATT, ids=rid)
def test_attention_parity(lens, rows, n_q, n_kv, hd, page, dtype, e4m3, causal, window, order):
    p = Paged(lens, rows, n_kv, hd, page, dtype, e4m3, seed=sum(lens) + hd, spread=16)
    q = rows_tensor(p.n_rows, n_q, hd, dtype, 3, extra=2, order=order, size=1.5)
    out, lse, status = run_attention(p, q, causal=causal, window=window)
    assert status == 0
    check_attention(p, q, out, lse, causal, window)


@pytest.mark.parametrize("length", [300, 900, 1500, 2600, 4100, 20000])
@pytest.mark.parametrize("rows,n_q,hd,dtype,e4m3", [(1, 3, 128, BF, False), (9, 5, 64, FH, True), (50, 4, 128, BF, True)])
def test_attention_joins_a_request_cut_into_few_and_many_parts(length, rows, n_q, hd, dtype, e4m3):
    """One KV head: its key tiles, 3 to 157 of them, are all there is to cut."""
    p = Paged([length], [rows], 1, hd, 64, dtype, e4m3, seed=length)
    q = rows_tensor(p.n_rows, n_q, hd, dtype, 3, extra=1, size=1.5)
    out, lse, status = run_attention(p, q)
    assert status == 0
    check_attention(p, q, out, lse)


def test_attention_without_lse_and_with_another_scale():
    p = Paged([400], [20], 2, 64, 32)
    q = rows_tensor(p.n_rows, 6, 64, BF, 3)
    out, lse, status = run_attention(p, q, lse=False, scale=0.7)
    assert status == 0 and lse is None
    check_attention(p, q, out, None, scale=0.7)


@pytest.mark.parametrize("dtype,left", [(BF, 2.0 ** -13), (FH, 2.0 ** -16)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_over_codes_keeps_queries_far_below_the_largest_of_their_row(dtype, left, hd):
    """Each row sees one key, so lse is its score.  The largest query, 192,
    meets a key of 0; all the others are below 2^-10.  As 8-bit terms a query
    may lose `left` (largest in [128, 256)); beside that, hd products are
    summed, 2 half steps each, and the scale and the logarithm take a few."""
    n = 12
    p = Paged([1] * n, [1] * n, 1, hd, 16, dtype, True, seed=4, garbage=False)
    codes = p.pages[0].view(torch.uint8)
    codes &= 0x7F                                     # positive keys
    codes[..., 0] = 0
    q = rows_tensor(n, 2, hd, dtype, 5)
    q.copy_((0.45 + 0.45 * torch.rand(q.shape, device="cuda")) * 2.0 ** -10)
    q[..., 0] = 192
    out, lse, status = run_attention(p, q, scale=1.0)
    assert status == 0
    kp, _, ks, _ = p.host()
    e = 2.0 ** -24
    for b in range(n):
        k = ot.sequence(kp, ks, p.table_np[b], 1, 16, True)[0, 0]
        want = to64(q)[b] @ k
        bound = left * k.sum() + (2 * (hd + 4) + 8) * e * np.abs(want) + 8 * e
        assert (np.abs(to64(lse)[b] - want) <= bound).all()
        assert (bound < 0.5 * want).all()             # what terms of 4 bits alone would lose


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_outputs_are_not_too_large_or_small_on_average(dtype, e4m3):
    """Roundings of weights and outputs go either way.  A rounding's error is
    evenly spread over half a step, its mean over the 1,024 softmaxes of this
    call about 0.6 u / 32, u / 50 a standard deviation for the weights and less
    for the outputs.  Over codes the weights of one key, which many rows may
    heed most, lean by up to 3.8e-4 one way, u / 10 in bf16.  Within u / 8 of
    the formula's size, then, whichever type."""
    p = Paged([500, 300], [128, 128], 4, 128, 64, dtype, e4m3, seed=8, garbage=False)
    q = rows_tensor(p.n_rows, 4, 128, dtype, 3)
    out, lse, status = run_attention(p, q, causal=False)
    assert status == 0
    check_attention(p, q, out, lse, causal=False)
    want = attention_reference(p, q, False, 0, 128 ** -0.5)[0]
    got = to64(out)
    assert abs((got * want).sum() / (want * want).sum() - 1.0) <= HALF_STEP[dtype] / 8


@pytest.mark.parametrize("e4m3", [False, True])
def test_attention_of_queries_that_are_zero_under_a_tiny_scale(e4m3):
    """All scores vanish: the plain mean of what a row sees, masked keys out."""
    p = Paged([200, 9], [70, 9], 2, 64, 16, e4m3=e4m3)
    q = rows_tensor(p.n_rows, 4, 64, BF, 3)
    q[::2] = 0
    for scale in (1e-9, 1e-30):
        out, lse, status = run_attention(p, q, scale=scale)
        assert status == 0
        check_attention(p, q, out, lse, scale=scale)


def test_attention_with_scores_of_hundreds_and_one_key_far_above_the_rest():
    """The running maximum grows late and by a lot; scores reach far beyond
    what exp holds."""
    p = Paged([900], [5], 1, 128, 64, garbage=False)
    for at, f in ((10, 2.0), (300, 8.0), (850, 30.0)):
        pid = p.table_np[0][at // 64]
        p.pages[0][pid, 0, at % 64] *= f
    q = rows_tensor(p.n_rows, 4, 128, BF, 3, size=6.0)
    out, lse, status = run_attention(p, q)
    assert status == 0
    check_attention(p, q, out, lse)


def test_attention_makes_the_cache_maps_itself_if_the_caller_keeps_none():
    import ctypes
    p = Paged([300, 40], [8, 3], 2, 64, 32, e4m3=True)
    q = rows_tensor(p.n_rows, 8, 64, BF, 3)
    want, _, _ = run_attention(p, q)
    out = torch.zeros_like(q)
    ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(8, 2, 64, 8))
    rows = [dfl.dflash_rows(t.data_ptr(), t.stride(0), t.stride(1)) for t in (q, out)]
    b = dfl.dflash_paged_batch(p.row_start.data_ptr(), p.kv_len.data_ptr(), p.table.data_ptr(), p.width, 2, p.width, p.n_rows)
    c = p.cache.struct
    assert not c.maps
    call = dfl.lib().dflash_paged_attention
    args = [ctypes.byref(b), 0, 8, ctypes.byref(rows[0]), ctypes.byref(rows[1]), None, 8, 0.125, 1, 0, ws.data_ptr(),
            ws.numel(), torch.cuda.current_stream().cuda_stream]
    assert call(ctypes.byref(c), *args) == 0
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want))
    # the maps of this cache do for no other
    other = Paged([300, 40], [8, 3], 2, 64, 32, e4m3=True, seed=1)
    run_attention(other, q)
    c.maps = ctypes.addressof(other.cache._maps[1])
    assert call(ctypes.byref(c), *args) == -1
    c.maps = None


def test_attention_shares_pages_between_requests():
    p = Paged([200, 200, 130], [8, 8, 8], 2, 64, 16)
    p.table_np[1, :8] = p.table_np[0, :8]
    p.table_np[2, :8] = p.table_np[0, :8]
    p.table.copy_(torch.from_numpy(p.table_np))
    q = rows_tensor(p.n_rows, 8, 64, BF, 3)
    out, lse, status = run_attention(p, q)
    assert status == 0
    check_attention(p, q, out, lse)


def test_attention_is_the_same_on_every_run_and_reuses_its_workspace():
    p = Paged([3000, 700, 40], [16, 3, 16], 2, 128, 64, e4m3=True)
    q = rows_tensor(p.n_rows, 10, 128, BF, 3)
    ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(10, 2, 128, 16))
    first = run_attention(p, q, ws=ws)
    ws[256:].fill_(255)       # what lies in the workspace is scratch
    second = run_attention(p, q, ws=ws)
    assert first[2] == second[2] == 0
    assert torch.equal(bits(first[0]), bits(second[0])) and torch.equal(bits(first[1]), bits(second[1]))


def test_attention_leaves_out_requests_that_do_not_fit():
    lens, rows = [100, 50, 60, 70], [4, 9, 5, 6]
    p = Paged(lens, rows, 2, 64, 16)
    q = rows_tensor(p.n_rows, 4, 64, BF, 3)
    out, lse, status = run_attention(p, q, max_rows=6)           # request 1 has 9 rows
    assert status == -2
    check_attention(p, q, out, lse, only=(0, 2, 3))
    p.kv_len[2] = 16 * p.width + 1                               # longer than its page table
    out, lse, status = run_attention(p, q)
    assert status == -2
    check_attention(p, q, out, lse, only=(0, 1, 3))
    p.kv_len[2] = -1
    out, lse, status = run_attention(p, q)
    assert status == -2
    check_attention(p, q, out, lse, only=(0, 1, 3))
    p.kv_len[2] = 60
    p.row_start[4] = p.n_rows + 1                                # past the row tensors
    out, lse, status = run_attention(p, q)
    assert status == -2
    check_attention(p, q, out, lse, only=(0, 1, 2))


def test_attention_reads_zeros_for_pages_outside_the_cache():
    p = Paged([100, 50], [4, 9], 2, 64, 16)
    p.table[0, 1] = p.n_pages
    p.table[1, 0] = -1
    q = rows_tensor(p.n_rows, 4, 64, BF, 3)
    out, lse, status = run_attention(p, q)
    assert status == -1
    # the oracle with those pages present and zero
    for b, i in ((0, 1), (1, 0)):
        for t in p.pages:
            t[p.table_np[b][i]] = 0
    want, _, b_out, _ = attention_reference(p, q, True, 0, 0.125)
    assert (np.abs(to64(out) - want) <= b_out).all()


def test_move_reports_bad_pages_and_lengths():
    for e4m3 in (False, True):
        p = Paged([40, 40, 40], [4, 4, 4], 1, 64, 16, e4m3=e4m3)
        ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
        k, v = (rows_tensor(p.n_rows, 1, 64, BF, s) for s in (1, 2))
        before = p.host()
        table = p.table.clone()
        table[1, 2] = p.n_pages
        lens = p.kv_len.clone()
        lens[2] = 1 << 40
        dfl.dflash_paged_append(p.cache, k, v, p.row_start, lens, table, ws)
        torch.cuda.synchronize()
        assert dfl.dflash_read_status(ws) in (-1, -2)
        after = p.host()
        for i in range(2):
            same = np.ones(before[i].shape[0:1] + (1, 16), dtype=bool)
            for n, b, _, pid, at in ot.places(p.start_np, p.lens, p.table_np, 16):
                if b == 0:
                    same[pid, :, at] = False
            same = np.broadcast_to(same, before[i].shape[:3])
            np.testing.assert_array_equal(before[i][same], after[i][same])
            assert (before[i][~same] != after[i][~same]).any()
        kk, vv = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
        ws.zero_()
        dfl.dflash_paged_gather(p.cache, kk, vv, p.row_start, lens, table, ws)
        torch.cuda.synchronize()
        assert dfl.dflash_read_status(ws) in (-1, -2)
        assert (kk[4:8] == 0).all() and (kk[8:] == 7.0).all() and not (kk[:4] == 7.0).any()


# ------------------------------------------------------------------ logits

def logit_inputs(B, G, V, dtype, seed, slots=None, pad=0):
    rng = np.random.default_rng(seed)
    slots = slots or B
    words = (V + 31) // 32
    z = torch.from_numpy(rng.normal(size=(B, G, V + pad)).astype(np.float32) * 3).to(dtype).cuda()[:, :, :V]
    counts = np.zeros((slots, V), dtype=np.int32)
    for s in range(slots):
        np.add.at(counts[s], rng.integers(0, V, size=V // 3 + 1), 1)
    prompt = rng.random((slots, words * 32)) < 0.2
    allow = rng.random((B, G, words * 32)) < 0.5
    draft = rng.integers(0, V, size=(B, max(G - 1, 1))).astype(np.int32)[:, :G - 1]
    if G > 3:
        draft[:, 2] = draft[:, 0]
        draft[0, 1] = -1
        draft[B - 1, 1] = V
    n = [int(x) for x in rng.integers(0, 700, size=B)]
    n[0] = 0 if B > 1 else n[0]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    ids = rng.integers(0, V, size=start[-1]).astype(np.int32)
    ids[1::2] = ids[:-1:2][:len(ids[1::2])]          # ids that come twice
    vals = rng.normal(size=start[-1]).astype(np.float32)
    par = {k: (rng.random(B) * w + o).astype(np.float32) for k, w, o in
           (("repetition", 0.5, 0.8), ("frequency", 1.0, -0.2), ("presence", 1.0, -0.3))}
    return z, counts, prompt, allow, draft, start, ids, vals, par


def words_of(flags):
    w = np.packbits(flags, axis=-1, bitorder="little").view(np.int32)
    return torch.from_numpy(np.ascontiguousarray(w)).cuda()


@pytest.mark.parametrize("B,G,V,dtype,pad,use", [
    (1, 1, 1, torch.float32, 0, "counts prompt bias allow par"),
    (2, 2, 31, torch.float32, 1, "counts draft prompt bias allow par"),
    (3, 5, 5003, BF, 21, "counts draft prompt bias allow par"),
    (2, 8, 4096, torch.float32, 0, "counts draft prompt bias allow par"),
    (2, 8, 4097, FH, 3, "draft bias par"),
    (1, 16, 8200, torch.float32, 0, "counts draft par"),
    (2, 3, 12288, torch.float32, 4, "allow"),
    (2, 3, 777, BF, 1, "prompt par"),
    (1, 8, 151936, torch.float32, 0, "counts draft prompt bias allow par"),
    (1, 64, 300, torch.float32, 0, "draft par"),
    (2, 3, 500, torch.float32, 0, ""),
])
def test_logits_adjust_parity(B, G, V, dtype, pad, use):
    slots = B + 2
    z, counts, prompt, allow, draft, start, ids, vals, par = logit_inputs(B, G, V, dtype, B * 10 + G, slots, pad)
    use = use.split()
    slot = np.arange(B)[::-1].astype(np.int32) + 1
    kw, ref = {}, {}
    if "counts" in use:
        kw["counts"], ref["counts"] = torch.from_numpy(counts).cuda(), counts
    if "prompt" in use:
        kw["prompt_mask"], ref["prompt"] = words_of(prompt), prompt[:, :V]
    if "counts" in use or "prompt" in use:
        kw["req_slot"], ref["slot"] = torch.from_numpy(slot).cuda(), slot
    if "draft" in use:
        kw["draft"], ref["draft"] = torch.from_numpy(draft).cuda(), draft
    if "allow" in use:
        kw["allow"], ref["allow"] = words_of(allow), allow[:, :, :V]
    if "bias" in use:
        kw.update(bias_start=torch.from_numpy(start).cuda(), bias_ids=torch.from_numpy(ids).cuda(),
                  bias_vals=torch.from_numpy(vals).cuda())
        ref["bias"] = [(b, int(ids[e]), float(vals[e])) for b in range(B) for e in range(start[b], start[b + 1])]
    if "par" in use:
        for k, v in par.items():
            kw[k], ref[k] = torch.from_numpy(v).cuda(), v
    out = torch.full((G, B, V + 2), 7.0, device="cuda")
    view = out.transpose(0, 1)[:, :, :V]               # positions outermost, padded rows
    ws = dfl.workspace(dfl.dflash_logits_adjust_workspace_bytes())
    dfl.dflash_logits_adjust(z, view, ws, **kw)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    want, size = ot.adjust(to64(z), **ref)
    got = to64(view)
    np.testing.assert_array_equal(np.isinf(got), np.isinf(want))
    fine = np.isfinite(want)
    # quotient or product, two products and sums, and a sum per bias: each off
    # by half a step of float32 of what it adds up; 1 + 5 + the biases of an id
    most = 6 + (max(np.unique([v for _, v, _ in ref["bias"]], return_counts=True)[1], default=0) if "bias" in use and ref["bias"] else 0)
    assert (np.abs(got[fine] - want[fine]) <= most * 2.0 ** -24 * size[fine]).all()
    assert (out[:, :, V:] == 7.0).all()
    if dtype == torch.float32:                          # in place
        dfl.dflash_logits_adjust(z, z, ws, **kw)
        torch.cuda.synchronize()
        assert torch.equal(bits(z), bits(view))


def test_logits_adjust_masks_everything_and_keeps_infinities():
    B, G, V = 2, 2, 700
    z = torch.randn(B, G, V, device="cuda")
    z[0, 0, 5], z[0, 0, 6], z[1, 1, 7] = float("inf"), float("-inf"), float("nan")
    allow = np.ones((B, G, 704), dtype=bool)
    allow[0, 1] = False
    out = torch.empty_like(z)
    ws = dfl.workspace(dfl.dflash_logits_adjust_workspace_bytes())
    dfl.dflash_logits_adjust(z, out, ws, allow=words_of(allow))
    torch.cuda.synchronize()
    assert (out[0, 1] == -float("inf")).all()
    # a NaN stays a NaN; which one, CUDA's additions do not say
    for b, i in ((0, 0), (1, 0), (1, 1)):
        np.testing.assert_array_equal(to64(out[b, i]), to64(z[b, i]))


@pytest.mark.parametrize("V", [700, 701])
def test_logits_adjust_takes_negative_counts_by_the_formula_whoever_computes_an_id(V):
    """Every id through the chunk's pass, and again with each named by a bias
    of 0: the same bits, and the formula's values."""
    G = 3
    z = torch.randn(1, G, V, device="cuda")
    counts = torch.arange(V, dtype=torch.int32, device="cuda").reshape(1, V) % 7 - 3
    par = dict(repetition=torch.tensor([1.25], device="cuda"), frequency=torch.tensor([0.5], device="cuda"),
               presence=torch.tensor([0.75], device="cuda"))
    ws = dfl.workspace(dfl.dflash_logits_adjust_workspace_bytes())
    out, again = torch.empty_like(z), torch.empty_like(z)
    dfl.dflash_logits_adjust(z, out, ws, counts=counts, **par)
    dfl.dflash_logits_adjust(z, again, ws, counts=counts, bias_start=torch.tensor([0, V], dtype=torch.int32, device="cuda"),
                             bias_ids=torch.arange(V, dtype=torch.int32, device="cuda"), bias_vals=torch.zeros(V, device="cuda"), **par)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    assert torch.equal(out, again)
    c, l = to64(counts)[0], to64(z)[0]
    l1 = np.where(c > 0, np.where(l > 0, l / 1.25, l * 1.25), l)
    want = l1 - (0.5 * c + 0.75 * (c > 0))
    # at most two roundings of the quotient and one each of the two others
    size = np.abs(l1) + 0.5 * np.abs(c) + 0.75
    assert (np.abs(to64(out)[0] - want) <= 4 * 2.0 ** -24 * size).all()


def test_logits_adjust_reports_bad_slots_and_ids():
    B, G, V = 3, 2, 100
    z = torch.randn(B, G, V, device="cuda")
    counts = torch.ones(B, V, dtype=torch.int32, device="cuda")
    f = torch.ones(B, device="cuda")
    out = torch.empty_like(z)
    ws = dfl.workspace(dfl.dflash_logits_adjust_workspace_bytes())
    slot = torch.tensor([0, 3, -1], dtype=torch.int32, device="cuda")
    dfl.dflash_logits_adjust(z, out, ws, counts=counts, req_slot=slot, frequency=f)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == -1
    assert torch.equal(out[0], z[0] - 1) and torch.equal(out[1:], z[1:])
    for start, ids in (([0, 2, 4, 4], [1, 100, -1, 2]), ([0, 5, 4, 4], [1, 2, 3, 4]), ([0, 1, 2, 9], [1, 2, 3, 4])):
        ws.zero_()
        dfl.dflash_logits_adjust(z, out, ws, bias_start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                                 bias_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"),
                                 bias_vals=torch.ones(4, device="cuda"))
        torch.cuda.synchronize()
        assert dfl.dflash_read_status(ws) == -1
        want = z.clone()
        for b in range(B):
            for e in range(start[b], start[b + 1]) if 0 <= start[b] <= start[b + 1] <= 4 else ():
                if 0 <= ids[e] < V:
                    want[b, :, ids[e]] += 1
        assert torch.equal(out, want)
