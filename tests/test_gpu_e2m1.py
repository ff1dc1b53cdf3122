"""A paged cache in 4 bits: rows written and read back, and attention over it."""

import threading

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import e2m1
from paged4_testutil import BF, F16, Paged4, check, kv_rows, run
from target_testutil import rows_tensor, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


# ------------------------------------------------------------ rows in and out

def expected(p, x, pages, side):
    """The pages after the batch's rows x were written."""
    want = pages[side].copy()
    rec = e2m1.pack(x[side].float().cpu().numpy())
    for b, length in enumerate(p.lens):
        n = p.rows[b]
        for j in range(n):
            s = length - n + j
            want[p.table_np[b, s // p.page], :, s % p.page] = rec[p.start_np[b] + j]
    return want


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("hd,n_kv,page,order", [(64, 2, 16, "rhd"), (128, 3, 32, "hrd"), (128, 8, 128, "wide"), (64, 1, 64, "rhd")])
def test_rows_are_written_and_read_back(dtype, hd, n_kv, page, order):
    lens, rows = [300, 1, 77, 500, 40], [129, 1, 0, 300, 40]
    p = Paged4(lens, rows, n_kv, hd, page, dtype, spread=48)
    x = [rows_tensor(p.n_rows, n_kv, hd, dtype, 3 + i, extra=5, order=order, size=3.0) for i in range(2)]
    before = p.host()
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append(p.cache, x[0], x[1], *p.batch, ws)
    back = [torch.full((p.n_rows + 5, n_kv, hd), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    dfl.dflash_paged_gather(p.cache, back[0], back[1], *p.batch, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    for side in range(2):
        np.testing.assert_array_equal(p.host()[side], expected(p, x, before, side))
        want = torch.from_numpy(e2m1.unpack(e2m1.pack(x[side].float().cpu().numpy()))).to(dtype)
        assert torch.equal(back[side][:p.n_rows].cpu(), want[:p.n_rows])
        assert (back[side][p.n_rows:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F16])
def test_values_that_round_oddly(dtype):
    """Ties, zeros of either sign, the type's ends, blocks of one value, NaN and
    infinities, whole and in one block of a row."""
    hd, lens = 128, [64]
    p = Paged4(lens, lens, 1, hd, 16, dtype, garbage=False)
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 1, hd)).astype(np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i in range(8):                                   # exact ties under scales of few bits
        x[i, 0] = np.resize(np.concatenate([mids, -mids]), hd) * 2.0 ** (i - 4)
        x[i, 0, 15::16] = 6 * 2.0 ** (i - 4)
    x[8] = 0
    x[9] = -0.0
    x[10] = np.where(np.arange(hd) == 70, 5.0, 0)
    x[11] = torch.finfo(dtype).max
    x[12] = torch.finfo(dtype).tiny
    x[13] = -torch.finfo(dtype).tiny * (np.arange(hd) % 7) / 4
    x[14, 0, ::16] = torch.finfo(dtype).max
    x[15] = torch.finfo(dtype).smallest_normal * 2.0 ** -(7 if dtype is BF else 10)
    x[16, 0, 33] = np.nan
    x[17, 0, 50] = np.inf
    x[18, 0, ::16] = -np.inf
    x[19] = np.nan
    x = torch.from_numpy(x).to(dtype)
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append(p.cache, x.cuda(), x.flip(0).cuda(), *p.batch, ws)
    back = [torch.empty_like(x).cuda() for _ in range(2)]
    dfl.dflash_paged_gather(p.cache, back[0], back[1], *p.batch, ws)
    rec = e2m1.pack(x.float().numpy())
    want, scales = e2m1.unpack(rec), e2m1.split(rec)[1]
    got_rec = p.host()[0][p.table_np[0, np.arange(64) // 16], :, np.arange(64) % 16]
    codes, got_scales = e2m1.split(got_rec)
    np.testing.assert_array_equal(got_scales, scales)
    fine = np.repeat(np.isfinite(scales), 16, -1)        # the codes of other blocks do not matter
    np.testing.assert_array_equal(codes[fine], e2m1.split(rec)[0][fine])
    want = torch.from_numpy(want).to(dtype)
    for got, w in ((back[0].cpu(), want), (back[1].cpu(), want.flip(0))):
        assert torch.equal(got.isnan(), w.isnan()) and torch.equal(got.nan_to_num(0.0), w.nan_to_num(0.0))
        assert torch.equal(got.signbit()[~w.isnan()], w.signbit()[~w.isnan()])


@pytest.mark.parametrize("dtype", [BF, F16])
def test_borders_under_every_scale(dtype):
    """Blocks of every significand that a largest value has, with the values next to each
    border between two codes and on it, for exponents over the type's range: codes and
    scales as the oracle's, bit for bit."""
    hd = 128
    exps = [-132, -110, -101, -100, -99, -60, 0, 60, 99, 100, 101, 102, 103, 120, 127] if dtype is BF else [-20, -10, 0, 15]
    bits = 7 if dtype is BF else 10
    mant = 1 + np.arange(0, 1 << bits, 1 if dtype is BF else 5) / (1 << bits)
    top = torch.from_numpy(np.outer(2.0 ** np.array(exps), mant).reshape(-1)).to(dtype)
    n = top.numel()
    scale = e2m1.split(e2m1.pack(np.repeat(top.float().numpy()[:, None], 16, -1)))[1].astype(np.float64)  # [n, 1]
    on = torch.from_numpy(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * scale).to(dtype)  # where representable
    near = torch.cat([on, (on.view(torch.int16) + 1).view(dtype), (on.view(torch.int16) - 1).clamp_min(0).view(dtype),
                      on[:, :5] * 0.5, on[:, 2:] * 0.25], 1)                                     # [n, 31]
    near = torch.cat([near, -near], 1)[:, :60].minimum(top[:, None]).maximum(-top[:, None])
    x = torch.stack([torch.cat([top[:, None], near[:, 15 * b:15 * b + 15]], 1) for b in (0, 1, 2, 3)] * 2, 1)
    x = x.reshape(n, 1, hd)
    p = Paged4([n], [n], 1, hd, 16, dtype, garbage=False)
    dfl.dflash_paged_append(p.cache, x.cuda(), x.flip(0).cuda(), *p.batch, dfl.workspace(dfl.dflash_paged_workspace_bytes()))
    for side, rows in ((0, x), (1, x.flip(0))):
        got = p.host()[side][p.table_np[0, np.arange(n) // 16], :, np.arange(n) % 16]
        want = e2m1.split(e2m1.pack(rows.float().numpy()))
        np.testing.assert_array_equal(e2m1.split(got)[1], want[1])
        np.testing.assert_array_equal(e2m1.split(got)[0], want[0])


def test_pages_that_are_none_and_requests_that_do_not_fit():
    lens, rows = [40, 33, 50], [20, 10, 30]
    p = Paged4(lens, rows, 2, 64, 16, BF, garbage=False)
    x = [kv_rows(p.n_rows, 2, 64, BF, 9 + i) for i in range(2)]
    before = p.host()
    table = p.table.clone()
    table[0, 2] = p.n_pages
    table[2, 1] = -3
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append(p.cache, x[0], x[1], p.row_start, p.kv_len, table, ws)
    back = [torch.full_like(t, 7.0) for t in x]
    assert dfl.dflash_read_status(ws) == -1
    dfl.dflash_paged_gather(p.cache, back[0], back[1], p.row_start, p.kv_len, table, ws)
    for side in range(2):
        want = expected(p, x, before, side)
        want[p.table_np[0, 2]] = before[side][p.table_np[0, 2]]
        want[p.table_np[2, 1]] = before[side][p.table_np[2, 1]]
        np.testing.assert_array_equal(p.host()[side], want)
        got = to64(back[side])
        for b in range(3):
            for j in range(rows[b]):
                s, bad = lens[b] - rows[b] + j, {0: 2, 2: 1}.get(b)
                if s // 16 == bad:
                    assert (got[p.start_np[b] + j] == 0).all()
    too_long = torch.tensor([40, 16 * p.width + 1, 50], device="cuda")
    for f in (dfl.dflash_paged_append, dfl.dflash_paged_gather):
        ws.zero_()
        # (what append writes are other rows than gather's outputs start from)
        y = [t.clone() if f is dfl.dflash_paged_append else torch.full_like(t, 7.0) for t in x]
        f(p.cache, y[0], y[1], p.row_start, too_long, p.table, ws)
        assert dfl.dflash_read_status(ws) == -2
        if f is dfl.dflash_paged_gather:
            assert (y[0][20:30] == 7.0).all() and not (y[0][:20] == 7.0).all()


# ------------------------------------------------------------------ attention

CASES = [
    # lens, new rows, n_q, n_kv, hd, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [1], 40, 8, 128, 64),
    ([1000], [1], 40, 8, 128, 64),
    ([127, 128, 129, 300], [1, 1, 1, 1], 5, 1, 128, 32),
    ([8, 16, 500, 4097], [8, 8, 8, 8], 10, 2, 128, 128),
    ([200, 0, 77, 64], [3, 0, 0, 64], 14, 2, 64, 16),
    ([700, 40], [13, 40], 7, 1, 64, 16),                    # 91 and 280 packed rows
    ([513, 900], [17, 100], 8, 2, 128, 64),                 # 68, 400
    ([260], [260], 4, 4, 64, 32),
    ([2000, 33], [16, 1], 16, 2, 64, 128),                  # 128 packed rows, and 8
    ([5, 3000], [5, 30], 6, 3, 128, 16),
    ([800, 300, 64, 1, 700], [129, 300, 2, 1, 0], 2, 2, 128, 32),   # items of 129, 256 and 44, 2 and 1 rows
    ([1500, 90], [400, 90], 5, 1, 64, 128),
]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("lens,rows,n_q,n_kv,hd,page", CASES)
def test_attention(lens, rows, n_q, n_kv, hd, page, dtype):
    p = Paged4(lens, rows, n_kv, hd, page, dtype, seed=len(lens) + hd)
    q = rows_tensor(p.n_rows, n_q, hd, dtype, 4, extra=3)
    out, lse, status = run(p, q)
    assert status == 0
    check(p, q, out, lse)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 100), (False, 64), (True, 1000), (False, 3000)])
@pytest.mark.parametrize("rows", [[1, 4, 9], [30, 70, 200]])
def test_masks(rows, causal, window):
    """Windows under which rows of an item see their first key tiles after others
    have, and rows that see nothing."""
    p = Paged4([600, 1500, 333], rows, 2, 128, 32, BF, seed=3)
    q = rows_tensor(p.n_rows, 10, 128, BF, 4)
    out, lse, _ = run(p, q, causal=causal, window=window)
    check(p, q, out, lse, causal, window)


def test_rows_that_see_nothing():
    """kv_len below the new rows: rows before position 0 see no key when causal."""
    p = Paged4([3, 0, 20], [8, 4, 20], 2, 64, 16, F16)
    q = rows_tensor(p.n_rows, 4, 64, F16, 4)
    out, lse, _ = run(p, q)
    assert (out[:5] == 0).all() and (lse[:5] == -np.inf).all() and (out[8:12] == 0).all() and (lse[8:12] == -np.inf).all()
    got = to64(out)
    k = e2m1.sequence(p.host()[0], p.table_np[0], 3, 16)
    v = e2m1.sequence(p.host()[1], p.table_np[0], 3, 16)
    for j in range(5, 8):
        for h in range(4):
            z = k[:j - 4, h // 2] @ to64(q)[j, h] / 8
            w = np.exp(z - z.max())
            want = (w / w.sum()) @ v[:j - 4, h // 2]
            assert np.abs(got[j, h] - want).max() <= 2.0 ** -9 * np.abs(v).max()


@pytest.mark.parametrize("n_q,lens,rows", [(8, [60000], [1]), (40, [20000], [8]), (40, [9000, 100], [30, 2])])
def test_items_cut_between_ctas(n_q, lens, rows):
    n_kv = 1 if n_q == 8 else 8
    p = Paged4(lens, rows, n_kv, 128, 64, BF, seed=11)
    q = rows_tensor(p.n_rows, n_q, 128, BF, 4)
    out, lse, _ = run(p, q)
    check(p, q, out, lse)
    again, lse2, _ = run(p, q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows", [2, 40, 200])
def test_tail_behind_a_dominant_key(dtype, rows):
    """One key takes nine tenths of every row; its values are tiny, so that the
    others, 2^-15 of its weight each, are the output."""
    n, hd = 20000, 64
    rng = np.random.default_rng(2)
    k = np.zeros((n, 1, hd), dtype=np.float32)
    k[:, 0, 0] = 0.01 * rng.standard_normal(n)
    k[777, 0, 0] = 4.0
    v = rng.standard_normal((n, 1, hd)).astype(np.float32) + 1.0
    v[777] = 2.0 ** -14 * rng.standard_normal((1, hd))
    k, v = (torch.from_numpy(t).to(dtype).float().numpy() for t in (k, v))
    p = Paged4([n], [rows], 1, hd, 64, dtype, values=[[k], [v]])
    q = torch.zeros(rows, 2, hd, dtype=dtype, device="cuda")
    q[..., 0] = (np.log(9.0 * n)) * 8.0 / 4.0            # over sqrt(64), times the key's 4
    out, lse, _ = run(p, q, causal=False)
    check(p, q, out, lse, causal=False)


def test_scores_that_grow_and_magnitudes_of_any_size():
    """Keys sorted so that every tile passes the references of the one before;
    queries and rows from 2^-60 to 2^60."""
    n, hd = 3000, 128
    rng = np.random.default_rng(4)
    k = rng.standard_normal((n, 2, hd)).astype(np.float32) * np.linspace(0.1, 30, n, dtype=np.float32)[:, None, None]
    v = rng.standard_normal((n, 2, hd)).astype(np.float32) * np.exp2(rng.integers(-30, 30, (n, 2, 1))).astype(np.float32)
    k, v = (torch.from_numpy(t).to(BF).float().numpy() for t in (k, v))
    p = Paged4([n], [30], 2, hd, 32, BF, values=[[k], [v]])
    q = rows_tensor(30, 6, hd, BF, 4)
    out, lse, _ = run(p, q)
    check(p, q, out, lse)
    # more rows share a power with 32 positions: sizes that differ less
    v = rng.standard_normal((n, 2, hd)).astype(np.float32) * np.exp2(rng.integers(-8, 8, (n, 2, 1))).astype(np.float32)
    v = torch.from_numpy(v).to(BF).float().numpy()
    many = Paged4([n], [300], 2, hd, 32, BF, values=[[k], [v]])
    q = rows_tensor(300, 6, hd, BF, 4)
    out, lse, _ = run(many, q)
    check(many, q, out, lse)
    big = Paged4([n], [9], 2, hd, 32, BF, values=[[k * 2.0 ** 50], [v * 2.0 ** 60]])
    q = rows_tensor(9, 6, hd, BF, 4) * 2.0 ** -50
    out, lse, _ = run(big, q)
    check(big, q, out, lse)
    small = Paged4([n], [9], 2, hd, 32, BF, values=[[k * 2.0 ** -60], [v]])
    q = rows_tensor(9, 6, hd, BF, 4) * 2.0 ** 60
    out, lse, _ = run(small, q)
    check(small, q, out, lse)


@pytest.mark.parametrize("n", [20, 60])
def test_rows_do_not_reach_into_one_another(n):
    """A row that is not finite, one of huge values and one of zeros among others
    of its item; a cache row that is not finite voids its head only."""
    p = Paged4([500, 400], [n, n], 2, 128, 64, BF, seed=8)
    q = rows_tensor(2 * n, 10, 128, BF, 4)
    clean, lse0, _ = run(p, q)
    check(p, q, clean, lse0)
    q2 = q.clone()
    q2[3, 2, 5] = float("nan")
    q2[4, 1] = float("inf")
    q2[5, 0] = 1e30
    q2[6, 7] = 0
    out, lse, _ = run(p, q2)
    same = torch.ones(2 * n, 10, dtype=torch.bool, device="cuda")
    for r, h in ((3, 2), (4, 1), (5, 0), (6, 7)):
        same[r, h] = False
    assert torch.equal(out[same], clean[same]) and torch.equal(lse[same], lse0[same])
    assert out[3, 2].isnan().all() and out[4, 1].isnan().all()
    pages = p.pages[1]
    pid = int(p.table_np[0, 2])
    pages[pid, 1, 7, 64:66] = 0xFF                       # NaN scale of one block of V, KV head 1, position 135
    out, lse, _ = run(p, q)
    assert torch.equal(out[n:], clean[n:]) and torch.equal(out[:n, :5], clean[:n, :5])
    assert torch.equal(lse[:n, :5], lse0[:n, :5])


def test_bad_pages_read_as_zeros_and_requests_that_do_not_fit_stay():
    p = Paged4([300, 300, 300], [4, 4, 4], 2, 64, 16, BF, seed=5)
    q = rows_tensor(12, 4, 64, BF, 4)
    clean, _, _ = run(p, q)
    table = p.table.clone()
    table[1, 3], table[1, 5] = p.n_pages + 4, -1
    ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(4, 2, 64, 4))
    out = torch.full_like(q, 7.0)
    dfl.dflash_paged_attention(p.cache, q, out, p.row_start, p.kv_len, table, 4, ws)
    assert dfl.dflash_read_status(ws) == -1
    assert torch.equal(out[:4], clean[:4]) and torch.equal(out[8:], clean[8:]) and out[4:8].isfinite().all()
    kp, vp = p.host()
    k, v = (e2m1.sequence(t, p.table_np[1], 300, 16) for t in (kp, vp))
    for s in (3, 5):
        k[16 * s:16 * s + 16] = v[16 * s:16 * s + 16] = 0
    z = k[:297, 0] @ to64(q)[4, 0] / 8
    w = np.exp(z - z.max())
    want = (w / w.sum()) @ v[:297, 0]
    assert np.abs(to64(out)[4, 0] - want).max() <= 2.0 ** -8 * np.abs(v).max()
    ws.zero_()
    out = torch.full_like(q, 7.0)
    lens = torch.tensor([300, 16 * p.width + 1, 300], device="cuda")
    dfl.dflash_paged_attention(p.cache, q, out, p.row_start, lens, p.table, 4, ws)
    assert dfl.dflash_read_status(ws) == -2
    assert torch.equal(out[:4], clean[:4]) and torch.equal(out[8:], clean[8:]) and (out[4:8] == 7.0).all()


@pytest.mark.parametrize("order", ["hrd", "wide"])
def test_strides_spread_pages_and_scales(order):
    p = Paged4([300, 70], [20, 70], 3, 64, 32, F16, seed=6, spread=16 * 7)
    q = rows_tensor(p.n_rows, 6, 64, F16, 4, order=order)
    out = torch.full_like(q, 7.0)
    for scale in (1.0, 0.01, 3.7):
        run(p, q, out=out, lse=False, scale=scale)
        check(p, q, out, None, scale=scale)


def test_lengths_in_between_and_max_rows_above_the_batchs():
    """max_rows says no request has more: one far above what the batch has changes
    nothing but the workspace."""
    p = Paged4([1000, 50, 8], [1, 6, 2], 2, 128, 64, BF, seed=7)
    q = rows_tensor(9, 10, 128, BF, 4, extra=200)
    a = run(p, q)
    b = run(p, q, max_rows=200)
    check(p, q, *a[:2])
    check(p, q, *b[:2], max_rows=200)


@pytest.mark.parametrize("rows", [8, 40])
def test_streams_threads_and_a_captured_graph(rows):
    p = Paged4([3000, 400, 77], [rows] * 3, 2, 128, 64, BF, seed=9)
    q = rows_tensor(3 * rows, 10, 128, BF, 4)
    want, lse, _ = run(p, q)
    need = dfl.dflash_paged_attention_workspace_bytes(10, 2, 128, rows)
    got = []

    def other(i):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ws = dfl.workspace(need)
        s.wait_stream(torch.cuda.default_stream())
        out = torch.empty_like(q)
        for _ in range(5):
            dfl.dflash_paged_attention(p.cache, q, out, *p.batch, rows, ws, stream=s)
        s.synchronize()
        got.append(out)
    threads = [threading.Thread(target=other, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 3 and all(torch.equal(o, want) for o in got)
    ws, out = dfl.workspace(need), torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dfl.dflash_paged_attention(p.cache, q, out, *p.batch, rows, ws)
    for n in (3000, 2500, 3, 0):
        p.kv_len[0] = n
        out.zero_()
        graph.replay()
        eager, _, _ = run(p, q)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
