"""Rotary positions on the way into the paged cache, and beside it on queries."""

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import e2m1, quant, rotary
from oracle import target as ot
from paged4_testutil import BF, F16, Paged4, check, kv_rows
from target_testutil import HALF_STEP, Paged, to64

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


def make(fmt, lens, rows, n_kv, hd, page, dtype, seed=0, **kw):
    if fmt == "e2m1":
        return Paged4(lens, rows, n_kv, hd, page, dtype, seed=seed, garbage=False, **kw)
    return Paged(lens, rows, n_kv, hd, page, dtype, e4m3=fmt == "e4m3", seed=seed, garbage=False, **kw)


def cached(p, fmt, side, b, s):
    """Row s of request b in the cache, float64 [heads, hd], and the steps between
    neighbouring values of its format there."""
    pages = to64(p.pages[side])[p.table_np[b, s // p.page], :, s % p.page]
    if fmt == "e2m1":
        codes, sc = e2m1.split(pages)
        v, sc = np.abs(e2m1.value(codes)), np.repeat(sc, 16, -1)
        return e2m1.unpack(pages), np.select([v < 2, v < 4], [0.5, 1.0], 2.0) * sc, np.abs(sc)
    if fmt == "e4m3":
        sc = to64(p.scale[side])[p.table_np[b, s // p.page], :, s % p.page][:, None]
        v = quant.e4m3_value(pages)
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -9))), -6) - 3)
        return v * sc, step * sc, np.broadcast_to(np.abs(sc), v.shape)
    return pages, None, None


def turned_bound(x, rope_dim, layout, factor):
    """Sum of the magnitudes that go into every rotated value, [.., hd], times factor."""
    a = np.abs(x)
    out = a.copy()
    half = rope_dim // 2
    i, j = (np.arange(half), half + np.arange(half)) if layout == 0 else (2 * np.arange(half), 2 * np.arange(half) + 1)
    out[..., i] = out[..., j] = (a[..., i] + a[..., j]) * abs(factor)
    return out


CASES = [
    # format, dtype, hd, n_kv, n_q, page, rotary_dim, layout, factor, positions
    ("16", BF, 128, 8, 40, 64, 128, 0, 1.0, None),
    ("16", F16, 64, 2, 14, 16, 32, 1, 1.2, "far"),
    ("16", BF, 64, 1, 3, 128, 64, 1, 1.0, "odd"),
    ("e4m3", BF, 128, 2, 10, 32, 96, 0, 1.0, None),
    ("e4m3", F16, 64, 3, 3, 16, 64, 0, 0.7, "far"),
    ("e4m3", F16, 128, 2, 2, 16, 64, 1, 1.0, None),
    ("e2m1", BF, 128, 8, 40, 64, 128, 0, 1.0, None),
    ("e2m1", F16, 128, 1, 5, 16, 32, 1, -1.5, "odd"),
    ("e2m1", BF, 64, 2, 0, 128, 32, 0, 1.0, None),
    ("e2m1", F16, 64, 4, 8, 32, 64, 1, 1.0, "far"),
    ("e2m1", BF, 128, 2, 4, 64, 96, 0, 1.0, "odd"),
]


@pytest.mark.parametrize("fmt,dtype,hd,n_kv,n_q,page,rot,layout,factor,pos", CASES)
def test_keys_and_queries_are_turned(fmt, dtype, hd, n_kv, n_q, page, rot, layout, factor, pos):
    """Bounds, before any run: cos and sin of an angle that is off by 2^-27 of a
    half turn and their own 2 ulp, e = 2^-24 each, times the factor, two products
    and a sum: 8 e of the magnitudes that meet; then the format's half step (of
    the value that was stored: its neighbours may be twice as far on one side)."""
    lens, rows = [700, 1, 77, 300], [33, 1, 0, 129]
    p = make(fmt, lens, rows, n_kv, hd, page, dtype, seed=hd + rot)
    n = p.n_rows
    k, v = kv_rows(n, n_kv, hd, dtype, 1, 4), kv_rows(n, n_kv, hd, dtype, 2, 4)
    q = kv_rows(n, n_q, hd, dtype, 3, 4) if n_q else None
    q_out = torch.full_like(q, 7.0) if n_q else None
    g = torch.Generator().manual_seed(5)
    positions = None
    where = np.concatenate([np.arange(l - r, l) for l, r in zip(lens, rows)])
    if pos:
        positions = torch.randint(-1000, 2 ** 31 if pos == "far" else 5000, (n + 4,), generator=g)
        positions[:3] = torch.tensor([0, -1, 2 ** 32 - 1])
        where = positions[:n].numpy()
        positions = positions.cuda()
    freq = dfl.dflash_rope_frequencies(rot, 1e4 if rot < 64 else 1e6, stretch=4.0, trained=0 if layout else 4096.0)
    rope = dfl.dflash_rope_init(freq, layout, factor)
    before = [to64(t) for t in p.pages]
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append_rope(p.cache, k, v, *p.batch, rope, ws, q=q, q_out=q_out, positions=positions)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    u = HALF_STEP[dtype]
    if n_q:
        want = rotary.rotate(to64(q)[:n], where, freq, layout, float(np.float32(factor)))
        size = turned_bound(to64(q)[:n], rot, layout, factor)
        b = 8 * E * size + u * (np.abs(want) + 8 * E * size) + 2.0 ** -25
        assert (np.abs(to64(q_out)[:n] - want) <= b).all()
        assert torch.equal(q_out[:n, :, rot:], q[:n, :, rot:]) and (q_out[n:] == 7.0).all()
    want_k = rotary.rotate(to64(k)[:n], where, freq, layout, float(np.float32(factor)))
    size = 8 * E * turned_bound(to64(k)[:n], rot, layout, factor)
    written = np.zeros(before[0].shape[:1] + before[0].shape[2:3], dtype=bool)
    for b in range(len(lens)):
        for j in range(rows[b]):
            s, r = lens[b] - rows[b] + j, p.start_np[b] + j
            written[p.table_np[b, s // page], s % page] = True
            got, step, scale = cached(p, fmt, 0, b, s)
            if step is None:
                lim = size[r] + u * (np.abs(want_k[r]) + size[r]) + 2.0 ** -25
            else:       # half a step, of the larger neighbour, and what saturates
                lim = size[r] + step / 2 * (1 + 2.0 ** -7) + (np.abs(want_k[r]) * 2.0 ** -8 if fmt == "e2m1" else 2.0 ** -20 * np.abs(want_k[r]))
            assert (np.abs(got - want_k[r]) <= lim).all(), (b, j)
            # values are written as append writes them
            got, _, _ = cached(p, fmt, 1, b, s)
            x = v[r].float().cpu().numpy()
            if fmt == "e2m1":
                np.testing.assert_array_equal(got, e2m1.unpack(e2m1.pack(x)))
            elif fmt == "e4m3":
                codes, sc = ot.quantize(x)
                np.testing.assert_array_equal(got, quant.e4m3_value(codes) * sc.astype(np.float64)[:, None])
            else:
                np.testing.assert_array_equal(got, x.astype(np.float64))
    for side in range(2):
        after = np.moveaxis(to64(p.pages[side]), 1, 2)[~written]
        np.testing.assert_array_equal(after, np.moveaxis(before[side], 1, 2)[~written])


@pytest.mark.parametrize("fmt", ["16", "e4m3", "e2m1"])
def test_position_zero_and_factor_one_are_append(fmt):
    """Angles of zero leave rows as they are: the bytes are append's."""
    lens, rows, hd = [200, 50], [90, 50], 128
    a, b = (make(fmt, lens, rows, 2, hd, 32, BF, seed=4) for _ in range(2))
    k, v = kv_rows(140, 2, hd, BF, 1), kv_rows(140, 2, hd, BF, 2)
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    rope = dfl.dflash_rope_init(dfl.dflash_rope_frequencies(128, 1e4))
    q = kv_rows(140, 4, hd, BF, 3)
    q_out = torch.empty_like(q)
    zero = torch.zeros(140, dtype=torch.int64, device="cuda")
    dfl.dflash_paged_append(a.cache, k, v, *a.batch, ws)
    dfl.dflash_paged_append_rope(b.cache, k, v, *b.batch, rope, ws, q=q, q_out=q_out, positions=zero)
    for side in range(2):
        assert torch.equal(a.pages[side].view(torch.uint8) if fmt == "e4m3" else a.pages[side],
                           b.pages[side].view(torch.uint8) if fmt == "e4m3" else b.pages[side])
        if fmt == "e4m3":
            assert torch.equal(a.scale[side], b.scale[side])
    assert torch.equal(q, q_out)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_keys_of_any_size(fmt):
    """At position 0 with factor 1 nothing turns: rows of every size from bfloat16's
    smallest on get the codes and scales that append gives them.  A factor that takes them
    where a scale would be 0 makes zeros of them, under scales of 1."""
    n, n_kv, hd = 512, 2, 128
    rng = np.random.default_rng(3)
    size = 2.0 ** np.linspace(-133, 127, n)
    x = rng.uniform(0.3, 1.0, (n, n_kv, hd)) * rng.choice([-1.0, 1.0], (n, n_kv, hd)) * size[:, None, None]
    x[:, :, ::37] = 0
    x = torch.from_numpy(x.clip(-3e38, 3e38)).to(BF)
    x[x == 0] = 0                                        # no -0
    k, zero = x.cuda(), torch.zeros(n, dtype=torch.int64, device="cuda")
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    freq = dfl.dflash_rope_frequencies(hd, 1e6)
    p, q = (make(fmt, [n], [n], n_kv, hd, 16, BF) for _ in range(2))
    dfl.dflash_paged_append(p.cache, k, k.flip(0), *p.batch, ws)
    dfl.dflash_paged_append_rope(q.cache, k, k.flip(0), *q.batch, dfl.dflash_rope_init(freq), ws, positions=zero)
    assert all(torch.equal(p.pages[i].view(torch.uint8), q.pages[i].view(torch.uint8)) for i in range(2))
    if fmt == "e4m3":
        assert all(torch.equal(p.scale[i], q.scale[i]) for i in range(2))
    k = torch.full_like(k, 2.0 ** -133)
    k[:, :, 5::9] = 0
    back = [torch.full_like(k, 7.0) for _ in range(2)]
    dfl.dflash_paged_append_rope(q.cache, k, k, *q.batch, dfl.dflash_rope_init(freq, factor=2.0 ** -12), ws, positions=zero)
    dfl.dflash_paged_gather(q.cache, *back, *q.batch, ws)
    assert (back[0] == 0).all()
    # values as they came: 2^-133 / 448 is a float32, 2^-133 / 6 below half of bfloat16's smallest, 2^-133
    assert torch.equal(back[1], k if fmt == "e4m3" else torch.zeros_like(k))
    if fmt == "e4m3":
        assert (q.scale[0][q.table_np[0].tolist()] == 1).all()


def test_in_place_slices_and_strides():
    """Queries turned in place, and slices of one projection's output."""
    lens, rows, hd, n_kv, n_q = [100, 30], [20, 30], 64, 2, 6
    qkv = kv_rows(50, n_q + 2 * n_kv, hd, BF, 7)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    rope = dfl.dflash_rope_init(dfl.dflash_rope_frequencies(64, 1e4))
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    outs = []
    for how in ("new", "place", "hrd", "wide", "beside"):
        p = make("16", lens, rows, n_kv, hd, 16, BF)
        kk, vv = k, v
        if how == "new":
            x, o = q.contiguous(), torch.empty_like(q.contiguous())
        elif how == "place":
            x = o = q.clone()
        elif how == "beside":
            both = torch.cat([q, torch.zeros_like(q)], 1)
            x, o = both[:, :n_q], both[:, n_q:]
        else:
            x, kk, vv = (t.contiguous().transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)) if how == "hrd" else (q, k, v)
            big = torch.zeros(50, n_q + 3, hd + 8, dtype=BF, device="cuda")
            o = big[:, 1:n_q + 1, :hd]
        dfl.dflash_paged_append_rope(p.cache, kk, vv, *p.batch, rope, ws, q=x, q_out=o)
        torch.cuda.synchronize()
        outs.append((o.clone(), p.pages[0].clone(), p.pages[1].clone()))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
    assert dfl.dflash_read_status(ws) == 0


@pytest.mark.parametrize("fmt", ["16", "e4m3", "e2m1"])
def test_padded_and_ill_formed_batches(fmt):
    """Rows behind the last request, requests that do not fit, pages that are none,
    rows before position 0: nothing of them is written but, for a bad page alone,
    the query."""
    hd, page = 64, 16
    lens, rows = [40, 33, 5, 50], [20, 10, 8, 30]        # the third: 3 rows before position 0
    p = make(fmt, lens, rows, 2, hd, page, BF)
    n = p.n_rows
    k, v, q = kv_rows(n, 2, hd, BF, 1, 30), kv_rows(n, 2, hd, BF, 2, 30), kv_rows(n, 4, hd, BF, 3, 30)
    rope = dfl.dflash_rope_init(dfl.dflash_rope_frequencies(32, 1e4))
    table = p.table.clone()
    table[0, 2] = p.n_pages
    lens_dev = p.kv_len.clone()
    lens_dev[1] = page * p.width + 1
    before = [to64(t) for t in p.pages]
    q_out = torch.full_like(q, 7.0)
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append_rope(p.cache, k, v, p.row_start, lens_dev, table, rope, ws, q=q, q_out=q_out)
    assert dfl.dflash_read_status(ws) in (-1, -2)
    got = to64(q_out)
    untouched = list(range(20, 30)) + list(range(30, 33)) + list(range(n, n + 30))
    assert (got[untouched] == 7.0).all()
    done = [r for r in range(n) if r not in untouched]
    assert not (got[done] == 7.0).all(axis=(1, 2)).any()
    after = [to64(t) for t in p.pages]
    owned = np.zeros(before[0].shape[:1] + before[0].shape[2:3], dtype=bool)
    for b, first, last in ((0, 20, 32), (2, 0, 5), (3, 20, 50)):
        for s in range(first, last):
            owned[p.table_np[b, s // page], s % page] = True
    for side in range(2):
        x, y = np.moveaxis(before[side], 1, 2), np.moveaxis(after[side], 1, 2)
        np.testing.assert_array_equal(x[~owned], y[~owned])
        assert (x[owned] != y[owned]).any(axis=(1, 2)).all()


def test_rows_that_are_not_finite():
    p = make("e2m1", [32], [32], 1, 64, 16, BF)
    k, v = kv_rows(32, 1, 64, BF, 1), kv_rows(32, 1, 64, BF, 2)
    k[3, 0, 5] = float("nan")
    v[4, 0, 40] = float("inf")
    k[7] = 3e38                                          # whose rotation leaves float32
    rope = dfl.dflash_rope_init(dfl.dflash_rope_frequencies(64, 1e4), factor=4.0)
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append_rope(p.cache, k, v, *p.batch, rope, ws)
    back = [torch.empty_like(k) for _ in range(2)]
    dfl.dflash_paged_gather(p.cache, back[0], back[1], *p.batch, ws)
    bad = back[0].isnan()[:, 0]
    assert bad[3, 0:16].all() and bad[3, 32:48].all() and bad[3].sum() == 32          # both blocks of the pair
    assert bad[7].any() and not bad[[i for i in range(32) if i not in (3, 7)]].any()
    bad = back[1].isnan()[:, 0]
    assert bad[4, 32:48].all() and bad.sum() == 16


def test_many_rows_of_one_call():
    """Blocks of several rows, ends inside a block, far more rows than blocks."""
    lens, rows = [6001, 5, 2500], [6001, 1, 2499]
    p = make("16", lens, rows, 1, 64, 64, BF)
    n = p.n_rows
    k, v, q = (kv_rows(n, h, 64, BF, i) for i, h in ((1, 1), (2, 1), (3, 3)))
    rope = dfl.dflash_rope_init(dfl.dflash_rope_frequencies(64, 1e4))
    q_out = torch.empty_like(q)
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append_rope(p.cache, k, v, *p.batch, rope, ws, q=q, q_out=q_out)
    pos = torch.cat([torch.arange(l - r, l) for l, r in zip(lens, rows)]).double()
    w = torch.tensor(rotary.frequencies(64, 1e4), dtype=torch.float64)
    turn = torch.polar(torch.ones(n, 32, dtype=torch.float64), pos[:, None] * w)[:, None]
    x = q.double().cpu()
    z = torch.complex(x[..., :32], x[..., 32:]) * turn
    want = torch.cat([z.real, z.imag], -1)
    size = torch.from_numpy(turned_bound(x.numpy(), 64, 0, 1.0))
    assert ((q_out.double().cpu() - want).abs() <= 8 * E * size + 2.0 ** -8 * (want.abs() + 8 * E * size)).all()


def test_a_step_eager_and_captured():
    """Rows turned, written in 4 bits, attended; as a user's step, and as one graph
    replayed over growing lengths with the lengths and rows changed in between."""
    lens, rows, hd, n_kv, n_q = [300, 40, 1000], [8, 8, 8], 128, 2, 10
    rope = dfl.dflash_rope_init(dfl.dflash_rope_frequencies(128, 1e6))

    def setup():
        p = make("e2m1", [l + 24 for l in lens], rows, n_kv, hd, 64, BF, seed=1)
        p.kv_len.copy_(torch.tensor(lens))
        x = {h: torch.empty(24, n, hd, dtype=BF, device="cuda") for h, n in (("k", n_kv), ("v", n_kv), ("q", n_q), ("turned", n_q), ("out", n_q))}
        ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(n_q, n_kv, hd, 8))

        def step():
            dfl.dflash_paged_append_rope(p.cache, x["k"], x["v"], *p.batch, rope, ws, q=x["q"], q_out=x["turned"])
            dfl.dflash_paged_attention(p.cache, x["turned"], x["out"], *p.batch, 8, ws)
            p.kv_len.add_(8)
        return p, x, ws, step
    p, x, ws, step = setup()
    p2, x2, ws2, step2 = setup()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step2()
    for i in range(3):
        for h, n in (("k", n_kv), ("v", n_kv), ("q", n_q)):
            x[h].copy_(kv_rows(24, n, hd, BF, 10 * i + n + (h == "v")))
            x2[h].copy_(x[h])
        step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x["out"], x2["out"]) and torch.equal(x["turned"], x2["turned"])
        assert all(torch.equal(a, b) for a, b in zip(p.pages, p2.pages)) and torch.equal(p.kv_len, p2.kv_len)
        # against the oracle, from what the cache holds
        p.lens = (p.kv_len - 8).tolist()
        out = x["out"].clone()
        check(p, x["turned"], out, None)
    assert dfl.dflash_read_status(ws) == 0 and dfl.dflash_read_status(ws2) == 0
