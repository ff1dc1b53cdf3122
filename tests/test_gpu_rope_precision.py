"""What rotated rows are quantised under, and how exact their sines and cosines are."""

import math

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import e2m1, rotary
from paged4_testutil import BF, F16, Paged4, kv_rows
from target_testutil import Paged, to64

E = 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,hd,rot,layout,factor", [
    ("e4m3", BF, 128, 128, 0, 1.0), ("e4m3", F16, 128, 96, 1, 0.7), ("e4m3", BF, 64, 32, 0, 1.2), ("e4m3", F16, 64, 64, 1, 1.0),
    ("e2m1", BF, 128, 128, 0, 1.0), ("e2m1", F16, 128, 96, 1, 0.7), ("e2m1", BF, 64, 32, 0, -1.5), ("e2m1", F16, 64, 64, 1, 1.0)])
def test_scales_are_those_of_the_turned_rows(fmt, dtype, hd, rot, layout, factor):
    """A scale is max / 448 of the row, or max / 6 of 16 values, as they are after the turn.
    Bounds, before any run: a turned value is off by 8 e of the magnitudes that meet in it
    (e = 2^-24: sine, cosine, factor, two products and a sum), so the largest of several by
    8 e of the largest such sum; the quotient e of itself, and in bfloat16 2^-8 of itself."""
    lens, rows = [700, 1, 77, 300], [33, 1, 0, 129]
    n_kv, page = 2, 32
    p = Paged4(lens, rows, n_kv, hd, page, dtype, garbage=False) if fmt == "e2m1" else \
        Paged(lens, rows, n_kv, hd, page, dtype, e4m3=True, garbage=False)
    n = p.n_rows
    k = kv_rows(n, n_kv, hd, dtype, 1)
    where = torch.randint(0, 2 ** 31, (n,), generator=torch.Generator().manual_seed(5))
    freq = dfl.dflash_rope_frequencies(rot, 1e5)
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append_rope(p.cache, k, k, *p.batch, dfl.dflash_rope_init(freq, layout, factor), ws, positions=where.cuda())
    assert dfl.dflash_read_status(ws) == 0
    x = to64(k)
    want = np.abs(rotary.rotate(x, where.tolist(), freq, layout, float(np.float32(factor))))
    size, half = np.abs(x).copy(), rot // 2
    i, j = (np.arange(half), half + np.arange(half)) if layout == 0 else (2 * np.arange(half), 2 * np.arange(half) + 1)
    size[..., i] = size[..., j] = (size[..., i] + size[..., j]) * abs(factor)
    group, most, own = (16, 6.0, 2.0 ** -8) if fmt == "e2m1" else (hd, 448.0, E)
    want, size = (t.reshape(n, n_kv, -1, group).max(-1) for t in (want, size))
    want = want / most
    lim = 8 * E * size / most + (own + 2 * E) * (want + 8 * E * size / most)
    for b in range(len(lens)):
        for r in range(rows[b]):
            s, at = lens[b] - rows[b] + r, p.start_np[b] + r
            place = p.table_np[b, s // page], slice(None), s % page
            got = e2m1.split(to64(p.pages[0])[place])[1] if fmt == "e2m1" else to64(p.scale[0])[place][:, None]
            assert (np.abs(got - want[at]) <= lim[at]).all(), (b, r)


# ------------------------------------------------------------------------- sines

ROT, PAIRS = 128, 64
BIG = 4096.0                       # the second value of every pair
LIMIT = 1.06                       # see test_sines_and_cosines_are_rounded_about_once


def exact_angles(rope, pos, device):
    """Angles of [n, PAIRS], float64 in [-pi, pi): positions times the table, modulo a turn,
    in wrapping 64-bit integers."""
    turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in list(rope.turns)[:PAIRS]], dtype=torch.int64, device=device)
    return (pos[:, None] * turns).double() * (2 * math.pi / 2.0 ** 64)


def pairs_that_cancel(t):
    """First values x of pairs (x, BIG) that turn to nearly 0: x = BIG tan t, to 11 bits, so
    that x cos t - BIG sin t is at most 2^-12 of either term and shows what those are off
    by.  Where tan t leaves [2^-4, 2^4] the pair is left out."""
    tan = t.tan()
    fine = (tan.abs() >= 2.0 ** -4) & (tan.abs() <= 15.0)
    return torch.where(fine, BIG * tan, torch.zeros_like(tan)).half(), fine


def deviation(got, x, t, fine):
    """Root mean square of what x cos t - BIG sin t is off by, in 2^-24ths of BIG sin t."""
    want = x.double() * t.cos() - BIG * t.sin()
    d = ((got.double() - want) / (BIG * t.sin()))[fine] / E
    return float(d.square().mean().sqrt())


def model(x, t, cos, sin):
    """The same from given float32 cosines and sines: BIG sin t is exact, the product with x
    and the sum are rounded together, then to 16 bits."""
    return (x.double() * cos.double() - BIG * sin.double()).float().half()


def positions(n, device):
    return torch.randint(0, 2 ** 31, (n,), generator=torch.Generator().manual_seed(11)).to(device)


@pytest.mark.gpu
def test_sines_and_cosines_are_rounded_about_once():
    """Against float32 sines and cosines that are the nearest ones.  Their own rounding is
    0.42 in 2^-24ths of themselves (half a unit in the last place, evenly spread), twice; a
    sine here may be off by another 0.23 units in the last place where all its roundings
    meet, so by some 0.1 as a root mean square, a cosine by less: 1.03 times as much in all
    at most.  An angle kept in one float32 makes 1.15 times as much."""
    n = 20000
    p = Paged([n], [n], 1, ROT, 128, F16, garbage=False)
    freq = dfl.dflash_rope_frequencies(ROT, 1e6)
    rope = dfl.dflash_rope_init(freq)
    where = positions(n, "cuda")
    t = exact_angles(rope, where, "cuda")
    x, fine = pairs_that_cancel(t)
    q = torch.cat([x, torch.where(fine, BIG, 0.0).half()], 1)[:, None].contiguous()
    out = torch.empty_like(q)
    k = torch.zeros(n, 1, ROT, dtype=F16, device="cuda")
    ws = dfl.workspace(dfl.dflash_paged_workspace_bytes())
    dfl.dflash_paged_append_rope(p.cache, k, k, *p.batch, rope, ws, q=q, q_out=out, positions=where)
    assert dfl.dflash_read_status(ws) == 0 and int(fine.sum()) > 10 ** 6
    got = deviation(out[:, 0, :PAIRS], x, t, fine)
    best = deviation(model(x, t, t.cos().float(), t.sin().float()), x, t, fine)
    assert got <= LIMIT * best, f"{got / best:.3f} of what rounding once makes"


def test_the_measure_tells_an_angle_in_one_float32():
    """The same measure of the mistakes that the limit has to tell: the angle beside the
    nearest quarter turn rounded to a float32, and sines off by up to 2 units."""
    dfl.declared_functions()
    rope = dfl.dflash_rope()
    for j, w in enumerate(rotary.frequencies(ROT, 1e6)):
        u = w / (2 * math.pi)
        rope.turns[j] = int((u - math.floor(u)) * 2.0 ** 64) % (1 << 64)
    t = exact_angles(rope, positions(8000, "cpu"), "cpu")
    x, fine = pairs_that_cancel(t)
    best = deviation(model(x, t, t.cos().float(), t.sin().float()), x, t, fine)
    quarter = torch.round(t / (math.pi / 2))
    one = (t - quarter * (math.pi / 2)).float().double() + quarter * (math.pi / 2)
    off = deviation(model(x, t, one.cos().float(), one.sin().float()), x, t, fine)
    assert off > 1.05 * LIMIT * best, f"{off / best:.3f}"
    g = torch.Generator().manual_seed(3)
    wrong = t.sin() * (1 + 2 * E * (2 * torch.rand(t.shape, generator=g, dtype=torch.float64) - 1))
    off = deviation(model(x, t, t.cos().float(), wrong.float()), x, t, fine)
    assert off > 1.05 * LIMIT * best, f"{off / best:.3f}"
