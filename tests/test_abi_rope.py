"""Host-side refusals of the rotary positions and of caches in 4 bits: every bad
argument is turned away before anything is launched (no call here reaches a GPU)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from block_speculative_decoding_ctx_gb300 import build as dbuild
from oracle import rotary
from test_abi_target import BAD_BATCH, BAD_CACHE, BAD_ROWS, FAKE, P, batch, cache, ref, rows

REC = 2 * 64 * 80      # a page of 2 heads of 64 records of 80 bytes


@pytest.fixture(scope="module")
def L():
    dbuild.build()
    return dfl.lib()


def cache4(**kw):
    return cache(**{**dict(format=4, k_page_stride=REC, v_page_stride=REC), **kw})


BAD_CACHE4 = [(dict(head_dim=96), -4), (dict(page_size=8), -4), (dict(n_pages=0), -2), (dict(k_page_stride=REC - 16), -2),
              (dict(v_page_stride=REC + 8), -3), (dict(k_pages=4104), -3), (dict(v_pages=None), -1)]


@pytest.mark.parametrize("name", ["dflash_paged_append", "dflash_paged_gather"])
def test_move_refusals_of_a_cache_in_4_bits(L, name):
    f = getattr(L, name)

    def call(c=cache4(), t=0, k=rows(), v=rows(), ws=FAKE, n=256):
        return f(ref(c), ref(batch()), t, ref(k), ref(v), ws, n, None)
    for bad, code in BAD_CACHE4:
        assert call(c=cache4(**bad)) == code, bad
    assert call(t=2) == -1 and call(ws=None) == -7 and call(n=255) == -7
    assert call(t=1, ws=None) == -7                    # either 16-bit type of rows
    assert call(c=cache4(k_page_stride=REC + 16, v_page_stride=1 << 38), ws=None) == -7
    assert call(c=cache4(v_page_stride=(1 << 38) + 16), ws=None) == -2


def test_attention_refusals_of_a_cache_in_4_bits(L):
    need = dfl.dflash_paged_attention_workspace_bytes(10, 2, 128, 8)

    def call(c=cache4(), t=0, n_q=10, max_rows=8, ws=FAKE, n=need):
        x = rows(row_stride=2048)
        return L.dflash_paged_attention(ref(c), ref(batch()), t, n_q, ref(x), ref(x), None, max_rows, 0.1, 1, 0, ws, n, None)
    for bad, code in BAD_CACHE4:
        assert call(c=cache4(**bad)) == code, bad
    assert call(n=need - 1) == -7 and call(n_q=9) == -2 and call(t=2) == -1
    assert call(max_rows=0) == 0
    # B * ceil(R / 128) items: 2^30 of them and no more
    many = dict(rows=1 << 30, max_pages=1, table_stride=1)
    x = rows(row_stride=1024)
    for B, code in ((128, -7), (129, -2)):
        assert L.dflash_paged_attention(ref(cache4()), ref(batch(B=B, **many)), 0, 2, ref(x), ref(x), None, 1 << 30, 0.1, 1, 0, None,
                                        0, None) == code
    maps = dfl.dflash_paged_maps()
    assert L.dflash_paged_cache_maps(ref(cache4()), ref(maps)) == 0
    assert call(c=cache4(maps=ctypes.addressof(maps)), max_rows=0) == 0
    assert call(c=cache4(maps=ctypes.addressof(maps), n_pages=11), max_rows=0) == -1


def good_rope(n=128, layout=0):
    return dfl.dflash_rope_init(rotary.frequencies(n, 1e4), layout)


def test_append_rope_refusals(L):
    def call(c=cache(), b=batch(), t=0, k=rows(), v=rows(), n_q=10, q=rows(ptr=1 << 24, row_stride=2048),
             o=rows(ptr=1 << 26, row_stride=2048), rope=good_rope(), pos=None, ws=FAKE, n=256):
        return L.dflash_paged_append_rope(ref(c), ref(b), t, ref(k), ref(v), n_q, ref(q), ref(o), ref(rope), pos, ws, n, None)
    for bad, code in BAD_CACHE:
        assert call(c=cache(**bad)) == code, bad
    for bad, code in BAD_CACHE4:
        assert call(c=cache4(**bad)) == code, bad
    for bad, code in BAD_BATCH:
        assert call(b=batch(**bad)) == code, bad
    for bad, code in BAD_ROWS:
        for which in ("k", "v", "q", "o"):
            assert call(**{which: rows(**bad)}) == code, (which, bad)
    assert call(c=None) == -1 and call(b=None) == -1 and call(k=None) == -1 and call(rope=None) == -1
    assert call(t=2) == -1 and call(t=1) == -1
    assert call(n_q=-1) == -2 and call(n_q=65536) == -2
    # queries come whole or not at all
    assert call(q=None) == -1 and call(o=None) == -1 and call(n_q=0) == -1 and call(q=None, o=None) == -1
    assert call(n_q=0, q=None, o=None, ws=None) == -7
    assert call(n_q=3, ws=None) == -7                  # no multiple of the KV heads is asked for
    for bad, code in ((dict(rotary_dim=0), -2), (dict(rotary_dim=48), -2), (dict(rotary_dim=160), -2), (dict(rotary_dim=-32), -2),
                      (dict(layout=2), -1), (dict(factor=math.inf), -1), (dict(factor=math.nan), -1)):
        r = good_rope()
        for k, v in bad.items():
            setattr(r, k, v)
        assert call(rope=r) == code, bad
    small = dict(head_dim=64, k_page_stride=2 * 64 * 64, v_page_stride=2 * 64 * 64)
    assert call(c=cache(**small)) == -2 and call(c=cache(**small), rope=good_rope(64), ws=None) == -7   # more than the head has
    assert call(pos=P(4100)) == -3
    assert call(ws=None) == -7 and call(ws=P(1000)) == -7 and call(n=255) == -7
    # q_out: q itself, beside it in one buffer, or elsewhere (16 rows and 10 heads of 128)
    assert call(o=rows(ptr=1 << 24, row_stride=2048), ws=None) == -7
    assert call(o=rows(ptr=(1 << 24) + 16, row_stride=2048)) == -1
    assert call(o=rows(ptr=1 << 24, row_stride=4096)) == -1
    wide = dict(row_stride=4096)
    assert call(q=rows(ptr=1 << 24, **wide), o=rows(ptr=(1 << 24) + 2 * 1280, **wide), ws=None) == -7
    assert call(q=rows(ptr=1 << 24, **wide), o=rows(ptr=(1 << 24) + 2 * 1272, **wide)) == -1
    assert call(q=rows(ptr=1 << 24, **wide), o=rows(ptr=(1 << 24) + 2 * 4096, **wide)) == -1       # the next row's
    assert call(q=rows(ptr=1 << 24, **wide), o=rows(ptr=(1 << 24) + 2 * (4096 + 1280), **wide), ws=None) == -7
    assert call(q=rows(ptr=1 << 24, **wide), o=rows(ptr=(1 << 24) + 2 * 2824, **wide)) == -1       # into the next row
    assert call(b=batch(rows=0), k=rows(ptr=None), v=rows(ptr=None), q=rows(ptr=None), o=rows(ptr=None), ws=None) == -7


def test_frequencies_follow_the_formula(L):
    for n in (32, 64, 96, 128):
        for kw in (dict(), dict(stretch=8.0), dict(stretch=4.0, trained=8192.0), dict(stretch=0.5, trained=1e6, slow=-2.0, fast=32.0)):
            got = dfl.dflash_rope_frequencies(n, 5e5, **kw)
            np.testing.assert_allclose(got, rotary.frequencies(n, 5e5, **kw), rtol=1e-14)
    for bad, code in ((dict(rotary_dim=16), "SHAPE"), (dict(rotary_dim=(1 << 31) - 32), "SHAPE"), (dict(rotary_dim=160), "SHAPE"), (dict(rotary_dim=-32), "SHAPE"),
                      (dict(theta=0.0), "ARG"), (dict(theta=math.inf), "ARG"), (dict(stretch=0.0), "ARG"),
                      (dict(stretch=math.nan), "ARG"), (dict(trained=-1.0), "ARG"), (dict(trained=8.0, slow=4.0), "ARG"),
                      (dict(trained=8.0, slow=math.nan), "ARG"), (dict(trained=8.0, fast=math.inf), "ARG")):
        with pytest.raises(dfl.DflashError, match=code):
            dfl.dflash_rope_frequencies(**{**dict(rotary_dim=64, theta=1e4), **bad})
    assert L.dflash_rope_frequencies(64, 1e4, 1.0, 0.0, 0.0, 0.0, None) == -1


def test_rotation_counts_in_turns(L):
    """Each entry of the table is its frequency in 2^-64ths of a turn, to one of
    them and what a double's frequency leaves open."""
    from fractions import Fraction
    freq = rotary.frequencies(64, 1e6) + [-1.0, -1e-12, 3.0, 2.0 ** 20, -2.0 ** 20, 6.283185307179586, 12345.678, 0.0] * 2
    r = dfl.dflash_rope_init(freq[:32] + freq[32:48], dfl.DFLASH_ROPE_INTERLEAVED, factor=1.5)
    assert r.rotary_dim == 96 and r.layout == 1 and r.factor == 1.5
    for j, w in enumerate(freq[:48]):
        t = Fraction(w) / rotary.TWO_PI
        want = round((t - math.floor(t)) * 2 ** 64) % 2 ** 64
        off = (r.turns[j] - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 2, (j, w)
    for bad in ([math.nan] * 32, [math.inf] * 32, [2.0 ** 20 * 1.01] * 32):
        with pytest.raises(dfl.DflashError, match="ARG"):
            dfl.dflash_rope_init(bad)
    with pytest.raises(dfl.DflashError, match="SHAPE"):
        dfl.dflash_rope_init([1.0] * 24)
    with pytest.raises(dfl.DflashError, match="SHAPE"):
        dfl.dflash_rope_init([])
    with pytest.raises(dfl.DflashError, match="ARG"):
        dfl.dflash_rope_init([1.0] * 32, layout=2)
    with pytest.raises(dfl.DflashError, match="ARG"):
        dfl.dflash_rope_init([1.0] * 32, factor=math.inf)


def test_binding_checks_of_a_cache_in_4_bits():
    pages = torch.zeros(3, 2, 16, 40, dtype=torch.uint8)
    E = dfl.DFLASH_CACHE_E2M1
    c = dfl.paged_cache(pages, pages, format=E)
    assert (c.struct.head_dim, c.struct.format, c.struct.k_page_stride) == (64, 4, 2 * 16 * 40)
    wide = torch.zeros(3, 2, 2, 16, 80, dtype=torch.uint8)
    c = dfl.paged_cache(wide[:, 0], wide[:, 1], format=E)
    assert (c.struct.head_dim, c.struct.k_page_stride) == (128, 2 * 2 * 16 * 80)
    for bad in (lambda: dfl.paged_cache(pages.to(torch.bfloat16), pages.to(torch.bfloat16), format=E),
                lambda: dfl.paged_cache(pages[..., :39], pages[..., :39], format=E),
                lambda: dfl.paged_cache(pages, pages, torch.zeros(3, 2, 16), torch.zeros(3, 2, 16), format=E),
                lambda: dfl.paged_cache(pages, pages, format=dfl.DFLASH_CACHE_BF16),
                lambda: dfl.paged_cache(pages, pages)):
        with pytest.raises(ValueError):
            bad()
    assert dfl.paged_cache(pages, pages, torch.zeros(3, 2, 16), torch.zeros(3, 2, 16), format=dfl.DFLASH_CACHE_E4M3).struct.format == 2


def test_binding_checks_of_append_rope():
    pages = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    c = dfl.paged_cache(pages, pages)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    r = good_rope(64)

    def call(k=k, v=k, rope=r, **kw):
        dfl.dflash_paged_append_rope(c, k, v, None, None, None, rope, None, **kw)
    for bad, text in ((dict(v=k[:4]), "k and v"), (dict(k=k.float(), v=k.float()), "no rows"), (dict(q=q), "together"),
                      (dict(q_out=q), "together"), (dict(q=q[:4], q_out=q[:4]), "q and q_out"),
                      (dict(q=q.half(), q_out=q.half()), "q and q_out"), (dict(q=q, q_out=q.half()), "q and q_out"),
                      (dict(q=q[:, :0], q_out=q[:, :0]), "q and q_out"), (dict(q=q[..., :32], q_out=q[..., :32]), "q and q_out"),
                      (dict(rope=[1.0] * 32), "rope"), (dict(q=q, q_out=q), "CUDA")):
        with pytest.raises(ValueError, match=text):
            call(**bad)
