"""Host-side refusals of the target-side entry points: every bad argument is
turned away before anything is launched (no call here reaches a GPU)."""

import ctypes

import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from block_speculative_decoding_ctx_gb300 import build as dbuild

P = ctypes.c_void_p
FAKE = P(1 << 20)          # never dereferenced


@pytest.fixture(scope="module")
def L():
    dbuild.build()
    return dfl.lib()


def cache(**kw):
    c = dict(k_pages=4096, v_pages=4096, k_scale=None, v_scale=None, k_page_stride=2 * 64 * 128, v_page_stride=2 * 64 * 128,
             n_pages=10, n_kv_heads=2, page_size=64, head_dim=128, format=0)
    c.update(kw)
    return dfl.dflash_paged_cache(**c)


def batch(**kw):
    c = dict(row_start=4096, kv_len=4096, page_table=4096, table_stride=8, B=3, max_pages=8, rows=20)
    c.update(kw)
    return dfl.dflash_paged_batch(**c)


def rows(ptr=4096, row_stride=1024, head_stride=128):
    return dfl.dflash_rows(ptr, row_stride, head_stride)


BAD_CACHE = [
    (dict(format=3), -1), (dict(head_dim=96), -4), (dict(page_size=8), -4), (dict(page_size=256), -4),
    (dict(n_pages=0), -2), (dict(n_kv_heads=0), -2), (dict(k_page_stride=100), -2), (dict(k_pages=None), -1),
    (dict(v_pages=4100), -3), (dict(v_page_stride=2 * 64 * 128 + 4), -3),
    (dict(format=2), -1), (dict(format=2, k_scale=4096, v_scale=4100), -3),
    (dict(format=2, k_scale=4096, v_scale=4096, k_page_stride=2 * 64 * 128 + 8), -3),
]
BAD_BATCH = [
    (dict(B=0), -2), (dict(B=65536), -2), (dict(max_pages=0), -2), (dict(rows=-1), -2), (dict(table_stride=7), -2),
    (dict(max_pages=1 << 24, table_stride=1 << 24), -2), (dict(row_start=None), -1), (dict(kv_len=4100), -3),
]
BAD_ROWS = [(dict(ptr=None), -1), (dict(ptr=4104), -3), (dict(row_stride=1028), -3), (dict(head_stride=64), -2),
            (dict(row_stride=-8), -2)]


def ref(x):
    return ctypes.byref(x) if x is not None else None


@pytest.mark.parametrize("name", ["dflash_paged_append", "dflash_paged_gather"])
def test_move_refusals(L, name):
    f = getattr(L, name)

    def call(c=cache(), b=batch(), t=0, k=rows(), v=rows(), ws=FAKE, n=256):
        return f(ref(c), ref(b), t, ref(k), ref(v), ws, n, None)
    for bad, code in BAD_CACHE:
        assert call(c=cache(**bad)) == code, bad
    for bad, code in BAD_BATCH:
        assert call(b=batch(**bad)) == code, bad
    for bad, code in BAD_ROWS:
        assert call(k=rows(**bad)) == code and call(v=rows(**bad)) == code, bad
    assert call(c=None) == -1 and call(b=None) == -1 and call(k=None) == -1
    assert call(t=2) == -1 and call(t=1) == -1 and call(c=cache(format=1)) == -1    # type against the cache's
    assert call(ws=None) == -7 and call(ws=P(1000)) == -7 and call(n=255) == -7


def test_attention_refusals(L):
    need = dfl.dflash_paged_attention_workspace_bytes(10, 2, 128, 8)
    assert need >= 256

    def call(c=cache(), b=batch(), t=0, n_q=10, q=rows(row_stride=2048), o=rows(row_stride=2048), lse=None, max_rows=8,
             scale=0.1, causal=1, window=0, ws=FAKE, n=need):
        return L.dflash_paged_attention(ref(c), ref(b), t, n_q, ref(q), ref(o), lse, max_rows, scale, causal, window, ws, n,
                                        None)
    for bad, code in BAD_CACHE:
        assert call(c=cache(**bad)) == code, bad
    for bad, code in BAD_BATCH:
        assert call(b=batch(**bad)) == code, bad
    for bad, code in BAD_ROWS:
        assert call(q=rows(**bad)) == code and call(o=rows(**bad)) == code, bad
    assert call(n_q=9) == -2 and call(n_q=0) == -2
    assert call(max_rows=-1) == -2 and call(max_rows=21) == -2
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == -1
    assert call(causal=2) == -1 and call(window=-1) == -1
    assert call(lse=P(4098)) == -3
    assert call(ws=None) == -7 and call(n=need - 1) == -7
    wrong = dfl.dflash_paged_maps()                    # of no cache, let alone of this one
    assert call(c=cache(maps=ctypes.addressof(wrong))) == -1
    assert call(b=batch(max_pages=1 << 23, table_stride=1 << 23), c=cache(n_kv_heads=4096, k_page_stride=1 << 26, v_page_stride=1 << 26),
                n_q=4096) == -2                        # more key tiles than 32 bits count
    assert call(max_rows=0) == 0                       # nothing to do, nothing launched
    assert call(b=batch(rows=0), max_rows=0, q=rows(ptr=None), o=rows(ptr=None)) == 0
    assert dfl.dflash_paged_attention_workspace_bytes(9, 2, 128, 8) == 0
    assert dfl.dflash_paged_attention_workspace_bytes(8, 2, 96, 8) == 0


def test_rows_that_would_be_written_twice_are_refused(L):
    """20 rows of 2 heads of 128, and of 10 heads for attention."""
    for n_q, f in ((2, "gather k"), (2, "gather v"), (10, "attention")):
        span = (n_q - 1) * 128 + 128
        tight = 19 * 128 + 128
        for r, h, ok in ((span, 128, True), (span - 8, 128, False), (128, tight, True), (128, tight - 8, False), (128, 128, False),
                         (256, 19 * 256 + 128, True), (256, 19 * 256 + 120, False), (1 << 41, 128, False), (128, 1 << 41, False)):
            x, y = rows(row_stride=r, head_stride=h), rows(row_stride=2048)
            if f == "attention":    # no workspace: a layout that passes is refused for that
                code = L.dflash_paged_attention(ref(cache()), ref(batch()), 0, n_q, ref(y), ref(x), None, 8, 0.1, 1, 0, None, 0, None)
            else:
                kv = (x, y) if f == "gather k" else (y, x)
                code = L.dflash_paged_gather(ref(cache()), ref(batch()), 0, ref(kv[0]), ref(kv[1]), None, 0, None)
            assert code == (-7 if ok else -2), (f, r, h)
    same = rows(row_stride=128, head_stride=128)       # rows that are only read may lie anywhere
    assert L.dflash_paged_append(ref(cache()), ref(batch()), 0, ref(same), ref(same), None, 0, None) == -7


def test_maps_refusals(L):
    out = dfl.dflash_paged_maps()
    for bad, code in BAD_CACHE:
        assert L.dflash_paged_cache_maps(ref(cache(**bad)), ref(out)) == code, bad
    assert L.dflash_paged_cache_maps(None, ref(out)) == -1 and L.dflash_paged_cache_maps(ref(cache()), None) == -1


def test_maps_of_a_cache_are_made_once_however_many_threads_ask(monkeypatch):
    """The address of one thread's maps must not be another's to free."""
    import threading
    import time
    made = []

    class Slow:
        def dflash_paged_cache_maps(self, cache, maps):
            time.sleep(0.05)
            made.append(maps)
            return 0
    monkeypatch.setattr(dfl, "lib", lambda: Slow())
    c = dfl.PagedCache(cache(), (), 0)
    got = []
    threads = [threading.Thread(target=lambda: got.append(c._with_maps())) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and len(got) == 4 and all(g is got[0] for g in got)


def test_logits_refusals(L):
    def call(B=2, G=4, V=100, t=2, z=P(1 << 20), l=(400, 100), out=P(1 << 22), o=(400, 100), ws=FAKE, n=256, none=False, **r):
        rules = dfl.dflash_logit_rules(**r)
        return L.dflash_logits_adjust(B, G, V, t, z, l[0], l[1], out, o[0], o[1], None if none else ref(rules), ws, n, None)
    assert call(B=0) == -2 and call(G=65) == -2 and call(V=0) == -2 and call(V=(1 << 18) + 1) == -2 and call(B=65536) == -2
    assert call(t=3) == -1 and call(z=None) == -1 and call(out=None) == -1 and call(none=True) == -1
    assert call(z=P((1 << 20) + 2)) == -3 and call(out=P((1 << 22) + 2)) == -3
    assert call(o=(400, 99)) == -2 and call(o=(399, 100)) == -2 and call(l=(-1, 100)) == -2
    assert call(counts=4096, slots=0) == -2 and call(counts=4098, slots=2) == -3
    assert call(bias_start=4096, n_bias=3) == -1 and call(bias_start=4096, n_bias=-1) == -2
    assert call(G=1, draft=4096) == -2
    # overlapping, but not the same tensor
    assert call(out=P((1 << 20) + 400)) == -1 and call(out=P(1 << 20), t=0) == -1 and call(out=P(1 << 20), o=(800, 200)) == -1
    assert call(ws=None) == -7 and call(n=255) == -7


def test_binding_checks_shapes_and_types():
    pages = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dfl.paged_cache(pages, pages[:2])
    with pytest.raises(ValueError):
        dfl.paged_cache(pages.float(), pages.float())
    with pytest.raises(ValueError):
        dfl.paged_cache(pages.transpose(1, 2), pages.transpose(1, 2))
    with pytest.raises(ValueError):
        dfl.paged_cache(pages, pages, torch.zeros(3, 2, 16), torch.zeros(3, 2, 16))
    codes = torch.zeros(3, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        dfl.paged_cache(codes, codes)
    with pytest.raises(ValueError):
        dfl.paged_cache(codes, codes, torch.zeros(3, 2, 8), torch.zeros(3, 2, 16))
    c = dfl.paged_cache(pages, pages)
    assert c.struct.page_size == 16 and c.struct.k_page_stride == 2 * 16 * 64 and c.struct.format == dfl.DFLASH_CACHE_BF16
    wide = torch.zeros(3, 2, 2, 16, 64, dtype=torch.bfloat16)
    c = dfl.paged_cache(wide[:, 0], wide[:, 1])
    assert c.struct.k_page_stride == 2 * 2 * 16 * 64
    with pytest.raises(ValueError):       # not on a GPU
        dfl.dflash_paged_append(c, torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 64, dtype=torch.bfloat16),
                                torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64),
                                torch.zeros(1, 1, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8))


@pytest.mark.parametrize("window,max_rows", [(1 << 32, 1), ((1 << 32) + 5, 1), (-1, 1), (0, (1 << 32) + 1), (0, -1)])
def test_binding_refuses_what_a_c_int_does_not_hold(window, max_rows):
    """ctypes would pass the lower 32 bits on: another window."""
    c = dfl.PagedCache(cache(), (), 0)
    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="max_rows and window"):
        dfl.dflash_paged_attention(c, q, q.clone(), None, None, None, max_rows, None, window=window)
