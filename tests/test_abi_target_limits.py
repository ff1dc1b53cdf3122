"""Host-side limits of the target-side entry points (no call here reaches a
GPU)."""

import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl


@pytest.mark.parametrize("shape", [(1, 1, (1 << 32) + 100), (1, (1 << 32) + 2, 100), ((1 << 32) + 1, 1, 100), (1, 1, 1 << 31)])
def test_binding_refuses_logits_whose_sizes_a_c_int_does_not_hold(shape):
    """ctypes would pass the lower 32 bits on: part of the logits."""
    z = torch.empty(shape, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        dfl.dflash_logits_adjust(z, z, torch.zeros(256, dtype=torch.uint8))


def test_binding_refuses_a_workspace_question_whose_sizes_a_c_int_does_not_hold():
    for args in ((8, 2, 64, (1 << 32) + 1), ((1 << 32) + 8, 2, 64, 1), (8, 2, (1 << 32) + 64, 1), (8, 2, 64, -(1 << 32))):
        with pytest.raises(ValueError, match="2\\^31"):
            dfl.dflash_paged_attention_workspace_bytes(*args)


def test_binding_refuses_biases_without_all_their_parts():
    """Half a rule would be dropped, and its values with it."""
    z = torch.empty(2, 3, 100, device="meta")
    parts = dict(bias_start=torch.zeros(3, dtype=torch.int32), bias_ids=torch.zeros(4, dtype=torch.int32), bias_vals=torch.zeros(4))
    for left_out in (("bias_start",), ("bias_ids",), ("bias_vals",), ("bias_start", "bias_vals"), ("bias_ids", "bias_vals")):
        with pytest.raises(ValueError, match="bias_start, bias_ids and bias_vals"):
            dfl.dflash_logits_adjust(z, z, torch.zeros(256, dtype=torch.uint8),
                                     **{k: v for k, v in parts.items() if k not in left_out})


def test_limits_that_the_header_names_are_the_ones_that_are_kept():
    """At a limit a call gets as far as its workspace (none here: -7), past it
    the size is refused (-2)."""
    import ctypes
    L, ref = dfl.lib(), ctypes.byref
    P = ctypes.c_void_p

    def paged(call, n_kv=2, stride=1 << 20, B=3, pages=8, rows=20, row_stride=1 << 20, n_q=None, max_rows=8):
        c = dfl.dflash_paged_cache(4096, 4096, None, None, stride, stride, 10, n_kv, 16, 64, 0, None)
        b = dfl.dflash_paged_batch(4096, 4096, 4096, pages, B, pages, rows)
        x = dfl.dflash_rows(4096, row_stride, 64)
        if call == "attention":
            return L.dflash_paged_attention(ref(c), ref(b), 0, n_q or n_kv, ref(x), ref(x), None, max_rows, 0.1, 1, 0, None, 0, None)
        return L.dflash_paged_append(ref(c), ref(b), 0, ref(x), ref(x), None, 0, None)

    for call in ("append", "attention"):
        for at, past in ((dict(n_kv=4096, stride=1 << 22), dict(n_kv=4097, stride=1 << 24)),
                         (dict(stride=1 << 38), dict(stride=(1 << 38) + 8)), (dict(B=65535), dict(B=65536)),
                         (dict(pages=(1 << 26) - 1), dict(pages=1 << 26)), (dict(rows=1 << 30), dict(rows=(1 << 30) + 1)),
                         (dict(row_stride=1 << 40), dict(row_stride=(1 << 40) + 8))):
            assert paged(call, **at) == -7 and paged(call, **past) == -2, (call, past)
    assert paged("attention", n_kv=1, n_q=65535, row_stride=1 << 23) == -7
    assert paged("attention", n_kv=1, n_q=65536, row_stride=1 << 23) == -2
    assert paged("attention", n_q=4, rows=1 << 30, max_rows=1 << 29) == -7
    assert paged("attention", n_q=4, rows=1 << 30, max_rows=(1 << 29) + 1) == -2

    def adjust(B=1, G=1, V=100, l=1 << 20, **r):
        rules = dfl.dflash_logit_rules(**r)
        return L.dflash_logits_adjust(B, G, V, 2, P(1 << 40), l, l, P(1 << 50), 1 << 20, (1 << 20) * B, ref(rules), None, 0, None)

    for at, past in ((dict(G=64), dict(G=65)), (dict(B=65535), dict(B=65536)), (dict(B=1024, G=63), dict(B=1024, G=64)),
                     (dict(V=1 << 18), dict(V=(1 << 18) + 1)), (dict(l=1 << 40), dict(l=(1 << 40) + 1)),
                     (dict(G=2, draft=4096), dict(G=1, draft=4096))):
        assert adjust(**at) == -7 and adjust(**past) == -2, past


def test_binding_takes_a_page_table_of_one_column_whatever_its_stride():
    """A column's stride says nothing where there is one column."""
    start, lens = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    table = torch.tensor([[3, 0, 2]], dtype=torch.int32)
    assert table.t().stride() == (1, 3)
    packed = dfl._batch(start, lens, table.t(), 5, -1)
    assert packed == dfl._PACK_BATCH(start.data_ptr(), lens.data_ptr(), table.data_ptr(), 1, 3, 1, 5)
    with pytest.raises(ValueError):
        dfl._batch(start, lens, torch.zeros(2, 3, dtype=torch.int32).t(), 5, -1)
