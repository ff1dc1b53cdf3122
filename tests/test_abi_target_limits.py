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
