"""Calls of the 8-bit base that would leave the adapter out (no GPU)."""

import pytest

from bit_nf4_quantized_19_amd import ops


def test_an_adapter_without_its_alpha_is_refused():
    """With A and B and a default alpha of zero, Y would be the base's alone."""
    import torch
    bf = dict(dtype=torch.bfloat16)
    w = ops.Int8Weight.empty(64, 128, "cpu")
    X, A, B = torch.zeros(4, 128, **bf), torch.zeros(8, 128, **bf), torch.zeros(64, 8, **bf)
    with pytest.raises(ValueError, match="lora_alpha"):
        ops.linear_fwd_int8(w, X, A, B)
    # given, also as zero: the next check, that of the device
    for alpha in (16.0, 0.0):
        with pytest.raises(ValueError, match="CUDA tensor"):
            ops.linear_fwd_int8(w, X, A, B, alpha)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.linear_fwd_int8(w, X)
