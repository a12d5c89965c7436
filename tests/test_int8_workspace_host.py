"""A workspace of the 8-bit base serves every shorter batch (no GPU)."""

import pytest

from bit_nf4_quantized_19_amd import ops

SHAPES = [(64, 64), (8, 4096), (520, 1088), (4096, 4096), (11008, 4096), (4096, 11008),
          (8192, 22016), (1000, 131072), (131072, 192)]


@pytest.mark.parametrize("d,k", SHAPES)
@pytest.mark.parametrize("r", [0, 16, 128])
@pytest.mark.parametrize("op", [ops.OP_FWD, ops.OP_BWD])
def test_sizes_do_not_fall_with_more_tokens(op, d, k, r):
    tokens = sorted({m + o for m in [1, 16, 32, 64, 96, 128, 192] + list(range(256, 2305, 128)) +
                     [4096, 8192, 65536, 1 << 20] for o in (-1, 0, 1) if 1 <= m + o <= 1 << 20})
    sizes = [ops.int8_workspace_bytes(op, d, k, M, r) for M in tokens]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), [
        (tokens[i], sizes[i], tokens[i + 1], sizes[i + 1]) for i in range(len(sizes) - 1)
        if sizes[i] > sizes[i + 1]]


@pytest.mark.parametrize("d,k", SHAPES)
@pytest.mark.parametrize("M", [1, 17, 65, 300, 2048])
@pytest.mark.parametrize("op", [ops.OP_FWD, ops.OP_BWD])
def test_sizes_do_not_fall_with_more_ranks(op, d, k, M):
    sizes = [ops.int8_workspace_bytes(op, d, k, M, r) for r in range(129)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
