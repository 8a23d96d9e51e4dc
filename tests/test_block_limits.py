"""Limits of the block cache's entry points without a GPU: what they refuse, and the workspace sizes of
what they refuse. Every call here is refused on the host, before any CUDA call."""
import ctypes as C

import pytest

from mtp_speculative_draft_lm_b200 import _lib as L
from test_block_abi import UNS, append, attn, cache, lib  # noqa: F401 (lib: builds and loads)


@pytest.mark.parametrize("num_blocks,stride", [((1 << 31) - 1, (1 << 39) - 16), ((1 << 31) - 1, 1 << 38), (1 << 30, 1 << 32),
                                               (1 << 22, (1 << 39) - 16)])
def test_codes_past_64_bit_offsets(num_blocks, stride):
    """Block strides whose product with the blocks passes 2^60 bytes, 2^64 too."""
    c = cache(num_blocks=num_blocks, block_stride=stride)
    assert append(c) == attn(c) == attn(c, sel=0x20000, n_sel=4) == UNS
