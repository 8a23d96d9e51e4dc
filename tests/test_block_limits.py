"""Limits of the block cache's entry points without a GPU: what they refuse, and the workspace sizes of
what they refuse. Every call here is refused on the host, before any CUDA call."""
import ctypes as C

import pytest

from mtp_speculative_draft_lm_b200 import _lib as L
from test_block_abi import UNS, WS, append, attn, cache, lib, select  # noqa: F401 (lib: builds and loads)


@pytest.mark.parametrize("num_blocks,stride", [((1 << 31) - 1, (1 << 39) - 16), ((1 << 31) - 1, 1 << 38), (1 << 30, 1 << 32),
                                               (1 << 22, (1 << 39) - 16)])
def test_codes_past_64_bit_offsets(num_blocks, stride):
    """Block strides whose product with the blocks passes 2^60 bytes, 2^64 too."""
    c = cache(num_blocks=num_blocks, block_stride=stride)
    assert append(c) == attn(c) == attn(c, sel=0x20000, n_sel=4) == UNS


def attn_ws(c, B, T, nq, n_table, mass=0):
    return L.load().mtp_block_attn_ws_bytes(C.byref(c), B, T, nq, n_table, mass)


def sparse_ws(c, B, T, nq, n_sel):
    return L.load().mtp_block_sparse_attn_ws_bytes(C.byref(c), B, T, nq, n_sel)


def test_attention_past_its_line():
    """1,024 sequences of 8 heads: 2^13 units of one row tile, whose tiles and 12 more each stay below 2^31."""
    c, most = cache(), (1 << 18) - 13
    assert attn_ws(c, 1024, 1, 64, most) > 0 and attn(c, nb=1024, T=1, n_table=most, ws=None) == WS
    for nbytes in (None, 0, 1 << 62):
        assert attn(c, nb=1024, T=1, n_table=most + 1, nbytes=nbytes) == UNS
    assert attn_ws(c, 1024, 1, 64, most + 1) == attn_ws(c, 1024, 1, 64, most + 1, 1) == 0
    # listed blocks: a unit for each token and head
    assert sparse_ws(c, 256, 4, 64, most) > 0 and attn(c, nb=256, T=4, sel=0x20000, n_sel=most, ws=None) == WS
    for nbytes in (None, 0, 1 << 62):
        assert attn(c, nb=256, T=4, sel=0x20000, n_sel=most + 1, nbytes=nbytes) == UNS
    assert sparse_ws(c, 256, 4, 64, most + 1) == 0


def test_rows_past_32_bits():
    wide = dict(stride=1 << 17, n_table=1)
    for nkv, fits in ((32, True), (33, False)):  # 16 query heads each: 65,535 x 64 x 512 rows are the most
        c, nq = cache(nkv=nkv), 16 * nkv
        assert (attn_ws(c, 65535, 64, nq, 1) > 0) == (sparse_ws(c, 65535, 64, nq, 1) > 0) == fits
        for f in (attn, lambda c, **kw: attn(c, sel=0x20000, n_sel=1, **kw)):
            for nbytes in (0, 1 << 62) if not fits else (0,):
                assert f(c, nb=65535, T=64, nq=nq, nbytes=nbytes, **wide) == (WS if fits else UNS)
    for nkv, fits in ((512, True), (513, False)):
        c = cache(nkv=nkv)
        assert (L.load().mtp_block_select_ws_bytes(C.byref(c), 65535, 64, 10) > 0) == fits
        for nbytes in (0, 1 << 62) if not fits else (0,):
            assert select(c, nb=65535, T=64, nq=nkv, nbytes=nbytes, stride=1 << 17) == (WS if fits else UNS)
