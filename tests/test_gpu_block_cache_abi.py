"""The block cache's entry points through the ctypes binding (_lib), as programs without api.py call them:
the same bits as api.py's calls."""
import math

import numpy as np
import pytest
import torch

from mtp_speculative_draft_lm_b200 import _lib as L
from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache import err_word
from test_gpu_block_cache_use import bits, outputs, step, step_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("other_stream", [False, True])
def test_the_binding_gives_the_same_bits(other_stream):
    rng = np.random.default_rng(4)
    st = outputs(step_state(rng, B=3, T=2, nq=12, nkv=2, hd=64, lens=(400, 18, 77)))
    ca, q, tab, lens, o = st["cache"], st["q"], st["table"], st["lens"], st["o"]
    base = bits(*ca.tensors())
    step(st, None)
    torch.cuda.synchronize()
    want = bits(*o.values(), *ca.tensors())
    for t, b in zip(ca.tensors(), base):
        t.copy_(b)
    for t in o.values():
        t.zero_()
    err = err_word()
    B, T, nq, hd = q.shape
    n_table, n_sel, scale = tab.shape[1], 4, 1.0 / math.sqrt(hd)
    need = [L.mtp_block_attn_ws_bytes(ca.desc, B, T, nq, n_table, True), L.mtp_block_select_ws_bytes(ca.desc, B, T, n_table),
            L.mtp_block_sparse_attn_ws_bytes(ca.desc, B, T, nq, n_sel)]
    ws = [torch.empty((n,), dtype=torch.uint8, device="cuda") for n in need]
    s = torch.cuda.Stream() if other_stream else None
    torch.cuda.synchronize()
    L.mtp_block_append(ca.desc, st["k"], st["v"], st["k"].stride(1), B, T, lens, None, tab, n_table, err, s)
    L.mtp_block_attn(ca.desc, q, nq * hd, B, T, nq, lens, None, tab, n_table, scale, o["out"], o["lse"], st["mass"], o["mass"], err,
                     ws[0], need[0], s)
    L.mtp_block_select(ca.desc, q, nq * hd, B, T, nq, lens, None, tab, n_table, n_sel, 1, 1, o["sel"], err, ws[1], need[1], s)
    L.mtp_block_sparse_attn(ca.desc, q, nq * hd, B, T, nq, lens, None, tab, n_table, o["sel"], n_sel, scale, o["sparse"], None, err,
                            ws[2], need[2], s)
    L.mtp_block_evict(B, tab, n_table, lens, o["mass"], 16, 3, 1, 1, o["table"], o["lens"], o["left"], o["freed"], o["n_freed"], s)
    torch.cuda.synchronize()
    for a, b in zip(bits(*o.values(), *ca.tensors()), want):
        assert torch.equal(a, b)
    assert int(err.item()) == 0
    for n, name in ((need[0], "attn"), (need[2], "sparse_attn")):
        with pytest.raises(L.MtpError) as e:
            args = (o["sel"], n_sel, scale) if name == "sparse_attn" else (scale,)
            outs = (o["out"], None) if name == "sparse_attn" else (o["out"], None, st["mass"], o["mass"])
            getattr(L, "mtp_block_" + name)(ca.desc, q, nq * hd, B, T, nq, lens, None, tab, n_table, *args, *outs, err, ws[0], n - 16, s)
        assert e.value.status == L.MTP_ERR_WORKSPACE
    assert api.BlockCache.of(*ca.tensors()).desc.num_blocks == ca.desc.num_blocks
