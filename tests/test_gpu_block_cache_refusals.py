"""Refused calls of the block cache's helpers launch nothing: the error word, every output that was
given and the cache are as they were."""
import numpy as np
import pytest
import torch

from mtp_speculative_draft_lm_b200 import _lib as L
from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache import err_word, i32
from test_gpu_block_cache_use import bits, outputs, step_state

pytestmark = pytest.mark.gpu


def test_nothing_changes_where_a_call_is_refused():
    st = outputs(step_state(np.random.default_rng(11)))
    ca, q, tab, lens, o, mass = st["cache"], st["q"], st["table"], st["lens"], st["o"], st["mass"]
    k, v = st["k"], st["v"]
    # every call below would flag the missing block if it ran
    tab = tab.clone()
    tab[:, 0] = -1
    err = err_word()
    for t in o.values():
        t.fill_(7)
    kw = dict(dev_err=err)
    at = dict(out=o["out"], out_lse=o["lse"], mass=mass, out_mass=o["mass"], **kw)
    ev = dict(out_table=o["table"], out_lens=o["lens"], out_mass=o["left"], freed=o["freed"], n_freed=o["n_freed"])
    no_means = api.BlockCache.of(ca.k, ca.v, ca.k_scale, ca.v_scale)
    small = torch.empty((1,), dtype=torch.uint8, device="cuda")
    value = [
        lambda: api.block_append(ca, k, v[:, :1], tab, lens, **kw), lambda: api.block_append(ca, k, v.float(), tab, lens, **kw),
        lambda: api.block_append(ca, q, q, tab, lens, **kw), lambda: api.block_append(ca, k, v, tab.long(), lens, **kw),
        lambda: api.block_append(ca, k, v, tab, lens, q_lens=lens[:1], **kw), lambda: api.block_append(ca, k, None, tab, lens, **kw),
        lambda: api.block_attn(ca, q, tab, lens[:2], **at), lambda: api.block_attn(ca, q, tab, lens.float(), **at),
        lambda: api.block_attn(ca, q.float(), tab, lens, **at), lambda: api.block_attn(ca, q, tab[:, :1], lens, **at),
        lambda: api.block_attn(ca, q, tab, lens, **{**at, "out_lse": mass}), lambda: api.block_attn(ca, q, tab, lens, **{**at, "mass": o["lens"]}),
        lambda: api.block_attn(ca, q, tab, lens, **{**at, "out": o["sel"]}),
        lambda: api.block_select(ca, q, tab, lens, 5, out=o["sel"], **kw), lambda: api.block_select(ca, q.half(), tab, lens, 4, out=o["sel"], **kw),
        lambda: api.block_sparse_attn(ca, q, tab, lens, o["sel"].long(), out=o["sparse"], **kw),
        lambda: api.block_sparse_attn(ca, q, tab, lens, o["sel"][0], out=o["sparse"], **kw),
        lambda: api.block_evict(tab, lens, mass, 16, 3, **{**ev, "freed": o["lens"]}),
        lambda: api.block_evict(tab, lens, mass.half(), 16, 3, **ev)]
    status = [
        lambda: api.block_attn(ca, q, tab, lens, **{**at, "out_mass": None}), lambda: api.block_attn(ca, q, tab, lens, scale=-1.0, **at),
        lambda: api.block_attn(ca, q, tab, lens, scale=float("nan"), ws=small, **at), lambda: api.block_attn(ca, q[:, :, :7], tab, lens, **kw),
        lambda: api.block_select(no_means, q, tab, lens, 4, out=o["sel"], **kw),
        lambda: api.block_select(ca, q, tab, lens, 4, n_first=3, n_last=2, out=o["sel"], **kw),
        lambda: api.block_select(ca, q, tab, lens, 4, n_first=-1, out=o["sel"], **kw),
        lambda: api.block_sparse_attn(ca, q, tab, lens, o["sel"], scale=float("inf"), out=o["sparse"], **kw),
        lambda: api.block_evict(tab, lens, mass, 16, 1, **ev), lambda: api.block_evict(tab, lens, mass, 0, 3, **ev),
        lambda: api.block_evict(tab, lens, mass, 16, 3, n_last=0, **ev)]
    torch.cuda.synchronize()
    watched = [err, tab, lens, mass, q, k, v, *o.values(), *ca.tensors()]
    before = bits(*watched)
    for kind, calls in ((ValueError, value), (L.MtpError, status)):
        for i, f in enumerate(calls):
            with pytest.raises(kind):
                f()
                pytest.fail(f"{kind.__name__} call {i} was not refused")
            torch.cuda.synchronize()
            for a, b in zip(watched, before):
                assert torch.equal(a, b), (kind, i)
    # and the same error word and outputs do change where a call runs
    api.block_attn(ca, q, tab, lens, **at)
    api.block_evict(tab, i32(lens.tolist()), mass, 16, 3, **ev)
    torch.cuda.synchronize()
    assert int(err.item()) == L.MTP_DEVFLAG_BAD_SLOT
    assert not bool((o["out"] == 7).all()) and not bool((o["freed"] == 7).all())
