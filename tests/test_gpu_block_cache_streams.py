"""The block cache's helpers with a `stream` argument: whose memory the outputs are, and what is kept while
the call still uses it."""
import numpy as np
import pytest
import torch

from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache_use import bits, outputs, step, step_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("current", ["default", "other"])
def test_address_zero_is_the_default_stream(current):
    """Outputs of a call on address 0 are the default stream's memory: what it gives back it hands out next."""
    n = 37 << 20
    with torch.cuda.stream(torch.cuda.Stream() if current == "other" else torch.cuda.default_stream()):
        t = api._new((n,), torch.uint8, 0, 0)
    at = t.data_ptr()
    torch.cuda.synchronize()
    del t
    assert torch.empty((n,), dtype=torch.uint8, device="cuda").data_ptr() == at
    st = outputs(step_state(np.random.default_rng(1)))
    step(st, None)
    torch.cuda.synchronize()
    want = bits(*st["o"].values())
    out, _ = api.block_attn(st["cache"], st["q"], st["table"], st["lens"], stream=0)
    sel, _ = api.block_select(st["cache"], st["q"], st["table"], st["lens"], 4, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(sel, want[3])


@pytest.mark.parametrize("by", ["object", "address"])
def test_inputs_let_go_while_the_call_waits(by):
    """Inputs and workspaces let go after calls on a stream that is still busy: their
    memory is not handed out again before the calls have read it."""
    rng = np.random.default_rng(3)
    st = outputs(step_state(rng, B=2, T=3, nq=16, nkv=2, hd=128, lens=(900, 333)))
    o, mk = st["o"], lambda: {k: st[k].clone() for k in ("q", "k", "v", "table", "lens", "mass")}  # noqa: E731
    base = [None if t is None else t.clone() for t in st["cache"].tensors()]
    step(st, None)
    torch.cuda.synchronize()
    want = bits(*o.values()) + bits(*st["cache"].tensors())
    s = torch.cuda.Stream()
    arg = s if by == "object" else s.cuda_stream
    for _ in range(3):
        cache, a = api.BlockCache(*(t.clone() for t in base)), mk()
        ws = torch.empty((32 << 20,), dtype=torch.uint8, device="cuda")
        for t in o.values():
            t.zero_()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)  # some 50 ms
        api.block_append(cache, a["k"], a["v"], a["table"], a["lens"], stream=arg)
        api.block_attn(cache, a["q"], a["table"], a["lens"], out=o["out"], out_lse=o["lse"], mass=a["mass"], out_mass=o["mass"],
                       ws=ws, stream=arg)
        api.block_select(cache, a["q"], a["table"], a["lens"], 4, out=o["sel"], ws=ws, stream=arg)
        api.block_sparse_attn(cache, a["q"], a["table"], a["lens"], o["sel"], out=o["sparse"], ws=ws, stream=arg)
        mass = o["mass"].clone()  # (the current stream's: zeros, as the calls wait)
        api.block_evict(a["table"], a["lens"], mass, 16, 3, out_table=o["table"], out_lens=o["lens"], out_mass=o["left"],
                        freed=o["freed"], n_freed=o["n_freed"], stream=arg)
        codes = list(cache.tensors())
        sizes = [(t.shape, t.dtype) for t in a.values()] + [(ws.shape, ws.dtype), (mass.shape, mass.dtype)]
        del cache, a, ws, mass
        # what the allocator would hand out in their place, overwritten on the current stream
        junk = [torch.full(shape, 1, dtype=dt, device="cuda") for shape, dt in sizes for _ in range(2)]
        torch.cuda.synchronize()
        got = bits(*(o[n] for n in ("out", "lse", "mass", "sel", "sparse"))) + bits(*codes)
        for x, y in zip(got, want[:5] + want[10:]):
            assert torch.equal(x, y)
        del junk, codes
