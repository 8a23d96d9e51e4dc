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
