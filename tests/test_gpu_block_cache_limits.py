"""The block cache's calls at the largest sizes that the header allows."""
import numpy as np
import pytest
import torch

from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache import bf16, err_word, i32, make_cache, to_gpu

pytestmark = pytest.mark.gpu


def test_select_over_the_longest_table():
    """2^26 blocks of 16, the longest table: one sequence that fills it, one short one."""
    rng = np.random.default_rng(0)
    hd, bs, n = 64, 16, 1 << 26
    c = make_cache(rng, 4, 1, bs, hd)
    c["mean"][0], c["mean"][1], c["mean"][2], c["mscale"][:] = 0, 127, 50, 0.01
    table = torch.zeros((2, n), dtype=torch.int32, device="cuda")
    for at, block in ((5_000_000, 2), (66_000_000, 1), (n - 2, 1)):
        table[0, at] = block
    table[1, 300], table[1, 7000] = 1, 2
    q, _ = bf16(np.ones((2, 1, 2, hd)))
    err = err_word()
    sel, _ = api.block_select(to_gpu(c), q, table, i32([n * bs, 7100 * bs - 3]), 8, dev_err=err)
    want = [[0, 1, 2, 3, 5_000_000, 66_000_000, n - 2, n - 1], [0, 1, 2, 3, 4, 300, 7000, 7099]]
    assert sel[:, 0, 0].tolist() == want and int(err.item()) == 0
