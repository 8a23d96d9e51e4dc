"""Strides that say nothing (dimensions of one element) and layouts of the block cache's inputs."""
import numpy as np
import pytest
import torch

import block_ref as R
from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache import batch, bf16, i32, make_cache, same_cache, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,nkv", [(1, 1, 2), (1, 1, 1), (1, 5, 1), (3, 1, 1), (1, 5, 2), (3, 1, 2)])
def test_append_of_tensors_of_different_strides(B, T, nkv):
    """k and v whose strides differ in dimensions of one element alone: rows of a wider buffer and packed ones."""
    rng = np.random.default_rng(B + T + nkv)
    hd, bs, lens = 64, 16, [20 + T + b for b in range(B)]
    N = 4 * B
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    k, kf = bf16(rng.normal(0, 1, (B, T, nkv, hd)))
    v, vf = bf16(rng.normal(0, 1, (B, T, nkv, hd)))
    wide = [n + 3 if n == 1 else n for n in (B, T, nkv)]
    big = torch.zeros((*wide, hd), dtype=torch.bfloat16, device="cuda")
    # (dimensions longer than one keep k's strides: only those of one element differ)
    odd = torch.as_strided(big, (B, T, nkv, hd), [s if n > 1 else s * 8 + 8 for n, s in zip((B, T, nkv, hd), k.stride())])
    odd.copy_(v)
    assert odd.stride() != k.stride()
    cache = to_gpu(c)
    api.block_append(cache, k, odd, i32(table), i32(lens))
    R.append(c, kf, vf, table, lens)
    same_cache(cache, c)


def test_append_refuses_strides_that_differ():
    rng = np.random.default_rng(0)
    c = to_gpu(make_cache(rng, 4, 2, 16, 64))
    table, lens = i32([[0, 1], [2, 3]]), i32([5, 7])
    k = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16, device="cuda")
    fused = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    for v in (fused[:, :, :2], k[:, :2], k.float(), k.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            api.block_append(c, k, v, table, lens)
