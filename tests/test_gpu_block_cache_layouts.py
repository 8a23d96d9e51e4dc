"""Strides that say nothing (dimensions of one element) and layouts of the block cache's inputs."""
import numpy as np
import pytest
import torch

import block_ref as R
from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache import batch, bf16, check_attn, i32, make_cache, run_attn, same_cache, to_gpu

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


def laid_out(c, how):
    """The cache c in one of the layouts that byte strides describe."""
    N, nkv, bs, hd = c["k"].shape
    k, v = torch.from_numpy(c["k"].copy()).cuda(), torch.from_numpy(c["v"].copy()).cuda()
    if how == "interleaved":  # K and V of a block side by side
        both = torch.stack((k, v), 1)
        k, v = both[:, 0], both[:, 1]
    elif how == "padded":  # rows of hd + 16 bytes, an unused block before the first
        both = torch.zeros((2, N + 1, nkv, bs, hd + 16), dtype=torch.uint8, device="cuda")
        both[0, 1:, ..., :hd], both[1, 1:, ..., :hd] = k, v
        k, v = both[0, 1:, ..., :hd], both[1, 1:, ..., :hd]
    elif how == "heads_first":  # all blocks of a head together
        k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v))
    elif how == "tokens_fused":  # [block, row, K and V, head, hd]
        both = torch.stack((k.transpose(1, 2), v.transpose(1, 2)), 2).contiguous()
        k, v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    f = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    return api.BlockCache(k, v, f(c["ks"]), f(c["vs"]), f(c["mean"]), f(c["mscale"]))


@pytest.mark.parametrize("hd,bs", [(64, 16), (128, 32), (256, 16)])
@pytest.mark.parametrize("how", ["interleaved", "padded", "heads_first", "tokens_fused"])
def test_layouts_of_the_cache(hd, bs, how):
    """Append, attention and attention over listed blocks where the codes' strides are not a plain tensor's."""
    rng = np.random.default_rng(hd + bs)
    B, T, nq, nkv, lens = 2, 3, 6, 3, [5 * bs + 4, 2 * bs]
    N = 9
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    cache = laid_out(c, how)
    kv, x = bf16(rng.normal(0, 1, (B, T, 2, nkv, hd)))
    api.block_append(cache, kv[:, :, 0], kv[:, :, 1], i32(table), i32(lens))
    R.append(c, x[:, :, 0], x[:, :, 1], table, lens)
    same_cache(cache, c)
    q, qf = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
    out, lse, om, err = run_attn(cache, q, table, lens, with_mass=True)
    check_attn(out, lse, R.attend(c, qf, table, lens), om)
    sel, _ = api.block_select(cache, q, i32(table), i32(lens), 3)
    want = R.select(c, qf, table, lens, 3, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want) and err == 0
    out, lse, _, err = run_attn(cache, q, table, lens, sel=sel)
    check_attn(out, lse, R.attend(c, qf, table, lens, sel=want))
    assert err == 0
