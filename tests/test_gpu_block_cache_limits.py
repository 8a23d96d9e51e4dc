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


def test_the_most_sequences():
    """65,535 sequences of 0 to 40 positions over a few shared blocks: the same bits as the sequence of that
    length alone; and each with a block of its own that a token is appended to."""
    rng = np.random.default_rng(1)
    B, nkv, hd, bs = 65535, 1, 64, 16
    c = make_cache(rng, 6, nkv, bs, hd)
    cache = to_gpu(c)
    row = np.array([4, 0, 3], np.int32)
    table = i32(row[None]).expand(B, 3).contiguous()
    n = rng.integers(0, 41, B)
    lens = i32(n)
    q1, _ = bf16(rng.normal(0, 1.5, (1, 1, 2, hd)))
    q = q1.expand(B, 1, 2, hd).contiguous()
    om = torch.empty((B, 3), device="cuda")
    out, ws = api.block_attn(cache, q, table, lens, out_mass=om)
    sel, ws = api.block_select(cache, q, table, lens, 2, ws=ws)
    sp, ws = api.block_sparse_attn(cache, q, table, lens, sel, ws=ws)
    t2, l2, m2, freed, nf = api.block_evict(table, lens, om, bs, 2)
    for length in (0, 1, 16, 17, 40):
        who = torch.from_numpy(np.flatnonzero(n == length)).cuda()
        one = torch.empty((1, 3), device="cuda")
        t, le = i32(row[None]), i32([length])
        o, _ = api.block_attn(cache, q1, t, le, out_mass=one)
        s, _ = api.block_select(cache, q1, t, le, 2)
        p, _ = api.block_sparse_attn(cache, q1, t, le, s)
        ev = api.block_evict(t, le, one, bs, 2)
        # (the parts of a sequence that several CTAs share are joined in another order: a bf16 step)
        for many, alone in ((out, o), (sp, p)):
            assert float((many[who].float() - alone.float()).abs().max()) <= 2.0 ** -7 * float(alone.float().abs().max())
        assert float((om[who] - one).abs().max()) <= 1e-5
        assert bool((sel[who] == s).all())
        for many, alone in zip((t2, l2, freed, nf), (ev[0], ev[1], ev[3], ev[4])):
            assert bool((many[who] == alone).all())
    own = api.BlockCache.empty(B, nkv, hd, bs)
    x, _ = bf16(rng.normal(0, 1, (B, 1, nkv, hd)))
    api.block_append(own, x, x, torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(), i32(np.full(B, 1)))
    got = own.k[:, 0, 0].view(torch.float8_e4m3fn).float() * own.k_scale
    want = x[:, 0, 0].float()
    # half a step of E4M3, 2^-4, or 2^-10 of the scale near zero
    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -4 + own.k_scale * 2.0 ** -10).all())
    assert bool((own.k[:, 0, 1:] == 0).all())
