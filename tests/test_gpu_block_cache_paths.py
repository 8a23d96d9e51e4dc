"""Paths of the block attention that other tests pass by: listed blocks of more sequences than a warp looks
at at once, and codes that are NaN for every head width and call."""
import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_block_cache import batch, bf16, check_attn, make_cache, run_attn, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,nq,nkv,hd,bs,n_sel", [(33, 1, 8, 2, 64, 16, 40), (70, 3, 6, 3, 64, 32, 12), (50, 2, 16, 1, 128, 16, 9),
                                                    (40, 1, 2, 2, 256, 64, 5), (300, 1, 4, 2, 64, 16, 8)])
def test_listed_blocks_of_many_sequences(B, T, nq, nkv, hd, bs, n_sel):
    """Ragged token counts, empty slots, lists with gaps; one long list among short ones, so that units are
    split over several CTAs."""
    rng = np.random.default_rng(B + hd)
    q_lens = [int(rng.integers(0, T + 1)) if b % 4 else T for b in range(B)]
    lens = [max(q_lens[b], int(rng.integers(0, 12 * bs)) if b % 7 else 3) for b in range(B)]
    lens[B // 2] = n_sel * bs + 5
    lens[5] = q_lens[5] = 0
    N = sum(-(-n // bs) for n in lens) + 2
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    sel = np.full((B, T, nkv, n_sel), -1, np.int32)
    for b in range(B):
        nb = -(-lens[b] // bs)
        for t in range(T):
            for g in range(nkv):
                pick = rng.permutation(nb)[:n_sel] if nb else np.zeros(0, int)
                at = np.sort(rng.permutation(n_sel)[:len(pick)])
                sel[b, t, g, at] = pick
    q, qf = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
    out, lse, _, err = run_attn(to_gpu(c), q, table, lens, q_lens, sel=torch.from_numpy(sel).cuda())
    ref = R.attend(c, qf, table, lens, q_lens, sel=sel)
    check_attn(out, lse, ref)
    assert err == 0
    dead = ~torch.from_numpy(ref["live"]).cuda()
    assert bool((out[dead] == 7.0).all()) and bool((lse[dead] == 7.0).all())


@pytest.mark.parametrize("hd,nq,nkv", [(64, 8, 2), (64, 2, 1), (128, 12, 2), (256, 8, 2), (256, 16, 1), (64, 26, 2)])
@pytest.mark.parametrize("sparse", [False, True], ids=["dense", "listed"])
def test_nan_codes_reach_the_rows_that_see_them(hd, nq, nkv, sparse):
    """NaN codes behind the sequences and in rows that earlier tokens do not see: every dimension of V in turn
    has one, at positions over the whole tile."""
    rng = np.random.default_rng(hd + nq)
    B, T, bs, G = 2, 8, 16, nq // nkv
    lens = [16 * 5, 16 * 2 + 11]
    c = make_cache(rng, 9, nkv, bs, hd)
    table = batch(rng, lens, bs, 9, n_table=6)
    for b, n in enumerate(lens):
        if n % bs:
            c["k"][table[b, n // bs], :, n % bs:] = 0x7F
            c["v"][table[b, n // bs], :, n % bs:] = 0xFF
    clean = {k: a.copy() for k, a in c.items()}
    # sequence 0: dimension d of V has a NaN at position 72 + d % 8, its token d % 8's own row, on the last kv head
    # (tokens are positions 72 .. 79); K has one in token 6's row of kv head 0 where there are two heads
    for d in range(hd):
        p = 72 + d % 8
        c["v"][table[0, p // bs], nkv - 1, p % bs, d] = 0x7F if d % 2 else 0xFF
    if nkv > 1:
        c["k"][table[0, 78 // bs], 0, 78 % bs, hd - 3] = 0xFF
    # sequence 1: its tile's rows 0, 3, .. of the last block (positions 35 .. 42 are tokens): position 40
    c["v"][table[1, 40 // bs], 0, 40 % bs, :: 3] = 0x7F
    sel = None
    if sparse:
        lists = np.full((B, T, nkv, 7), -1, np.int32)
        lists[0, :, :, 1:6] = np.arange(5)
        lists[1, :, :, 2:5] = np.arange(3)
        sel = torch.from_numpy(lists).cuda()
    q, qf = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
    out, lse, _, err = run_attn(to_gpu(c), q, table, lens, sel=sel)
    ref = R.attend(clean, qf, table, lens)
    hit = np.zeros((B, T, nq, hd), bool)
    for d in range(hd):
        hit[0, d % 8:, (nkv - 1) * G:, d] = True
    hit[1, 40 - 35:, :G, :: 3] = True
    no_lse = np.zeros((B, T, nq), bool)
    if nkv > 1:
        hit[0, 6:, :G], no_lse[0, 6:, :G] = True, True
    o = out.float().cpu().numpy()
    assert np.isnan(o[hit]).all() and np.isfinite(o[~hit]).all()
    ref["out"][hit], ref["out_tol"][hit] = 0, np.inf
    o[hit] = 0
    l = lse.cpu().numpy()
    assert np.isnan(l[no_lse]).all()
    l[no_lse], ref["lse"][no_lse] = 0, 0
    check_attn(torch.from_numpy(o), torch.from_numpy(l), ref)
    assert err == 0
