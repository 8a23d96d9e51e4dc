"""Small softmax weights of blocks whose V scales lie below an earlier block's: what each block adds
keeps its accuracy in the dimensions that it alone fills."""
import math

import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_block_cache import batch, bf16, run_attn, to_gpu

pytestmark = pytest.mark.gpu


def sink_cache(rng, nb, nkv, hd, bs, sink, top, scales):
    """Blocks of small K and random V. Row 3 of block `sink` has a key `top` nats above the rest, and that
    block's V is zero in the first half of the dimensions. V scales: 1 there, `scales` in turn elsewhere."""
    k = R.encode(rng.uniform(-0.25, 0.25, (nb, nkv, bs, hd)))
    v = R.encode(rng.uniform(64, 448, (nb, nkv, bs, hd)) * rng.choice([-1.0, 1.0], (nb, nkv, 1, hd)))
    k[sink, :, 3] = R.encode(np.full((nkv, hd), top))
    v[sink, :, :, :hd // 2] = 0
    vs = np.array([scales[n % len(scales)] for n in range(nb)], np.float32)[:, None].repeat(nkv, 1)
    vs[sink] = 1.0
    return dict(k=k, v=v, ks=np.ones((nb, nkv), np.float32), vs=vs, mean=np.zeros((nb, nkv, hd), np.int8),
                mscale=np.zeros((nb, nkv), np.float32))


@pytest.mark.parametrize("hd,G,T", [(64, 1, 1), (64, 8, 5), (128, 8, 1), (128, 12, 1), (128, 16, 2), (256, 4, 1), (256, 16, 1)])
@pytest.mark.parametrize("nb,sink,top,exps", [
    (2, 0, 12.0, (-9,)), (2, 1, 12.0, (-9,)), (40, 0, 12.0, (-10, -9, -3)), (40, 17, 10.0, (-40, -41)), (300, 5, 14.0, (-5, -7, -2)),
    (12, 3, 12.0, (0,))])
def test_small_weights_of_small_scales(hd, G, T, nb, sink, top, exps):
    rng = np.random.default_rng(hd + G + nb)
    nkv, bs = 2, 16
    c = sink_cache(rng, nb, nkv, hd, bs, sink, top, [2.0 ** e for e in exps])
    n = nb * bs
    table = np.arange(nb, dtype=np.int32)[None]
    q, qf = bf16(rng.uniform(0.9, 1.1, (1, T, nkv * G, hd)))
    scale = 1.0 / hd
    lists = np.tile(np.arange(nb, dtype=np.int32), (1, T, nkv, 1))
    for sel in (None, torch.from_numpy(lists).cuda()):
        out, lse, _, _ = run_attn(to_gpu(c), q, table, [n], sel=sel, scale=scale)
        got = out.float().cpu().numpy().astype(np.float64)
        K = R.decode(c["k"]).astype(np.float64)
        V = R.decode(c["v"]).astype(np.float64) * c["vs"][..., None, None]
        for t in range(T):
            lim = n - T + t + 1
            for i in range(nkv * G):
                g = i // G
                k, v = K[:, g].reshape(n, hd)[:lim], V[:, g].reshape(n, hd)[:lim]
                s = scale * (k @ qf[0, t, i].astype(np.float64))
                m = s.max()
                w = np.exp(s - m)
                l = w.sum()
                want = (w / l) @ v
                # a score: hd products and sums in fp32, its scales; 2^x of a difference, to 2^-22
                e = ((hd + 8) * 2.0 ** -23 * scale * (np.abs(k) @ np.abs(qf[0, t, i])) + 2.0 ** -22 * (np.abs(s - m) + 1)).max()
                # weights: at least four times their size in f16's range, so half a step is 2^-11 of a
                # weight or 2^-27 of the row's largest one, in units of the block's own scale
                lim_e = (2.0 ** -8 * np.abs(want) + ((w / l) @ np.abs(v)) * (2.0 ** -11 + 4 * e + 4 * (lim + 64) * 2.0 ** -24)
                         + 2.0 ** -27 / l * np.abs(v).sum(0) + 1e-37)
                err = np.abs(got[0, t, i] - want)
                assert np.all(err <= lim_e), (sel is not None, t, i, int((err / lim_e).argmax()), (err / lim_e).max())
        assert math.isfinite(float(lse.sum()))


def test_scales_at_the_ends_of_fp32():
    """V scales from the least normal number on, and below it: finite, and right where bf16 has a value."""
    rng = np.random.default_rng(2)
    nkv, hd, bs, nb = 1, 64, 16, 6
    for lo in (2.0 ** -126, 2.0 ** -140, 2.0 ** 100):
        c = sink_cache(rng, nb, nkv, hd, bs, 2, 1.0, [lo, lo * 4])
        c["vs"][2] = lo * 2
        table = np.arange(nb, dtype=np.int32)[None]
        q, qf = bf16(rng.uniform(0.9, 1.1, (1, 1, 4, hd)))
        out, lse, _, _ = run_attn(to_gpu(c), q, table, [nb * bs], scale=1.0 / hd)
        ref = R.attend(c, qf, table, [nb * bs], scale=1.0 / hd)
        err = np.abs(out.float().cpu().numpy() - ref["out"])
        # (sums of values below the normal range have steps of 2^-149 each)
        assert np.all(err <= ref["out_tol"] + nb * bs * 2.0 ** -149), (lo, err.max())


def test_tables_of_scattered_blocks():
    """The same through a shuffled table and a ragged batch whose sequences have sinks of their own."""
    rng = np.random.default_rng(5)
    nkv, hd, bs, B = 2, 128, 16, 5
    lens = [16 * 40, 16 * 7 + 3, 5, 16 * 90, 33]
    N = sum(-(-n // bs) for n in lens)
    table = batch(rng, lens, bs, N)
    c = sink_cache(rng, N, nkv, hd, bs, int(table[0, 0]), 12.0, [2.0 ** -8, 2.0 ** -6, 2.0 ** -9])
    for b in range(1, B):
        s = int(table[b, 0])
        c["vs"][s], c["v"][s, :, :, :hd // 2] = 1.0, 0
        c["k"][s, :, 3] = R.encode(np.full((nkv, hd), 12.0))
    q, qf = bf16(rng.uniform(0.9, 1.1, (B, 1, 16, hd)))
    out, _, _, _ = run_attn(to_gpu(c), q, table, lens, scale=1.0 / hd)
    ref = R.attend(c, qf, table, lens, scale=1.0 / hd)
    err = np.abs(out.float().cpu().numpy() - ref["out"])
    assert np.all(err <= ref["out_tol"]), (err / ref["out_tol"]).max()
