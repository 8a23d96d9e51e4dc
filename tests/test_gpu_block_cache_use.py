"""The block-scaled cache's calls as programs make them: captured in graphs that share a workspace,
on other streams, two at a time, over caches past 4 GiB, tables past what a CTA holds, batches of
many sequences, the most rows; and what the helpers refuse before anything is launched."""
import numpy as np
import pytest
import torch

import block_ref as R
from mtp_speculative_draft_lm_b200 import _lib as L
from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache import batch, bf16, check_attn, err_word, i32, make_cache, run_attn, same_cache, to_gpu

pytestmark = pytest.mark.gpu


def bits(*ts):
    return [t.detach().clone() for t in ts]


def step_state(rng, B=3, T=2, nq=8, nkv=2, hd=128, bs=16, lens=(150, 64, 33)):
    N = sum(-(-n // bs) for n in lens) + 2
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    kv, _ = bf16(rng.normal(0, 1, (2, B, T, nkv, hd)))
    q, _ = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
    return dict(cache=to_gpu(c), table=i32(table), lens=i32(lens), k=kv[0].contiguous(), v=kv[1].contiguous(), q=q,
                mass=torch.rand(table.shape, device="cuda"))


def step(st, ws):
    """One step of a server: append, attention with weights, selection, attention over it, eviction."""
    o = st["o"]
    api.block_append(st["cache"], st["k"], st["v"], st["table"], st["lens"])
    api.block_attn(st["cache"], st["q"], st["table"], st["lens"], out=o["out"], out_lse=o["lse"], mass=st["mass"], out_mass=o["mass"],
                   ws=ws)
    api.block_select(st["cache"], st["q"], st["table"], st["lens"], 4, out=o["sel"], ws=ws)
    api.block_sparse_attn(st["cache"], st["q"], st["table"], st["lens"], o["sel"], out=o["sparse"], ws=ws)
    api.block_evict(st["table"], st["lens"], o["mass"], 16, 3, out_table=o["table"], out_lens=o["lens"], out_mass=o["left"],
                    freed=o["freed"], n_freed=o["n_freed"])


def outputs(st):
    B, T, nq, hd = st["q"].shape
    z = lambda s, t: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    tab = st["table"].shape
    st["o"] = dict(out=z(st["q"].shape, torch.bfloat16), lse=z((B, T, nq), torch.float32), mass=z(tab, torch.float32),
                   sel=z((B, T, st["cache"].desc.nkv, 4), torch.int32), sparse=z(st["q"].shape, torch.bfloat16),
                   table=z(tab, torch.int32), lens=z((B,), torch.int32), left=z(tab, torch.float32), freed=z(tab, torch.int32),
                   n_freed=z((B,), torch.int32))
    return st


def test_captured_steps_share_a_workspace():
    """Two captured steps of different shapes on one workspace, replayed in turn after their inputs
    changed in place (lengths too): the same bits as eager calls."""
    rng = np.random.default_rng(0)
    sts = [outputs(step_state(rng)), outputs(step_state(rng, B=1, T=5, nq=32, nkv=4, hd=64, lens=(700,)))]
    ws = torch.empty((64 << 20,), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for st in sts:
            step(st, ws)
    torch.cuda.synchronize()
    graphs = []
    for st in sts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(st, ws)
        graphs.append(g)
    for turn in range(3):
        for st, g in zip(sts, graphs):
            st["k"].mul_(1.5)
            st["q"].add_(0.125)
            st["lens"].sub_(1)
            before = [t.clone() for t in (st["cache"].k, st["cache"].v, st["cache"].k_scale, st["cache"].v_scale)]
            g.replay()
            torch.cuda.synchronize()
            got = bits(*st["o"].values(), st["cache"].k, st["cache"].v, st["cache"].k_scale, st["cache"].v_scale, st["cache"].k_mean)
            for t, b in zip((st["cache"].k, st["cache"].v, st["cache"].k_scale, st["cache"].v_scale), before):
                t.copy_(b)
            for t in st["o"].values():
                t.zero_()
            step(st, ws)
            torch.cuda.synchronize()
            want = bits(*st["o"].values(), st["cache"].k, st["cache"].v, st["cache"].k_scale, st["cache"].v_scale, st["cache"].k_mean)
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_other_streams_and_two_at_once():
    """On a stream given as an argument, on the current one, and two calls at once with a workspace
    each: the same bits."""
    rng = np.random.default_rng(1)
    st = outputs(step_state(rng))
    step(st, None)
    torch.cuda.synchronize()
    want = bits(*st["o"].values())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a, _ = api.block_attn(st["cache"], st["q"], st["table"], st["lens"])
        b, _ = api.block_attn(st["cache"], st["q"], st["table"], st["lens"], stream=s2)
        c, _ = api.block_sparse_attn(st["cache"], st["q"], st["table"], st["lens"], st["o"]["sel"], stream=s1)
        d, _ = api.block_select(st["cache"], st["q"], st["table"], st["lens"], 4, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[0]) and torch.equal(c, want[4]) and torch.equal(d, want[3])


def test_same_bits_every_time():
    rng = np.random.default_rng(2)
    c = make_cache(rng, 800, 2, 16, 64)
    lens = [5000, 1, 3333, 900]
    table = i32(batch(rng, lens, 16, 800))
    q, _ = bf16(rng.normal(0, 1.5, (4, 3, 14, 64)))
    cache, first = to_gpu(c), None
    for _ in range(4):
        out, lse, om, _ = run_attn(cache, q, table.cpu().numpy(), lens, with_mass=True)
        if first is None:
            first = bits(out, lse, om)
        for a, b in zip((out, lse, om), first):
            assert torch.equal(a, b)


def test_cache_past_4_gib():
    """Blocks whose codes lie past 2^32 bytes: the same bits as in a small cache."""
    rng = np.random.default_rng(3)
    nkv, hd, bs, n = 8, 128, 16, 500
    big_n = (1 << 32) // (nkv * bs * hd) + 4000  # 4.35 GB of K, the same of V
    small, big = api.BlockCache.empty(40, nkv, hd, bs), api.BlockCache.empty(big_n, nkv, hd, bs)
    k, _ = bf16(rng.normal(0, 1, (1, n, nkv, hd)))
    q, _ = bf16(rng.normal(0, 1.5, (1, 1, 16, hd)))
    perm = rng.permutation(40)[: -(-n // bs)].astype(np.int32)
    got = []
    for cache, off in ((small, 0), (big, big_n - 40)):
        table, lens = i32(perm[None] + off), i32([n])
        api.block_append(cache, k, k, table, lens)
        out, _ = api.block_attn(cache, q, table, lens)
        sel, _ = api.block_select(cache, q, table, lens, 6)
        sp, _ = api.block_sparse_attn(cache, q, table, lens, sel)
        torch.cuda.synchronize()
        got.append(bits(out, sel, sp, cache.k[off + perm[3]], cache.k_mean[off + perm[3]]))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("nb,n_sel", [(600, 100), (2500, 64), (9000, 700), (20000, 33)])
def test_select_of_long_tables(nb, n_sel):
    """Up to what a CTA's registers hold and past it, with many equal scores."""
    rng = np.random.default_rng(nb)
    nkv, hd, bs = 1, 64, 16
    c = make_cache(rng, 50, nkv, bs, hd)  # 50 blocks many times over: every score is shared
    table = rng.integers(0, 50, (2, nb)).astype(np.int32)
    lens = [nb * bs, nb * bs - 5 * bs - 3]
    q, qf = bf16(rng.normal(0, 1.5, (2, 1, 2, hd)))
    sel, _ = api.block_select(to_gpu(c), q, i32(table), i32(lens), n_sel, n_first=2, n_last=3)
    assert np.array_equal(sel.cpu().numpy(), R.select(c, qf, table, lens, n_sel, 2, 3))


@pytest.mark.parametrize("n_table,keep", [(2100, 2000), (8192, 10), (9000, 4000), (30000, 29999), (17000, 8500)])
def test_evict_of_long_tables(n_table, keep):
    rng = np.random.default_rng(n_table)
    B, bs = 2, 16
    lens = [n_table * bs, (n_table - 77) * bs + 1]
    table = rng.permutation(B * n_table).astype(np.int32).reshape(B, n_table)
    mass = rng.integers(0, 40, (B, n_table)).astype(np.float32)  # many equal
    want = R.evict(table, lens, mass, bs, keep, 3, 2)
    t, l, m = i32(table), i32(lens), torch.from_numpy(mass).cuda()
    for kw in ({}, dict(out_table=t, out_lens=l, out_mass=m)):  # the second in place
        got = api.block_evict(t, l, m, bs, keep, 3, 2, **kw)
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), w)


def test_select_extreme_products():
    """The largest whole-number sums there are, 127 127 256, of both signs."""
    nkv, hd, bs, nb = 1, 256, 16, 40
    rng = np.random.default_rng(5)
    c = make_cache(rng, nb, nkv, bs, hd)
    c["mean"][:] = 127
    c["mean"][::2] = -127
    c["mean"][7, 0, 3], c["mean"][8, 0, 200] = 126, -126
    c["mscale"][:] = 0.01
    table = np.arange(nb, dtype=np.int32)[None]
    q, qf = bf16(np.full((1, 1, 1, hd), 3.0))
    sel, _ = api.block_select(to_gpu(c), q, i32(table), i32([nb * bs]), 21, n_first=0, n_last=1)
    assert np.array_equal(sel.cpu().numpy(), R.select(c, qf, table, [nb * bs], 21, 0, 1))


def test_many_sequences():
    """More sequences than a warp looks at at once, most of them empty or short."""
    rng = np.random.default_rng(6)
    B, nq, nkv, hd, bs = 150, 4, 2, 64, 16
    lens = [int(n) for n in rng.integers(0, 40, B) * (rng.random(B) < 0.6)]
    lens[77] = 900
    N = sum(-(-n // bs) for n in lens) + 1
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    q, qf = bf16(rng.normal(0, 1.5, (B, 1, nq, hd)))
    out, lse, om, err = run_attn(to_gpu(c), q, table, lens, with_mass=True)
    check_attn(out, lse, R.attend(c, qf, table, lens), om)
    assert err == 0


@pytest.mark.parametrize("T,nq,nkv,hd", [(64, 16, 1, 64), (64, 16, 1, 256), (50, 11, 1, 128), (3, 40, 5, 64), (5, 8, 1, 64), (4, 24, 4, 128)])
def test_many_rows(T, nq, nkv, hd):
    """Many query rows per kv head: every number of row tiles and columns."""
    rng = np.random.default_rng(T + nq)
    bs, lens, q_lens = 32, [190, 64], [T, max(1, T - 2)]
    lens = [max(a, b) for a, b in zip(lens, q_lens)]
    c = make_cache(rng, 12, nkv, bs, hd)
    table = batch(rng, lens, bs, 12)
    q, qf = bf16(rng.normal(0, 1.5, (2, T, nq, hd)))
    out, lse, om, _ = run_attn(to_gpu(c), q, table, lens, q_lens, with_mass=True)
    check_attn(out, lse, R.attend(c, qf, table, lens, q_lens), om)
    n_sel = 4
    sel = torch.full((2, T, nkv, n_sel), -2, dtype=torch.int32, device="cuda")
    api.block_select(to_gpu(c), q, i32(table), i32(lens), n_sel, q_lens=i32(q_lens), out=sel)
    want = R.select(c, qf, table, lens, n_sel, 1, 1, q_lens)
    assert np.array_equal(sel.cpu().numpy(), want)
    out, lse, _, _ = run_attn(to_gpu(c), q, table, lens, q_lens, sel=sel)
    check_attn(out, lse, R.attend(c, qf, table, lens, q_lens, sel=want))


def test_append_of_a_prompt_by_chunks():
    """A prompt appended whole, in chunks that end inside blocks, and token by token, where the scales
    do not have to grow: the same bytes."""
    rng = np.random.default_rng(9)
    nkv, hd, bs, n = 2, 128, 32, 300
    x = rng.normal(0, 1, (1, n, nkv, hd))
    x[0, ::bs] = np.sign(x[0, ::bs]) * 4.5  # the largest value of a block comes first
    x = np.clip(x, -4.5, 4.5)
    t, xf = bf16(x)
    table = i32(rng.permutation(12)[:10].astype(np.int32)[None])
    caches = []
    for sizes in ([n], [100, 7, 93, 64, 36], [1] * n):
        cache, at = api.BlockCache.empty(12, nkv, hd, bs), 0
        for m in sizes:
            at += m
            chunk = t[:, at - m:at]
            api.block_append(cache, chunk, chunk, table, i32([at]))
        caches.append(cache)
    torch.cuda.synchronize()
    for other in caches[1:]:
        for f in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale"):
            assert torch.equal(getattr(caches[0], f), getattr(other, f)), f
    ref = {k: getattr(api.BlockCache.empty(12, nkv, hd, bs), f).cpu().numpy().copy() for k, f in (
        ("k", "k"), ("v", "v"), ("ks", "k_scale"), ("vs", "v_scale"), ("mean", "k_mean"), ("mscale", "k_mean_scale"))}
    R.append(ref, xf, xf, table.cpu().numpy(), [n])
    same_cache(caches[0], ref)


def test_a_scale_no_append_wrote():
    """Rows before the new ones under a scale that is no power of two (a cache from elsewhere)."""
    rng = np.random.default_rng(10)
    nkv, hd, bs = 2, 64, 16
    c = make_cache(rng, 4, nkv, bs, hd)
    c["ks"][:], c["vs"][:] = np.float32(0.037), np.float32(3.3)
    table = np.array([[2, 0]], np.int32)
    x, xf = bf16(rng.normal(0, 4, (1, 5, nkv, hd)) * np.array([1, 1, 50, 1, 1]).reshape(1, 5, 1, 1))
    cache = to_gpu(c)
    api.block_append(cache, x, x, i32(table), i32([20]))
    R.append(c, xf, xf, table, [20])
    same_cache(cache, c)


def test_helpers_refuse_before_launching():
    rng = np.random.default_rng(11)
    st = outputs(step_state(rng))
    ca, q, tab, lens = st["cache"], st["q"], st["table"], st["lens"]
    bad = [
        lambda: api.block_attn(ca, q.cpu(), tab, lens), lambda: api.block_attn(ca, q, tab.cpu(), lens),
        lambda: api.block_attn(ca, q, tab.long(), lens), lambda: api.block_attn(ca, q, tab, lens.long()),
        lambda: api.block_attn(ca, q, tab, lens[:2]), lambda: api.block_attn(ca, q, tab[:2], lens),
        lambda: api.block_attn(ca, q[..., :64].contiguous(), tab, lens), lambda: api.block_attn(ca, q.float(), tab, lens),
        lambda: api.block_attn(ca, q, tab, lens, q_lens=lens.float()), lambda: api.block_attn(ca, q, tab, lens, out=q[:1]),
        lambda: api.block_attn(ca, q, tab, lens, out=q.float()), lambda: api.block_attn(ca, q, tab, lens, out_lse=st["mass"]),
        lambda: api.block_attn(ca, q, tab, lens, out_mass=st["mass"][:, :2].contiguous()),
        lambda: api.block_attn(ca, q, tab, lens, dev_err=lens), lambda: api.block_attn(ca, q, tab.t().contiguous().t(), lens),
        lambda: api.block_sparse_attn(ca, q, tab, lens, st["o"]["sel"][:, :1].contiguous()),
        lambda: api.block_sparse_attn(ca, q, tab, lens, st["o"]["sel"].long()),
        lambda: api.block_select(ca, q, tab, lens, 4, out=st["o"]["sel"][:1]),
        lambda: api.block_append(ca, st["k"], st["v"][:, :1], tab, lens), lambda: api.block_append(ca, q, q, tab, lens),
        lambda: api.block_append(ca, st["k"].cpu(), st["v"].cpu(), tab, lens),
        lambda: api.block_evict(tab.cpu(), lens, st["mass"], 16, 3), lambda: api.block_evict(tab, lens, st["mass"].double(), 16, 3),
        lambda: api.block_evict(tab, lens[:1], st["mass"], 16, 3),
        lambda: api.BlockCache.of(ca.k, ca.v.cpu(), ca.k_scale, ca.v_scale),
        lambda: api.BlockCache.of(ca.k, ca.v, ca.k_scale[:1], ca.v_scale), lambda: api.BlockCache.of(ca.k.float(), ca.v, ca.k_scale, ca.v_scale)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    no_means = api.BlockCache.of(ca.k, ca.v, ca.k_scale, ca.v_scale)
    for f, status in ((lambda: api.block_select(no_means, q, tab, lens, 4), L.MTP_ERR_INVALID_ARG),
                      (lambda: api.block_evict(tab, lens, st["mass"], 16, 1), L.MTP_ERR_INVALID_ARG),
                      (lambda: api.block_attn(ca, q.expand(3, 2, 8, 128)[:, :, :7], tab, lens), L.MTP_ERR_INVALID_ARG)):
        with pytest.raises(L.MtpError) as e:
            f()
        assert e.value.status == status
    assert int(err_word().item()) == 0
