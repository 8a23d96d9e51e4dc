"""The block-scaled paged cache on the GPU against plain references: append (bit for bit),
attention (64-bit, with bounds derived from the stated roundings), block selection and
eviction (exactly), and a run of them together."""
import numpy as np
import pytest
import torch

import block_ref as R
from mtp_speculative_draft_lm_b200 import _lib as L
from mtp_speculative_draft_lm_b200 import api, synth

pytestmark = pytest.mark.gpu


def bf16(x):
    """fp32 array -> (bf16 tensor on the GPU, its fp32 values)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy()


def make_cache(rng, N, nkv, bs, hd, scale_exp=(-8, -4), spread=40.0):
    """A cache full of codes, scales powers of two (numpy dict)."""
    c = dict(k=R.encode(rng.normal(0, spread, (N, nkv, bs, hd))), v=R.encode(rng.normal(0, spread, (N, nkv, bs, hd))))
    for n in ("ks", "vs"):
        c[n] = np.exp2(rng.integers(scale_exp[0], scale_exp[1] + 1, (N, nkv))).astype(np.float32)
    c["mean"] = rng.integers(-127, 128, (N, nkv, hd)).astype(np.int8)
    c["mscale"] = rng.uniform(0.001, 0.01, (N, nkv)).astype(np.float32)
    return c


def to_gpu(c, rows_first=False):
    """An api.BlockCache of a numpy cache; rows_first: stored [block, row, head, hd]."""
    def codes(a):
        t = torch.from_numpy(a.copy()).cuda()
        return t.transpose(1, 2).contiguous().transpose(1, 2) if rows_first else t

    f = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    return api.BlockCache(codes(c["k"]), codes(c["v"]), f(c["ks"]), f(c["vs"]), f(c["mean"]), f(c["mscale"]))


def batch(rng, lens, bs, N, n_table=None):
    """A table over shuffled blocks, -1 behind each sequence."""
    nb = [-(-max(n, 0) // bs) for n in lens]
    n_table = max(1, max(nb)) if n_table is None else n_table
    perm = rng.permutation(N).astype(np.int32)
    table = np.full((len(lens), n_table), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        n = min(n, n_table)
        table[b, :n] = perm[at:at + n]
        at += n
    assert at <= N
    return table


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def err_word():
    return torch.zeros((1,), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ append
def same_cache(cache, ref):
    torch.cuda.synchronize()
    for n, t in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scale), ("vs", cache.v_scale), ("mean", cache.k_mean),
                 ("mscale", cache.k_mean_scale)):
        got, want = t.cpu().contiguous().numpy(), ref[n]
        if got.dtype == np.float32:
            got, want = got.view(np.int32), want.view(np.int32)
        bad = np.argwhere(got != want)
        assert bad.size == 0, (n, len(bad), bad[0], got[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("B,T,nkv,hd,bs,base", [
    (1, 1, 1, 64, 16, 0), (3, 1, 2, 128, 16, 37), (5, 4, 3, 64, 32, 61), (2, 7, 2, 256, 64, 0), (4, 33, 2, 128, 16, 5),
    (1, 200, 4, 128, 32, 9), (2, 130, 1, 256, 16, 15), (3, 17, 5, 64, 64, 63)])
@pytest.mark.parametrize("rows_first", [False, True], ids=["head", "row"])
def test_append_matches(B, T, nkv, hd, bs, base, rows_first):
    rng = np.random.default_rng(B * 1000 + T + hd + bs)
    q_lens = [T if b % 2 == 0 else max(0, T - b) for b in range(B)]
    lens = [base + 11 * b + q for b, q in enumerate(q_lens)]
    N = sum(-(-n // bs) for n in lens) + 2
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    grow = np.exp2(rng.integers(-6, 7, (B, T, nkv, 1)))
    kv, x = bf16(rng.normal(0, 1, (B, T, 2, nkv, hd)) * grow[:, :, None])
    cache, err = to_gpu(c, rows_first), err_word()
    api.block_append(cache, kv[:, :, 0], kv[:, :, 1], i32(table), i32(lens), q_lens=i32(q_lens), dev_err=err)
    flags = R.append(c, x[:, :, 0], x[:, :, 1], table, lens, q_lens)
    same_cache(cache, c)
    assert int(err.item()) == flags == 0


def test_append_step_by_step():
    """Tokens one at a time into empty blocks: the same scales as the rows' largest value, and
    every row within the roundings it went through."""
    rng = np.random.default_rng(3)
    nkv, hd, bs, n = 2, 128, 16, 40
    x = rng.normal(0, 1, (1, n, nkv, hd)) * np.exp2(rng.integers(-3, 4, (1, n, nkv, 1)))
    t, xf = bf16(x)
    cache = api.BlockCache.empty(5, nkv, hd, bs)
    ref = {k: a.cpu().numpy().copy() for k, a in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scale), ("vs", cache.v_scale),
                                                  ("mean", cache.k_mean), ("mscale", cache.k_mean_scale))}
    table = np.array([[3, 0, 4]], np.int32)
    for p in range(n):
        step = t[:, p:p + 1].contiguous()
        api.block_append(cache, step, step, i32(table), i32([p + 1]))
        R.append(ref, xf[:, p:p + 1], xf[:, p:p + 1], table, [p + 1])
    same_cache(cache, ref)
    whole = {k: np.zeros_like(a) for k, a in ref.items()}
    R.append(whole, xf, xf, table, [n])
    assert np.array_equal(whole["ks"], ref["ks"])
    got = R.decode(ref["k"][table[0]]) * ref["ks"][table[0]][..., None, None]
    got = got.transpose(0, 2, 1, 3).reshape(-1, nkv, hd)[:n]
    # one rounding (2^-4) for each of the block's binades at most; 2^-10 of the scale below normals
    lim = np.abs(xf[0]) * 2.0 ** -4 + 2.0 ** -10 * np.repeat(ref["ks"][table[0]], bs, 0)[:n][..., None] * 4
    assert np.all(np.abs(got - xf[0]) <= lim)


def test_append_odd_values():
    """Zeros, infinities, NaN, the largest and the smallest magnitudes, exact borders of the scale."""
    rng = np.random.default_rng(5)
    nkv, hd, bs = 1, 64, 16
    x = np.zeros((1, 8 * 16, nkv, hd), np.float32)
    x[0, 16:32] = 448.0 * 2.0 ** 3              # a scale that divides exactly
    x[0, 32:48] = 450.0 * 2.0 ** 3              # one bf16 step more: twice the scale
    x[0, 48:64] = rng.normal(0, 1, (16, 1, hd))
    x[0, 50, 0, 3], x[0, 51, 0, 4], x[0, 52, 0, 5] = np.inf, -np.inf, np.nan
    x[0, 64:80] = 3.3e38
    x[0, 80:96] = 1e-40
    x[0, 96:112, :, ::2] = -0.0
    x[0, 112:128, 0, 0] = np.inf                # nothing finite but zeros
    t, xf = bf16(x)
    c = make_cache(rng, 9, nkv, bs, hd)
    cache, table = to_gpu(c), np.arange(8, dtype=np.int32)[None]
    api.block_append(cache, t, t, i32(table), i32([128]))
    R.append(c, xf, xf, table, [128])
    same_cache(cache, c)
    assert c["ks"][1, 0] == 8.0 and c["ks"][2, 0] == 16.0


def test_append_missing_blocks_and_padding():
    """A table that is too short, blocks out of range, more tokens than positions, empty slots:
    the rest is written, nothing else touched, the flag set."""
    rng = np.random.default_rng(8)
    nkv, hd, bs, B, T = 2, 64, 16, 6, 40
    lens, q_lens = [50, 40, 33, 0, -5, 10], [40, 40, 0, 40, 3, 20]
    c = make_cache(rng, 30, nkv, bs, hd)
    table = batch(rng, lens, bs, 30, n_table=3)
    table[1, 1] = 30
    x, xf = bf16(rng.normal(0, 1, (B, T, nkv, hd)))
    cache, err = to_gpu(c), err_word()
    api.block_append(cache, x, x, i32(table), i32(lens), q_lens=i32(q_lens), dev_err=err)
    flags = R.append(c, xf, xf, table, lens, q_lens)
    same_cache(cache, c)
    assert int(err.item()) == flags == L.MTP_DEVFLAG_BAD_SLOT


# ------------------------------------------------------------------------------ attention
def check_attn(got_out, got_lse, ref, got_mass=None, mass_in=None):
    live = ref["live"]
    out, lse = got_out.float().cpu().numpy().astype(np.float64), got_lse.cpu().numpy().astype(np.float64)
    e = np.abs(out - ref["out"])[live]
    assert np.all(e <= ref["out_tol"][live]), (e.max(), (e / ref["out_tol"][live]).max())
    same_inf = lse[live] == ref["lse"][live]
    with np.errstate(invalid="ignore"):
        e = np.abs(lse[live] - ref["lse"][live])
    assert np.all(same_inf | (e <= ref["lse_tol"][live])), np.nanmax(e)
    if got_mass is not None:
        want = ref["mass"] + (0 if mass_in is None else mass_in)
        e = np.abs(got_mass.cpu().numpy() - want)
        lim = ref["mass_tol"] + 2.0 ** -23 * np.abs(want)
        assert np.all(e <= lim), (e.max(), (e / lim).max())


def run_attn(cache, q, table, lens, q_lens=None, sel=None, mass=None, with_mass=False, **kw):
    B, T, nq, hd = q.shape
    out = torch.full((B, T, nq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, nq), 7.0, device="cuda")
    err = err_word()
    kw.update(q_lens=None if q_lens is None else i32(q_lens), out=out, out_lse=lse, dev_err=err)
    om = None
    if sel is not None:
        api.block_sparse_attn(cache, q, i32(table), i32(lens), sel, **kw)
    else:
        om = torch.full(table.shape, 7.0, device="cuda") if with_mass else None
        api.block_attn(cache, q, i32(table), i32(lens), mass=mass, out_mass=om, **kw)
    torch.cuda.synchronize()
    return out, lse, om, int(err.item())


@pytest.mark.parametrize("B,T,nq,nkv,hd,bs,top", [
    (1, 1, 1, 1, 64, 16, 1), (1, 1, 8, 8, 128, 16, 17), (2, 1, 64, 8, 128, 16, 700), (3, 2, 6, 2, 64, 32, 300),
    (11, 5, 8, 2, 64, 16, 130), (2, 8, 16, 1, 256, 64, 257), (4, 3, 14, 2, 256, 16, 100), (2, 3, 32, 2, 128, 32, 90),
    (1, 64, 2, 1, 128, 16, 200), (2, 33, 32, 2, 64, 16, 70), (1, 1, 16, 1, 128, 64, 5000), (40, 1, 4, 4, 64, 16, 60),
    (3, 7, 21, 7, 128, 16, 333)])
@pytest.mark.parametrize("rows_first", [False, True], ids=["head", "row"])
def test_attention_matches(B, T, nq, nkv, hd, bs, top, rows_first):
    rng = np.random.default_rng(B + 10 * T + nq + hd + top)
    q_lens = [T if b % 3 != 1 else max(0, T - b % T - 1) for b in range(B)]
    lens = [max(q_lens[b], top if b == 0 else int(rng.integers(0, top + 1))) for b in range(B)]
    if B > 8:
        lens[4], q_lens[4], lens[6] = 0, 0, 0  # an empty slot; tokens of a sequence without positions
    N = sum(-(-n // bs) for n in lens) + 3
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N, n_table=max(1, -(-max(lens) // bs)) + 2)
    q, qf = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
    mass = rng.uniform(0, 3, table.shape).astype(np.float32)
    out, lse, om, err = run_attn(to_gpu(c, rows_first), q, table, lens, q_lens, mass=torch.from_numpy(mass).cuda(), with_mass=True)
    ref = R.attend(c, qf, table, lens, q_lens)
    check_attn(out, lse, ref, om, mass)
    assert err == 0
    dead = ~torch.from_numpy(ref["live"]).cuda()
    assert bool((out[dead] == 7.0).all()) and bool((lse[dead] == 7.0).all())


def test_attention_masked_garbage():
    """NaN codes behind each sequence's end and in the rows that a step's earlier tokens do not
    see yet, NaN scales of blocks that no table names: outputs as without them. A NaN that a
    token does see reaches that token and the later ones alone."""
    rng = np.random.default_rng(21)
    B, T, nq, nkv, hd, bs = 2, 6, 8, 2, 128, 16
    lens = [70, 38]
    c = make_cache(rng, 12, nkv, bs, hd)
    table = batch(rng, lens, bs, 10)
    used = set(table[table >= 0].tolist())
    for n in set(range(12)) - used:
        c["ks"][n] = c["vs"][n] = np.nan
    for b, n in enumerate(lens):
        ph = table[b, n // bs]
        c["k"][ph, :, n % bs:] = 0x7F
        c["v"][ph, :, n % bs:] = 0xFF
    clean = {k: a.copy() for k, a in c.items()}
    # position 67 is token 3 of sequence 0: tokens 0 .. 2 do not see it
    c["v"][table[0, 67 // bs], 1, 67 % bs, 5] = 0x7F
    c["k"][table[0, 69 // bs], 0, 69 % bs, 9] = 0xFF  # seen by token 5 alone
    q, qf = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
    out, lse, om, err = run_attn(to_gpu(c), q, table, lens)
    ref = R.attend(clean, qf, table, lens)
    o = out.float().cpu().numpy()
    hit = np.zeros(o.shape, bool)
    hit[0, 3:, nq // 2:, 5] = True   # V's NaN: one dimension of kv head 1
    hit[0, 5, :nq // 2] = True       # K's NaN: every dimension of kv head 0
    assert np.isnan(o[hit]).all() and np.isfinite(o[~hit]).all()
    ref["out"][hit], ref["out_tol"][hit] = 0, np.inf
    ref["lse_tol"][0, 5, :nq // 2] = np.inf
    o[hit] = 0
    l = lse.cpu()
    l[0, 5, :nq // 2] = 0
    check_attn(torch.from_numpy(o), l, ref)
    assert err == 0


def test_attention_scales_far_apart():
    """V scales over 60 binades, zero scales, K scales that make scores large: each block's part
    keeps its accuracy."""
    rng = np.random.default_rng(4)
    nkv, hd, bs, n = 2, 64, 16, 400
    c = make_cache(rng, 30, nkv, bs, hd, spread=2.0)
    c["vs"] = np.exp2(rng.integers(-30, 31, c["vs"].shape)).astype(np.float32)
    c["ks"] = np.exp2(rng.integers(-2, 2, c["ks"].shape)).astype(np.float32)
    c["vs"][rng.random(c["vs"].shape) < 0.2] = 0
    c["ks"][rng.random(c["ks"].shape) < 0.2] = 0
    c["vs"][3] *= np.float32(1.3)  # not a power of two
    table = batch(rng, [n], bs, 30)
    q, qf = bf16(rng.normal(0, 3, (1, 1, 8, hd)))
    out, lse, om, _ = run_attn(to_gpu(c), q, table, [n], with_mass=True)
    check_attn(out, lse, R.attend(c, qf, table, [n]), om)


def test_attention_missing_blocks():
    """Short tables, blocks out of range, lengths past the table: read where there is something."""
    rng = np.random.default_rng(6)
    nkv, hd, bs = 2, 128, 16
    lens, T = [100, 90, 5000, 30], 2
    c = make_cache(rng, 20, nkv, bs, hd)
    table = batch(rng, [min(n, 80) for n in lens], bs, 20, n_table=5)
    table[0, 2], table[3] = 20, -1  # out of range; a sequence with nothing
    q, qf = bf16(rng.normal(0, 1, (4, T, 4, hd)))
    out, lse, om, err = run_attn(to_gpu(c), q, table, lens, with_mass=True)
    ref = R.attend(c, qf, table, lens)
    check_attn(out, lse, ref, om)
    assert err == ref["flags"] == L.MTP_DEVFLAG_BAD_SLOT
    assert bool((out[3] == 0).all()) and bool(torch.isinf(lse[3]).all())


def test_attention_q_slices_scale_and_infinite_q():
    """q as a slice of a fused projection, another scale, scale 0 (a plain mean), a head of q with an infinity."""
    rng = np.random.default_rng(7)
    B, T, nq, nkv, hd, bs = 2, 3, 4, 2, 64, 16
    lens = [120, 77]
    c = make_cache(rng, 14, nkv, bs, hd)
    table = batch(rng, lens, bs, 14)
    fused, ff = bf16(rng.normal(0, 1, (B, T, (nq + 2 * nkv) * hd)))
    q = fused[..., :nq * hd].unflatten(-1, (nq, hd))
    qf = ff[..., :nq * hd].reshape(B, T, nq, hd)
    for sc in (0.02, 0.0, 1.0):
        out, lse, _, _ = run_attn(to_gpu(c), q, table, lens, scale=sc)
        check_attn(out, lse, R.attend(c, qf, table, lens, scale=sc))
    q2 = q.clone()
    q2[1, 2, 3, 7] = float("inf")
    out, lse, _, _ = run_attn(to_gpu(c), q2.contiguous(), table, lens)
    o = out.float().cpu()
    assert bool(torch.isnan(o[1, 2, 3]).all())
    o[1, 2, 3] = 0
    assert bool(torch.isfinite(o).all())


def test_attention_of_the_prefill_cache():
    """The cache that prefill_kv writes, read with its two scales."""
    d = synth.prefill_inputs(seed=85, R=300, vocab=700, h=512, nkv=4, hd=128)
    d["k_scale"], d["v_scale"] = 0.5, 2.0
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    nb = int(d["num_blocks"])
    kc = torch.zeros((nb, 16, 4, 128), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    api.prefill_kv(dev, kc, vc, chunk_rows=256)
    q, qf = bf16(np.random.default_rng(2).normal(0, 1, (1, 1, 16, 128)))
    table = d["block_table"].numpy()[None]
    out, lse, _, err = run_attn(api.BlockCache.of_prefill(kc, vc, 0.5, 2.0), q, table, [300])
    hw = lambda t: t.cpu().transpose(1, 2).contiguous().numpy()  # noqa: E731
    c = dict(k=hw(kc), v=hw(vc), ks=np.full((nb, 4), 0.5, np.float32), vs=np.full((nb, 4), 2.0, np.float32))
    check_attn(out, lse, R.attend(c, qf, table, [300]))
    one, _ = api.paged_decode_attn(q[0, 0], 4, kc, vc, dev["block_table"], 300, k_scale=0.5, v_scale=2.0)
    assert err == 0
    assert float((one.float() - out[0, 0].float()).abs().max()) <= 2.0 ** -7 * float(out.float().abs().max())


# ------------------------------------------------------------------------------ selected blocks
@pytest.mark.parametrize("B,T,nq,nkv,hd,bs,top,n_sel", [
    (1, 1, 8, 1, 64, 16, 100, 3), (2, 1, 64, 8, 128, 16, 3000, 40), (3, 4, 6, 2, 256, 32, 700, 9), (2, 3, 32, 2, 128, 64, 900, 50),
    (10, 2, 3, 3, 64, 16, 500, 16)])
def test_select_and_sparse_attention(B, T, nq, nkv, hd, bs, top, n_sel):
    rng = np.random.default_rng(B + T + top)
    q_lens = [T if b % 3 != 1 else max(0, T - 1) for b in range(B)]
    lens = [max(q_lens[b], top if b == 0 else int(rng.integers(0, top + 1))) for b in range(B)]
    N = sum(-(-n // bs) for n in lens) + 1
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    q, qf = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
    cache = to_gpu(c)
    sel = torch.full((B, T, nkv, n_sel), -2, dtype=torch.int32, device="cuda")
    err = err_word()
    api.block_select(cache, q, i32(table), i32(lens), n_sel, q_lens=i32(q_lens), out=sel, dev_err=err)
    want = R.select(c, qf, table, lens, n_sel, 1, 1, q_lens)
    assert np.array_equal(sel.cpu().numpy(), want) and int(err.item()) == 0
    out, lse, _, e2 = run_attn(cache, q, table, lens, q_lens, sel=sel)
    check_attn(out, lse, R.attend(c, qf, table, lens, q_lens, sel=want))
    assert e2 == 0


def test_select_ties_forced_and_odd_scores():
    """Equal scores take the lowest blocks; forced blocks count; NaN, infinite and missing ones come last."""
    rng = np.random.default_rng(9)
    nkv, hd, bs, nb = 2, 64, 16, 60
    c = make_cache(rng, nb, nkv, bs, hd)
    c["mean"][:] = c["mean"][0]
    c["mscale"][:] = 0.01
    c["mscale"][20:23] = 0.0
    table = np.arange(nb, dtype=np.int32)[None].copy()
    q, qf = bf16(rng.normal(0, 1, (1, 1, 4, hd)))
    sel, _ = api.block_select(to_gpu(c), q, i32(table), i32([nb * bs]), 20, n_first=3, n_last=5)
    assert np.array_equal(sel.cpu().numpy(), R.select(c, qf, table, [nb * bs], 20, 3, 5))
    c["mscale"][5], c["mscale"][6] = np.nan, np.inf
    table[0, 30] = -1
    err = err_word()
    sel, _ = api.block_select(to_gpu(c), q, i32(table), i32([nb * bs]), 57, n_first=0, n_last=1, dev_err=err)
    got = sel.cpu().numpy()[0, 0]
    for g in range(nkv):
        assert 5 not in got[g] and 30 not in got[g] and len(set(got[g])) == 57
    assert int(err.item()) == L.MTP_DEVFLAG_BAD_SLOT
    q[0, 0, 0, 3] = float("inf")  # that head does not count
    qf[0, 0, 0, 3] = np.inf
    c = make_cache(rng, nb, nkv, bs, hd)
    table = np.arange(nb, dtype=np.int32)[None]
    sel, _ = api.block_select(to_gpu(c), q, i32(table), i32([nb * bs]), 20)
    assert np.array_equal(sel.cpu().numpy(), R.select(c, qf, table, [nb * bs], 20, 1, 1))


def test_sparse_attention_odd_lists():
    """Lists in any order, with -1 among them, a block twice (counts twice), blocks the token does not
    see, blocks past the table (flagged), nothing at all."""
    rng = np.random.default_rng(12)
    nkv, hd, bs = 2, 128, 32
    lens, B, T = [300, 40], 2, 3
    c = make_cache(rng, 14, nkv, bs, hd)
    table = batch(rng, lens, bs, 14)
    sel = np.full((B, T, nkv, 6), -1, np.int32)
    sel[0, 0, 0] = [7, -1, 2, 2, 0, 9]
    sel[0, 1, 0] = [9, 8, 7, 3, -5, 1]
    sel[0, 2, 1] = [4, -1, -1, 4, -1, 4]
    sel[1, :, :, 0] = 1
    sel[1, 2, 1, 2:4] = [5, 0]
    q, qf = bf16(rng.normal(0, 1.5, (B, T, 6, hd)))
    out, lse, _, err = run_attn(to_gpu(c), q, table, lens, sel=torch.from_numpy(sel).cuda())
    ref = R.attend(c, qf, table, lens, sel=sel)
    check_attn(out, lse, ref)
    assert err == 0 and bool((out[0, 2, :3] == 0).all()) and bool(torch.isinf(lse[0, 2, :3]).all())
    # past the table: block 10 of a 400-position sequence whose table has 10 entries
    sel[0, 0, 0, 1] = 10
    out, lse, _, err = run_attn(to_gpu(c), q, table, [400, 40], sel=torch.from_numpy(sel).cuda())
    ref = R.attend(c, qf, table, [400, 40], sel=sel)
    check_attn(out, lse, ref)
    assert err == ref["flags"] == L.MTP_DEVFLAG_BAD_SLOT


# ------------------------------------------------------------------------------ eviction
@pytest.mark.parametrize("B,n_table,bs,keep,n_first,n_last", [
    (1, 1, 16, 1, 0, 1), (4, 40, 16, 8, 1, 1), (3, 1500, 32, 700, 4, 2), (2, 5000, 16, 33, 0, 1), (6, 100, 64, 100, 2, 3), (2, 9, 1, 5, 2, 3)])
def test_evict_matches(B, n_table, bs, keep, n_first, n_last):
    rng = np.random.default_rng(n_table + keep)
    lens = [int(rng.integers(0, n_table * bs + 1)) for _ in range(B)]
    lens[0] = n_table * bs - (bs > 1)
    table = rng.permutation(B * n_table).astype(np.int32).reshape(B, n_table)
    mass = rng.random((B, n_table)).astype(np.float32) ** 4
    mass[:, ::3] = mass[:, :1]  # ties
    if n_table > 30:
        mass[0, 7], mass[0, 8], mass[0, 9] = np.nan, np.inf, -0.0
    want = R.evict(table, lens, mass, bs, keep, n_first, n_last)
    t, l, m = i32(table), i32(lens), torch.from_numpy(mass).cuda()
    got = api.block_evict(t, l, m, bs, keep, n_first, n_last)
    inplace = api.block_evict(t, l, m, bs, keep, n_first, n_last, out_table=t, out_lens=l, out_mass=m)
    torch.cuda.synchronize()
    for g in (got, inplace):
        for a, w in zip(g, want):
            assert np.array_equal(a.cpu().numpy(), w, equal_nan=a.dtype.is_floating_point)


# ------------------------------------------------------------------------------ together
def test_run_together():
    """A server's steps on a small pool: prompts appended, then tokens one to three at a time, each attending
    (every block, then selected ones) with the weights accumulated, and sequences cut to a bound, whose
    freed blocks the next appends take. Every result against the references on the same state."""
    rng = np.random.default_rng(31)
    B, nq, nkv, hd, bs, N, n_table, keep = 3, 8, 2, 64, 16, 60, 16, 9
    cache = api.BlockCache.empty(N, nkv, hd, bs)
    ref = {k: a.cpu().numpy().copy() for k, a in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scale), ("vs", cache.v_scale),
                                                  ("mean", cache.k_mean), ("mscale", cache.k_mean_scale))}
    free = list(range(N))
    table, lens = np.full((B, n_table), -1, np.int32), np.zeros(B, np.int64)
    mass = np.zeros((B, n_table), np.float32)
    for step in range(12):
        T = 120 if step == 0 else 1 + step % 3
        q_lens = [T - 13 * b if step == 0 else max(1, T - b) for b in range(B)]
        for b in range(B):
            for j in range(-(-int(lens[b]) // bs), -(-int(lens[b] + q_lens[b]) // bs)):
                table[b, j] = free.pop(0)
        lens = lens + np.array(q_lens)
        k, kf = bf16(rng.normal(0, 1 + step, (B, T, nkv, hd)))
        v, vf = bf16(rng.normal(0, 1, (B, T, nkv, hd)))
        api.block_append(cache, k, v, i32(table), i32(lens), q_lens=i32(q_lens))
        R.append(ref, kf, vf, table, lens, q_lens)
        same_cache(cache, ref)
        if step == 0:
            continue
        q, qf = bf16(rng.normal(0, 1.5, (B, T, nq, hd)))
        out, lse, om, err = run_attn(cache, q, table, lens, q_lens, mass=torch.from_numpy(mass).cuda(), with_mass=True)
        check_attn(out, lse, R.attend(ref, qf, table, lens, q_lens), om, mass)
        mass = om.cpu().numpy()
        sel = torch.full((B, T, nkv, 5), -2, dtype=torch.int32, device="cuda")
        api.block_select(cache, q, i32(table), i32(lens), 5, q_lens=i32(q_lens), out=sel)
        want = R.select(ref, qf, table, lens, 5, 1, 1, q_lens)
        assert np.array_equal(sel.cpu().numpy(), want)
        out, lse, _, _ = run_attn(cache, q, table, lens, q_lens, sel=sel)
        check_attn(out, lse, R.attend(ref, qf, table, lens, q_lens, sel=want))
        got = [a.cpu().numpy() for a in api.block_evict(i32(table), i32(lens), torch.from_numpy(mass).cuda(), bs, keep)]
        for a, w in zip(got, R.evict(table, lens, mass, bs, keep, 1, 1)):
            assert np.array_equal(a, w)
        table, lens, mass = got[0], got[1].astype(np.int64), got[2]
        for b in range(B):
            free += [int(x) for x in got[3][b][:got[4][b]]]
    assert len(free) + int((table >= 0).sum()) == N
