"""The block-scaled cache's calls where a launch takes another shape: appends whose CTAs hold
several heads, selections for more rows than the SMs hold at once; and its native calls: wrong
arguments, and threads that call at once."""
import threading

import numpy as np
import pytest
import torch

import block_ref as R
from mtp_speculative_draft_lm_b200 import _lib as L
from mtp_speculative_draft_lm_b200 import api
from test_gpu_block_cache import batch, bf16, err_word, i32, make_cache, same_cache, to_gpu
from test_gpu_block_cache_use import outputs, step_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,nkv,hd,bs", [
    (300, 1, 1, 64, 16), (110, 1, 3, 64, 16), (70, 2, 5, 128, 16), (60, 5, 5, 64, 32), (200, 17, 2, 64, 16), (61, 1, 5, 256, 32),
    (75, 9, 4, 64, 64), (130, 65, 2, 64, 16), (40, 64, 1, 64, 16)])
def test_append_of_many_sequences(B, T, nkv, hd, bs):
    """A CTA's warps take heads of their own, the last CTA fewer of them; some sequences empty or
    without tokens, some without their blocks."""
    rng = np.random.default_rng(B + T)
    q_lens = [int(n) for n in rng.integers(0, T + 1, B)]
    lens = [int(n) + q for n, q in zip(rng.integers(0, 3 * bs, B), q_lens)]
    N = sum(-(-n // bs) for n in lens) + 2
    c = make_cache(rng, N, nkv, bs, hd)
    table = batch(rng, lens, bs, N)
    table[5::17, 0] = -1
    kv, x = bf16(rng.normal(0, 1, (B, T, 2, nkv, hd)) * np.exp2(rng.integers(-6, 7, (B, T, 1, nkv, 1))))
    cache, err = to_gpu(c), err_word()
    api.block_append(cache, kv[:, :, 0], kv[:, :, 1], i32(table), i32(lens), q_lens=i32(q_lens), dev_err=err)
    flags = R.append(c, x[:, :, 0], x[:, :, 1], table, lens, q_lens)
    same_cache(cache, c)
    assert int(err.item()) == flags


@pytest.mark.parametrize("B,T,nkv,nb,n_sel", [(80, 2, 2, 600, 70), (40, 1, 8, 1100, 32), (300, 1, 1, 513, 500), (2, 3, 50, 2048, 9)])
def test_select_for_many_rows(B, T, nkv, nb, n_sel):
    rng = np.random.default_rng(nb)
    hd, bs = 64, 16
    c = make_cache(rng, 300, nkv, bs, hd)
    table = rng.integers(0, 300, (B, nb)).astype(np.int32)
    lens = [int(n) for n in rng.integers(0, nb * bs + 1, B)]
    lens[0], lens[1] = nb * bs, T
    q, qf = bf16(rng.normal(0, 1.5, (B, T, 2 * nkv, hd)))
    sel, _ = api.block_select(to_gpu(c), q, i32(table), i32(lens), n_sel, n_first=1, n_last=2)
    want, got = R.select(c, qf, table, lens, n_sel, 1, 2), sel.cpu().numpy()
    for b in range(B):  # (tokens before a sequence's first position have nothing)
        assert np.array_equal(got[b], want[b]), b


def test_native_calls_refuse_what_is_no_tensor():
    st = outputs(step_state(np.random.default_rng(3)))
    ca, q, tab, lens, mass = st["cache"], st["q"], st["table"], st["lens"], st["mass"]
    for f in (lambda: api.block_append(ca, q, None, tab, lens), lambda: api.block_attn(ca, q, None, lens, out=q),
              lambda: api.block_attn(ca, q, tab, [1, 2, 3], out=q), lambda: api.block_attn(ca, q, tab, lens, out=q, ws=7),
              lambda: api.block_attn(ca, q[0], tab, lens, out=q), lambda: api.block_attn(ca, q, tab[0], lens, out=q),
              lambda: api.block_attn(ca, q, tab, lens, out=q, mass=mass.cpu()), lambda: api.block_attn(ca, q, tab, lens, ws=mass.cpu().new_empty(1 << 24)),
              lambda: api.block_select(ca, q, tab, lens, -1, out=st["o"]["sel"]), lambda: api.block_select(ca, q, tab, lens, 1 << 40, out=st["o"]["sel"]),
              lambda: api.block_sparse_attn(ca, q, tab, lens, st["o"]["sel"][0], out=q),
              lambda: api.block_evict(tab, lens, mass, 16, 3, freed=mass), lambda: api.block_evict(tab, None, mass, 16, 1 << 33)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: api.block_attn(ca, q, tab, lens, out=q, scale="1"), lambda: api.block_select(ca, q, tab, lens, 4.5, out=st["o"]["sel"])):
        with pytest.raises(TypeError):
            f()


def test_refused_sizes_raise():
    """Fewer query heads than kv heads, too many tokens: an error from the call, with a workspace or
    without one."""
    st = outputs(step_state(np.random.default_rng(6)))
    ca, q, tab, lens = st["cache"], st["q"], st["table"], st["lens"]
    wide = torch.zeros((3, 65, 8, 128), dtype=torch.bfloat16, device="cuda")
    for x, status in ((q[:, :, :1].contiguous(), L.MTP_ERR_INVALID_ARG), (wide, L.MTP_ERR_UNSUPPORTED)):
        sel = torch.zeros((3, x.shape[1], 2, 4), dtype=torch.int32, device="cuda")
        for ws in (None, torch.empty(1 << 20, dtype=torch.uint8, device="cuda")):
            for f in (lambda: api.block_attn(ca, x, tab, lens, ws=ws), lambda: api.block_select(ca, x, tab, lens, 4, ws=ws),
                      lambda: api.block_sparse_attn(ca, x, tab, lens, sel, ws=ws)):
                with pytest.raises(L.MtpError) as e:
                    f()
                assert e.value.status == status


def test_threads_call_at_once():
    """Each thread with a stream and outputs of its own, on one cache that all of them read."""
    st = step_state(np.random.default_rng(4))
    ca, q, tab, lens = st["cache"], st["q"], st["table"], st["lens"]
    want, _ = api.block_attn(ca, q, tab, lens)
    sel, _ = api.block_select(ca, q, tab, lens, 4)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ws = ws2 = None
            for _ in range(50):
                out, ws = api.block_attn(ca, q, tab, lens, ws=ws)
                got, ws2 = api.block_select(ca, q, tab, lens, 4, ws=ws2)
                s.synchronize()
                if not (torch.equal(out, want) and torch.equal(got, sel)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "address"])
def test_new_outputs_are_the_streams_own(raw):
    """A call on another stream does not write into memory that the current stream's work, still
    to run, has yet to write."""
    st = step_state(np.random.default_rng(8))
    ca, q, tab, lens = st["cache"], st["q"], st["table"], st["lens"]
    want, ws = api.block_attn(ca, q, tab, lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        late = [torch.empty_like(want) for _ in range(4)]
        torch.cuda._sleep(20_000_000)  # (10 ms)
        for t in late:
            t.fill_(7)
        del late, t
        out, _ = api.block_attn(ca, q, tab, lens, ws=ws, stream=s.cuda_stream if raw else s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
