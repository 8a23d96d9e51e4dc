"""The block-scaled cache's entry points without a GPU: every refusal happens on the host before
any CUDA call, and the Python helpers refuse layouts that the C ABI cannot describe."""
import ctypes as C

import pytest
import torch

from mtp_speculative_draft_lm_b200 import _lib as L
from mtp_speculative_draft_lm_b200 import api
from mtp_speculative_draft_lm_b200 import build as B

INV, UNS, WS = L.MTP_ERR_INVALID_ARG, L.MTP_ERR_UNSUPPORTED, L.MTP_ERR_WORKSPACE
A, X, OUT, WSP = 0x10000, 0x20000, 0x30000, 0x40000


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return L.load()


def cache(**kw):
    d = dict(nkv=8, hd=128, block_size=16, reserved=0, num_blocks=100, block_stride=8 * 16 * 128, head_stride=16 * 128,
             row_stride=128, k=A, v=A, k_scale=A, v_scale=A, k_mean=A, k_mean_scale=A)
    d.update(kw)
    return L.mtp_block_cache(*(d[n] for n, _ in L.mtp_block_cache._fields_))


BAD_CACHES = [
    (dict(nkv=0), INV), (dict(hd=0), INV), (dict(hd=96), UNS), (dict(block_size=0), INV), (dict(block_size=24), UNS),
    (dict(block_size=128), UNS), (dict(reserved=1), INV), (dict(num_blocks=0), INV), (dict(num_blocks=1 << 31), UNS),
    (dict(nkv=4097), UNS), (dict(k_mean=None), INV), (dict(k_mean_scale=None), INV), (dict(k_mean=A + 8), INV),
    (dict(k_mean_scale=A + 2), INV)]
BAD_CODES = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k_scale=None), INV), (dict(v_scale=None), INV), (dict(k=A + 8), INV),
    (dict(v=A + 4), INV), (dict(k_scale=A + 2), INV), (dict(block_stride=0), INV), (dict(head_stride=8), INV),
    (dict(row_stride=64), INV), (dict(row_stride=136), INV), (dict(block_stride=-16), INV), (dict(row_stride=1 << 39), UNS)]


def append(c, k=X, v=X, stride=1024, nb=2, T=3, lens=X, q_lens=None, table=X, n_table=10, err=None):
    return L.raw_status("mtp_block_append", C.byref(c) if c else None, k, v, stride, nb, T, lens, q_lens, table, n_table, err, None)


def attn(c, q=X, stride=8192, nb=2, T=3, nq=64, lens=X, q_lens=None, table=X, n_table=10, scale=0.1, out=OUT, lse=None,
         mass=None, out_mass=None, err=None, ws=WSP, nbytes=None, sel=None, n_sel=0):
    p = C.byref(c) if c else None
    if sel is None:
        nbytes = L.load().mtp_block_attn_ws_bytes(p, nb, T, nq, n_table, int(out_mass is not None)) if nbytes is None else nbytes
        return L.raw_status("mtp_block_attn", p, q, stride, nb, T, nq, lens, q_lens, table, n_table, scale, out, lse, mass,
                            out_mass, err, ws, nbytes, None)
    nbytes = L.load().mtp_block_sparse_attn_ws_bytes(p, nb, T, nq, n_sel) if nbytes is None else nbytes
    return L.raw_status("mtp_block_sparse_attn", p, q, stride, nb, T, nq, lens, q_lens, table, n_table, sel or None, n_sel,
                        scale, out, lse, err, ws, nbytes, None)


def select(c, q=X, stride=8192, nb=2, T=3, nq=64, lens=X, q_lens=None, table=X, n_table=10, n_sel=4, first=1, last=1, sel=OUT,
           ws=WSP, nbytes=None):
    p = C.byref(c) if c else None
    nbytes = L.load().mtp_block_select_ws_bytes(p, nb, T, n_table) if nbytes is None else nbytes
    return L.raw_status("mtp_block_select", p, q, stride, nb, T, nq, lens, q_lens, table, n_table, n_sel, first, last, sel,
                        None, ws, nbytes, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES + BAD_CODES)
def test_bad_descriptors(bad, status):
    for f in (append, attn, lambda c: attn(c, sel=X, n_sel=4)):
        assert f(cache(**bad)) == status, bad
    if (bad, status) in BAD_CACHES:
        assert select(cache(**bad)) == status, bad


def test_no_descriptor():
    assert append(None) == attn(None) == select(None) == attn(None, sel=X, n_sel=4) == INV
    assert L.load().mtp_block_attn_ws_bytes(None, 1, 1, 8, 10, 0) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(nb=0), INV), (dict(T=0), INV), (dict(lens=None), INV), (dict(table=None), INV), (dict(n_table=0), INV),
    (dict(lens=X + 2), INV), (dict(q_lens=X + 1), INV), (dict(table=X + 2), INV), (dict(nb=65536), UNS),
    (dict(n_table=(1 << 26) + 1), UNS)])
def test_bad_batches(bad, status):
    for f in (append, attn, select, lambda c, **kw: attn(c, sel=X, n_sel=4, **kw)):
        assert f(cache(), **bad) == status, bad


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INV), (dict(q=X + 8), INV), (dict(nq=0), INV), (dict(nq=60), INV), (dict(stride=8191), INV),
    (dict(stride=8196), INV), (dict(nq=136, stride=136 * 128), UNS), (dict(T=65), UNS)])
def test_bad_queries(bad, status):
    for f in (attn, select, lambda c, **kw: attn(c, sel=X, n_sel=4, **kw)):
        assert f(cache(), **bad) == status, bad


def test_append_refuses():
    assert append(cache(), k=None) == append(cache(), v=None) == append(cache(), k=X + 8) == INV
    assert append(cache(), stride=1016) == append(cache(), stride=1028) == INV
    assert append(cache(), err=X + 2) == INV
    assert append(cache(), T=(1 << 30) + 1) == UNS


def test_attn_refuses():
    for f in (attn, lambda c, **kw: attn(c, sel=X, n_sel=4, **kw)):
        assert f(cache(), out=None) == f(cache(), out=OUT + 8) == f(cache(), lse=OUT + 2) == INV
        assert f(cache(), scale=-1.0) == f(cache(), scale=float("nan")) == f(cache(), scale=float("inf")) == INV
        assert f(cache(), ws=None) == f(cache(), ws=WSP + 4) == f(cache(), nbytes=0) == WS
    assert attn(cache(), mass=X) == INV  # mass needs out_mass
    assert attn(cache(), out_mass=X + 2) == INV
    need = L.load().mtp_block_attn_ws_bytes(C.byref(cache()), 2, 3, 64, 10, 1)
    assert need > L.load().mtp_block_attn_ws_bytes(C.byref(cache()), 2, 3, 64, 10, 0) > 0
    assert attn(cache(), out_mass=X, nbytes=need - 16) == WS
    assert attn(cache(), sel=0, n_sel=4) == attn(cache(), sel=X, n_sel=0) == attn(cache(), sel=X + 2, n_sel=4) == INV
    assert attn(cache(), sel=X, n_sel=(1 << 26) + 1, nbytes=0) == UNS


def test_select_refuses():
    assert select(cache(k_mean=None, k_mean_scale=None)) == INV
    assert select(cache(k=None, v=None, k_scale=None, v_scale=None), ws=None) == WS  # codes are not needed
    for bad in (dict(sel=None), dict(sel=OUT + 2), dict(n_sel=1), dict(first=-1), dict(last=0), dict(first=4), dict(n_sel=0)):
        assert select(cache(), **bad) == INV, bad
    assert select(cache(), nbytes=16) == select(cache(), ws=WSP + 8) == WS


def test_evict_refuses():
    def ev(nb=2, table=X, n_table=10, lens=X, mass=X, bs=16, keep=4, first=1, last=1, ot=OUT, ol=OUT, om=OUT, fr=OUT, nf=OUT):
        return L.raw_status("mtp_block_evict", nb, table, n_table, lens, mass, bs, keep, first, last, ot, ol, om, fr, nf, None)

    for bad in (dict(nb=0), dict(table=None), dict(n_table=0), dict(lens=None), dict(mass=None), dict(bs=0), dict(keep=1),
                dict(keep=0), dict(first=-1), dict(last=0), dict(ot=None), dict(ol=None), dict(om=None), dict(fr=None),
                dict(nf=None), dict(mass=X + 2), dict(ot=OUT + 1), dict(first=2**31 - 1)):
        assert ev(**bad) == INV, bad
    assert ev(nb=65536) == ev(n_table=(1 << 26) + 1) == UNS


def test_python_layouts():
    t = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    assert api._token_stride(t) == 256
    fused = torch.zeros((2, 3, 12 * 64), dtype=torch.bfloat16)
    assert api._token_stride(fused[..., 256:512].unflatten(-1, (4, 64))) == 768
    assert api._token_stride(fused[:, :1, :256].unflatten(-1, (4, 64))) == 3 * 768
    for bad in (t.float(), t.transpose(1, 2), fused[:, :2, :256].unflatten(-1, (4, 64)), t[..., ::2]):
        with pytest.raises(ValueError):
            api._token_stride(bad)


def test_workspace_sizes_of_refused_calls():
    """Sizes that a call refuses (fewer query heads than kv heads among them) need no workspace."""
    lib, c = L.load(), C.byref(cache())
    assert lib.mtp_block_attn_ws_bytes(c, 2, 3, 64, 10, 0) > 0 and lib.mtp_block_sparse_attn_ws_bytes(c, 2, 3, 64, 4) > 0
    for nq in (-8, 0, 1, 4, 7, 60, 136):
        assert lib.mtp_block_attn_ws_bytes(c, 2, 3, nq, 10, 1) == lib.mtp_block_sparse_attn_ws_bytes(c, 2, 3, nq, 4) == 0
    for B, T, n in ((0, 3, 10), (65536, 3, 10), (2, 0, 10), (2, 65, 10), (2, 3, 0), (2, 3, (1 << 26) + 1), (-1, 3, 10)):
        assert lib.mtp_block_attn_ws_bytes(c, B, T, 64, n, 0) == lib.mtp_block_select_ws_bytes(c, B, T, n) == 0
        assert lib.mtp_block_sparse_attn_ws_bytes(c, B, T, 64, n) == 0
