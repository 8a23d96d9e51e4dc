"""Torch-facing helpers over the C ABI: they allocate device buffers with torch
(memory and streams are torch's job here) and call the ``mtp_*`` entry points.
No arithmetic of the method happens in Python."""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass, field

import torch

from . import _lib as L


def _u16(t: torch.Tensor) -> torch.Tensor:
    assert t.dtype in (torch.bfloat16, torch.int16, torch.uint16)
    return t


@dataclass
class Table:
    """A [n, k] weight table on the device in one of the three formats."""
    fmt: int
    n: int
    k: int
    data: torch.Tensor
    row_scale: torch.Tensor | None = None
    block_scale: torch.Tensor | None = None
    global_scale: torch.Tensor | None = None
    desc: L.mtp_weight = field(init=False)

    def __post_init__(self):
        self.desc = L.weight(self.fmt, self.n, self.k, self.data, self.row_scale,
                             self.block_scale, self.global_scale)

    def nbytes(self) -> int:
        b = self.data.numel() * self.data.element_size()
        for t in (self.row_scale, self.block_scale, self.global_scale):
            if t is not None:
                b += t.numel() * t.element_size()
        return b


def bf16_table(w: torch.Tensor) -> Table:
    n, k = w.shape
    return Table(L.MTP_FMT_BF16, n, k, _u16(w.contiguous()))


def quantize_fp8(w: torch.Tensor, stream=None) -> Table:
    n, k = w.shape
    codes = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    scale = torch.empty((n,), dtype=torch.float32, device=w.device)
    L.mtp_quantize_fp8(w, n, k, codes, scale, stream)
    return Table(L.MTP_FMT_FP8_ROW, n, k, codes, row_scale=scale)


def quantize_nvfp4(w: torch.Tensor, ws: torch.Tensor | None = None, stream=None) -> Table:
    n, k = w.shape
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    bscale = torch.empty((n, L.mtp_nvfp4_scale_pitch(k)), dtype=torch.uint8, device=w.device)
    g = torch.empty((1,), dtype=torch.float32, device=w.device)
    nbytes = L.mtp_quantize_nvfp4_ws_bytes(n, k)
    if ws is None:
        ws = torch.zeros((nbytes,), dtype=torch.uint8, device=w.device)
    L.mtp_quantize_nvfp4(w, n, k, codes, bscale, g, ws, ws.numel(), stream)
    return Table(L.MTP_FMT_NVFP4, n, k, codes, block_scale=bscale, global_scale=g)


class LmHead:
    """The fused sweep + argmax over a table, with its zeroed workspace."""

    def __init__(self, table: Table, n_eff: int | None = None, max_m: int = 32):
        self.table = table
        self.n_eff = table.n if n_eff is None else int(n_eff)
        dev = table.data.device
        # room for the host-input entry point's copy of x as well
        nbytes = L.mtp_lm_head_host_ws_bytes(table.desc, self.n_eff, max_m)
        self.ws = torch.zeros((nbytes,), dtype=torch.uint8, device=dev)
        self.dev_err = torch.zeros((1,), dtype=torch.int32, device=dev)

    def bytes_per_call(self, M: int, mask_words: int = 0, rows: int | None = None) -> int:
        """Algorithmic bytes of one sweep: the table rows it must read (all n_eff rows, or
        `rows` of them under a grammar mask), the inputs, the mask words and the
        outputs."""
        t = self.table
        frac = (self.n_eff if rows is None else rows) / t.n
        return int(t.nbytes() * frac) + M * t.k * 2 + mask_words * 4 + M * 8

    def __call__(self, x: torch.Tensor, out_idx: torch.Tensor, out_val=None, out_logits=None,
                 mask=None, mask_words=0, mask_stride_words=0, stream=None, out_logprob=None):
        M = x.shape[0]
        if out_logprob is None:
            L.mtp_lm_head_argmax(self.table.desc, self.n_eff, x, M, mask, mask_words,
                                 mask_stride_words, out_idx, out_val, out_logits, self.dev_err,
                                 self.ws, self.ws.numel(), stream)
        else:
            L.mtp_lm_head_argmax_lp(self.table.desc, self.n_eff, x, M, mask, mask_words,
                                    mask_stride_words, out_idx, out_val, out_logprob,
                                    out_logits, self.dev_err, self.ws, self.ws.numel(), stream)

    def argmax_host(self, x_host: torch.Tensor, out_host: torch.Tensor, mask=None, mask_words=0,
                    mask_stride_words=0, stream=None):
        """One draft step from pinned host memory to pinned host memory: x_host bf16
        [M, k] pinned; out_host int32 [2M] pinned receives the indices, then the values
        (float32 bits). Valid once the stream has synchronised."""
        M = x_host.shape[0]
        L.mtp_lm_head_argmax_host(self.table.desc, self.n_eff, x_host, M, mask, mask_words,
                                  mask_stride_words, out_host, self.dev_err, self.ws,
                                  self.ws.numel(), stream)

    def argmax(self, x: torch.Tensor, mask=None, mask_words=0, mask_stride_words=0,
               logits=False, stream=None, logprob=False):
        """Returns (idx, val, logits or None), plus the top-1 log-probabilities when
        logprob is true."""
        M = x.shape[0]
        dev = x.device
        idx = torch.empty((M,), dtype=torch.int32, device=dev)
        val = torch.empty((M,), dtype=torch.float32, device=dev)
        lg = torch.empty((M, self.n_eff), dtype=torch.bfloat16, device=dev) if logits else None
        lp = torch.empty((M,), dtype=torch.float32, device=dev) if logprob else None
        self(x, idx, val, lg, mask, mask_words, mask_stride_words, stream, out_logprob=lp)
        return (idx, val, lg, lp) if logprob else (idx, val, lg)


def table_rows(table: Table, r0: int, r1: int) -> Table:
    """Rows [r0, r1) of a table as a table of its own (views: rows are contiguous, so a
    vocab shard is a base-pointer offset and a smaller n)."""
    rs = table.row_scale[r0:r1] if table.row_scale is not None else None
    bs = table.block_scale[r0:r1] if table.block_scale is not None else None
    return Table(table.fmt, r1 - r0, table.k, table.data[r0:r1], row_scale=rs, block_scale=bs,
                 global_scale=table.global_scale)


def shard_range(n: int, world: int, rank: int, align: int = 16) -> tuple[int, int]:
    """(row_offset, rows) of rank's vocab shard: equal contiguous ranges in units of
    `align` rows (the sweep's 16-row tiles), the last one shorter; empty when there are
    more ranks than units."""
    units = -(-n // align)
    per = -(-units // world) * align
    off = min(n, rank * per)
    return off, min(n, off + per) - off


#: a shard partial: {f32 max logit, i32 global row (INT32_MAX: none allowed), f32 sum of
#: exp(l - max), unused}, stored as 4 float32 words per input row
EMPTY_PARTIAL = (float("-inf"), 2147483647, 0.0)


def exchange_partials(local: torch.Tensor, group=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """All-gathers every rank's [M, 4] partials into [world, M, 4] (rank-major), the one
    collective of the vocab-sharded sweep (NCCL over NVLink on GPUs)."""
    import torch.distributed as dist

    world = dist.get_world_size(group)
    if out is None:
        out = torch.empty((world,) + tuple(local.shape), dtype=local.dtype, device=local.device)
    # gathered along dim 0 ([world * M, 4]); viewed back as [world, M, 4]
    flat = out.view((world * local.shape[0],) + tuple(local.shape[1:]))
    dist.all_gather_into_tensor(flat, local.contiguous(), group=group)
    return out


class ShardedLmHead:
    """The lm_head sweep + argmax split by vocab over the ranks of a process group: each
    rank sweeps its own rows (mtp_lm_head_shard_partial), the 16-byte partials are
    all-gathered, and every rank merges them (mtp_argmax_merge_partials)."""

    def __init__(self, shard: Table | None, row_offset: int, group=None, max_m: int = 32):
        self.shard = shard
        self.row_offset = int(row_offset)
        self.group = group
        self.head = LmHead(shard, max_m=max_m) if shard is not None and shard.n > 0 else None
        self._bufs = {}

    def _buffers(self, M: int, dev):
        import torch.distributed as dist

        if M not in self._bufs:
            world = dist.get_world_size(self.group)
            self._bufs[M] = dict(
                local=torch.empty((M, 4), dtype=torch.float32, device=dev),
                parts=torch.empty((world, M, 4), dtype=torch.float32, device=dev),
                idx=torch.empty((M,), dtype=torch.int32, device=dev),
                val=torch.empty((M,), dtype=torch.float32, device=dev),
                lp=torch.empty((M,), dtype=torch.float32, device=dev),
                err=torch.zeros((1,), dtype=torch.int32, device=dev), world=world)
        return self._bufs[M]

    def argmax(self, x: torch.Tensor, mask=None, mask_words=0, mask_stride_words=0,
               logprob=False, stream=None):
        """Returns (idx, val, err) or (idx, val, logprob, err): the merged result, the
        same on every rank; err is the merge's device error word. The returned tensors
        are reused by the next call with the same M."""
        M = x.shape[0]
        b = self._buffers(M, x.device)
        local = b["local"]
        if self.head is None:  # no rows here: an empty partial
            local.zero_()
            local[:, 0] = EMPTY_PARTIAL[0]
            local.view(torch.int32)[:, 1] = EMPTY_PARTIAL[1]
        else:
            L.mtp_lm_head_shard_partial(self.shard.desc, self.shard.n, self.row_offset, x, M, mask,
                                        mask_words, mask_stride_words, local, None,
                                        self.head.dev_err, self.head.ws, self.head.ws.numel(),
                                        stream)
        exchange_partials(local, self.group, out=b["parts"])
        b["err"].zero_()
        lp = b["lp"] if logprob else None
        L.mtp_argmax_merge_partials(b["parts"], b["world"], M, b["idx"], b["val"], lp, b["err"],
                                    stream)
        return (b["idx"], b["val"], lp, b["err"]) if logprob else (b["idx"], b["val"], b["err"])


def combine(embed, token_ids, hidden, w_norm_embed, w_norm_hidden, eps, fc: Table,
            out=None, dev_err=None, stream=None, norm_mode=L.MTP_NORM_W):
    M, h = hidden.shape
    if out is None:
        out = torch.empty((M, h), dtype=torch.bfloat16, device=hidden.device)
    L.mtp_combine(embed, embed.shape[0], token_ids, hidden, M, h, w_norm_embed, w_norm_hidden,
                  eps, norm_mode, fc.desc, out, dev_err, stream)
    return out


def draft_step(embed, token_ids, hidden, w_norm_embed, w_norm_hidden, eps, fc, head,
               n_eff=None, mask=None, mask_words=0, mask_stride_words=0, out_y=None,
               out_idx=None, out_val=None, dev_err=None, stream=None, norm_mode=L.MTP_NORM_W):
    """One whole draft step (combiner + lm_head sweep + argmax) for a small BF16 head in
    one launch: returns (idx, val, y)."""
    M, h = hidden.shape
    dev = hidden.device
    n = head.shape[0] if n_eff is None else int(n_eff)
    out_y = torch.empty((M, h), dtype=torch.bfloat16, device=dev) if out_y is None else out_y
    out_idx = torch.empty((M,), dtype=torch.int32, device=dev) if out_idx is None else out_idx
    out_val = torch.empty((M,), dtype=torch.float32, device=dev) if out_val is None else out_val
    L.mtp_draft_step(embed, embed.shape[0], token_ids, hidden, M, h, w_norm_embed, w_norm_hidden,
                     eps, norm_mode, fc, head, n, mask, mask_words, mask_stride_words, out_y,
                     out_idx, out_val, dev_err, stream)
    return out_idx, out_val, out_y


def paged_decode_attn(q, nkv, k_cache, v_cache, block_table, seq_len, k_scale=1.0, v_scale=1.0,
                      scale=None, out=None, ws=None, dev_err=None, stream=None):
    """Single-token decode attention of q [nq, hd] (bf16) over cache rows 0 .. seq_len - 1 of
    a paged E4M3 cache [num_blocks, block_size, nkv, hd]; returns (out, ws)."""
    nq, hd = q.shape
    num_blocks, block_size = k_cache.shape[0], k_cache.shape[1]
    scale = 1.0 / float(hd) ** 0.5 if scale is None else float(scale)
    if out is None:
        out = torch.empty((nq, hd), dtype=torch.bfloat16, device=q.device)
    nbytes = L.mtp_paged_decode_attn_ws_bytes(nq, hd, seq_len)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty((nbytes,), dtype=torch.uint8, device=q.device)
    L.mtp_paged_decode_attn(q, nq, nkv, hd, k_cache, v_cache, block_table, block_table.numel(),
                            block_size, num_blocks, seq_len, k_scale, v_scale, scale, out, dev_err,
                            ws, ws.numel(), stream)
    return out, ws


def _need(device: int, dtype, numel: int, *tensors):
    """Raises unless each tensor (None: left out) is contiguous, of this type and size, on this device."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.numel() != numel or t.get_device() != device
                              or not t.is_contiguous()):
            raise ValueError(f"expected a contiguous {dtype} tensor of {numel} elements on device {device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")


@dataclass(frozen=True, eq=False)  # (desc holds the tensors' addresses: another tensor is another cache)
class BlockCache:
    """A block-scaled paged cache: E4M3 codes k, v with logical shape [num_blocks, nkv,
    block_size, hd] (uint8, any strides with hd contiguous), fp32 scales [num_blocks, nkv] and,
    for block selection, 8-bit mean keys [num_blocks, nkv, hd] with their scales.

    The block_* calls run on the current stream, or on their argument `stream` (a torch stream or
    its address): the caller orders that one behind what writes their inputs and before what
    reads their outputs; any tensor of the call may be let go as soon as it returns. Token slots
    that q_lens leaves empty are not written: in an output that a call makes itself (out=None) they
    hold whatever its memory held."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_mean: torch.Tensor | None = None
    k_mean_scale: torch.Tensor | None = None
    desc: L.mtp_block_cache = field(init=False)
    device: int = field(init=False)

    def __post_init__(self):
        nb, nkv, bs, hd = self.k.shape
        object.__setattr__(self, "device", self.k.get_device())
        if self.k.dtype is not torch.uint8 or self.v.dtype is not torch.uint8 or self.v.shape != self.k.shape:
            raise ValueError("k and v: uint8 codes of one shape")
        if self.k.stride() != self.v.stride() or self.k.stride(3) != 1 or self.v.get_device() != self.device:
            raise ValueError("k and v: one layout with hd contiguous, on one device")
        _need(self.device, torch.float32, nb * nkv, self.k_scale, self.v_scale, self.k_mean_scale)
        _need(self.device, torch.int8, nb * nkv * hd, self.k_mean)
        object.__setattr__(self, "desc", L.mtp_block_cache(
            nkv, hd, bs, 0, nb, self.k.stride(0), self.k.stride(1), self.k.stride(2),
            *(L._ptr(t) for t in self.tensors())))

    def tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale, self.k_mean, self.k_mean_scale

    @classmethod
    def empty(cls, num_blocks: int, nkv: int, hd: int, block_size: int = 16, device="cuda"):
        """A cache with its codes, scales and means zero, one block's rows of a head contiguous."""
        z = lambda shape, t: torch.zeros(shape, dtype=t, device=device)  # noqa: E731
        n = (num_blocks, nkv)
        return cls(z(n + (block_size, hd), torch.uint8), z(n + (block_size, hd), torch.uint8),
                   z(n, torch.float32), z(n, torch.float32), z(n + (hd,), torch.int8),
                   z(n, torch.float32))

    @classmethod
    def of(cls, k, v, k_scale, v_scale, k_mean=None, k_mean_scale=None):
        """Over tensors the caller has."""
        return cls(k, v, k_scale, v_scale, k_mean, k_mean_scale)

    @classmethod
    def of_prefill(cls, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float = 1.0,
                   v_scale: float = 1.0):
        """Over the [num_blocks, block_size, nkv, hd] cache that prefill_kv writes, every block
        and head at the call's one scale. It has no means (block_select needs them)."""
        nb, _, nkv, _ = k_cache.shape
        ks = torch.full((nb, nkv), float(k_scale), dtype=torch.float32, device=k_cache.device)
        return cls(k_cache.transpose(1, 2), v_cache.transpose(1, 2), ks,
                   torch.full_like(ks, float(v_scale)))


_calls = None


def _block():
    """The module that makes the block cache's calls (csrc/block_calls.cpp), with the library's
    functions. It checks each tensor (type, size, contiguity, device) before the call."""
    global _calls
    if _calls is None:
        lib = L.load()
        from . import _block as m

        m.init(*(C.cast(getattr(lib, n), C.c_void_p).value for n in (
            "mtp_block_append", "mtp_block_attn_ws_bytes", "mtp_block_attn",
            "mtp_block_select_ws_bytes", "mtp_block_select", "mtp_block_sparse_attn_ws_bytes",
            "mtp_block_sparse_attn", "mtp_block_evict")))
        _calls = m
    return _calls


def _token_stride(x: torch.Tensor) -> int:
    """Elements between the tokens of x [B, T, heads, hd], whose heads are packed."""
    return _block().token_stride(x)


def _torch_stream(stream, device: torch.device):
    """A stream argument (a torch stream or an address; 0 is the default stream) as torch's object."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    address = L._stream(stream)
    # (torch takes an external address of 0 for none at all, and gives a stream of its pool)
    return torch.cuda.ExternalStream(address, device=device) if address else torch.cuda.default_stream(device)


def _new(shape, dtype, device: int, stream):
    """A tensor that a call on `stream` writes (None: the current one): that stream's memory, whose
    earlier use its work comes after, and not given back before the current stream's use ends."""
    if device < 0:
        raise ValueError("the tensors must be on a GPU")
    dev = torch.device("cuda", device)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(_torch_stream(stream, dev)):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _used_on(stream, device: int, *tensors):
    """Tells the allocator that a call on `stream` (None: the current one, as any torch call) uses these
    tensors: one that the caller lets go while the call runs is not handed out before it has ended."""
    if stream is not None:
        s = _torch_stream(stream, torch.device("cuda", device))
        for t in tensors:
            if t is not None:
                t.record_stream(s)


def _with_ws(where: str, call, cache: BlockCache, head: tuple, tail: tuple, ws, stream):
    """Makes a call whose last argument is its workspace, with a new one if ws is None or too
    small (the call then says how large, and launches nothing); returns the workspace."""
    args = _call(cache, *head, stream) + tail
    r = call(*args, ws)
    if r > 0:
        ws = _new((r,), torch.uint8, cache.device, stream)
        r = call(*args, ws)
    if r:
        raise L.MtpError(-r, where)
    if stream is not None:
        _used_on(stream, cache.device, *cache.tensors(), *(t for t in (*head, *tail, ws) if isinstance(t, torch.Tensor)))
    return ws


def _call(cache: BlockCache, x, block_table, seq_lens, q_lens, dev_err, stream) -> tuple:
    """What every call over a cache begins with."""
    return (C.addressof(cache.desc), cache.device, x, block_table, seq_lens, q_lens, dev_err,
            _address(stream))


def _address(stream):
    """The stream as _block takes it (None: the current one, which it looks up itself)."""
    return None if stream is None else L._stream(stream)


def block_append(cache: BlockCache, k, v, block_table, seq_lens, q_lens=None, dev_err=None,
                 stream=None):
    """Writes the new rows k, v [B, T, nkv, hd] (bf16, slices of a projection allowed) at the end
    of each sequence (seq_lens counts them already) and updates scales and means."""
    r = _block().append(*_call(cache, k, block_table, seq_lens, q_lens, dev_err, stream), v)
    if r:
        raise L.MtpError(-r, "mtp_block_append")
    if stream is not None:
        _used_on(stream, cache.device, *cache.tensors(), k, v, block_table, seq_lens, q_lens, dev_err)


def block_attn(cache: BlockCache, q, block_table, seq_lens, q_lens=None, scale=None, out=None,
               out_lse=None, mass=None, out_mass=None, ws=None, dev_err=None, stream=None):
    """Attention of q [B, T, nq, hd] over each sequence's cached positions (causal among the T
    tokens); out_mass [B, n_table] accumulates each block's softmax weight. Returns (out, ws); a
    ws that is passed in again saves its allocation. (With out_mass it takes 4 B T nq bytes for
    every 16 positions of block_table's width: mtp_block_attn_ws_bytes tells.)"""
    out = _new(q.shape, torch.bfloat16, cache.device, stream) if out is None else out
    ws = _with_ws("mtp_block_attn", _block().attn, cache, (q, block_table, seq_lens, q_lens, dev_err),
                  (scale, out, out_lse, mass, out_mass), ws, stream)
    return out, ws


def block_select(cache: BlockCache, q, block_table, seq_lens, n_sel, n_first=1, n_last=1,
                 q_lens=None, out=None, ws=None, dev_err=None, stream=None):
    """The n_sel blocks that each token and kv head attends to, by the 8-bit product of its
    query heads with the blocks' mean keys: (sel [B, T, nkv, n_sel] i32, ws)."""
    if out is None:
        out = _new((*q.shape[:2], cache.desc.nkv, n_sel), torch.int32, cache.device, stream)
    ws = _with_ws("mtp_block_select", _block().select, cache, (q, block_table, seq_lens, q_lens, dev_err),
                  (n_sel, n_first, n_last, out), ws, stream)
    return out, ws


def block_sparse_attn(cache: BlockCache, q, block_table, seq_lens, sel, q_lens=None, scale=None,
                      out=None, out_lse=None, ws=None, dev_err=None, stream=None):
    """block_attn over the blocks that sel [B, T, nkv, n_sel] lists. Returns (out, ws)."""
    out = _new(q.shape, torch.bfloat16, cache.device, stream) if out is None else out
    ws = _with_ws("mtp_block_sparse_attn", _block().sparse_attn, cache, (q, block_table, seq_lens, q_lens, dev_err),
                  (sel, scale, out, out_lse), ws, stream)
    return out, ws


def block_evict(block_table, seq_lens, mass, block_size, keep, n_first=1, n_last=1, out_table=None,
                out_lens=None, out_mass=None, freed=None, n_freed=None, stream=None):
    """Bounds each sequence to `keep` blocks by accumulated weight: (out_table, out_lens,
    out_mass, freed, n_freed). Outputs may be the inputs (in place)."""
    B, n_table = block_table.shape
    dev = block_table.get_device()
    out_table = _new((B, n_table), torch.int32, dev, stream) if out_table is None else out_table
    out_lens = _new((B,), torch.int32, dev, stream) if out_lens is None else out_lens
    out_mass = _new((B, n_table), torch.float32, dev, stream) if out_mass is None else out_mass
    freed = _new((B, n_table), torch.int32, dev, stream) if freed is None else freed
    n_freed = _new((B,), torch.int32, dev, stream) if n_freed is None else n_freed
    r = _block().evict(block_table, seq_lens, mass, block_size, keep, n_first, n_last, out_table,
                       out_lens, out_mass, freed, n_freed, _address(stream))
    if r:
        raise L.MtpError(-r, "mtp_block_evict")
    _used_on(stream, dev, block_table, seq_lens, mass, out_table, out_lens, out_mass, freed, n_freed)
    return out_table, out_lens, out_mass, freed, n_freed


def aligned_empty(nbytes: int, align: int, device) -> torch.Tensor:
    """A uint8 device buffer of nbytes whose address is a multiple of align (torch only
    promises 512 bytes)."""
    raw = torch.empty((nbytes + align,), dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % align
    return raw[off: off + nbytes]


def prefill_kv(inputs: dict, k_cache: torch.Tensor, v_cache: torch.Tensor, chunk_rows: int = 2048,
               ws: torch.Tensor | None = None, dev_err: torch.Tensor | None = None, stream=None):
    """Drafter-context prefill over device tensors named as in synth.prefill_inputs (plus the
    optional "norm_mode", "k_norm" [hd] and "in_norm" [h] entries)."""
    d = inputs
    R, h = d["hidden"].shape
    nkv, hd = int(d["nkv"]), int(d["hd"])
    chunk = min(int(chunk_rows), R)
    nbytes = L.mtp_prefill_ws_bytes(chunk, h, nkv, hd)
    if ws is None:
        ws = aligned_empty(nbytes, 1024, k_cache.device)
    L.mtp_prefill_kv(d["embed"], d["embed"].shape[0], d["tokens"], d["hidden"], R, h,
                     d["w_norm_embed"], d["w_norm_hidden"], d["eps"], int(d.get("norm_mode", 0)),
                     d["fc"], d["wk"], d["wv"], d.get("k_norm"), d.get("in_norm"), nkv, hd, d["rope_base"],
                     d["rope_pos"], int(d["cache_start"]),
                     d["block_table"], d["block_table"].numel(), int(d["block_size"]), k_cache,
                     v_cache, k_cache.shape[0], d["k_scale"], d["v_scale"], chunk, ws, ws.numel(),
                     dev_err, stream)
    return ws
