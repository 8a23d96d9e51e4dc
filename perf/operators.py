"""Cases of the block-scaled paged cache: append, attention, block selection, attention over selected
blocks, eviction. Each has a plain torch form (`own` false) and the library's call (`own` true).

A cache holds K and V of `nkv` heads of `hd` in blocks of `bs` tokens as E4M3 codes with one fp32 scale
for each block and head; a sequence's positions are found through its block table. The batch's lengths
follow from a case alone, every value from the seed.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
GOLD = 0.6180339887498949


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: every sequence appends one token to a block it may share
        # with 0 .. 15 earlier ones
        dict(name="append_step", op="append", B=24, T=1, max_len=4096, nkv=8, hd=128, bs=16),
        # a whole prompt into an empty cache: the drafter's 32,768 rows of 8 heads x 128
        dict(name="append_prompt_32k", op="append", B=1, T=32768, max_len=32768, nkv=8, hd=128, bs=16),
        # one draft token of one user over a short prompt: latency
        dict(name="attn_draft_1k", op="attn", B=1, T=1, max_len=1000, nq=64, nkv=8, hd=128, bs=16, mass=False),
        # one draft token over the 32,768-row prompt
        dict(name="attn_draft_32k", op="attn", B=1, T=1, max_len=32768, nq=64, nkv=8, hd=128, bs=16, mass=False),
        # a padded batch that verifies up to five draft tokens, ragged, 64-wide heads, blocks of 32
        dict(name="attn_verify_ragged", op="attn", B=31, T=5, max_len=8191, nq=32, nkv=4, hd=64, bs=32, mass=True),
        # a serving batch of long contexts, one token each, with the weights that eviction goes by
        dict(name="attn_batch_32k", op="attn", B=32, T=1, max_len=32768, nq=64, nkv=8, hd=128, bs=16, mass=True),
        # the blocks one token reads of a 32,768-row context
        dict(name="select_32k", op="select", B=1, T=1, max_len=32768, nq=64, nkv=8, hd=128, bs=16, n_sel=128),
        # the same for a batch of up to 131,072 rows, two tokens each
        dict(name="select_batch_128k", op="select", B=16, T=2, max_len=131072, nq=64, nkv=8, hd=128, bs=16, n_sel=256),
        # one token over 128 of its 2,048 blocks
        dict(name="sparse_32k", op="sparse", B=1, T=1, max_len=32768, nq=64, nkv=8, hd=128, bs=16, n_sel=128),
        # a batch of four-token steps over 256 blocks each of long contexts
        dict(name="sparse_batch_64k", op="sparse", B=24, T=4, max_len=65536, nq=64, nkv=8, hd=128, bs=16, n_sel=256),
        # a few short sequences over their bound
        dict(name="evict_small", op="evict", B=8, max_len=8000, bs=16, keep=256),
        # a full server's sequences cut to half
        dict(name="evict_batch", op="evict", B=256, max_len=131072, bs=16, keep=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "select", "sparse", "evict"])
    bs = rng.choice([16, 16, 32, 64])
    if op == "evict":
        B, ml = _log(rng, 1, 256), _log(rng, 500, 131072)
        return dict(op=op, B=B, max_len=ml, bs=bs, keep=max(4, int(ml / bs * rng.uniform(0.2, 0.9))))
    nkv, hd = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    B = _log(rng, 1, 32)
    if op == "append":
        T = _log(rng, 1, max(1, 32768 * 8 * 128 // (B * nkv * hd)))
        return dict(op=op, B=B, T=T, max_len=T + rng.randrange(0, 2000), nkv=nkv, hd=hd, bs=bs)
    T = rng.choice([1, 1, 2, 3, 5, 8])
    G = rng.choice([1, 3, 4, 7, 8, 16])
    # at most the largest listed case's cache bytes, and its work where many rows share them
    most = 32 * 32768 * 8 * 128 // (2 * B * nkv * hd * max(1, G * T // 16))
    ml = _log(rng, 30, max(31, min(131072, most)))
    c = dict(op=op, B=B, T=T, max_len=ml, nq=nkv * G, nkv=nkv, hd=hd, bs=bs)
    if op == "attn":
        return dict(c, mass=rng.random() < 0.5)
    # padded lists are kept small enough for the plain form's gathered copies
    return dict(c, n_sel=min(_log(rng, 4, 256), max(4, 200000000 // (B * T * nkv * hd * bs))))


def _lens(c):
    """Lengths of the batch after this step's tokens, and how many tokens each sequence has in it: the
    first at its most, the others spread, one slot of a larger batch empty."""
    B, T, ml = c["B"], c.get("T", 1), c["max_len"]
    lens = [ml] + [1 + int((ml - 1) * ((b * GOLD) % 1.0)) for b in range(1, B)]
    q = [T if b % 3 != 1 else max(1, T - b % T) for b in range(B)]
    lens = [max(a, n) for a, n in zip(lens, q)]
    if B > 8:
        lens[5], q[5] = 0, 0
    return lens, q


def work(c):
    lens, q = _lens(c)
    bs = c["bs"]
    nb = [-(-n // bs) for n in lens]
    if c["op"] == "evict":
        # mass and table read; table, mass and the freed list written; lengths
        return dict(bytes=4 * sum(5 * n for n in nb) + 12 * c["B"], flops=sum(nb))
    nkv, hd, T = c["nkv"], c["hd"], c["T"]
    if c["op"] == "append":
        touched = sum(-(-n // bs) - (n - k) // bs for n, k in zip(lens, q) if k)
        # new rows in bf16 read, codes written; the rows before them in their first block read; scales, means
        old = sum((n - k) % bs for n, k in zip(lens, q) if k)
        return dict(bytes=nkv * (sum(q) * hd * 6 + old * hd + touched * (hd + 12 + 4)), flops=sum(q) * nkv * hd * 6)
    nq = c["nq"]
    qo = sum(q) * nq * hd * 2
    if c["op"] == "attn":
        extra = sum(nb) * 8 if c["mass"] else 0
        return dict(bytes=sum(lens) * nkv * hd * 2 + sum(nb) * (nkv * 8 + 4) + 2 * qo + extra,
                    flops=4 * hd * nq * sum(n * k for n, k in zip(lens, q)))
    if c["op"] == "select":
        return dict(bytes=sum(nb) * (nkv * (hd + 4) + 4) + qo + sum(q) * nkv * c["n_sel"] * 4,
                    flops=2 * hd * nq * sum(n * k for n, k in zip(nb, q)))
    rows = sum(k * min(n, c["n_sel"] * bs) for n, k in zip(lens, q))
    return dict(bytes=rows * nkv * (hd * 2 + 12 / bs) + 2 * qo, flops=4 * hd * nq * rows)


# ------------------------------------------------------------------------------ inputs
def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    lens, q = _lens(c)
    B, bs = c["B"], c["bs"]
    NB = -(-c["max_len"] // bs)
    nb = torch.tensor([-(-n // bs) for n in lens], device=dev)
    pool = int(sum(-(-n // bs) for n in lens)) + 3
    j = torch.arange(NB, device=dev)
    have = j[None, :] < nb[:, None]
    at = torch.cumsum(nb, 0) - nb
    perm = torch.randperm(pool, generator=g, device=dev)
    table = torch.where(have, perm[torch.where(have, at[:, None] + j[None, :], 0)], -1).to(torch.int32)
    st = dict(c=c, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if c["op"] == "evict":
        # accumulated weights: a few blocks hold most, many nearly nothing
        m = torch.rand((B, NB), generator=g, device=dev).clamp_min(1e-6).pow(-0.7) * 0.01
        st["mass"] = torch.where(have, m, 0.0)
        st["out"] = dict(table=torch.empty_like(table), lens=torch.empty_like(st["lens"]), mass=torch.empty_like(st["mass"]),
                         freed=torch.empty_like(table), n_freed=torch.empty_like(st["lens"]))
        return st
    T, nkv, hd = c["T"], c["nkv"], c["hd"]
    st["q_lens"] = torch.tensor(q, dtype=torch.int32, device=dev)
    shape = (pool, nkv, bs, hd)

    def codes():
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float16).mul_(40.0).to(F8)

    def scales(lo, hi):  # powers of two, as an append leaves them
        return torch.exp2(torch.randint(lo, hi + 1, (pool, nkv), generator=g, device=dev).float())

    st["vs"], st["ks"] = scales(-8, -4), scales(-7, -5)
    if c["op"] == "append":
        st["k"], st["v"] = codes(), codes()
        # new rows as slices of one projection's output; later rows of a sequence are larger, so that scales grow
        kv = torch.randn((B, T, 2 * nkv * hd), generator=g, device=dev)
        grow = torch.exp2(torch.randint(-3, 3, (B, T, 1), generator=g, device=dev).float())
        kv = (kv * grow).to(torch.bfloat16)
        st["new_k"] = kv[..., : nkv * hd].unflatten(-1, (nkv, hd))
        st["new_v"] = kv[..., nkv * hd:].unflatten(-1, (nkv, hd))
        st["mean"] = torch.zeros((pool, nkv, hd), dtype=torch.int8, device=dev)
        st["mean_scale"] = torch.zeros((pool, nkv), device=dev)
        return st
    st["q"] = (torch.randn((B, T, c["nq"], hd), generator=g, device=dev) * 1.5).to(torch.bfloat16)
    if c["op"] == "select":
        st["mean"] = torch.randint(-127, 128, (pool, nkv, hd), generator=g, device=dev, dtype=torch.int8)
        st["mean_scale"] = torch.rand((pool, nkv), generator=g, device=dev) * 0.01 + 0.002
        # the selection reads the means alone: the codes need no values
        st["k"] = st["v"] = torch.empty(shape, dtype=torch.uint8, device=dev).view(F8)
        st["out"] = torch.full((B, T, nkv, c["n_sel"]), -1, dtype=torch.int32, device=dev)
        return st
    st["k"], st["v"] = codes(), codes()
    st["out"] = torch.zeros((B, T, c["nq"], hd), dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.zeros((B, T, c["nq"]), device=dev)
    if c["op"] == "attn":
        if c["mass"]:
            st["mass"] = torch.where(have, torch.rand((B, NB), generator=g, device=dev) * 10.0, 0.0)
            st["out_mass"] = torch.empty_like(st["mass"])
        return st
    # sparse: per token and head the first block, the last one its token sees, and others at random, ascending
    lim = (st["lens"][:, None] - st["q_lens"][:, None] + torch.arange(T, device=dev)[None, :] + 1).clamp_min(0)
    nbt = (lim + bs - 1) // bs  # [B, T]
    key = torch.rand((B, T, nkv, NB), generator=g, device=dev)
    key = torch.where(j < nbt[:, :, None, None], key, 2.0)
    key = torch.where((j == 0) | (j == nbt[:, :, None, None] - 1), key - 1.0, key)
    n = min(c["n_sel"], NB)
    sel = torch.argsort(key, dim=-1)[..., :n]
    sel = torch.where(sel < nbt[:, :, None, None], sel, NB + 1).sort(-1).values
    st["sel"] = torch.full((B, T, nkv, c["n_sel"]), -1, dtype=torch.int32, device=dev)
    st["sel"][..., :n] = torch.where(sel < NB, sel, -1).to(torch.int32)
    return st


# ------------------------------------------------------------------------------ plain forms (32 bits)
def _live(st):
    """[B, T]: whether slot t holds a token, and how many positions it sees."""
    T = st["c"]["T"]
    t = torch.arange(T, device=st["lens"].device)[None, :]
    lim = st["lens"][:, None] - st["q_lens"][:, None] + t + 1
    return t < st["q_lens"][:, None], lim.clamp_min(0)


def _pow2_scale(a):
    """The least power of two >= a / 448; 0 for 0."""
    m, e = torch.frexp(a.double() / 448.0)
    s = torch.ldexp(torch.ones_like(m), e - (m == 0.5).int())
    return torch.where(a > 0, s.clamp(2.0 ** -110, 2.0 ** 120), 0.0).float()


def _plain_append(st):
    c = st["c"]
    B, T, nkv, hd, bs = (c[k] for k in ("B", "T", "nkv", "hd", "bs"))
    dev = st["lens"].device
    end = st["lens"].long()
    beg = end - st["q_lens"].long()
    J = T // bs + 2  # blocks that a sequence's tokens can touch
    lb = (beg // bs)[:, None] + torch.arange(J, device=dev)[None, :]
    hit = lb * bs < end[:, None]
    hit &= (st["q_lens"] > 0)[:, None]
    spare = st["k"].shape[0] - 1
    phys = st["table"].long().gather(1, lb.clamp(0, st["table"].shape[1] - 1))
    # slots that nothing goes to rewrite one block with what it holds: a block no table names or an untouched one
    touched = torch.zeros(spare + 1, device=dev).index_put((phys.clamp_min(0),), hit.float(), accumulate=True)
    idle = torch.argmin(touched)
    phys = torch.where(hit, phys, idle)
    pos = lb[:, :, None] * bs + torch.arange(bs, device=dev)  # [B, J, bs]
    new = (pos >= beg[:, None, None]) & (pos < end[:, None, None]) & hit[:, :, None]
    old = (pos < beg[:, None, None]) & hit[:, :, None]
    b = torch.arange(B, device=dev)[:, None, None]
    t = (pos - beg[:, None, None]).clamp(0, T - 1)
    rows = (new | old).sum(-1).float()[:, :, None]  # [B, J, 1]

    def one(x, cache, scale):
        x = x[b, t].float()  # [B, J, bs, nkv, hd]
        x = torch.where(new[..., None, None], x, 0.0).transpose(2, 3)  # [B, J, nkv, bs, hd]
        a = torch.where(x.isfinite(), x.abs(), 0.0).amax((-1, -2))
        s_old = torch.where(old.any(-1)[..., None], scale[phys], 0.0)
        s = torch.maximum(s_old, _pow2_scale(a))  # [B, J, nkv]
        by = torch.where(s > 0, s, 1.0)
        was = cache[phys].float()
        m_old, m_new = old[:, :, None, :, None], new[:, :, None, :, None]
        val = torch.where(m_old, was * (s_old / by)[..., None, None], x / by[..., None, None]).clamp(-448.0, 448.0).to(F8)
        put = torch.where((m_old | m_new), val.float(), was).to(F8)
        cache[phys] = put
        scale[phys] = torch.where(hit[..., None], s, scale[phys])
        return torch.where(m_old | m_new, val.float(), 0.0), s

    val, s = one(st["new_k"], st["k"], st["ks"])
    one(st["new_v"], st["v"], st["vs"])
    S = val.sum(-2)  # exact: multiples of 2^-9 below 2^15
    ms = S.abs().amax(-1) / 127.0
    code = torch.round(S / torch.where(ms > 0, ms, 1.0)[..., None]).clamp(-127, 127).to(torch.int8)
    st["mean"][phys] = torch.where(hit[:, :, None, None], code, st["mean"][phys])
    st["mean_scale"][phys] = torch.where(hit[..., None], ms * s / rows.clamp_min(1.0), st["mean_scale"][phys])
    return st["k"], st["v"], st["ks"], st["vs"], st["mean"], st["mean_scale"]


def _attend(q, K, V, seen, scale):
    """q [..., R, hd], K, V [..., P, hd], seen [..., R, P] -> out, natural log-sum-exp, weights."""
    s = torch.matmul(q, K.transpose(-1, -2)) * scale
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(s - torch.where(m.isfinite(), m, 0.0)), 0.0)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    return torch.matmul(p, V), torch.where(l > 0, m + torch.log(l), -math.inf)[..., 0], p


def _plain_attn(st):
    c = st["c"]
    B, T, nq, nkv, hd, bs = (c[k] for k in ("B", "T", "nq", "nkv", "hd", "bs"))
    G = nq // nkv
    at = st["table"].long().clamp_min(0)
    NB = at.shape[1]
    live, lim = _live(st)
    pos = torch.arange(NB * bs, device=at.device)
    inside = (pos[None, :] < st["lens"][:, None])[:, None, :, None]

    def rows(cache, scale):
        x = cache[at].float() * scale[at][..., None, None]  # [B, NB, nkv, bs, hd]
        return torch.where(inside, x.transpose(1, 2).reshape(B, nkv, NB * bs, hd), 0.0)

    q = st["q"].float().view(B, T, nkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, nkv, T * G, hd)
    seen = (pos < torch.where(live, lim, 0)[..., None])[:, None, :, None, :].expand(B, 1, T, G, NB * bs).reshape(B, 1, T * G, NB * bs)
    out, lse, p = _attend(q, rows(st["k"], st["ks"]), rows(st["v"], st["vs"]), seen, 1.0 / math.sqrt(hd))
    out = out.view(B, nkv, T, G, hd).permute(0, 2, 1, 3, 4).reshape(B, T, nq, hd)
    lse = lse.view(B, nkv, T, G).permute(0, 2, 1, 3).reshape(B, T, nq)
    out = torch.where(live[..., None, None], out, 0.0).to(torch.bfloat16)
    lse = torch.where(live[..., None], lse, 0.0)
    if not c["mass"]:
        return out, lse
    return out, lse, st["mass"] + p.sum((1, 2)).view(B, NB, bs).sum(-1)


def _plain_select(st):
    c = st["c"]
    B, T, nq, nkv, hd, bs, n = (c[k] for k in ("B", "T", "nq", "nkv", "hd", "bs", "n_sel"))
    at = st["table"].long().clamp_min(0)
    NB = at.shape[1]
    live, lim = _live(st)
    q = st["q"].float().view(B, T, nkv, nq // nkv, hd)
    sq = q.abs().amax(-1) / 127.0
    q8 = torch.round(q / torch.where(sq > 0, sq, 1.0)[..., None])
    mean = st["mean"][at].float()  # [B, NB, nkv, hd]
    dot = torch.einsum("btgih,bngh->btgin", q8, mean)  # whole numbers below 2^24
    sk = st["mean_scale"][at].transpose(1, 2)[:, None, :, None, :]
    score = (dot * (sq[..., None] * sk)).amax(3)  # [B, T, nkv, NB]
    nbt = ((lim + bs - 1) // bs)[:, :, None, None]
    j = torch.arange(NB, device=at.device)
    score = torch.where(j < nbt, score, -math.inf)
    score = torch.where((j < 1) | ((j >= nbt - 1) & (j < nbt)), math.inf, score)
    score = torch.where(j < nbt, score, -math.inf)
    k = min(n, NB)
    top = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    top = torch.where(top < nbt, top, NB).sort(-1).values
    out = torch.full((B, T, nkv, n), -1, dtype=torch.int32, device=at.device)
    out[..., :k] = torch.where((top < NB) & live[:, :, None, None], top, -1).to(torch.int32)
    return out


def _plain_sparse(st):
    c = st["c"]
    B, T, nq, nkv, hd, bs, n = (c[k] for k in ("B", "T", "nq", "nkv", "hd", "bs", "n_sel"))
    live, lim = _live(st)
    sel = st["sel"].long()
    phys = st["table"].long().gather(1, sel.clamp_min(0).view(B, -1)).clamp_min(0).view(B, T, nkv, n)
    g = torch.arange(nkv, device=sel.device)[:, None]
    pos = (sel[..., None] * bs + torch.arange(bs, device=sel.device)).view(B, T, nkv, n * bs)
    ok = ((sel >= 0)[..., None].expand(B, T, nkv, n, bs).reshape(B, T, nkv, n * bs)
          & (pos < torch.where(live, lim, 0)[..., None, None]))

    def rows(cache, scale):
        x = cache[phys, g].float() * scale[phys, g][..., None, None]  # [B, T, nkv, n, bs, hd]
        return torch.where(ok[..., None], x.view(B, T, nkv, n * bs, hd), 0.0)

    q = st["q"].float().view(B, T, nkv, nq // nkv, hd)
    out, lse, _ = _attend(q, rows(st["k"], st["ks"]), rows(st["v"], st["vs"]), ok[..., None, :], 1.0 / math.sqrt(hd))
    out = torch.where(live[..., None, None, None], out, 0.0).to(torch.bfloat16).view(B, T, nq, hd)
    return out, torch.where(live[..., None, None], lse, 0.0).view(B, T, nq)


def _plain_evict(st):
    c = st["c"]
    bs, keep = c["bs"], c["keep"]
    table, mass, lens = st["table"], st["mass"], st["lens"]
    B, NB = table.shape
    j = torch.arange(NB, device=table.device)
    nb = ((lens + bs - 1) // bs)[:, None]
    go = (nb - keep).clamp_min(0)  # how many leave
    may = (j >= 1) & (j < nb - 1)
    order = torch.sort(torch.where(may, mass, math.inf), dim=-1, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand(B, NB).contiguous())
    gone = may & (rank < go)
    stay = (j < nb) & ~gone

    def packed(x, by, fill):
        to = torch.where(by, torch.cumsum(by, 1) - 1, NB)
        return torch.full((B, NB + 1), fill, dtype=x.dtype, device=x.device).scatter_(1, to, x)[:, :NB]

    return (packed(table, stay, -1), (lens - go[:, 0] * bs).to(torch.int32), packed(mass, stay, 0.0),
            packed(table, gone, -1), go[:, 0].to(torch.int32))


# ------------------------------------------------------------------------------ the library's calls
def _cache(st):
    from mtp_speculative_draft_lm_b200 import api

    if "cache" not in st:
        st["cache"] = api.BlockCache.of(st["k"].view(torch.uint8), st["v"].view(torch.uint8), st["ks"], st["vs"],
                                        st.get("mean"), st.get("mean_scale"))
        st["ws"] = None
    return api, st["cache"]


def run(st):
    c = st["c"]
    op = c["op"]
    if not own:
        return dict(append=_plain_append, attn=_plain_attn, select=_plain_select, sparse=_plain_sparse, evict=_plain_evict)[op](st)
    if op == "evict":
        from mtp_speculative_draft_lm_b200 import api

        o = st["out"]
        api.block_evict(st["table"], st["lens"], st["mass"], c["bs"], c["keep"], out_table=o["table"], out_lens=o["lens"],
                        out_mass=o["mass"], freed=o["freed"], n_freed=o["n_freed"])
        return o["table"], o["lens"], o["mass"], o["freed"], o["n_freed"]
    api, cache = _cache(st)
    if op == "append":
        api.block_append(cache, st["new_k"], st["new_v"], st["table"], st["lens"], q_lens=st["q_lens"])
        return st["k"], st["v"], st["ks"], st["vs"], st["mean"], st["mean_scale"]
    if op == "select":
        _, st["ws"] = api.block_select(cache, st["q"], st["table"], st["lens"], c["n_sel"], q_lens=st["q_lens"], out=st["out"],
                                       ws=st["ws"])
        return st["out"]
    if op == "sparse":
        _, st["ws"] = api.block_sparse_attn(cache, st["q"], st["table"], st["lens"], st["sel"], q_lens=st["q_lens"], out=st["out"],
                                            out_lse=st["lse"], ws=st["ws"])
        return st["out"], st["lse"]
    _, st["ws"] = api.block_attn(cache, st["q"], st["table"], st["lens"], q_lens=st["q_lens"], out=st["out"], out_lse=st["lse"],
                                 mass=st.get("mass"), out_mass=st.get("out_mass"), ws=st["ws"])
    return (st["out"], st["lse"], st["out_mass"]) if c["mass"] else (st["out"], st["lse"])


# ------------------------------------------------------------------------------ 64 bits, sequence by sequence
def exact(c, seed):
    st = prepare(c, seed)
    lens, qn = _lens(c)
    op, bs = c["op"], c["bs"]
    if op == "select":
        return None  # whole numbers alone
    if op == "evict":
        return [None, None, _exact_evicted_mass(st, c, lens), None, None]
    nkv, hd, T = c["nkv"], c["hd"], c["T"]
    tab = st["table"].long()
    if op == "append":
        k, v, ks, vs = (st[n].double() for n in ("k", "v", "ks", "vs"))
        msc = st["mean_scale"].double()
        for b, (n, m) in enumerate(zip(lens, qn)):
            if m == 0:
                continue
            beg = n - m
            first, last = beg // bs, (n - 1) // bs
            ph = tab[b, first:last + 1]
            had = beg - first * bs
            for X, S, new in ((k, ks, st["new_k"]), (v, vs, st["new_v"])):
                x = torch.zeros(((last + 1 - first) * bs, nkv, hd), dtype=torch.float64, device=new.device)
                x[had:had + m] = new[b, :m].double()
                x = x.view(-1, bs, nkv, hd).transpose(1, 2)
                amax = x.abs().amax((2, 3))
                s = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / 448.0) - 1e-12)), 0.0)
                full = X[ph]
                if had:
                    s_old = S[ph[0]].clone()
                    s[0] = torch.maximum(s[0], s_old)
                    full[0, :, :had] *= (s_old / s[0])[:, None, None]
                y = x / torch.where(s > 0, s, 1.0)[:, :, None, None]
                r = torch.arange((last + 1 - first) * bs, device=y.device).view(-1, 1, bs, 1)
                full = torch.where((r >= had) & (r < had + m), y, full)
                X[ph], S[ph] = full, s
                if X is k:
                    rows = ((r < had + m).to(torch.float64)).sum(2)
                    val = full.float().to(F8).double() * (r < had + m)
                    msc[ph] = val.sum(2).abs().amax(-1) / 127.0 * s / rows[:, :, 0]
        return k, v, ks, vs, None, msc
    nq = c["nq"]
    G = nq // nkv
    if sum(lens) * nkv * hd > 1.2e9 and op == "attn":
        return None
    out = torch.zeros((c["B"], T, nq, hd), dtype=torch.float64, device=tab.device)
    lse = torch.zeros((c["B"], T, nq), dtype=torch.float64, device=tab.device)
    mass = st["mass"].double() if c.get("mass") else None
    for b, (n, m) in enumerate(zip(lens, qn)):
        nblk = -(-n // bs)
        for t in range(m):
            lim = n - m + t + 1
            q = st["q"][b, t].double().view(nkv, G, hd)
            if op == "attn":
                ph = tab[b, :nblk]
                if t == 0:
                    K = (st["k"][ph].double() * st["ks"][ph].double()[..., None, None]).transpose(0, 1).reshape(nkv, -1, hd)
                    V = (st["v"][ph].double() * st["vs"][ph].double()[..., None, None]).transpose(0, 1).reshape(nkv, -1, hd)
                w = torch.einsum("gih,gph->gip", q, K[:, :lim]) / math.sqrt(hd)
                L = torch.logsumexp(w, -1)
                w = torch.exp(w - L[..., None])
                o = torch.einsum("gip,gph->gih", w, V[:, :lim])
                if mass is not None:
                    full = torch.zeros(nblk * bs, dtype=torch.float64, device=tab.device)
                    full[:lim] = w.sum((0, 1))
                    mass[b, :nblk] += full.view(nblk, bs).sum(1)
            else:
                sel = st["sel"][b, t].long()  # [nkv, n]
                ph = tab[b][sel.clamp_min(0)].clamp_min(0)
                g = torch.arange(nkv, device=tab.device)[:, None]
                K = (st["k"][ph, g].double() * st["ks"][ph, g].double()[..., None, None]).reshape(nkv, -1, hd)
                V = (st["v"][ph, g].double() * st["vs"][ph, g].double()[..., None, None]).reshape(nkv, -1, hd)
                p = (sel[..., None] * bs + torch.arange(bs, device=tab.device)).view(nkv, 1, -1)
                w = torch.einsum("gih,gph->gip", q, K) / math.sqrt(hd)
                w = w.masked_fill((p >= lim) | (sel < 0).repeat_interleave(bs, 1)[:, None, :], -math.inf)
                L = torch.logsumexp(w, -1)
                w = torch.exp(w - L[..., None])
                o = torch.einsum("gip,gph->gih", w, V)
            out[b, t], lse[b, t] = o.reshape(nq, hd), L.reshape(nq)
    return (out, lse, mass) if mass is not None else (out, lse)


def _exact_evicted_mass(st, c, lens):
    got = torch.zeros_like(st["mass"], dtype=torch.float64)
    m = st["mass"].cpu().numpy()
    for b, n in enumerate(lens):
        nb = -(-n // c["bs"])
        leave = max(0, nb - c["keep"])
        inner = sorted(range(1, nb - 1), key=lambda i: (m[b, i], i))[:leave]
        stay = torch.tensor(sorted(set(range(nb)) - set(inner)), dtype=torch.long, device=got.device)
        got[b, : len(stay)] = st["mass"][b].double()[stay]
    return got
