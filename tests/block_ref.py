"""Plain references of the block-scaled cache's operators on the CPU: codes, scales, means,
lists and tables exactly (fp32 steps rounded to nearest, as the header states them), attention
in 64 bits with the error each output may have, derived from the stated roundings."""
import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn
BAD_SLOT = 4


def encode(x: np.ndarray) -> np.ndarray:
    """fp32 -> E4M3 codes, to nearest even, saturating; NaN becomes 0x7F."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).clamp(-448.0, 448.0)
    c = t.to(F8).view(torch.uint8).numpy().copy()
    c[np.isnan(x)] = 0x7F
    return c


def decode(c: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(c)).view(F8).float().numpy()


def pow2_scale(a: float) -> float:
    if a == 0:
        return 0.0
    m, e = math.frexp(a / 448.0)  # exact where it matters: a has 8 bits and 448 = 7 2^6
    return float(min(max(2.0 ** (e - (1 if m == 0.5 else 0)), 2.0 ** -110), 2.0 ** 120))


def steps(seq_lens, q_lens, T):
    for b, n in enumerate(seq_lens):
        n = max(int(n), 0)
        yield b, n, (min(max(int(q_lens[b]), 0), T) if q_lens is not None else T)


def append(c, x_k, x_v, table, seq_lens, q_lens=None):
    """c: dict of numpy arrays k, v [N, nkv, bs, hd] u8, ks, vs [N, nkv] f32, mean i8, mscale f32
    (changed in place); x_k, x_v fp32 [B, T, nkv, hd]. Returns the flags."""
    N, nkv, bs, hd = c["k"].shape
    flags = 0
    f32 = np.float32
    for b, n, ql in steps(seq_lens, q_lens, x_k.shape[1]):
        beg = n - ql
        if ql == 0:
            continue
        if beg < 0 and n > 0:
            flags |= BAD_SLOT
        for lb in range(max(beg, 0) // bs, (n + bs - 1) // bs):
            ph = int(table[b, lb]) if lb < table.shape[1] else -1
            if not 0 <= ph < N:
                flags |= BAD_SLOT
                continue
            r0, r1 = max(beg, lb * bs) - lb * bs, min(n, lb * bs + bs) - lb * bs
            r0 = max(r0, 0)
            t0 = lb * bs + r0 - beg
            for g in range(nkv):
                for codes, scales, x in ((c["k"], c["ks"], x_k), (c["v"], c["vs"], x_v)):
                    new = x[b, t0:t0 + r1 - r0, g]
                    fin = np.abs(new[np.isfinite(new)])
                    s = f32(pow2_scale(float(fin.max()) if fin.size else 0.0))
                    if r0 > 0:
                        s_old = scales[ph, g]
                        s = max(s, s_old)
                        if s != s_old:
                            codes[ph, g, :r0] = encode(decode(codes[ph, g, :r0]) * (s_old / s))
                    with np.errstate(all="ignore"):
                        codes[ph, g, r0:r1] = encode(new / s if s > 0 else new)
                    scales[ph, g] = s
                if c.get("mean") is not None:
                    S = decode(c["k"][ph, g, :r1]).astype(np.float64).sum(0)
                    S = np.where(np.isnan(S), 0.0, S).astype(f32)
                    ms = f32(np.abs(S).max()) * (f32(1.0) / f32(127.0))
                    c["mean"][ph, g] = np.rint(S / ms).astype(np.int8) if ms > 0 else 0
                    c["mscale"][ph, g] = f32(f32(ms * c["ks"][ph, g]) / f32(r1))
    return flags


def attend(c, q, table, seq_lens, q_lens=None, scale=None, sel=None):
    """fp64 attention. q fp32 [B, T, nq, hd]. Returns dict(out, lse, mass, and the bound of each
    one's error: out_tol, lse_tol, mass_tol; live [B, T]; flags)."""
    N, nkv, bs, hd = c["k"].shape
    B, T, nq, _ = q.shape
    G = nq // nkv
    scale = 1.0 / math.sqrt(hd) if scale is None else scale
    n_table = table.shape[1]
    z = lambda *s: np.zeros(s)  # noqa: E731
    r = dict(out=z(B, T, nq, hd), lse=np.full((B, T, nq), -np.inf), mass=z(B, n_table), out_tol=z(B, T, nq, hd),
             lse_tol=z(B, T, nq), mass_tol=z(B, n_table), live=np.zeros((B, T), bool), flags=0)
    K, V = decode(c["k"]).astype(np.float64), decode(c["v"]).astype(np.float64)
    for b, n, ql in steps(seq_lens, q_lens, T):
        for t in range(ql):
            r["live"][b, t] = True
            lim = n - ql + t + 1
            for g in range(nkv):
                lbs = range((max(lim, 0) + bs - 1) // bs) if sel is None else [int(j) for j in sel[b, t, g] if j >= 0]
                k, v, blk = [], [], []
                for j in lbs:
                    rows = min(bs, lim - j * bs)
                    if rows <= 0:
                        continue
                    ph = int(table[b, j]) if j < n_table else -1
                    if not 0 <= ph < N:
                        r["flags"] |= BAD_SLOT
                        continue
                    k.append(K[ph, g, :rows] * c["ks"][ph, g])
                    v.append(V[ph, g, :rows] * c["vs"][ph, g])
                    blk += [j] * rows
                if not k:
                    continue
                k, v, blk = np.concatenate(k), np.concatenate(v), np.array(blk)
                P = len(blk)
                for i in range(g * G, g * G + G):
                    qi = q[b, t, i].astype(np.float64)
                    s = scale * (k @ qi)
                    m = s.max()
                    w = np.exp(s - m)
                    l = w.sum()
                    lse = m + math.log(l)
                    w /= l
                    r["out"][b, t, i] = w @ v
                    r["lse"][b, t, i] = lse
                    np.add.at(r["mass"][b], blk, w)
                    # a score: hd products and sums in fp32 (the matrix unit may truncate: a whole
                    # step each), its two scales, log2(e); then 2^x of a difference, to 2^-22
                    es = (hd + 8) * 2.0 ** -23 * scale * (np.abs(k) @ np.abs(qi)) + 2.0 ** -22 * (np.abs(s - m) + 1)
                    e = es.max()
                    sums = (P + 64) * 2.0 ** -24
                    # weights rounded to f16 (2^-11 relative, 2^-25 absolute below 2^-14 of the
                    # largest), numerator and denominator each; the output rounded to bf16
                    av = w @ np.abs(v)
                    r["out_tol"][b, t, i] = (2.0 ** -8 * np.abs(r["out"][b, t, i]) + av * (2.0 ** -10 + 4 * e + 4 * sums)
                                             + 2.0 ** -24 / l * (np.abs(v).sum(0) + P * av) + 1e-37)
                    r["lse_tol"][b, t, i] = e + sums + 2.0 ** -21 * (1 + abs(lse))
                    np.add.at(r["mass_tol"][b], blk, w * (2 * e + 2 * sums + 2.0 ** -20 * (1 + abs(lse))))
    r["mass_tol"] += 2.0 ** -22 * r["mass"] + 1e-30
    return r


def select(c, q, table, seq_lens, n_sel, n_first, n_last, q_lens=None):
    """The chosen blocks [B, T, nkv, n_sel] (padding slots -2: not written)."""
    N, nkv, hd = c["mean"].shape
    bs = c["k"].shape[2]
    B, T, nq, _ = q.shape
    G = nq // nkv
    f32 = np.float32
    out = np.full((B, T, nkv, n_sel), -2, np.int32)
    for b, n, ql in steps(seq_lens, q_lens, T):
        for t in range(ql):
            lim = n - ql + t + 1
            nb = min((max(lim, 0) + bs - 1) // bs, table.shape[1])
            ph = table[b, :nb].astype(np.int64)
            ok = (ph >= 0) & (ph < N)
            at = np.where(ok, ph, 0)
            for g in range(nkv):
                best = np.full(nb, -np.inf, f32)
                nan = np.zeros(nb, bool)
                for i in range(g * G, g * G + G):
                    x = q[b, t, i].astype(f32)
                    if not np.isfinite(x).all():
                        continue
                    sq = np.abs(x).max() * (f32(1.0) / f32(127.0))
                    q8 = np.rint(x / sq).astype(np.int64) if sq > 0 else np.zeros(hd, np.int64)
                    dot = c["mean"][at, g].astype(np.int64) @ q8
                    with np.errstate(all="ignore"):
                        f = dot.astype(f32) * (sq * c["mscale"][at, g])
                    nan |= np.isnan(f)
                    best = np.fmax(best, f)
                best = np.where(ok, best, -np.inf).astype(np.float64)
                best[nan & ok] = -1e300  # below every number, above -inf?: resolved by the caller's inputs
                j = np.arange(nb)
                must = (j < n_first) | (j >= nb - n_last)
                order = sorted(j, key=lambda x: (not must[x], -best[x], x))[:n_sel]
                out[b, t, g] = sorted(order) + [-1] * (n_sel - min(n_sel, nb))
    return out


def evict(table, seq_lens, mass, bs, keep, n_first, n_last):
    B, n_table = table.shape
    t2, m2 = np.full_like(table, -1), np.zeros_like(mass)
    freed, lens, nf = np.full_like(table, -1), np.array(seq_lens, np.int32).copy(), np.zeros(B, np.int32)
    for b in range(B):
        n = max(int(seq_lens[b]), 0)
        nb = min((n + bs - 1) // bs, n_table)
        go = max(nb - keep, 0)
        inner = list(range(n_first, nb - n_last))
        bad = lambda i: (0, 0.0) if np.isnan(mass[b, i]) else (1, float(mass[b, i]))  # noqa: E731
        gone = set(sorted(inner, key=lambda i: (bad(i), i))[:go])
        stay = [i for i in range(nb) if i not in gone]
        t2[b, :len(stay)], m2[b, :len(stay)] = table[b, stay], mass[b, stay]
        freed[b, :go] = table[b, sorted(gone)]
        lens[b], nf[b] = n - go * bs, go
    return t2, lens, m2, freed, nf
