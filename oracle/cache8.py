"""Double-precision restatement of the paged 8-bit K/V cache (numpy, lists).

A pool is a dict: codes k, v (uint8 [n_pages, H, page, d], int8 codes as their
two's complement bytes), fp32 scales k_scale, v_scale [n_pages, H, page / block]
and kind ("e4m3" or "int8").  Tables are lists of lists, refs a list.
"""

import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}


def _e4m3_values():
    """Value of each e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; S.1111.111 is NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.ldexp(m / 8.0, -6) if e == 0 else np.ldexp(1.0 + m / 8.0, e - 7)
        if e == 15 and m == 7:
            x = np.nan
        out[c] = -x if c & 128 else x
    return out


E4M3 = _e4m3_values()


def values(codes, kind):
    """float64 values of uint8 codes."""
    if kind == "e4m3":
        return E4M3[codes]
    return codes.astype(np.uint8).view(np.int8).astype(np.float64)


def encode(x, kind):
    """Codes of float64 x: nearest value, ties to even; beyond the range the largest value."""
    x = np.asarray(x, dtype=np.float64)
    if kind == "int8":
        y = np.clip(np.rint(np.nan_to_num(x, nan=0.0)), -127, 127)
        return y.astype(np.int8).view(np.uint8)
    grid = E4M3[:127]                                   # 0 .. 448, ascending codes
    a = np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=448.0))
    mid = (grid[1:] + grid[:-1]) / 2
    c = np.searchsorted(mid, a, side="left")            # first code whose upper midpoint >= a
    tie = (c < 126) & (a == mid[np.minimum(c, 125)])
    c = np.where(tie & (c % 2 == 1), c + 1, c)
    c = c.astype(np.uint8) | np.where(np.signbit(x), 128, 0).astype(np.uint8)
    return np.where(np.isnan(x), c | 127, c).astype(np.uint8)


def scale_for(amax, kind):
    """Smallest power of two s >= 2^-126 with amax <= s * TOP; 0 for amax = 0."""
    if amax == 0:
        return 0.0
    e = -126
    while amax > np.ldexp(TOP[kind], e):
        e += 1
    return float(np.ldexp(1.0, e))


def pool(n_pages, H, page, d, block, kind, rng=None, spread=1.0):
    """A pool; with rng filled by quantised normals whose blocks differ in size."""
    shape, sshape = (n_pages, H, page, d), (n_pages, H, page // block)
    p = {"kind": kind, "page": page, "block": block}
    for n in ("k", "v"):
        if rng is None:
            p[n], p[n + "_scale"] = np.zeros(shape, np.uint8), np.zeros(sshape, np.float32)
            continue
        x = rng.standard_normal(shape).reshape(n_pages, H, page // block, block * d)
        x *= np.exp2(np.round(rng.standard_normal(sshape) * spread))[..., None]
        s = np.array([scale_for(a, kind) for a in np.abs(x).max(-1).ravel()]).reshape(sshape)
        p[n] = encode(x / s[..., None], kind).reshape(shape)
        p[n + "_scale"] = s.astype(np.float32)
    return p


def append(p, table, lens, counts, k, v):
    """Append in place; k, v float64 [B, T, H, d]."""
    kind, page, block = p["kind"], p["page"], p["block"]
    for n, new in (("k", k), ("v", v)):
        H = new.shape[2]
        for b, (start, m) in enumerate(zip(lens, counts)):
            for first in range(start // block * block, start + m, block):
                lo, hi = max(first, start), min(first + block, start + m)
                pid, r0 = table[b][first // page], first % page
                for h in range(H):
                    x = new[b, lo - start:hi - start, h]
                    fin = np.abs(x[np.isfinite(x)])
                    amax = fin.max() if fin.size else 0.0
                    if amax == 0 and np.isinf(x).any():
                        amax = np.ldexp(1.0, -133)
                    old = lo - first
                    sc = p[n + "_scale"][pid, h]
                    s_old = float(sc[r0 // block]) if old else 0.0
                    s = max(scale_for(amax, kind), s_old)
                    codes = p[n][pid, h, r0:r0 + block]
                    if old and s > s_old:
                        codes[:old] = encode(values(codes[:old], kind) * s_old / s, kind)
                    with np.errstate(invalid="ignore"):
                        codes[old:hi - first] = encode(x / s if s else x * 0.0, kind)
                    sc[r0 // block] = s


def rows(p, name, table, b, n):
    """float64 [n, H, d]: rows 0 .. n - 1 of sequence b (NaN where a page is missing)."""
    H, d, page = p[name].shape[1], p[name].shape[3], p["page"]
    out = np.full((n, H, d), np.nan)
    for first in range(0, n, page):
        pid = table[b][first // page]
        if not 0 <= pid < p[name].shape[0]:
            continue
        s = np.repeat(p[name + "_scale"][pid].astype(np.float64), p["block"], axis=1)
        x = values(p[name][pid], p["kind"]) * s[..., None]
        m = min(page, n - first)
        out[first:first + m] = x[:, :m].transpose(1, 0, 2)
    return out


def decode(p, table, lens, q, scale, window=0, sinks=0):
    """q float64 [B, Hq, d] -> (o, bound): o float64 [B, Hq, d] and how far bf16 outputs of
    the kernel's arithmetic may be off, elementwise.

    Bound, in units of the row's largest weight w = 1, A = sum w |v| / sum w.
    A score is off by fp32 sums of d products (d 2^-24 of the sum of magnitudes, plus as
    much again for the operands' scaling) and by elements of q below 2^-14 of their row's
    largest value, off by 2^-25 of that; a weight by as much and the exponential's
    2^-21, in the numerator and in the sum: twice that of A.  In the numerator only, a
    weight is rounded to f16, by 2^-11 of itself; and fp32 sums of up to 512 terms (a
    warp's products, then its pieces) add 2^-15.  Weights enter as 2^7 times themselves,
    times their V scale over a reference at most 64 times that: below w = 2^-15 they may be
    under f16's 2^-14 and off by 2^-25 absolutely, 2^-26 of |v| each.  A block whose V scale
    lies more than 2^80 below the sequence's largest may be lost.  Then half a step of
    bf16, 2^-8.
    """
    B, Hq, d = q.shape
    H = p["k"].shape[1]
    o, bound = np.zeros((B, Hq, d)), np.full((B, Hq, d), 1e-30)
    for b, n in enumerate(lens):
        j = np.arange(n)
        see = np.ones(n, bool) if not window else (j >= n - window) | (j < sinks)
        kk, vv = rows(p, "k", table, b, n)[see], rows(p, "v", table, b, n)[see]
        there = ~np.isnan(kk[:, 0, 0])
        kk, vv = kk[there], vv[there]
        if not len(kk):
            continue
        for h in range(Hq):
            k, v = kk[:, h // (Hq // H)], vv[:, h // (Hq // H)]
            s = k @ q[b, h] * scale
            w = np.exp(s - s.max())
            o[b, h] = w @ v / w.sum()
            mag = (np.abs(k) @ np.abs(q[b, h]) * scale).max()
            off = 2.0 * d * 2.0 ** -24 * mag + 2.0 ** -21
            off += 2.0 ** -25 * np.abs(q[b, h]).max() * np.abs(k).sum(1).max() * scale
            av = np.abs(v)
            mean = w @ av / w.sum()
            small = 2.0 ** -26 * av[w < 2.0 ** -15].sum(0) / w.sum() + 2.0 ** -80 * av.max()
            bound[b, h] += 2.0 ** -8 * np.abs(o[b, h]) + (2 * off + 2.0 ** -11 + 2.0 ** -15) * mean + small
    return o, bound


def copy(p, moves):
    for a, b, n in moves:
        nb = -(-n // p["block"])
        for name in ("k", "v"):
            p[name][b, :, :n] = p[name][a, :, :n]
            p[name + "_scale"][b, :, :nb] = p[name + "_scale"][a, :, :nb]


def count(table, n_pages):
    refs = [0] * n_pages
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return refs


def resize(table, refs, lens, page):
    """In place; returns how many entries found no free page."""
    keep = [-(-n // page) for n in lens]
    for row, k in zip(table, keep):
        for s in range(k, len(row)):
            if row[s] >= 0:
                refs[row[s]] -= 1
                row[s] = -1
    missing = 0
    free = iter([i for i, r in enumerate(refs) if r <= 0])
    for row, k in zip(table, keep):
        for s in range(k):
            if row[s] < 0:
                e = next(free, None)
                missing += e is None
                row[s] = -1 if e is None else e
                if e is not None:
                    refs[e] = 1
    return missing


def fork(table, refs, lens, parents, page):
    """In place; returns the moves."""
    old, n_old = [list(r) for r in table], list(lens)
    children = {}
    for b, x in enumerate(parents):
        if x >= 0:
            children.setdefault(x, []).append(b)
    wants = []
    for b, x in enumerate(parents):
        if x == b:
            continue
        n = n_old[x] if x >= 0 else 0
        full = n // page
        heir = x >= 0 and x not in children[x] and children[x][0] == b
        row = [-1] * len(table[b])
        if x >= 0:
            row = list(old[x]) if heir else old[x][:full] + [-1] * (len(row) - full)
            if not heir and n % page:
                wants.append((b, old[x][full], full, n % page))
        table[b][:], lens[b] = row, n
    refs[:] = count(table, len(refs))
    free = iter([i for i, r in enumerate(refs) if r <= 0])
    moves = []
    for b, src, full, part in wants:
        e = next(free, None)
        if e is None:
            continue
        table[b][full], refs[e] = e, 1
        moves.append((src, e, part))
    return moves


def compact(table, refs, page):
    """In place; returns the moves."""
    n = sum(r > 0 for r in refs)
    src = [i for i, r in enumerate(refs) if r > 0 and i >= n]
    dst = [i for i, r in enumerate(refs) if r <= 0 and i < n]
    to = dict(zip(src, dst))
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    for row in table:
        for s, e in enumerate(row):
            row[s] = to.get(e, e)
    return [(a, b, page) for a, b in to.items()]
