"""Cases and plain forms of the operators of the paged 8-bit K/V cache.

A cache holds K and V in pages [n_pages, Hkv, page, d] of 8-bit values (e4m3 or
int8) with one fp32 scale for each block of tokens and head, [n_pages, Hkv,
page / block].  A table [B, M] names the pages of each sequence in order (-1: no
page) and refs [n_pages] counts the table entries that name a page.

  append    new K / V rows are quantised into the pages (the scale of a block is
            the smallest power of two that covers its rows; a block that was begun
            earlier is requantised when its scale grows)
  read      the rows of every sequence as bf16 [B, T, Hkv, d]
  decode    one query token per sequence against the pages (window, sinks, RoPE)
  fork      rows become copies of other rows: whole pages are shared, the last,
            partly filled page is copied
  turnover  sequences leave, the pages in use are moved together, others enter
"""

import math

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_DTYPE = {"f8": torch.float8_e4m3fn, "i8": torch.int8}


def _case(name, op, **sizes):
    return {"name": name, "op": op, **sizes}


def listed():
    return [
        # one user, short context, the head shape of the 32 / 8 workloads: latency
        _case("decode_b1_l1024", "decode", B=1, Hq=32, Hkv=8, d=128, Lmin=1024, Lmax=1024, page=64,
              block=64, kind="f8", window=0, sinks=0, theta=0.0),
        # the batched decode workload (64 ragged sequences), queries rotated on load
        _case("decode_b64_l8192", "decode", B=64, Hq=32, Hkv=8, d=128, Lmin=1024, Lmax=8192,
              page=64, block=16, kind="f8", window=0, sinks=0, theta=10000.0),
        # the same batch with a sliding window and sinks, int8
        _case("decode_b64_window", "decode", B=64, Hq=32, Hkv=8, d=128, Lmin=1024, Lmax=8192,
              page=32, block=32, kind="i8", window=2048, sinks=4, theta=0.0),
        # two long documents, 64 / 8 heads: few rows, a long axis
        _case("decode_b2_l131072", "decode", B=2, Hq=64, Hkv=8, d=128, Lmin=100000, Lmax=131072,
              page=128, block=64, kind="f8", window=0, sinks=0, theta=0.0),
        # one decode step's new token of each sequence of the batch
        _case("append_b64_t1", "append", B=64, T=1, Hkv=8, d=128, Lmin=1024, Lmax=8192, page=64,
              block=16, kind="f8"),
        # ragged prompts enter an empty or begun cache
        _case("append_b8_t4096", "append", B=8, T=4096, Hkv=8, d=128, Lmin=0, Lmax=100, page=64,
              block=64, kind="i8"),
        # the cached prefix of one sequence, before a further prompt chunk attends to it
        _case("read_b1_t1000", "read", B=1, T=1000, Hkv=8, d=128, Lmin=900, Lmax=1000, page=16,
              block=16, kind="i8"),
        # long ragged prefixes of a batch
        _case("read_b8_t8192", "read", B=8, T=8192, Hkv=8, d=128, Lmin=4096, Lmax=8192, page=64,
              block=32, kind="f8"),
        # one search with four beams
        _case("fork_b4", "fork", B=4, beam=4, Hkv=8, d=128, Lmin=300, Lmax=700, page=64, block=64,
              kind="f8"),
        # many searches at once
        _case("fork_b256", "fork", B=256, beam=8, Hkv=8, d=128, Lmin=1024, Lmax=8192, page=64,
              block=16, kind="f8"),
        # a small pool: two sequences leave, two enter
        _case("turnover_b8", "turnover", B=8, Hkv=2, d=64, Lmin=1, Lmax=500, page=16, block=16,
              kind="i8"),
        # a large pool: a quarter of 128 sequences leaves, another enters
        _case("turnover_b128", "turnover", B=128, Hkv=8, d=128, Lmin=512, Lmax=4096, page=64,
              block=64, kind="f8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "read", "fork", "turnover"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (8, 2), (32, 1), (8, 8), (28, 4), (12, 1), (32, 32)])
    page = rng.choice([16, 32, 48, 64, 128])
    block = rng.choice([b for b in (16, 32, 48, 64, 128) if page % b == 0])
    c = dict(op=op, Hkv=Hkv, d=rng.choice([64, 128]), page=page, block=block,
             kind=rng.choice(["f8", "f8", "i8"]))
    # rows of all sequences together, so that no case costs more than the largest listed one
    room = (1 << 28) // (Hkv * c["d"])
    if op == "decode":
        B = _log(rng, 1, 96)
        Lmax = min(_log(rng, 1, 131072), max(1, room // B))
        c.update(B=B, Hq=Hq, Lmin=rng.randint(0, Lmax), Lmax=Lmax,
                 window=rng.choice([0, 0, _log(rng, 1, 4096)]), sinks=0,
                 theta=rng.choice([0.0, 10000.0, 500000.0]))
        if c["window"]:
            c["sinks"] = rng.choice([0, 1, 4, 100])
    elif op == "append":
        B = _log(rng, 1, 64)
        T = rng.choice([1, min(_log(rng, 1, 4096), max(1, room // 3 // B))])
        c.update(B=B, T=T, Lmin=0, Lmax=min(_log(rng, 1, 8192), max(1, room // B)))
    elif op == "read":
        B = _log(rng, 1, 32)
        T = min(_log(rng, 1, 8192), max(1, room // 3 // B))
        c.update(B=B, T=T, Lmin=0, Lmax=T)
    elif op == "fork":
        beam = rng.randint(2, 8)
        B = beam * _log(rng, 1, 24)
        Lmax = min(_log(rng, 2, 8192), max(2, room * beam // B))
        c.update(B=B, beam=beam, Lmin=1, Lmax=Lmax)
    else:
        B = 4 * _log(rng, 1, 24)
        Lmax = min(_log(rng, 2, 4096), max(2, room // B))
        c.update(B=B, Lmin=1, Lmax=Lmax)
    return c


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _lengths(c, n, g):
    return torch.randint(c["Lmin"], c["Lmax"] + 1, (n,), generator=g, device=_DEV,
                         dtype=torch.int32)


def _pages_for(c):
    """Slots of a table row: enough for Lmax rows and, for append, T more."""
    return max(1, -(-(c["Lmax"] + (c["T"] if c["op"] == "append" else 0)) // c["page"]))


def _rows(c, shape, g, keys):
    """bf16 K or V rows [..., d]: unit normals; a few channels of K are larger, as in real keys."""
    x = torch.randn(shape, generator=g, device=_DEV)
    if keys:
        x[..., :: shape[-1] // 4] *= 6.0
    return x.to(torch.bfloat16)


def _pool(c, n_pages, g):
    """A filled cache: K, V pages and their scales."""
    pools, scales = [], []
    for keys in (True, False):
        x = _rows(c, (n_pages, c["Hkv"], c["page"], c["d"]), g, keys).float()
        nb = c["page"] // c["block"]
        s = _scale_for(x.unflatten(2, (nb, c["block"])).abs().amax((-1, -2)), c["kind"])
        y = x.unflatten(2, (nb, c["block"])) / s[..., None, None]
        pools.append(_to8(y, c["kind"]).flatten(2, 3))
        scales.append(s)
    return {"k": pools[0], "v": pools[1], "k_scale": scales[0], "v_scale": scales[1]}


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    M = _pages_for(c)
    if c["op"] in ("decode", "append", "read"):
        B = c["B"]
        n_pages = B * M + 3
        lens = _lengths(c, B, g)
        counts = None
        if c["op"] == "append":
            # ragged prompts; a decode step appends one row to each sequence
            counts = torch.randint(max(1, c["T"] // 4), c["T"] + 1, (B,), generator=g, device=_DEV,
                                   dtype=torch.int32)
        held = -(-(lens + (counts if counts is not None else 0)) // c["page"])
        table = torch.randperm(n_pages, generator=g, device=_DEV)[:B * M].view(B, M).to(torch.int32)
        table[torch.arange(M, device=_DEV)[None, :] >= held[:, None]] = -1
        st.update(_pool(c, n_pages, g), table=table, lens=lens)
        if c["op"] == "append":
            shape = (B, c["T"], c["Hkv"], c["d"])
            st.update(counts=counts, k_new=_rows(c, shape, g, True), v_new=_rows(c, shape, g, False))
        if c["op"] == "decode":
            st["q"] = torch.randn((B, c["Hq"], c["d"]), generator=g, device=_DEV).to(torch.bfloat16)
    elif c["op"] == "fork":
        # beams of one search share the whole pages of their common rows and
        # have a last page each; every beam continues one of its search's beams
        B, beam = c["B"], c["beam"]
        n = B // beam
        n_pages = n * M + 2 * B
        ids = torch.randperm(n_pages, generator=g, device=_DEV).to(torch.int32)
        lens = _lengths(c, n, g).repeat_interleave(beam)
        slot = torch.arange(M, device=_DEV, dtype=torch.int32)
        table = ids[: n * M].view(n, M).repeat_interleave(beam, 0)
        full = lens[:, None] // c["page"]
        last = ids[n * M: n * M + B][:, None]
        table = torch.where(slot < full, table, torch.where(
            (slot == full) & (lens[:, None] % c["page"] > 0), last, -1))
        base = (torch.arange(B, device=_DEV) // beam * beam).to(torch.int32)
        parents = base + torch.randint(0, beam, (B,), generator=g, device=_DEV, dtype=torch.int32)
        st.update(_pool(c, n_pages, g), table=table.contiguous(), lens=lens, parents=parents,
                  refs=_count(table, n_pages))
    else:
        # four groups of sequences, three of them in the pool; on every pass the
        # oldest leaves and the missing one enters
        B = c["B"]
        lens = _lengths(c, B, g)
        group = torch.arange(B, device=_DEV) % 4
        n_pages = 3 * (B // 4) * M + 1
        held = torch.where(group < 3, -(-lens // c["page"]), 0)
        order = torch.argsort(group, stable=True)
        cum = held[order].cumsum(0)
        first = torch.empty_like(cum)
        first[order] = cum - held[order]
        slot = torch.arange(M, device=_DEV)
        table = torch.where(slot < held[:, None], first[:, None] + slot, -1).to(torch.int32)
        turns = []
        for t in range(4):
            left = torch.where((group == t) | (group == (t + 3) % 4), 0, lens)
            turns.append((left, torch.where(group == t, 0, lens)))
        st.update(_pool(c, n_pages, g), table=table, refs=_count(table, n_pages), turns=turns,
                  turn=0)
    return st


def _count(table, n_pages):
    return torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)


# ------------------------------------------------------------- plain forms --

def _scale_for(amax, kind):
    """Smallest power of two s with amax <= s * (largest 8-bit value); 0 for amax = 0."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, 1/2 <= m < 1
    if kind == "f8":
        e = e - 9 + (m > 0.875).int()              # 448 = 0.875 * 2^9
    else:
        e = e - 7 + (m > 0.9921875).int()          # 127 = 0.9921875 * 2^7
    s = ((e.clamp(min=-126) + 127) << 23).view(torch.float32)          # 2^e, exactly
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _to8(x, kind):
    """x in units of its scale -> 8 bits, nearest even (x / 0 of an all-zero block is 0)."""
    x = torch.nan_to_num(x, nan=0.0)
    if kind == "f8":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return x.round().clamp(-127.0, 127.0).to(torch.int8)


def _gathered(st, name, idx):
    """fp32 rows [B, slots * page, Hkv, d] of the pages idx [B, slots] of K or V."""
    c = st["case"]
    x = st[name].view(torch.uint8)[idx].view(_DTYPE[c["kind"]]).float()    # [B, M, H, page, d]
    s = st[name + "_scale"][idx].repeat_interleave(c["block"], -1)          # [B, M, H, page]
    x = x * s[..., None]
    return x.permute(0, 1, 3, 2, 4).flatten(1, 2)


def _rotated(q, lens, theta):
    """RoPE of decode queries at position max(len - 1, 0), rounded to bf16."""
    d = q.shape[-1]
    pos = (lens - 1).clamp(min=0).double()
    ang = pos[:, None] * theta ** (-torch.arange(0, d, 2, device=q.device).double() / d)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    x = q.float()
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2).to(q.dtype)


def _decode(st):
    c = st["case"]
    q, lens = st["q"], st["lens"]
    if c["theta"]:
        q = _rotated(q, lens, c["theta"])
    idx = st["table"].clamp(min=0).long()
    k = _gathered(st, "k", idx).transpose(1, 2)                             # [B, H, L, d]
    qg = q.float().unflatten(1, (c["Hkv"], -1))
    s = qg @ k.transpose(-1, -2) * (1.0 / math.sqrt(c["d"]))
    j, n = torch.arange(s.shape[-1], device=q.device), lens[:, None]
    seen = j < n
    if c["window"]:
        seen = seen & ((j >= n - c["window"]) | (j < c["sinks"]))
    s = s.masked_fill(~seen[:, None, None, :], -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -torch.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = p @ _gathered(st, "v", idx).transpose(1, 2) / torch.where(total > 0, total, 1.0)
    return o.flatten(1, 2).to(q.dtype)


def _append_one(st, name, new):
    """Quantises the new rows of K or V into the pages, block by block."""
    c = st["case"]
    B, T, block, page = c["B"], c["T"], c["block"], c["page"]
    x8 = st[name].view(torch.uint8)
    scale = st[name + "_scale"]
    n = -(-T // block) + 1                                     # blocks that T rows can touch
    start, count = st["lens"].long(), st["counts"].long()
    row = torch.arange(n * block, device=new.device).view(n, block)
    pos = (start // block * block)[:, None, None] + row        # [B, n, block]
    t = pos - start[:, None, None]
    fresh = (t >= 0) & (t < count[:, None, None])
    touched = fresh.any(-1)
    old = (t < 0) & touched[..., None]
    # the blocks that get rows: their page, place in the page, and rows
    b = touched.nonzero()[:, 0]
    pos, t, fresh, old = pos[touched], t[touched], fresh[touched], old[touched]
    pid = st["table"][b, pos[:, 0] // page].long()
    blk = pos[:, 0] % page // block
    r = pos % page
    x = new[b[:, None], t.clamp(0, T - 1)].float() * fresh[..., None, None]      # [N, block, H, d]
    s_old = scale[pid, :, blk] * old.any(-1)[:, None]                            # [N, H]
    before = x8[pid[:, None], :, r].view(_DTYPE[c["kind"]]).float()
    before = before * s_old[:, None, :, None]
    s = torch.maximum(_scale_for(x.abs().amax((1, 3)), c["kind"]), s_old)
    y = torch.where(old[..., None, None], before, x) * (1.0 / s)[:, None, :, None]
    y = _to8(y, c["kind"]).view(torch.uint8)
    write = fresh | old
    pr = pid[:, None].expand_as(r)
    x8[pr[write], :, r[write]] = y[write]
    scale[pid, :, blk] = s


def _append(st):
    _append_one(st, "k", st["k_new"])
    _append_one(st, "v", st["v_new"])
    return _cache(st)


def _cache(st):
    return {n: st[n] for n in ("k", "v", "k_scale", "v_scale")}


def _read(st):
    c = st["case"]
    idx = st["table"].clamp(min=0).long()
    seen = torch.arange(c["T"], device=idx.device) < st["lens"][:, None]
    out = []
    for name in ("k", "v"):
        x = _gathered(st, name, idx)[:, : c["T"]]
        out.append(torch.where(seen[..., None, None], x, 0.0).to(torch.bfloat16))
    return out


def _copy(st, src, dst, rows):
    """Moves (src, dst, rows): the first rows of page src replace those of page dst."""
    c = st["case"]
    for name in ("k", "v"):
        x8, s = st[name].view(torch.uint8), st[name + "_scale"]
        r = torch.arange(c["page"], device=src.device)
        head = (r < rows[:, None])[:, None, :, None]
        x8[dst] = torch.where(head, x8[src], x8[dst])
        b = torch.arange(s.shape[-1], device=src.device) * c["block"]
        s[dst] = torch.where((b < rows[:, None])[:, None, :], s[src], s[dst])


def _fork(st):
    c = st["case"]
    table, lens, refs, parents = st["table"], st["lens"], st["refs"], st["parents"].long()
    me = torch.arange(c["B"], device=table.device)
    slot = torch.arange(table.shape[1], device=table.device)
    # one child goes on in its parent's last page: the parent's own row, or the first child
    claim = torch.where(parents == me, -1, me)
    best = torch.full_like(me, c["B"]).scatter_reduce(0, parents, claim, "amin")
    heir = best[parents] == claim
    n = lens[parents]
    full, part = (n // c["page"]).long(), n % c["page"]
    rows = torch.where(heir[:, None] | (slot < full[:, None]), table[parents], -1)
    refs.add_(_count(rows, refs.numel()) - _count(table, refs.numel()))
    need = ~heir & (part > 0)
    src = table[parents[need], full[need]].long()
    dst = (refs <= 0).nonzero()[:, 0][: src.numel()]
    rows[need, full[need]] = dst.to(torch.int32)
    refs[dst] = 1
    table.copy_(rows)
    lens.copy_(n)
    _copy(st, src, dst, part[need])
    return {"table": table, "lens": lens, "refs": refs, **_cache(st)}


def _resize(st, lens):
    table, refs = st["table"], st["refs"]
    keep = -(-lens // st["case"]["page"])[:, None]
    slot = torch.arange(table.shape[1], device=table.device)
    gone = (table >= 0) & (slot >= keep)
    refs.sub_(_count(torch.where(gone, table, -1), refs.numel()))
    table[gone] = -1
    need = (table < 0) & (slot < keep)
    free = (refs <= 0).nonzero()[:, 0][: need.sum()]
    table[need] = free.to(torch.int32)
    refs[free] = 1


def _compact(st):
    table, refs = st["table"], st["refs"]
    used = refs > 0
    ids = torch.arange(refs.numel(), device=refs.device)
    low = ids < used.sum()
    src, dst = (used & ~low).nonzero()[:, 0], (~used & low).nonzero()[:, 0]
    ids[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, ids[table.clamp(min=0).long()], -1))
    _copy(st, src, dst, torch.full_like(src, st["case"]["page"]))


def _turnover(st):
    left, entered = st["turns"][st["turn"] % 4]
    st["turn"] += 1
    _resize(st, left)
    _compact(st)
    _resize(st, entered)
    return {"table": st["table"], "refs": st["refs"], **_cache(st)}


_PLAIN = {"decode": _decode, "append": _append, "read": _read, "fork": _fork, "turnover": _turnover}


def _own(st):
    import grouped_query_attention_attn_b200 as gqa
    c, table = st["case"], st["table"]
    cache = gqa.Cache8(st["k"], st["v"], st["k_scale"], st["v_scale"])
    if c["op"] == "decode":
        return gqa.decode8(st["q"], cache, table, st["lens"], window=c["window"] or None,
                           sinks=c["sinks"], rope_theta=c["theta"] or None)
    if c["op"] == "append":
        gqa.cache8_append_(cache, table, st["lens"], st["k_new"], st["v_new"], counts=st["counts"])
        return _cache(st)
    if c["op"] == "read":
        return gqa.cache8_read(cache, table, st["lens"], c["T"])
    if c["op"] == "fork":
        moves = gqa.pages_fork_(table, st["refs"], st["lens"], st["parents"], c["page"])
        gqa.cache8_copy_(cache, moves)
        return {"table": table, "lens": st["lens"], "refs": st["refs"], **_cache(st)}
    left, entered = st["turns"][st["turn"] % 4]
    st["turn"] += 1
    gqa.pages_resize_(table, st["refs"], left, c["page"])
    gqa.cache8_copy_(cache, gqa.pages_compact_(table, st["refs"], c["page"]))
    gqa.pages_resize_(table, st["refs"], entered, c["page"])
    return {"table": table, "refs": st["refs"], **_cache(st)}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    mean = (c["Lmin"] + c["Lmax"]) / 2
    row = 2 * c["Hkv"] * (c["d"] + 4 / c["block"])              # K and V of one token, 8 bits
    M = _pages_for(c)
    if c["op"] == "decode":
        seen = mean
        if c["window"]:
            seen = min(mean, c["window"] + c["sinks"])
        return {"bytes": c["B"] * (seen * row + 4 * c["Hq"] * c["d"] + 4 + 4 * seen / c["page"]),
                "flops": 4 * c["B"] * seen * c["Hq"] * c["d"]}
    if c["op"] == "append":
        rows = c["B"] * (max(1, c["T"] // 4) + c["T"]) / 2
        return {"bytes": rows * (row + 4 * c["Hkv"] * c["d"]), "flops": 6 * rows * c["Hkv"] * c["d"]}
    if c["op"] == "read":
        return {"bytes": c["B"] * (mean * row + 4 * c["T"] * c["Hkv"] * c["d"]),
                "flops": 2 * c["B"] * mean * c["Hkv"] * c["d"]}
    if c["op"] == "fork":
        # rows that are not the first child of their parent copy half a page on average
        n = c["B"] / c["beam"]
        copies = c["B"] * (1 - 1 / c["beam"]) ** c["beam"]
        pool = n * M + 2 * c["B"]
        return {"bytes": copies * c["page"] * row + 8 * c["B"] * M + 8 * pool + 12 * c["B"],
                "flops": c["B"] * M}
    moved = c["B"] / 4 * mean / c["page"]
    pool = 3 * (c["B"] // 4) * M + 1
    return {"bytes": 2 * moved * c["page"] * row + 24 * c["B"] * M + 24 * pool, "flops": c["B"] * M}


# ------------------------------------------------------------------- exact --

def _exact_rows(st, name, b, n):
    """float64 [n, Hkv, d]: the first n rows of sequence b, page by page."""
    c = st["case"]
    out = []
    for i in range(-(-n // c["page"])):
        p = int(st["table_host"][b][i])
        s = st[name + "_scale"][p].double()
        x = st[name][p].double().reshape(c["Hkv"], -1, c["block"], c["d"]) * s[:, :, None, None]
        out.append(x.reshape(c["Hkv"], c["page"], c["d"]).transpose(0, 1))
    if not out:
        return torch.zeros((0, c["Hkv"], c["d"]), dtype=torch.float64, device=_DEV)
    return torch.cat(out)[:n]


def _exact_decode(st):
    c = st["case"]
    out = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float64, device=_DEV)
    for b, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        q = st["q"][b].double()
        if c["theta"]:
            pairs = torch.view_as_complex(q.reshape(c["Hq"], -1, 2))
            turn = (n - 1) * torch.exp(-math.log(c["theta"]) * 2 / c["d"] *
                                       torch.arange(c["d"] // 2, device=_DEV, dtype=torch.float64))
            pairs = pairs * torch.polar(torch.ones_like(turn), turn)
            # the rotated query is held in its own type
            q = torch.view_as_real(pairs).reshape(c["Hq"], c["d"]).to(torch.bfloat16).double()
        keys, values = _exact_rows(st, "k", b, n), _exact_rows(st, "v", b, n)
        if c["window"] and n > c["window"]:
            at = torch.arange(n, device=_DEV)
            at = at[(at >= n - c["window"]) | (at < c["sinks"])]
            keys, values = keys[at], values[at]
        share = c["Hq"] // c["Hkv"]
        for h in range(c["Hkv"]):
            w = torch.softmax(q[h * share:(h + 1) * share] @ keys[:, h].T / c["d"] ** 0.5, -1)
            out[b, h * share:(h + 1) * share] = w @ values[:, h]
    return out


_POWERS = torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=_DEV)


def _power(e):
    return _POWERS[(e + 200).clamp(0, 400).long()]


def _exact_power(amax, top):
    """Smallest power of two s with amax <= s * top, by search from an estimate below it."""
    e = torch.floor(torch.log2(torch.clamp(amax, min=1e-300) / top)) - 1
    for _ in range(4):
        e = torch.where(amax > top * _power(e), e + 1, e)
    return torch.where(amax > 0, _power(torch.clamp(e, min=-126)), 0.0)


def _exact_8(x, kind):
    """float64 values rounded to the nearest 8-bit value, ties to even."""
    if kind == "i8":
        return torch.round(x).clamp(-127, 127)
    size = torch.clamp(torch.floor(torch.log2(torch.clamp(x.abs(), min=1e-300))), min=-6)
    step = _power(size - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(st):
    c = st["case"]
    top = 448.0 if c["kind"] == "f8" else 127.0
    out = {}
    for name in ("k", "v"):
        pages = st[name].double()
        scales = st[name + "_scale"].double()
        for b, (n, m) in enumerate(zip(st["lens"].tolist(), st["counts"].tolist())):
            first = n // c["block"] * c["block"]
            x = st[name + "_new"][b, :m].double()
            pad = -(n + m) % c["block"]
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, n - first, pad))
            x = x.reshape(-1, c["block"], c["Hkv"], c["d"])           # whole blocks
            amax = x.abs().amax((1, 3))                                # [blocks, H]
            s = _exact_power(amax, top)
            for i in range(x.shape[0]):
                at = first + i * c["block"]
                p, r = int(st["table_host"][b][at // c["page"]]), at % c["page"]
                k = r // c["block"]
                kept = max(0, n - at)                                  # rows of earlier calls
                if kept:
                    was = scales[p, :, k].clone()
                    s[i] = torch.maximum(s[i], was)
                    x[i, :kept] = pages[p, :, r:r + kept].transpose(0, 1) * was[None, :, None]
                end = min(c["block"], n + m - at)
                y = x[i, :end] / torch.where(s[i] > 0, s[i], 1.0)[None, :, None]
                pages[p, :, r:r + end] = _exact_8(y, c["kind"]).transpose(0, 1)
                scales[p, :, k] = s[i]
        out[name], out[name + "_scale"] = pages, scales
    return {n: out[n] if c["kind"] == "f8" or "scale" in n else None
            for n in ("k", "v", "k_scale", "v_scale")}


def _exact_read(st):
    c = st["case"]
    out = []
    for name in ("k", "v"):
        x = torch.zeros((c["B"], c["T"], c["Hkv"], c["d"]), dtype=torch.float64, device=_DEV)
        for b, n in enumerate(st["lens"].tolist()):
            x[b, :n] = _exact_rows(st, name, b, n)
        out.append(x)
    return out


def _exact_moved(st, moves):
    """The cache in float64 after the moves (src, dst, rows); integers have no such value."""
    c = st["case"]
    out = {}
    for name in ("k", "v"):
        x, s = st[name].double(), st[name + "_scale"].double()
        for a, b, n in moves:
            x[b, :, :n] = x[a, :, :n]
            s[b, :, :-(-n // c["block"])] = s[a, :, :-(-n // c["block"])]
        out[name], out[name + "_scale"] = (x if c["kind"] == "f8" else None), s
    return {n: out[n] for n in ("k", "v", "k_scale", "v_scale")}


def _exact_fork(st):
    c = st["case"]
    rows, lens, parents = st["table_host"], st["lens"].tolist(), st["parents"].tolist()
    children = {}
    for b, p in enumerate(parents):
        children.setdefault(p, []).append(b)
    new, held, wants = [], [0] * st["refs"].numel(), []
    for b, p in enumerate(parents):
        keeps = (p if p in children[p] else children[p][0]) == b
        full, part = divmod(lens[p], c["page"])
        row = list(rows[p]) if keeps else rows[p][:full] + [-1] * (len(rows[p]) - full)
        if not keeps and part:
            wants.append((b, rows[p][full], full, part))
        for x in row:
            if x >= 0:
                held[x] += 1
        new.append(row)
    free = iter([i for i, n in enumerate(held) if n == 0])
    moves = [(src, next(free), part) for _, src, _, part in wants]
    return {"table": None, "lens": None, "refs": None, **_exact_moved(st, moves)}


def _exact_turnover(st):
    # the data only depends on the moves of the compaction, and those on the pages that stay
    left = st["turns"][0][0].tolist()
    pages = {x for row, n in zip(st["table_host"], left)
             for x in row[:-(-n // st["case"]["page"])] if x >= 0}
    high = sorted(x for x in pages if x >= len(pages))
    low = [x for x in range(len(pages)) if x not in pages]
    moves = [(a, b, st["case"]["page"]) for a, b in zip(high, low)]
    return {"table": None, "refs": None, **_exact_moved(st, moves)}


def exact(case, seed):
    st = prepare(case, seed)
    st["table_host"] = st["table"].tolist()
    return {"decode": _exact_decode, "append": _exact_append, "read": _exact_read,
            "fork": _exact_fork, "turnover": _exact_turnover}[case["op"]](st)
