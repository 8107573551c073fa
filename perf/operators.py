"""The paged 8-bit key/value cache's operators, as they are measured.

A case is one pass of one of four kinds:

  attend  one layer's attention of the new tokens of every row (one token, a drafted block,
          a draft tree, a chunk of a prompt) over the row's cached tokens and its own;
  append  one layer's new keys and values quantised into the cache, and read back;
  fork    rows copied for beams or samples (full pages shared, partial pages copied), read
          back, and the copies freed again;
  round   a speculative round on forked rows: fork, reserve, append in every layer, commit of
          the accepted nodes, read back, and the forks freed again.

The passes of the last two end in the state they began with, so they can be repeated.
The cache: k, v [layers, pages, heads, page, dim] in e4m3 with one fp32 scale per (layer,
page, head); table [rows, max_pages] of page ids (-1 past n_pages [rows]), len [rows],
refs [pages] (0: free).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EXP_MIN = -64  # smallest scale the cache writes is 2^-64


# ------------------------------------------------------------------ cases
def _attend(name, rows, T, lens, heads, group, dim, page=64, dtype="bf16", tree=False, window=0,
            sinks=0, fused=False):
    return dict(name=name, kind="attend", rows=rows, T=T, len_lo=lens[0], len_hi=lens[1],
                heads=heads, group=group, dim=dim, page=page, dtype=dtype, tree=tree,
                window=window, sinks=sinks, fused=fused, layers=1)


def listed():
    return [
        # One user, one token, a short chat: latency only.
        _attend("attend_one_token", 1, 1, (701, 701), 8, 4, 128),
        # Plain decoding of a batch of 64 chats of uneven length.
        _attend("attend_decode", 64, 1, (150, 8000), 8, 8, 128, page=64),
        # The benchmark's block: 64 requests, 8 drafted tokens and the last accepted one.
        _attend("attend_block9", 64, 9, (2000, 6000), 8, 4, 128, page=64, fused=True),
        # The benchmark's trees: 64 requests, 16 nodes.
        _attend("attend_tree16", 64, 16, (1000, 5000), 8, 8, 128, page=32, tree=True),
        # Two long documents, a drafted block of 4, an odd group, half precision.
        _attend("attend_long", 2, 5, (120001, 131071), 4, 7, 128, page=128, dtype="f16"),
        # Sliding-window layers with sink tokens under a long context, small pages and heads.
        _attend("attend_window", 32, 9, (3, 32000), 8, 8, 64, page=16, window=4096, sinks=4),
        # A chunk of a prompt behind earlier chunks, wide heads.
        _attend("attend_prompt", 2, 1023, (2049, 4100), 2, 8, 256, page=64),
        # One decoding layer's block of new tokens, sliced from a fused projection.
        dict(name="append_block9", kind="append", rows=64, T=9, len_lo=100, len_hi=8000, heads=8,
             dim=128, page=64, dtype="bf16", fused=True, layers=1),
        # One layer's prompts.
        dict(name="append_prompt", kind="append", rows=8, T=4093, len_lo=0, len_hi=300, heads=8,
             dim=128, page=64, dtype="bf16", fused=False, layers=1),
        # Beams of 16 prompts, four each, every layer.
        dict(name="fork_beams", kind="fork", rows=16, copies=3, len_lo=200, len_hi=4000, heads=8,
             dim=128, page=64, layers=32),
        # A short chain round on one forked row.
        dict(name="round_chain", kind="round", rows=1, T=5, len_lo=90, len_hi=130, heads=2,
             dim=64, page=16, dtype="bf16", tree=False, layers=2),
        # Tree rounds on 32 forked rows.
        dict(name="round_tree16", kind="round", rows=32, T=16, len_lo=500, len_hi=4000, heads=8,
             dim=128, page=64, dtype="bf16", tree=True, layers=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "attend", "append", "fork", "round"))
    page = rng.choice((16, 32, 64, 128))
    dim = rng.choice((64, 80, 96, 128, 128, 192, 256))
    heads = rng.choice((1, 2, 4, 8))
    if kind == "attend":
        T = rng.choice((1, 1, 2, 5, 9, 13, 16, 33, 150, 600))
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16)) if T <= 33 else rng.choice((1, 4, 8))
        hi = _log_int(rng, 20, 60000)
        # No more cached elements and products than the largest listed cases.
        hi = max(1, min(hi, 30_000_000_000 // (heads * dim * group * T) - T))
        rows = max(1, min(_log_int(rng, 1, 64), 200_000_000 // (hi * heads * dim),
                          30_000_000_000 // ((hi + T) * heads * dim * group * T)))
        tree = T <= 33 and rng.random() < 0.4
        window, sinks = (rng.choice((64, 1000, 4096)), rng.choice((0, 1, 4, 130))) \
            if rng.random() < 0.4 else (0, 0)
        return dict(kind=kind, rows=rows, T=T, len_lo=rng.randint(0, hi), len_hi=hi, heads=heads,
                    group=group, dim=dim, page=page, dtype=rng.choice(("bf16", "bf16", "f16")),
                    tree=tree, window=window, sinks=sinks, fused=rng.random() < 0.5, layers=1)
    if kind == "append":
        T = _log_int(rng, 1, 4000)
        rows = max(1, min(_log_int(rng, 1, 64), 33_000_000 // (T * heads * dim)))
        hi = _log_int(rng, 1, 4000)
        return dict(kind=kind, rows=rows, T=T, len_lo=rng.randint(0, hi), len_hi=hi, heads=heads,
                    dim=dim, page=page, dtype=rng.choice(("bf16", "bf16", "f16", "f32")),
                    fused=rng.random() < 0.5, layers=1)
    if kind == "fork":
        rows = _log_int(rng, 1, 16)
        hi = _log_int(rng, 1, 3000)
        layers = min(_log_int(rng, 1, 32), 64 * 128 * 32 // (page * dim))
        return dict(kind=kind, rows=rows, copies=rng.randint(1, 3), len_lo=rng.randint(0, hi),
                    len_hi=hi, heads=heads, dim=dim, page=page, layers=layers)
    hi, T, layers = _log_int(rng, 1, 3000), rng.randint(1, 33), rng.randint(1, 8)
    rows = max(1, min(_log_int(rng, 1, 32), 32 * 16 * 128 * 8 * 8 // (T * dim * heads * layers)))
    return dict(kind=kind, rows=rows, T=T, len_lo=rng.randint(0, hi), len_hi=hi, heads=heads,
                dim=dim, page=page, dtype=rng.choice(("bf16", "f16")), tree=rng.random() < 0.6,
                layers=layers)


# ------------------------------------------------------------------ inputs
def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9), not below 2^EXP_MIN."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(min=EXP_MIN)
    return torch.ldexp(torch.ones_like(amax), e)


def _quantise(x):
    s = _pow2_scale(x.abs().amax(dim=(-2, -1)))
    return (x / s[..., None, None]).to(F8), s


def _tree(rows, T, rnd):
    """Parent links of random draft trees."""
    return [[-1] + [rnd.randint(max(0, n - 4), n - 1) for n in range(1, T)] for _ in range(rows)]


def _lens(case):
    """Cached lengths of a case's rows: evenly over its range, the longest first."""
    lo, hi, R = case["len_lo"], case["len_hi"], case["rows"]
    return [hi - (hi - lo) * i // max(R - 1, 1) for i in range(R)]


def _n_new(case):
    """New tokens of a case's rows: full blocks and, for short ones, a third ragged."""
    T, R = case["T"], case["rows"]
    if case["kind"] == "append" or T > 33:
        return [T] * R
    return [1 + 5 * i % T if i % 3 == 1 else T for i in range(R)]


def _inputs(case, seed):
    """Tensors of a case, from the seed alone."""
    rnd = random.Random(seed * 7919 + 13)
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    R, H, D, ps, Ly = c["rows"], c["heads"], c["dim"], c["page"], c["layers"]
    T = c.get("T", 0)
    total = R * (2 if c["kind"] == "round" else 1 + c.get("copies", 0))
    lens = _lens(c) + [0] * (total - R)
    # Rows hold the pages of their tokens, and for attention and appending those of the new
    # ones too; page ids in random order, some pages free between them.
    hold = T if c["kind"] in ("attend", "append") else 0
    n_pages = [-(-(n + hold) // ps) if i < R else 0 for i, n in enumerate(lens)]
    max_pages = -(-(max(lens) + T) // ps) + 1
    spare = total * (-(-max(T, 1) // ps) + 2) + 7 if c["kind"] in ("fork", "round") else 3
    pages = sum(n_pages) + spare
    ids = list(range(pages))
    rnd.shuffle(ids)
    table = torch.full((total, max_pages), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for i, n in enumerate(n_pages):
        mine = torch.tensor(ids[at: at + n], dtype=torch.int32)
        table[i, :n] = mine
        refs[mine.long()] = 1
        at += n
    st = dict(case=c, lens=lens, total=total, table=table.to(DEV), refs=refs.to(DEV),
              n_pages=torch.tensor(n_pages, dtype=torch.int32, device=DEV),
              len=torch.tensor(lens, dtype=torch.int32, device=DEV))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    # Keys with a few strong channels per head; the first token of a row draws much of the
    # attention; queries lean towards it.
    chan = torch.exp(0.4 * randn(H, 1, D))
    chan[:, :, ::37] *= 4.0
    lean = randn(H, 1, D)
    st["k"] = torch.empty(Ly, pages, H, ps, D, dtype=F8, device=DEV)
    st["v"] = torch.empty_like(st["k"])
    st["k_scale"] = torch.empty(Ly, pages, H, device=DEV)
    st["v_scale"] = torch.empty(Ly, pages, H, device=DEV)
    first = table[:R, 0][torch.tensor(n_pages[:R]) > 0].long().to(DEV)
    for ly in range(Ly):
        x = randn(pages, H, ps, D) * chan
        if first.numel():
            x[first, :, 0] += 0.8 * lean[:, 0]
        st["k"][ly], st["k_scale"][ly] = _quantise(x)
        st["v"][ly], st["v_scale"][ly] = _quantise(randn(pages, H, ps, D) * torch.exp(
            0.5 * randn(H, 1, 1)))
    if c["kind"] == "fork":
        st["src"] = torch.arange(total, device=DEV, dtype=torch.int32) % R
        st["src_free"] = torch.where(torch.arange(total, device=DEV) < R,
                                     torch.arange(total, device=DEV), -1).to(torch.int32)
        full = [n // ps * ps for n in lens[:R]]
        st["start"] = torch.tensor([full[i % R] for i in range(total)], dtype=torch.int32,
                                   device=DEV)
        st["count"] = torch.tensor([lens[i % R] - full[i % R] for i in range(total)],
                                   dtype=torch.int32, device=DEV)
        return st
    dt = DTYPES[c["dtype"]]
    n_new = _n_new(c)
    par = None
    if c.get("tree"):
        par = _tree(R, T, rnd)
    if c["kind"] == "attend":
        G = c["group"]
        q = randn(R, T, H * G, D)
        q += 0.6 * lean[:, 0].repeat_interleave(G, 0)
        qkv = torch.empty(R, T, H * (G + 2) if c["fused"] else H * G, D, dtype=dt, device=DEV)
        qkv[:, :, :H * G] = q.to(dt)
        if c["fused"]:
            qkv[:, :, H * G:] = 0
        st["q"] = qkv[:, :, :H * G]
        st["scale"] = 1.0 / math.sqrt(D)
        st["n_new_host"] = n_new
        st["n_new"] = torch.tensor(n_new, dtype=torch.int32, device=DEV)
        st["parent_host"] = par
        st["parent"] = None if par is None else torch.tensor(par, dtype=torch.int32, device=DEV)
        return st
    # New keys and values of every layer, sliced from a fused projection or dense.
    st["new"] = []
    for _ in range(Ly):
        fused = torch.empty(total, T, 4 * H if c.get("fused") else 2 * H, D, dtype=dt, device=DEV)
        fused[:, :, -2 * H:-H] = (randn(total, T, H, D) * chan[:, 0]).to(dt)
        fused[:, :, -H:] = randn(total, T, H, D).to(dt)
        if c.get("fused"):
            fused[:, :, :2 * H] = 0
        k, v = fused[:, :, -2 * H:-H], fused[:, :, -H:]
        st["new"].append((k, v) if c.get("fused") else (k.contiguous(), v.contiguous()))
    if c["kind"] == "append":
        st["n_new"] = torch.tensor(n_new, dtype=torch.int32, device=DEV)
        st["start"], st["count"] = st["len"], st["n_new"]
        return st
    # Round: the forks are rows R .. 2R-1; the parents take no new tokens.
    st["src"] = torch.arange(total, device=DEV, dtype=torch.int32) % R
    st["src_free"] = torch.where(torch.arange(total, device=DEV) < R,
                                 torch.arange(total, device=DEV), -1).to(torch.int32)
    acc, path = [-1] * R, [[-1] * T for _ in range(total)]
    for i in range(R):
        nodes, at = [], 0
        while True:
            kids = [n for n in range(1, n_new[i]) if (par[i][n] if par else n - 1) == at]
            if not kids or rnd.random() < 0.2:
                break
            at = rnd.choice(kids)
            nodes.append(at)
        acc.append(len(nodes) if rnd.random() > 0.03 else -1)
        path[R + i][:len(nodes)] = nodes
    st["n_new"] = torch.tensor([0] * R + n_new, dtype=torch.int32, device=DEV)
    st["accepted"] = torch.tensor(acc, dtype=torch.int32, device=DEV)
    st["path"] = torch.tensor(path, dtype=torch.int32, device=DEV) if par else None
    st["start"] = torch.tensor([lens[i % R] for i in range(total)], dtype=torch.int32, device=DEV)
    st["count"] = st["accepted"] + 1
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import speculative_decoding_verification_79_gb300 as sv

        Ly, pages, H, ps, D = st["k"].shape
        c = sv.KVCache(Ly, pages, ps, H, D, st["total"], st["table"].shape[1], device=DEV)
        for f in ("k", "v", "k_scale", "v_scale", "table", "n_pages", "len", "refs"):
            getattr(c, f).copy_(st.pop(f))
        st["cache"] = c
        if case["kind"] in ("append",):
            st["start"] = c.len
    return st


# ------------------------------------------------------------------ the plain forms
def _tokens(st, pos):
    """Page id and slot of positions pos [rows, n] (clamped into the table)."""
    ps = st["k"].shape[3]
    j = (pos // ps).clamp(0, st["table"].shape[1] - 1)
    pid = st["table"].long().gather(1, j).clamp(min=0)
    return pid, pos % ps


def _read(st, start, count, T):
    pos = start.long()[:, None] + torch.arange(T, device=DEV)
    pid, slot = _tokens(st, pos)
    live = (torch.arange(T, device=DEV) < count[:, None])[None, :, :, None, None]
    out = []
    for x, s in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
        H = x.shape[2]
        val = x.view(torch.uint8)[:, pid[..., None], torch.arange(H, device=DEV), slot[..., None]]
        val = val.view(F8).float() * s[:, pid][..., None]
        out.append(torch.where(live, val, 0.0).to(torch.bfloat16))
    return out


def _free_order(refs):
    return torch.argsort((refs != 0).to(torch.int8), stable=True)


def _reserve(st, n_new):
    ps = st["k"].shape[3]
    need = ((st["len"] + n_new + ps - 1) // ps - st["n_pages"]).clamp(min=0).long()
    end = torch.cumsum(need, 0)
    j = torch.arange(st["table"].shape[1], device=DEV)[None]
    lo = st["n_pages"].long()[:, None]
    mine = (j >= lo) & (j < lo + need[:, None])
    rank = ((end - need)[:, None] + j - lo).clamp(0, st["refs"].numel() - 1)
    fresh = _free_order(st["refs"])[rank]
    st["table"] = torch.where(mine, fresh, st["table"].long()).to(torch.int32)
    st["refs"].index_add_(0, torch.where(mine, fresh, 0).flatten(), mine.flatten().to(torch.int32))
    st["n_pages"] = st["n_pages"] + need.to(torch.int32)


def _append(st, layer, k, v, n_new):
    ps = st["k"].shape[3]
    rows, T, H, D = k.shape
    J = (T + ps - 2) // ps + 1
    L = st["len"].long()
    # Tokens past a row's n_new, and pages they would need, repeat the row's first.
    t = torch.arange(T, device=DEV)
    t = torch.where(t[None] < n_new[:, None], t[None], 0)
    pos = L[:, None] + t
    pid, slot = _tokens(st, pos)
    jj = pos // ps - (L // ps)[:, None]
    j = torch.arange(J, device=DEV)[None]
    j = torch.where(j * ps < (L % ps)[:, None] + n_new[:, None], j, 0)
    ppid, _ = _tokens(st, ((L // ps)[:, None] + j) * ps)
    h = torch.arange(H, device=DEV)
    rows_hit = st["hit"] if "hit" in st else slice(None)
    for name, x in (("k", k), ("v", v)):
        pool, scale = st[name][layer], st[name + "_scale"][layer]
        x = x.float().gather(1, t[..., None, None].expand(-1, -1, H, D))
        a = torch.zeros(rows, J, H, device=DEV)
        a.scatter_reduce_(1, jj[..., None].expand(-1, -1, H), x.abs().amax(-1), "amax")
        s = _pow2_scale(a)
        old = scale[ppid[:, 0]]
        s[:, 0] = torch.where((L % ps > 0)[:, None], torch.maximum(s[:, 0], old), s[:, 0])
        # Older tokens of the first page, at its new scale.
        bytes_ = pool.view(torch.uint8)
        page0 = bytes_[ppid[:, 0]]
        re = (page0.view(F8).float() * (old / s[:, 0])[..., None, None]).to(F8).view(torch.uint8)
        keep = torch.arange(ps, device=DEV)[None] < (L % ps)[:, None]
        bytes_[ppid[rows_hit, 0]] = torch.where(keep[:, None, :, None], re, page0)[rows_hit]
        scale[ppid[rows_hit]] = s.gather(1, j[..., None].expand(rows, J, H))[rows_hit]
        q = (x / s.gather(1, jj[..., None].expand(-1, -1, H))[..., None]).to(F8)
        bytes_[pid[rows_hit][..., None], h, slot[rows_hit][..., None]] = \
            q.view(torch.uint8)[rows_hit]


def _commit(st, accepted, path, T):
    ps = st["k"].shape[3]
    hit = st["hit"]
    H = st["k"].shape[2]
    L = st["len"].long()
    n = (accepted + 1).long()
    if path is not None:
        # Dropped tokens repeat the first (the root, which stays where it is).
        i = torch.arange(T, device=DEV)
        i = torch.where(i[None] < n[:, None], i[None], 0)
        idx = torch.cat([torch.zeros_like(path[:, :1]), path[:, :-1]], 1).long().gather(1, i)
        spid, sslot = _tokens(st, L[:, None] + idx)
        dpid, dslot = _tokens(st, L[:, None] + i)
        J = (T + ps - 2) // ps + 1
        jj = (L[:, None] + i) // ps - (L // ps)[:, None]
        j = torch.arange(J, device=DEV)[None]
        j = torch.where(j <= jj.amax(1, keepdim=True), j, 0)
        ppid, _ = _tokens(st, ((L // ps)[:, None] + j) * ps)
        h = torch.arange(H, device=DEV)
        for name in ("k", "v"):
            for pool, scale in zip(st[name], st[name + "_scale"]):
                bytes_ = pool.view(torch.uint8)
                val = bytes_[spid[..., None], h, sslot[..., None]]
                src_s = scale[spid]
                s = torch.zeros(L.numel(), J, H, device=DEV)
                s.scatter_reduce_(1, jj[..., None].expand(-1, -1, H), src_s, "amax")
                old = scale[ppid]
                s[:, 0] = torch.where((L % ps > 0)[:, None], torch.maximum(s[:, 0], old[:, 0]),
                                      s[:, 0])
                page0 = bytes_[ppid[:, 0]]
                re = (page0.view(F8).float() * (old[:, 0] / s[:, 0])[..., None, None]).to(F8)
                keep = torch.arange(ps, device=DEV)[None] < (L % ps)[:, None]
                bytes_[ppid[hit, 0]] = torch.where(keep[:, None, :, None], re.view(torch.uint8),
                                                   page0)[hit]
                scale[ppid[hit]] = s.gather(1, j[..., None].expand(-1, -1, H))[hit]
                q = (val.view(F8).float()
                     * (src_s / s.gather(1, jj[..., None].expand(-1, -1, H)))[..., None]).to(F8)
                bytes_[dpid[hit][..., None], h, dslot[hit][..., None]] = \
                    q.view(torch.uint8)[hit]
    st["len"] = st["len"] + n.to(torch.int32)
    used = torch.minimum((st["len"] + ps - 1) // ps, st["n_pages"])
    drop = (torch.arange(st["table"].shape[1], device=DEV)[None] >= used[:, None]) \
        & (st["table"] >= 0)
    st["refs"].index_add_(0, st["table"].clamp(min=0).long().flatten(),
                          -drop.flatten().to(torch.int32))
    st["table"] = torch.where(drop, -1, st["table"])
    st["n_pages"] = used


def _fork(st, src):
    ps = st["k"].shape[3]
    n = src.numel()
    b = torch.arange(n, device=DEV)
    take = src.long()[None] == b[:, None]  # [old row, new row]
    m = take.sum(1)
    keeper = torch.where(take.diagonal(), b, take.to(torch.int8).argmax(1))
    full, tail = st["len"].long() // ps, st["len"] % ps
    j = torch.arange(st["table"].shape[1], device=DEV)[None]
    held = j < st["n_pages"][:, None]
    delta = torch.where(j < full[:, None], m[:, None] - 1,
                        torch.where(m[:, None] > 0, 0, -1)) * held
    st["refs"].index_add_(0, st["table"].clamp(min=0).long().flatten(),
                          delta.flatten().to(torch.int32))
    s = src.long().clamp(min=0)
    some = src >= 0
    keeps = some & (keeper[s] == b)
    copy = some & ~keeps & (tail[s] > 0)
    fresh = _free_order(st["refs"])[(torch.cumsum(copy, 0) - 1).clamp(min=0)]
    st["refs"].index_add_(0, torch.where(copy, fresh, 0), copy.to(torch.int32))
    old = st["table"].long()
    partial = old.gather(1, full[:, None].clamp(max=old.shape[1] - 1))[:, 0].clamp(min=0)[s]
    hit = st["copied"]
    if hit.numel() and st["forking"]:
        for name in ("k", "v"):
            x = st[name].view(torch.uint8)
            x[:, fresh[hit]] = x[:, partial[hit]]
            y = st[name + "_scale"]
            y[:, fresh[hit]] = y[:, partial[hit]]
    row = old[s]
    f = full[s][:, None]
    new = torch.where(j < f, row, torch.where(copy[:, None] & (j == f), fresh[:, None], -1))
    st["table"] = torch.where(keeps[:, None], row, torch.where(some[:, None], new, -1)).to(
        torch.int32)
    st["n_pages"] = torch.where(keeps, st["n_pages"][s],
                                torch.where(some, (f[:, 0] + copy).to(torch.int32), 0)).to(
        torch.int32)
    st["len"] = torch.where(some, st["len"][s], 0).to(torch.int32)


def _attend_plain(st):
    c = st["case"]
    R, T, H, G, D, ps = c["rows"], c["T"], c["heads"], c["group"], c["dim"], c["page"]
    o = torch.zeros(R, T, H * G, D, dtype=st["q"].dtype, device=DEV)
    lse = torch.full((R, T, H * G), -math.inf, device=DEV)
    i = torch.arange(T, device=DEV)
    if st["parent"] is not None:
        # Ancestor-or-self of every node.
        up = i.repeat(R, 1)
        sees = torch.eye(T, device=DEV, dtype=torch.bool).repeat(R, 1, 1)
        for _ in range(T - 1):
            up = torch.where(up > 0, st["parent"].long().gather(1, up.clamp(min=0)), -1)
            sees |= up[:, :, None] == i
    else:
        sees = (i[None] <= i[:, None]).expand(R, T, T)
    depths = sees.sum(2) - 1
    for b in range(R):
        n, L = st["n_new_host"][b], st["lens"][b]
        see, depth = sees[b], depths[b]
        pid = st["table"][b, : -(-(L + n) // ps)].long()
        k = (st["k"][0][pid].float() * st["k_scale"][0][pid][..., None, None])
        v = (st["v"][0][pid].float() * st["v_scale"][0][pid][..., None, None])
        k = k.transpose(0, 1).reshape(H, -1, D)[:, : L + n]
        v = v.transpose(0, 1).reshape(H, -1, D)[:, : L + n]
        pos = torch.cat([torch.arange(L, device=DEV), L + depth[:n]])
        mask = torch.ones(n, L + n, dtype=torch.bool, device=DEV)
        mask[:, L:] = see[:n, :n]
        if c["window"]:
            j = torch.arange(L + n, device=DEV)
            mask &= (((L + depth[:n])[:, None] - pos[None]) < c["window"]) | (j < c["sinks"])
        q = st["q"][b, :n].float().reshape(n, H, G, D).permute(1, 0, 2, 3).reshape(H, n * G, D)
        s = torch.matmul(q, k.transpose(1, 2)) * st["scale"]
        s = torch.where(mask.repeat_interleave(G, 0)[None], s, -math.inf)
        mx = s.amax(-1, keepdim=True)
        mx = torch.where(torch.isinf(mx), torch.zeros_like(mx), mx)
        p = torch.exp(s - mx)
        den = p.sum(-1, keepdim=True)
        out = torch.matmul(p, v) / torch.where(den > 0, den, 1.0)
        o[b, :n] = out.reshape(H, n, G, D).permute(1, 0, 2, 3).reshape(n, H * G, D).to(o.dtype)
        ls = (torch.log(den) + mx)[..., 0]
        lse[b, :n] = ls.reshape(H, n, G).permute(1, 0, 2).reshape(n, H * G)
    return o, lse


def _plain(st):
    c = st["case"]
    if c["kind"] == "attend":
        return _attend_plain(st)
    if c["kind"] == "append":
        _append(st, 0, *st["new"][0], st["n_new"])
        return _read(st, st["start"], st["count"], c["T"])
    R = c["rows"]
    if "hit" not in st:
        st["hit"] = torch.arange(R, st["total"], device=DEV)
        st["copied"] = torch.tensor([i for i in range(R, st["total"])
                                     if st["lens"][i % R] % c["page"]], device=DEV,
                                    dtype=torch.long)
    st["forking"] = True
    _fork(st, st["src"])
    if c["kind"] == "round":
        _reserve(st, st["n_new"])
        for ly, (k, v) in enumerate(st["new"]):
            _append(st, ly, k, v, st["n_new"])
        _commit(st, st["accepted"], st["path"], c["T"])
    k, v = _read(st, st["start"], st["count"], c["page"] if c["kind"] == "fork" else c["T"])
    state = [st[f].clone() for f in ("table", "n_pages", "len", "refs")]
    st["forking"] = False
    _fork(st, st["src_free"])
    return [k, v] + state


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import speculative_decoding_verification_79_gb300 as sv

    c, cache = st["case"], st["cache"]
    if c["kind"] == "attend":
        return sv.sv_kv_attend(cache, 0, st["q"], n_new=st["n_new"], parent=st["parent"],
                               scale=st["scale"], window=c["window"], sinks=c["sinks"],
                               want_lse=True)
    if c["kind"] == "append":
        sv.sv_kv_append(cache, 0, *st["new"][0], n_new=st["n_new"])
        return list(sv.sv_kv_read(cache, st["start"], c["T"], count=st["count"]))
    sv.sv_kv_fork(cache, st["src"])
    if c["kind"] == "round":
        sv.sv_kv_reserve(cache, st["n_new"])
        for ly, (k, v) in enumerate(st["new"]):
            sv.sv_kv_append(cache, ly, k, v, n_new=st["n_new"])
        sv.sv_kv_commit(cache, st["accepted"], c["T"], path=st["path"])
    k, v = sv.sv_kv_read(cache, st["start"], c["page"] if c["kind"] == "fork" else c["T"],
                         count=st["count"])
    state = [getattr(cache, f).clone() for f in ("table", "n_pages", "len", "refs")]
    sv.sv_kv_fork(cache, st["src_free"])
    return [k, v] + state


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    """Each cached token read once per key/value head, each input and output once."""
    c = case
    H, D, R, T = c["heads"], c["dim"], c["rows"], c.get("T", 0)
    eb = 4 if c.get("dtype") == "f32" else 2
    if c["kind"] == "attend":
        G, W, S = c["group"], c["window"], c["sinks"]
        tokens = pairs = 0
        for n, new in zip(_lens(c), _n_new(c)):
            if not W:
                tokens += n + new
                # A block's query sees about half of the block (a chain: exactly).
                pairs += new * n + new * (new + 1) // 2
            else:
                lo = max(0, n + 1 - W)  # the first query's oldest token
                tokens += n + new - lo + min(S, lo)
                for t in range(new):
                    pairs += min(n + t + 1, W) + min(S, max(0, n + t + 1 - W))
        kv = tokens * H * D * 2 + tokens / c["page"] * H * 8
        return {"bytes": int(kv + R * T * H * G * (D * eb * 2 + 4)),
                "flops": int(4 * pairs * G * H * D)}
    if c["kind"] == "append":
        n = R * T * H * D * 2
        return {"bytes": int(n * (eb + 1) + n * 1 + n * 2), "flops": int(2 * n)}
    Ly, ps = c["layers"], c["page"]
    tail = sum(n % ps for n in _lens(c))
    if c["kind"] == "fork":
        elems = tail * c["copies"] * H * D * 2 * Ly
        read = tail * (1 + c["copies"]) * H * D * 2 * Ly
        out = R * (1 + c["copies"]) * ps * H * D * 2 * Ly
        return {"bytes": int(2 * elems + read + 2 * out), "flops": int(out)}
    tail *= H * D * 2 * Ly
    new = sum(_n_new(c)) * H * D * 2 * Ly
    return {"bytes": int(2 * tail + new * (eb + 1) + 2 * 2 * R * T * H * D * 2 * Ly),
            "flops": int(3 * new)}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3(x):
    """Nearest e4m3 value (ties to even), saturating at 448, of float64 x."""
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(a)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def _scale64(a):
    """Smallest 2^e >= a / 448, e >= EXP_MIN."""
    e = EXP_MIN
    if a > 0:
        e = max(EXP_MIN, math.ceil(math.log2(a / 448.0)) - 1)
        while 448.0 * 2.0 ** e < a:
            e += 1
    return 2.0 ** e


def _exact_attend(c, st):
    R, T, H, G, D, ps = c["rows"], c["T"], c["heads"], c["group"], c["dim"], c["page"]
    o = torch.zeros(R, T, H * G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((R, T, H * G), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(R):
        n, L = st["n_new_host"][b], st["lens"][b]
        anc = []
        for t in range(n):
            up = t if st["parent_host"] is None else st["parent_host"][b][t]
            if st["parent_host"] is None:
                anc.append(list(range(t + 1)))
            else:
                anc.append((anc[up] if t else []) + [t])
        ids = st["table"][b, : -(-(L + n) // ps)].long()
        for h in range(H):
            def full(x, s):
                y = x[0][ids, h].double() * s[0][ids, h].double()[:, None, None]
                return y.reshape(-1, D)[: L + n]
            k, v = full(st["k"], st["k_scale"]), full(st["v"], st["v_scale"])
            allowed = torch.zeros(n, L + n, dtype=torch.bool)
            for t in range(n):
                p = L + len(anc[t]) - 1
                if c["window"]:
                    lo = max(0, p - c["window"] + 1)
                    allowed[t, lo:L] = True
                    allowed[t, : min(c["sinks"], L)] = True
                    for dpt, a in enumerate(anc[t]):
                        allowed[t, L + a] = p - (L + dpt) < c["window"] or L + a < c["sinks"]
                else:
                    allowed[t, :L] = True
                    allowed[t, [L + a for a in anc[t]]] = True
            q = st["q"][b, :n, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,jd->tgj", q, k) * st["scale"]
            s = s.masked_fill(~allowed.to(DEV)[:, None, :], -math.inf)
            l64 = torch.logsumexp(s, -1)
            w = torch.where(torch.isinf(l64)[..., None], torch.zeros_like(s),
                            torch.exp(s - l64[..., None]))
            o[b, :n, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", w, v)
            lse[b, :n, h * G:(h + 1) * G] = l64
    return o, lse


def exact(case, seed):
    c = case
    st = _inputs(case, seed)
    if c["kind"] == "attend":
        return _exact_attend(c, st)
    # The other kinds: rows as token lists on the host, pages kept as the definition says.
    R, total, ps, Ly, H, D = c["rows"], st["total"], c["page"], c["layers"], c["heads"], c["dim"]
    T = ps if c["kind"] == "fork" else c["T"]
    lens = list(st["lens"])
    refs = st["refs"].cpu().numpy().copy()
    width = st["table"].shape[1]
    rows = [[int(x) for x in r if x >= 0] for r in st["table"].cpu().tolist()]
    start, count = st["start"].cpu().tolist(), st["count"].cpu().tolist()
    copied = {}
    if c["kind"] != "append":
        take = [[i for i in range(total) if i % R == r] for r in range(R)]
        for r in range(R):
            f = lens[r] // ps
            for b in take[r][1:]:
                for p in rows[r][:f]:
                    refs[p] += 1
        for b in range(R, total):
            r, f = b % R, lens[b % R] // ps
            rows[b] = rows[r][:f]
            lens[b] = lens[r]
            if lens[r] % ps:
                p = int(np.flatnonzero(refs == 0)[0])
                refs[p] = 1
                copied[p] = rows[r][f]
                rows[b].append(p)
    if c["kind"] == "round":
        add = st["n_new"].cpu().tolist()
        for b in range(total):
            while len(rows[b]) * ps < lens[b] + add[b]:
                p = int(np.flatnonzero(refs == 0)[0])
                refs[p] = 1
                rows[b].append(p)
    else:
        add = st["n_new"].cpu().tolist() if c["kind"] == "append" else [0] * total
    acc = st["accepted"].cpu().tolist() if c["kind"] == "round" else [0] * total
    path = st["path"].cpu().tolist() if c["kind"] == "round" and st["path"] is not None else None
    outs = []
    for which in (0, 1):
        name = ("k", "v")[which]
        out = torch.zeros(Ly, total, T, H, D, dtype=torch.float64)
        for ly in range(Ly):
            scale = st[name + "_scale"][ly].double().cpu().numpy()
            new = None
            if add and c["kind"] != "fork":
                new = st["new"][ly][which].double().cpu().numpy()
            for b in range(total):
                if count[b] <= 0:
                    continue
                j0, end = start[b] // ps, lens[b] + add[b]
                ids = rows[b][j0: -(-max(end, start[b] + count[b]) // ps)]
                src = [copied.get(p, p) for p in ids]
                page = st[name][ly][torch.tensor(src, device=DEV)].double().cpu().numpy()
                s = scale[src]
                # page[i, h, slot]: e4m3 values of positions (j0 + i) ps + slot.
                for i in range(len(ids)):
                    lo, hi = max(lens[b], (j0 + i) * ps), min(end, (j0 + i + 1) * ps)
                    if hi <= lo:
                        continue
                    x = new[b, lo - lens[b]: hi - lens[b]]
                    for h in range(H):
                        t = _scale64(float(np.abs(x[:, h]).max()))
                        off = lo - (j0 + i) * ps
                        if off > 0:
                            t = max(t, s[i, h])
                            page[i, h, :off] = _e4m3(page[i, h, :off] * (s[i, h] / t))
                        s[i, h] = t
                        page[i, h, off: off + hi - lo] = _e4m3(x[:, h] / t)
                if c["kind"] == "round" and path is not None:
                    kept = [0] + path[b][: acc[b]]
                    val = [page[(lens[b] + n) // ps - j0, :, (lens[b] + n) % ps].copy()
                           for n in kept]
                    vs = [s[(lens[b] + n) // ps - j0].copy() for n in kept]
                    for i in range(len(ids)):
                        mine = [m for m in range(len(kept)) if (lens[b] + m) // ps - j0 == i]
                        if not mine:
                            continue
                        t = np.max([vs[m] for m in mine], axis=0)
                        off = max(0, lens[b] - (j0 + i) * ps)
                        if off > 0:
                            t = np.maximum(t, s[i])
                            page[i, :, :off] = _e4m3(page[i, :, :off] * (s[i] / t)[:, None, None])
                        s[i] = t
                        for m in mine:
                            page[i, :, (lens[b] + m) % ps] = _e4m3(val[m]
                                                                   * (vs[m] / t)[:, None])
                for t in range(count[b]):
                    p = start[b] + t
                    i = p // ps - j0
                    out[ly, b, t] = torch.from_numpy(page[i, :, p % ps] * s[i][:, None])
        outs.append(out.to(DEV))
    if c["kind"] == "append":
        return outs
    if c["kind"] == "round":
        for b in range(total):
            lens[b] += acc[b] + 1
            while len(rows[b]) > -(-lens[b] // ps):
                refs[rows[b].pop()] -= 1
    table = [r + [-1] * (width - len(r)) for r in rows]
    i32 = [torch.tensor(x, dtype=torch.int32, device=DEV)
           for x in (table, [len(r) for r in rows], lens, refs.tolist())]
    return outs + i32
