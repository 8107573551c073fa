"""Rotary positions and shared prefixes of the paged key/value cache, as they are measured.

A case is one pass of one of four kinds:

  rope    queries or keys rotated by their positions (half or interleaved pairs, the first
          `rot` components of a head, frequencies stretched for long contexts), or gradients
          rotated back;
  append  one layer's new keys rotated and quantised into the cache together with its values,
          and its queries rotated; what the cache then holds is read back;
  attend  one layer's attention of the new tokens of every row over its cache, where groups of
          rows (samples or beams of a prompt, chats behind one system prompt) hold the same
          pages for their first tokens;
  step    a round's attention layers on such rows: which pages groups share, then for every
          layer append with rotation and attention.

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
def _rope(name, rows, T, heads, dim, rot, dtype="bf16", interleaved=False, inverse=False,
          scaling="none", start=(0, 0), fused=False, tree=False):
    return dict(name=name, kind="rope", rows=rows, T=T, heads=heads, dim=dim, rot=rot, dtype=dtype,
                interleaved=interleaved, inverse=inverse, scaling=scaling, len_lo=start[0],
                len_hi=start[1], fused=fused, tree=tree)


def _append(name, rows, T, lens, heads, group, dim, rot, page=64, dtype="bf16",
            interleaved=False, scaling="none", tree=False, fused=True):
    return dict(name=name, kind="append", rows=rows, T=T, len_lo=lens[0], len_hi=lens[1],
                heads=heads, group=group, dim=dim, rot=rot, page=page, dtype=dtype, layers=1,
                interleaved=interleaved, scaling=scaling, tree=tree, fused=fused)


def _attend(name, groups, members, alone, T, prefix, tail, heads, group, dim, page=64,
            dtype="bf16", tree=False, window=0, sinks=0):
    return dict(name=name, kind="attend", groups=groups, members=members, alone=alone, T=T,
                pre_lo=prefix[0], pre_hi=prefix[1], tail_lo=tail[0], tail_hi=tail[1], heads=heads,
                group=group, dim=dim, page=page, dtype=dtype, tree=tree, window=window,
                sinks=sinks, layers=1)


def listed():
    return [
        # The queries of one user's next token: latency only.
        _rope("rope_one_token", 1, 1, 32, 128, 128, start=(701, 701)),
        # The queries of eight prompts, sliced from a fused projection.
        _rope("rope_prompt", 8, 4093, 32, 128, 128, fused=True),
        # Gradients of a training batch's keys, single precision, interleaved pairs of half a
        # head.
        _rope("rope_grad", 4, 2047, 12, 80, 40, dtype="f32", interleaved=True, inverse=True),
        # A token of every chat of a batch, queries too.
        _append("append_rope_decode", 64, 1, (150, 8000), 8, 8, 128, 128),
        # The benchmark's trees on a context stretched to 131,072 positions.
        _append("append_rope_tree16", 64, 16, (1000, 120000), 8, 4, 128, 128, scaling="turns",
                tree=True),
        # Prompts: one layer's keys, values and queries.
        _append("append_rope_prompt", 8, 4093, (0, 300), 8, 4, 128, 128, dtype="bf16"),
        # Four samples of one short prompt: latency only.
        _attend("shared_samples", 1, 4, 0, 1, (701, 701), (3, 40), 8, 4, 128),
        # 64 chats behind one system prompt.
        _attend("shared_chats", 1, 64, 0, 1, (8100, 8100), (60, 1500), 8, 8, 128),
        # Sixteen prompts with four beams each, trees of 16 nodes, and four rows alone.
        _attend("shared_tree16", 16, 4, 4, 16, (1000, 5000), (5, 300), 8, 8, 128, tree=True),
        # Samples of a long document, a drafted block of 5, an odd group, half precision.
        _attend("shared_long", 1, 8, 0, 5, (120001, 120001), (1, 900), 4, 7, 128, page=128,
                dtype="f16"),
        # Sliding-window layers with sink tokens, wide heads, small pages.
        _attend("shared_window", 2, 12, 1, 9, (5000, 9000), (10, 700), 4, 4, 192, page=16,
                window=4096, sinks=4),
        # A round of trees of nine nodes: four layers of rotation, cache and attention.
        dict(name="step_tree9", kind="step", groups=8, members=4, alone=2, T=9, pre_lo=700,
             pre_hi=2500, tail_lo=5, tail_hi=200, heads=8, group=4, dim=128, rot=128, page=64,
             dtype="bf16", tree=True, window=0, sinks=0, layers=4, interleaved=False,
             scaling="none"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("rope", "append", "attend", "attend", "attend", "step"))
    dim = rng.choice((64, 80, 96, 128, 128, 192, 256))
    page = rng.choice((16, 32, 64, 128))
    rot = rng.choice((dim, dim, dim // 2, dim // 8 * 2, 32))
    scaling = rng.choice(("none", "none", "linear", "turns", "index"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    T = rng.choice((1, 1, 2, 5, 9, 13, 16, 33))
    tree = T > 2 and rng.random() < 0.5
    inter = rng.random() < 0.4
    heads = rng.choice((1, 2, 4, 8))
    if kind == "rope":
        T = _log_int(rng, 1, 4093)
        n = rng.choice((1, 2, 5, 8, 12, 28, 32, 40, 64))
        hi = _log_int(rng, 1, 131000)
        return dict(kind=kind, rows=max(1, min(_log_int(rng, 1, 64), 130_000_000 // (T * n * dim))),
                    T=T, heads=n, dim=dim, rot=rot, dtype=rng.choice(("bf16", "f16", "f32")),
                    interleaved=inter, inverse=rng.random() < 0.4, scaling=scaling,
                    len_lo=rng.randint(0, hi), len_hi=hi, fused=rng.random() < 0.5,
                    tree=T <= 33 and tree)
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    if kind == "append":
        if rng.random() < 0.4:
            T, tree = _log_int(rng, 34, 4000), False
        hi = _log_int(rng, 1, 30000)
        rows = max(1, min(_log_int(rng, 1, 64), 33_000_000 // (T * heads * dim * (1 + group // 4))))
        return dict(kind=kind, rows=rows, T=T, len_lo=rng.randint(0, hi), len_hi=hi, heads=heads,
                    group=group, dim=dim, rot=rot, page=page,
                    dtype=rng.choice(("bf16", "bf16", "f16", "f32")), layers=1, interleaved=inter,
                    scaling=scaling, tree=tree, fused=rng.random() < 0.5)
    members = rng.choice((2, 2, 3, 4, 5, 8, 16, 40, 64))
    pre = _log_int(rng, 40, 60000 if kind == "attend" else 4000)
    tail = _log_int(rng, 1, 1500)
    # No more products and cached elements than the largest listed cases.
    pre = max(1, min(pre, 30_000_000_000 // (members * T * heads * group * dim) - tail))
    tail = max(1, min(tail, 30_000_000_000 // (members * T * heads * group * dim)))
    groups = max(1, min(_log_int(rng, 1, 16), 64 // members,
                        200_000_000 // ((pre + tail * members) * heads * dim),
                        30_000_000_000 // ((pre + tail) * members * T * heads * group * dim)))
    c = dict(kind=kind, groups=groups, members=members, alone=rng.choice((0, 0, 1, 3)), T=T,
             pre_lo=rng.randint(max(1, pre // 2), pre), pre_hi=pre, tail_lo=rng.randint(1, tail),
             tail_hi=tail, heads=heads, group=group, dim=dim, page=page, dtype=dtype, tree=tree)
    if kind == "attend":
        window, sinks = (rng.choice((64, 1000, 4096)), rng.choice((0, 1, 4, 130))) \
            if rng.random() < 0.25 else (0, 0)
        return dict(c, window=window, sinks=sinks, layers=1)
    return dict(c, window=0, sinks=0, layers=rng.randint(1, 4), rot=rot, interleaved=inter,
                scaling=scaling)


# ------------------------------------------------------------------ rotary frequencies
BASE, STRETCH, ORIGINAL = 500000.0, 8.0, 8192.0
TURNS = {"turns": (1.0, 4.0), "index": (1.0, 32.0)}  # low, high
GAIN = {"index": 0.1 * math.log(STRETCH) + 1.0}      # of cosine and sine


def _spread(lo, hi, i, n):
    """The i-th of n numbers from hi down to lo."""
    return hi - (hi - lo) * i // max(n - 1, 1)


def _tree(rows, T, rnd):
    """Parent links of random draft trees."""
    return [[-1] + [rnd.randint(max(0, n - 4), n - 1) for n in range(1, T)] for _ in range(rows)]


def _n_new(case):
    """New tokens of a case's rows: full blocks and, for short ones, a third ragged."""
    T, R = case["T"], _rows(case)
    if T > 33:
        return [T] * R
    return [1 + 5 * i % T if i % 3 == 1 else T for i in range(R)]


def _rows(c):
    return c["rows"] if "rows" in c else c["groups"] * c["members"] + c["alone"]


def _lens(c):
    """Cached lengths of the rows, and how many tokens (whole pages) row i shares with its group."""
    R = _rows(c)
    if "rows" in c:
        return [_spread(c["len_lo"], c["len_hi"], i, R) for i in range(R)], [0] * R
    G, N, ps = c["groups"], c["members"], c["page"]
    lens, shared = [], []
    for i in range(R):
        pre = _spread(c["pre_lo"], c["pre_hi"], i // N % max(G, 1), G)
        tail = _spread(c["tail_lo"], c["tail_hi"], i * 7 % R, R)
        shared.append(pre // ps * ps if i < G * N else 0)
        lens.append(pre + tail)
    return lens, shared


# ------------------------------------------------------------------ inputs
def _pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9), not below 2^EXP_MIN."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(min=EXP_MIN)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    s = _pow2_scale(x.abs().amax(dim=(-2, -1)))
    return (x / s[..., None, None]).to(F8), s


def _inputs(case, seed):
    """Tensors of a case, from the seed alone."""
    rnd = random.Random(seed * 6151 + 29)
    g = torch.Generator(device=DEV).manual_seed(seed)
    c, R, T, D = case, _rows(case), case["T"], case["dim"]
    lens, shared = _lens(c)
    n_new = _n_new(c)
    par = _tree(R, T, rnd) if c["tree"] else None
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    st = dict(case=c, lens=lens, n_new_host=n_new, parent_host=par, len=i32(lens),
              n_new=i32(n_new), parent=None if par is None else i32(par), scale=D ** -0.5)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if c["kind"] == "rope":
        # Projections, or their gradients, which are small.
        H, dt = c["heads"], DTYPES[c["dtype"]]
        x = torch.empty(R, T, H + 2 if c["fused"] else H, D, dtype=dt, device=DEV)
        x[:, :, H:] = 0
        x[:, :, :H] = (randn(R, T, H, D) * (1e-3 if c["inverse"] else 1.0)).to(dt)
        st["x"] = x[:, :, :H]
        return st
    H, G, ps, Ly, dt = c["heads"], c["group"], c["page"], c["layers"], DTYPES[c["dtype"]]
    # Rows hold the pages of their tokens and of the new ones; the first pages of a group's
    # rows are the same ones. Page ids in random order, some pages free between them.
    max_pages = max(-(-(n + T) // ps) for n in lens) + 1
    mine = [-(-(n + T) // ps) - s // ps for n, s in zip(lens, shared)]
    leader = [i // c["members"] * c["members"] if shared[i] else i for i in range(R)] \
        if "members" in c else list(range(R))
    pages = sum(mine) + sum(s // ps for i, s in enumerate(shared) if leader[i] == i) + 3
    ids = list(range(pages))
    rnd.shuffle(ids)
    ids, own_pages, held = iter(ids), [], []
    table = torch.full((R, max_pages), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    first = {}
    for i in range(R):
        if shared[i] and leader[i] not in first:
            first[leader[i]] = [next(ids) for _ in range(shared[i] // ps)]
        row = first.get(leader[i], []) + [next(ids) for _ in range(mine[i])]
        table[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
        refs[torch.tensor(row)] += 1
        held.append(len(row))
    st.update(table=table.to(DEV), refs=refs.to(DEV), n_pages=i32(held), max_pages=max_pages,
              group=i32(leader), shared=shared, leader=leader)
    # Keys with a few strong channels per head; the first token of a row draws much of the
    # attention; queries lean towards it.
    chan = torch.exp(0.4 * randn(H, 1, D))
    chan[:, :, ::37] *= 4.0
    lean = randn(H, 1, D)
    st["k"] = torch.empty(Ly, pages, H, ps, D, dtype=F8, device=DEV)
    st["v"] = torch.empty_like(st["k"])
    st["k_scale"] = torch.empty(Ly, pages, H, device=DEV)
    st["v_scale"] = torch.empty(Ly, pages, H, device=DEV)
    heads0 = table[:, 0].long().to(DEV)
    for ly in range(Ly):
        x = randn(pages, H, ps, D) * chan
        x[heads0, :, 0] += 0.8 * lean[:, 0]
        st["k"][ly], st["k_scale"][ly] = _quantise(x)
        st["v"][ly], st["v_scale"][ly] = _quantise(randn(pages, H, ps, D) * torch.exp(
            0.5 * randn(H, 1, 1)))
    # Every layer's queries, keys and values, sliced from a fused projection or dense.
    st["new"] = []
    for _ in range(Ly):
        qkv = torch.empty(R, T, H * (G + 2), D, dtype=dt, device=DEV)
        qkv[:, :, :H * G] = (randn(R, T, H * G, D)
                             + 0.6 * lean[:, 0].repeat_interleave(G, 0)).to(dt)
        qkv[:, :, H * G:-H] = (randn(R, T, H, D) * chan[:, 0]).to(dt)
        qkv[:, :, -H:] = randn(R, T, H, D).to(dt)
        parts = qkv[:, :, :H * G], qkv[:, :, H * G:-H], qkv[:, :, -H:]
        st["new"].append(parts if c.get("fused", True) else tuple(x.contiguous() for x in parts))
    return st


def _freqs(c):
    """Angle of each pair per position, in radians."""
    rot, low, high = c["rot"], *TURNS.get(c["scaling"], (0, 0))
    f = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if c["scaling"] == "linear":
        return [x / STRETCH for x in f]
    if c["scaling"] == "none":
        return f
    if c["scaling"] == "turns":  # kept share: by the turns over the original context
        keep = [min(1.0, max(0.0, (ORIGINAL * x / (2 * math.pi) - low) / (high - low))) for x in f]
    else:                        # by the pair's index between those of `high` and `low` turns
        at = lambda n: rot * math.log(ORIGINAL / (2 * math.pi * n)) / (2 * math.log(BASE))  # noqa: E731
        a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        keep = [1.0 - min(1.0, max(0.0, (i - a) / max(b - a, 1e-3))) for i in range(rot // 2)]
    return [x * (k + (1.0 - k) / STRETCH) for x, k in zip(f, keep)]


def prepare(case, seed):
    st = _inputs(case, seed)
    c = case
    if "rot" in c:
        st["freqs"] = torch.tensor(_freqs(c), dtype=torch.float64, device=DEV)
    if own:
        import speculative_decoding_verification_79_gb300 as sv

        if "rot" in c:
            low, high = TURNS.get(c["scaling"], (1.0, 2.0))
            st["rope"] = sv.Rope(c["rot"], base=BASE, interleaved=c["interleaved"],
                                 scaling=c["scaling"], stretch=STRETCH, original=ORIGINAL, low=low,
                                 high=high, gain=GAIN.get(c["scaling"], 1.0), device=DEV)
        if c["kind"] == "rope":
            return st
        Ly, pages, H, ps, D = st["k"].shape
        kv = sv.KVCache(Ly, pages, ps, H, D, _rows(c), st["max_pages"], device=DEV)
        for f in ("k", "v", "k_scale", "v_scale", "table", "n_pages", "len", "refs"):
            getattr(kv, f).copy_(st.pop(f))
        st["cache"] = kv
        if c["kind"] != "append":
            st["share"] = sv.KVShare(kv, c["T"], H * c["group"])
        if c["kind"] == "attend":
            sv.sv_kv_share(kv, st["share"], st["group"])
    return st


# ------------------------------------------------------------------ the plain forms
def _sees(st):
    """[rows, T, T]: which nodes of its block a token sees."""
    T = st["case"]["T"]
    i = torch.arange(T, device=DEV)
    if st["parent"] is None:
        return (i[None] <= i[:, None]).expand(_rows(st["case"]), T, T)
    up = (st["parent"][..., None] == i).float()  # node -> its parent (none for the first)
    up[:, 0] = 0
    return torch.linalg.matrix_power(up + torch.eye(T, device=DEV), T) > 0


def _positions(st):
    """[rows, T]: the first position plus the token's depth in its block."""
    if st["parent"] is None:
        return st["len"].long()[:, None] + torch.arange(st["case"]["T"], device=DEV)
    return st["len"].long()[:, None] + _sees(st).sum(2) - 1


def _rotate(st, x, sign=1.0):
    """x [rows, T, heads, dim] rotated by its positions, in float32."""
    c = st["case"]
    rot, x = c["rot"], x.float()
    angle = (_positions(st).double()[..., None] * st["freqs"])[:, :, None]
    gain = GAIN.get(c["scaling"], 1.0)
    cos, sin = (torch.cos(angle) * gain).float(), (torch.sin(angle) * (gain * sign)).float()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _live(st):
    """[rows, T]: is the token there?"""
    return torch.arange(st["case"]["T"], device=DEV) < st["n_new"][:, None]


def _blank(st, x):
    """x [rows, T, ...] with zeros for tokens that are not there."""
    live = _live(st)
    return torch.where(live.view(*live.shape, *[1] * (x.dim() - 2)), x, 0.0)


def _tokens(st, pos):
    """Page id and slot of positions pos [rows, n] (clamped into the table)."""
    ps = st["k"].shape[3]
    j = (pos // ps).clamp(0, st["table"].shape[1] - 1)
    return st["table"].long().gather(1, j).clamp(min=0), pos % ps


def _append_plain(st, layer, k, v):
    """k, v [rows, T, heads, dim] float32 into the pages behind the rows' tokens."""
    ps, n_new = st["k"].shape[3], st["n_new"]
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
    for name, x in (("k", k), ("v", v)):
        pool, scale = st[name][layer], st[name + "_scale"][layer]
        x = x.gather(1, t[..., None, None].expand(-1, -1, H, D))
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
        bytes_[ppid[:, 0]] = torch.where(keep[:, None, :, None], re, page0)
        scale[ppid] = s.gather(1, j[..., None].expand(rows, J, H))
        q = (x / s.gather(1, jj[..., None].expand(-1, -1, H))[..., None]).to(F8)
        bytes_[pid[..., None], h, slot[..., None]] = q.view(torch.uint8)


def _read_plain(st):
    """Every layer's new keys and values as the cache holds them."""
    pos = st["len"].long()[:, None] + torch.arange(st["case"]["T"], device=DEV)
    pid, slot = _tokens(st, pos)
    live, h = _live(st)[None, :, :, None, None], torch.arange(st["k"].shape[2], device=DEV)
    out = []
    for name in ("k", "v"):
        val = st[name].view(torch.uint8)[:, pid[..., None], h, slot[..., None]]
        val = val.view(F8).float() * st[name + "_scale"][:, pid][..., None]
        out.append(torch.where(live, val, 0.0).to(torch.bfloat16))
    return out


def _attend_plain(st, layer, q):
    """All rows at once, padded to the longest; q [rows, T, q_heads, dim] of the case's type."""
    c = st["case"]
    R, T, H, G, D, ps = _rows(c), c["T"], c["heads"], c["group"], c["dim"], c["page"]
    pid = st["table"].long().clamp(min=0)
    S = pid.shape[1] * ps
    j = torch.arange(S, device=DEV)
    L = st["len"].long()[:, None]
    held = (j < L + st["n_new"][:, None])[:, None, :, None]  # a row's own tokens
    k, v = ((st[n][layer][pid].float() * st[n + "_scale"][layer][pid][..., None, None])
            .transpose(1, 2).reshape(R, H, S, D) for n in ("k", "v"))
    q = q.float().reshape(R, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, T * G, D)
    s = torch.matmul(q, torch.where(held, k, 0.0).transpose(2, 3)) * st["scale"]
    pos = _positions(st)
    i = (j - L).clamp(0, T - 1)  # the block's node at a position
    see = torch.gather(_sees(st), 2, i[:, None].expand(R, T, S)) | (j < L)[:, None]
    see = see & (j < L + st["n_new"][:, None])[:, None] & _live(st)[..., None]
    if c["window"]:
        at = torch.where(j < L, j, torch.gather(pos, 1, i))
        see = see & ((pos[..., None] - at[:, None] < c["window"]) | (j < c["sinks"]))
    see = see.repeat_interleave(G, 1)[:, None]
    s = torch.where(see, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(s - top)
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(held, v, 0.0)) / torch.where(den > 0, den, 1.0)
    lse = (torch.log(den) + top)[..., 0]
    back = lambda x: x.reshape(R, H, T, G, *x.shape[3:]).transpose(1, 2).flatten(2, 3)  # noqa: E731
    return back(o).to(DTYPES[c["dtype"]]), back(lse)


def _plain(st):
    c = st["case"]
    if c["kind"] == "rope":
        x = st["x"]
        return _blank(st, _rotate(st, x, -1.0 if c["inverse"] else 1.0).to(x.dtype))
    if c["kind"] == "attend":
        return _attend_plain(st, 0, st["new"][0][0])
    out = []
    for ly, (q, k, v) in enumerate(st["new"]):
        _append_plain(st, ly, _rotate(st, k), v.float())
        q = _blank(st, _rotate(st, q).to(q.dtype))
        out.append(q if c["kind"] == "append" else _attend_plain(st, ly, q))
    return [out, _read_plain(st)]


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import speculative_decoding_verification_79_gb300 as sv

    c = st["case"]
    if c["kind"] == "rope":
        return sv.sv_rope(st["rope"], st["x"], start=st["len"], parent=st["parent"],
                          n_new=st["n_new"], inverse=c["inverse"])
    cache = st["cache"]
    if c["kind"] == "attend":
        return sv.sv_kv_attend_shared(cache, 0, st["new"][0][0], st["share"], n_new=st["n_new"],
                                      parent=st["parent"], scale=st["scale"], window=c["window"],
                                      sinks=c["sinks"], want_lse=True)
    if c["kind"] == "step":
        sv.sv_kv_share(cache, st["share"], st["group"])
    out = []
    for ly, (q, k, v) in enumerate(st["new"]):
        q = sv.sv_kv_append_rope(cache, ly, k, v, st["rope"], q=q, n_new=st["n_new"],
                                 parent=st["parent"])
        if c["kind"] == "step":
            q = sv.sv_kv_attend_shared(cache, ly, q, st["share"], n_new=st["n_new"],
                                       parent=st["parent"], scale=st["scale"], want_lse=True)
        out.append(q)
    return [out, list(sv.sv_kv_read(cache, cache.len, c["T"], count=st["n_new"]))]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    """Each cached token read once per key/value head (a group's common ones once), each input
    and output once."""
    c = case
    R, T, D, eb = _rows(c), c["T"], c["dim"], 4 if c["dtype"] == "f32" else 2
    if c["kind"] == "rope":
        n = sum(_n_new(c)) * c["heads"]
        return {"bytes": int(n * D * eb + R * T * c["heads"] * D * eb), "flops": int(3 * n * c["rot"])}
    H, G, Ly = c["heads"], c["group"], c["layers"]
    new = sum(_n_new(c))
    total = {"bytes": 0, "flops": 0}
    if c["kind"] in ("append", "step"):
        kv = new * H * D * 2
        total["bytes"] += Ly * (kv * eb + kv + 2 * R * T * H * D * 2 + kv)
        total["flops"] += Ly * (2 * kv + 3 * new * H * (G + 1) * c["rot"])
        if c["kind"] == "append":
            total["bytes"] += (new + R * T) * H * G * D * eb
    if c["kind"] in ("attend", "step"):
        W, S = c["window"], c["sinks"]
        lens, shared = _lens(c)
        tokens = pairs = 0
        first = {}  # oldest tokens that a group's rows see, by the group's number
        for i, (n, m) in enumerate(zip(lens, _n_new(c))):
            lo = max(0, n + 1 - W) if W else 0
            mine = max(n + m - max(lo, shared[i]), 0)
            if shared[i]:
                at = i // c["members"]
                first[at] = min(first.get(at, shared[i]), lo)
                if first[at] == lo:
                    first[at, "n"] = max(shared[i] - lo, 0) + min(S, lo)
            else:
                mine += min(S, lo)
            tokens += mine
            for t in range(m):
                pairs += min(n + t + 1, W) + min(S, max(0, n + t + 1 - W)) if W else n + t + 1
        tokens += sum(x for k, x in first.items() if isinstance(k, tuple))
        kv = tokens * H * D * 2 + tokens / c["page"] * H * 8
        total["bytes"] += Ly * (kv + R * T * H * G * (D * eb * 2 + 4))
        total["flops"] += Ly * 4 * pairs * G * H * D
    return {k: int(x) for k, x in total.items()}


# ------------------------------------------------------------------ the same in 64 bits
def _depth(par, t):
    """Ancestors of node t and itself, nearest first."""
    up = [t]
    while up[-1] > 0:
        up.append(par[up[-1]] if par else up[-1] - 1)
    return up


def _turned(c, x, positions, back=False):
    """x [T, heads, dim] float64 rotated by positions: complex numbers times unit vectors."""
    rot = c["rot"]
    f = torch.tensor(_freqs(c), dtype=torch.float64, device=DEV)
    angle = torch.tensor(positions, dtype=torch.float64, device=DEV)[:, None] * f
    unit = torch.polar(torch.full_like(angle, GAIN.get(c["scaling"], 1.0)),
                       -angle if back else angle)[:, None]
    y = x.clone()
    if c["interleaved"]:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * unit
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * unit
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exp2(e):
    """2^e in float64 of whole e, exactly, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """Nearest e4m3 value (3 bits of fraction, exponents from -6), ties to even."""
    _, e = torch.frexp(x)
    step = _exp2((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _scale64(a):
    """Smallest power of two s >= 2^EXP_MIN with a <= 448 s, of a float64 tensor."""
    _, e = torch.frexp(a)  # a < 2^e, so 2^(e - 8) is enough, and half of it may be
    s = _exp2(torch.where(a > 0, e - 8, EXP_MIN).clamp(min=EXP_MIN))
    return torch.where((a <= 224.0 * s) & (s > 2.0 ** EXP_MIN), s / 2, s)


def exact(case, seed):
    c, st = case, _inputs(case, seed)
    R, T, D, n_new, lens = _rows(c), c["T"], c["dim"], st["n_new_host"], st["lens"]
    par = st["parent_host"] or [None] * R
    ups = [[_depth(par[b], t) for t in range(n_new[b])] for b in range(R)]
    pos = [[lens[b] + len(u) - 1 for u in ups[b]] for b in range(R)]
    f64 = dict(dtype=torch.float64, device=DEV)
    if c["kind"] == "rope":
        out = torch.zeros(R, T, c["heads"], D, **f64)
        for b in range(R):
            out[b, :n_new[b]] = _turned(c, st["x"][b, :n_new[b]].double(), pos[b], c["inverse"])
        return out
    H, G, ps, Ly = c["heads"], c["group"], c["page"], c["layers"]
    read = [torch.zeros(Ly, R, T, H, D, **f64) for _ in range(2)]
    outs = []
    for ly, (q, k, v) in enumerate(st["new"]):
        o = torch.zeros(R, T, H * G, D, **f64)
        lse = torch.full((R, T, H * G), -math.inf, **f64)
        for b in range(R):
            n, L = n_new[b], lens[b]
            ids = st["table"][b, : -(-(L + n) // ps)].long()
            # The row's tokens, page by page: numbers [pages, heads, page, dim] and scales.
            val = [st[m][ly][ids].double() for m in ("k", "v")]
            sc = [st[m + "_scale"][ly][ids].double() for m in ("k", "v")]
            qb = q[b, :n].double()
            if c["kind"] != "attend":
                qb = _turned(c, qb, pos[b])
                new = _turned(c, k[b, :n].double(), pos[b]), v[b, :n].double()
                for p in range(L // ps, len(ids)):
                    lo, hi = max(L, p * ps), min(L + n, (p + 1) * ps)
                    for m in range(2):
                        x = new[m][lo - L: hi - L].transpose(0, 1)  # [heads, tokens, dim]
                        s = _scale64(x.abs().amax((1, 2)))
                        at = lo - p * ps
                        if at:
                            s = torch.maximum(s, sc[m][p])
                            val[m][p, :, :at] = _e4m3(val[m][p, :, :at]
                                                      * (sc[m][p] / s)[:, None, None])
                        val[m][p, :, at: at + hi - lo] = _e4m3(x / s[:, None, None])
                        sc[m][p] = s
            kk, vv = ((val[m] * sc[m][..., None, None]).transpose(0, 1).reshape(H, -1, D)[:, :L + n]
                      for m in range(2))
            if c["kind"] != "attend":
                read[0][ly, b, :n], read[1][ly, b, :n] = (x[:, L:].transpose(0, 1)
                                                          for x in (kk, vv))
            if c["kind"] == "append":
                o[b, :n] = qb
                continue
            qb = qb.to(DTYPES[c["dtype"]]).double() if c["kind"] == "step" else qb
            mask = np.zeros((n, L + n), dtype=bool)
            for t in range(n):
                j = np.arange(L)
                mask[t, :L] = (pos[b][t] - j < c["window"]) | (j < c["sinks"]) if c["window"] \
                    else True
                for steps, i in enumerate(ups[b][t]):
                    mask[t, L + i] = not c["window"] or steps < c["window"] or L + i < c["sinks"]
            mask = torch.from_numpy(mask).to(DEV)
            for h in range(H):
                s = torch.einsum("tgd,jd->tgj", qb[:, h * G:(h + 1) * G], kk[h]) * st["scale"]
                s = s.masked_fill(~mask[:, None], -math.inf)
                z = torch.logsumexp(s, -1)
                w = torch.where(torch.isinf(z)[..., None], 0.0, torch.exp(s - z[..., None]))
                o[b, :n, h * G:(h + 1) * G] = w @ vv[h]
                lse[b, :n, h * G:(h + 1) * G] = z
        outs.append(o if c["kind"] == "append" else (o, lse))
    return outs[0] if c["kind"] == "attend" else [outs, read]
