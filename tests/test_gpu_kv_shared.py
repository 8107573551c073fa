"""GPU parity of attention over shared pages with the plain float64 model of kv_ref, within the
bounds that test_gpu_kv derives for sv_kv_attend: the shared call rounds nothing more, but
joins one part more (an exponential and a product of float32, inside their 2^-19)."""
import math

import numpy as np
import pytest
import torch

import kv_ref
from test_gpu_kv import Both, bounds, check_attend, f64, i32, needs_cuda, rand_kv, tree

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


@pytest.fixture(autouse=True, params=[True, False], ids=["always", "rule"])
def always(request, sv):
    """Every group's common tokens read once, and only where the library finds that faster."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    prev = sv.set_share_always(request.param)
    yield request.param
    sv.set_share_always(prev)


def rows_of(groups, alone):
    """Rows of groups and lone rows, dealt out so that a group's rows are not neighbours: leader
    of each row."""
    sizes = [m for m, _ in groups]
    order, left = [], [list(range(m)) for m in sizes]
    while any(left):
        for g, x in enumerate(left):
            if x:
                x.pop()
                order.append(g)
    for i in range(len(alone)):
        order.insert(3 * i % (len(order) + 1), len(groups) + i)
    first = {}
    return [first.setdefault(g, b) for b, g in enumerate(order)], order


def grouped(sv, groups, alone, tails, heads, dim, page, T, seed=0, sigma=0.5):
    """A cache of forked rows: groups [(rows, common tokens)], lone rows [tokens], and for every
    row a tail of its own (tails, in turn)."""
    lead, order = rows_of(groups, alone)
    B = len(order)
    common = [p for _, p in groups] + list(alone)
    tail = [tails[b % len(tails)] for b in range(B)]
    longest = max(common[g] + t for g, t in zip(order, tail)) + T
    per = -(-longest // page) + 1
    need = sum(-(-c // page) for c in common) + sum(-(-(t + T + page) // page) + 1 for t in tail)
    both = Both(sv, 1, need + 4, page, heads, dim, B, per)
    both.fill([common[order[b]] if lead[b] == b else 0 for b in range(B)], seed, sigma)
    assert all(both.fork(lead))
    assert all(both.reserve(tail))
    k, v = rand_kv(both.r, max(tail + [1]), seed + 31, sigma)
    both.append(0, k, v, tail)
    both.commit([t - 1 for t in tail], max(tail + [1]))
    return both, lead


def block(both, T, seed, n, sigma=0.5):
    assert all(both.reserve(n))
    k, v = rand_kv(both.r, T, seed + 77, sigma)
    both.append(0, k, v, n)


def queries(both, T, group, dtype, seed, q_sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    q = torch.randn(both.r.batch, T, both.r.heads * group, both.r.dim, generator=g, device="cuda")
    return (q_sigma * q).to(dtype)


def case(sv, groups, alone=(), tails=(5,), T=1, heads=2, group=4, dim=64, page=16, dtype=BF,
         trees=False, window=0, sinks=0, seed=0, n=None, by_page=False, q_sigma=1.0, sigma=0.5,
         rows=None):
    both, lead = grouped(sv, groups, list(alone), list(tails), heads, dim, page, T, seed, sigma)
    B, rng = both.r.batch, np.random.default_rng(seed)
    if n is None:
        n = [int(x) for x in rng.integers(0, T + 1, B)]
        n[0] = T
    block(both, T, seed, n, sigma)
    par = [tree(rng, T) for _ in range(B)] if trees else None
    q = queries(both, T, group, dtype, seed, q_sigma)
    share = sv.KVShare(both.g, T, heads * group)
    sv.sv_kv_share(both.g, share, None if by_page else i32(lead))
    kw = dict(n_new=i32(n), parent=None if par is None else i32(par), window=window, sinks=sinks,
              want_lse=True)
    got = sv.sv_kv_attend_shared(both.g, 0, q, share, **kw)
    check_attend(both, 0, q, n, par, window=window, sinks=sinks, got=got, rows=rows)
    again = sv.sv_kv_attend_shared(both.g, 0, q, share, **kw)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    both.same()
    return both, q, n, par, share, kw, got


@needs_cuda
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim,page", [(16, 16), (64, 64), (80, 16), (128, 128), (128, 32),
                                      (192, 16), (256, 64)])
@pytest.mark.parametrize("T,trees", [(1, False), (9, True), (16, False)])
def test_sizes(sv, dim, page, T, trees, dtype):
    case(sv, [(3, 700), (4, 1500), (2, 130), (2, 100)], [900, 3], [5, 40, 200, 1], T, 2, 4, dim, page,
         dtype, trees, seed=T + dim)


@needs_cuda
@pytest.mark.parametrize("members,heads,group,T", [
    (2, 1, 1, 1), (2, 2, 16, 1), (3, 1, 11, 1), (4, 2, 8, 1), (5, 1, 13, 1), (8, 1, 8, 1),
    (9, 2, 15, 1), (16, 2, 8, 1), (17, 1, 8, 1), (33, 1, 7, 3), (64, 1, 8, 1), (12, 2, 8, 9),
    (2, 1, 128, 1), (3, 1, 100, 3), (40, 1, 1, 5)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups(sv, members, heads, group, T, dim):
    """Query tiles of every width, and groups of several."""
    case(sv, [(members, 1000), (2, 640)], [77], [3, 130, 60], T, heads, group, dim, 64,
         seed=members + T)


@needs_cuda
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (100, 1), (300, 130), (1000, 4),
                                          (4096, 700), (640, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("T,trees", [(1, False), (13, True), (16, False)])
def test_windows(sv, window, sinks, T, trees):
    """Windows that reach all, some or none of the common tokens, by row."""
    case(sv, [(4, 1300), (6, 700)], [500], [2, 300, 700, 90], T, 2, 8, 64, 16, trees=trees,
         window=window, sinks=sinks, seed=window % 1000 + T)


@needs_cuda
@pytest.mark.parametrize("common", [0, 1, 127, 128, 129, 255, 256, 257, 384])
@pytest.mark.parametrize("page", [16, 128])
def test_common_lengths(sv, common, page):
    """Around multiples of a key tile and of a page; rows without tokens of their own."""
    case(sv, [(6, common)], [40], [0, 1, 30, 0], 4, 1, 8, 64, page, seed=common, n=[4, 1, 0, 4, 2, 4, 3])
    case(sv, [(6, common)], [], [0], 1, 1, 8, 64, page, seed=common, n=[1] * 6)


@needs_cuda
def test_long_and_many(sv):
    """Common tokens cut between many CTAs; many groups; a large batch of small ones."""
    case(sv, [(8, 20000)], [9000], [3, 700], 5, 1, 7, 128, 128, HF, seed=1, n=[5] * 9)
    case(sv, [(3, 300 + 50 * g) for g in range(20)], [], [9], 2, 1, 8, 64, 32, seed=2)
    case(sv, [(2, 520)] * 150, [20] * 400, [3], 1, 1, 2, 16, 16, seed=3)


@needs_cuda
@pytest.mark.parametrize("q_sigma,sigma", [(0.0, 0.5), (0.01, 3.0), (30.0, 0.0), (30.0, 3.0)])
def test_score_ranges(sv, q_sigma, sigma):
    """Weights all alike, and scores far apart between the common and a row's own tokens.

    A weight times its value's scale is kept to 2^-28 of the row's largest such product (in all
    attention calls): with values of sizes as far apart as these, components that only small
    weights make up are off by that much times the sum of what multiplies it, the values over
    their scales."""
    both, q, n, par, share, kw, got = case(sv, [(20, 700), (3, 500)], [100], [40, 3], 3, 2, 8, 128, 64,
                                           seed=4, q_sigma=q_sigma, sigma=sigma, rows=[])
    r, scale, page = both.r, 128 ** -0.5, 64
    for b in range(r.batch):
        L = r.len[b] + n[b]
        k, v = r.values(0, 0, b, 0, L), r.values(1, 0, b, 0, L)
        o, ls, av, ab, qk = kv_ref.attend(f64(q[b]), k, v, r.len[b], n[b], scale)
        bo, bl = bounds(o, ls, av, ab, qk, scale, q.dtype)
        s = np.stack([r.s[1, 0, r.rows[b][j // page]] for j in range(L)])  # [L, heads]
        codes = (np.abs(v) / s[..., None]).sum(0)                           # [heads, dim]
        for t in range(n[b]):
            for h in range(16):
                w = np.exp(k[:r.len[b] + t + 1, h // 8] @ f64(q[b, t, h]) * scale - ls[t, h])
                floor = 2.0 ** -28 * (w * s[:r.len[b] + t + 1, h // 8]).max() * codes[h // 8]
                assert (np.abs(f64(got[0][b, t, h]) - o[t, h]) <= bo[t, h] + floor).all()
        assert (np.abs(f64(got[1][b]) - ls)[:n[b]] <= bl[:n[b]]).all()


@needs_cuda
def test_by_first_page(sv):
    """Without group numbers, rows whose first page is the same belong together."""
    a = case(sv, [(5, 700), (3, 300)], [400, 200], [9, 60], 2, 2, 8, 64, 16, seed=5, by_page=True)
    b = case(sv, [(5, 700), (3, 300)], [400, 200], [9, 60], 2, 2, 8, 64, 16, seed=5)
    assert torch.equal(a[-1][0], b[-1][0])


@needs_cuda
@pytest.mark.parametrize("T,group", [(1, 8), (9, 8)])
def test_no_groups(sv, T, group):
    """A new buffer, rows that are all alone, numbers that are out of range, and no new tokens."""
    both, q, n, par, share, kw, got = case(sv, [(4, 700)], [300], [9, 60], T, 2, group, 64, 16, seed=6)
    g, B = both.g, both.r.batch
    fresh = sv.KVShare(g, T, 2 * group)
    check_attend(both, 0, q, n, got=sv.sv_kv_attend_shared(g, 0, q, fresh, **kw))
    sv.sv_kv_share(g, fresh, i32([-1] * B))
    check_attend(both, 0, q, n, got=sv.sv_kv_attend_shared(g, 0, q, fresh, **kw))
    assert g.status(clear=True) == sv.SV_OK
    sv.sv_kv_share(g, fresh, i32([B, -2, 2 ** 31 - 1, -2 ** 31] + [1] * (B - 4)))
    assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
    check_attend(both, 0, q, n, got=sv.sv_kv_attend_shared(g, 0, q, fresh, **kw))
    sv.sv_kv_share(g, fresh, i32([0] * B))  # (rows with little in common)
    check_attend(both, 0, q, n, got=sv.sv_kv_attend_shared(g, 0, q, fresh, **kw))
    out, lse = sv.sv_kv_attend_shared(g, 0, q, share, n_new=i32([0] * B), want_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert g.status() == sv.SV_OK


@needs_cuda
def test_smaller_calls_on_a_buffer(sv):
    """Calls of fewer tokens and heads than the buffer was made for, in turn."""
    both, lead = grouped(sv, [(6, 700), (3, 400)], [90], [9, 60], 2, 64, 16, 9)
    share = sv.KVShare(both.g, 9, 32)
    sv.sv_kv_share(both.g, share, i32(lead))
    block(both, 9, 0, [9] * both.r.batch)
    for T, group in ((9, 16), (1, 4), (5, 16), (1, 16), (9, 2)):
        q = queries(both, T, group, BF, T)
        n = [T] * both.r.batch
        got = sv.sv_kv_attend_shared(both.g, 0, q, share, n_new=i32(n), want_lse=True)
        check_attend(both, 0, q, n, got=got)
    with pytest.raises(sv.SpecVerifyError):
        sv.sv_kv_attend_shared(both.g, 0, queries(both, 9, 32, BF, 0), share)
    both.same()


@needs_cuda
@pytest.mark.parametrize("what", ["table", "len", "n_pages", "count", "count_high", "tree", "own_page",
                                  "scale"])
def test_rows_with_wrong_data(sv, what, always):
    """A row that no longer holds what its group shares, or has other wrong data, is NaN; the
    others are right, and so is the row when the groups are found again."""
    if not always:
        pytest.skip("rows may be attended to by themselves")
    T = 6
    both, q, n, par, share, kw, want = case(sv, [(6, 2000), (3, 400)], [90], [20, 60], T, 2, 4, 64, 16,
                                            trees=True, seed=8, n=[6] * 10)
    g, bad = both.g, 5  # (of the first group, not its first row)
    old = [t.clone() for t in (g.table, g.len, g.n_pages, g.k_scale)]
    again = n
    if what == "table":
        g.table[bad, 3] = int(g.table[bad, 126])
    if what == "len":
        g.len[bad] = 30
    if what == "n_pages":
        g.n_pages[bad] = 2
    if what == "own_page":
        g.table[bad, 126] = -5
    if what == "scale":
        g.k_scale[0, int(g.table[bad, 127])] = math.inf
    if what.startswith("count"):
        again = [x if i != bad else (-1 if what == "count" else T + 1) for i, x in enumerate(n)]
    par2 = [list(p) for p in par]
    if what == "tree":
        par2[bad][3] = 3
    call = lambda p, m: sv.sv_kv_attend_shared(g, 0, q, share, **dict(  # noqa: E731
        kw, parent=i32(p), n_new=i32(m)))
    for _ in range(2):
        out, lse = call(par2, again)
        assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
        assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
        check_attend(both, 0, q, n, par, got=(out, lse), rows=[b for b in range(10) if b != bad])
    for t, o in zip((g.table, g.len, g.n_pages, g.k_scale), old):
        t.copy_(o)
    if what in ("table", "len", "n_pages"):
        assert torch.isnan(call(par, n)[0][bad].float()).all()
        g.status(clear=True)
    sv.sv_kv_share(g, share, i32(rows_of([(6, 2000), (3, 400)], [90])[0]))
    out, lse = call(par, n)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and g.status() == sv.SV_OK


@needs_cuda
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("members,group,window", [(3, 4, 0), (6, 8, 0), (20, 8, 0), (6, 8, 300)])
def test_stored_nan(sv, what, members, group, window):
    """A NaN in a common token reaches every row of the group that sees it, and no other."""
    both, q, n, par, share, kw, want = case(sv, [(members, 700), (2, 400)], [90], [20, 60], 2, 2, group,
                                            64, 16, seed=9, window=window,
                                            n=[2] * (members + 3))
    g, (lead, order) = both.g, rows_of([(members, 700), (2, 400)], [90])
    first = order.index(0)
    at = 650
    getattr(g, what).view(torch.uint8)[0, int(g.table[first, at // 16]), 1, at % 16, 7] = 0x7F
    out, lse = sv.sv_kv_attend_shared(g, 0, q, share, **kw)
    for b in range(both.r.batch):
        sees = order[b] == 0 and (not window or both.r.len[b] - at < window)
        h = group  # (heads of key/value head 1 come second)
        assert torch.equal(out[b, :, :h], want[0][b, :, :h])
        got = out[b, 0, h:].float()
        if sees:
            assert torch.isnan(got[..., 7] if what == "v" else got).all()
        else:
            assert torch.equal(out[b, 0, h:], want[0][b, 0, h:])
    assert g.status() == sv.SV_OK


@needs_cuda
@pytest.mark.parametrize("dim,T,group", [(128, 1, 8), (64, 9, 4), (128, 16, 8), (256, 9, 8)])
def test_gives_up(sv, dim, T, group):
    """Waits with a bound that they pass, at the first of them or later: the call ends, says
    SV_ERR_TIMEOUT, and the next call on the same buffer has the bits it had before."""
    both, q, n, par, share, kw, want = case(sv, [(7, 2000), (2, 500)], [300], [50, 9], T, 2, group, dim, 64,
                                            seed=T, n=[T] * 10)
    want = [t.clone() for t in want]
    for limit in (1, 300, 1000, 3000, 10000, 30000, 1):
        prev = sv.set_wait_limit(limit)
        try:
            sv.sv_kv_attend_shared(both.g, 0, q, share, **kw)
            torch.cuda.synchronize()
        finally:
            sv.set_wait_limit(prev)
        both.g.status(clear=True)
        got = sv.sv_kv_attend_shared(both.g, 0, q, share, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), limit
        assert both.g.status() == sv.SV_OK


@needs_cuda
def test_graph_and_streams(sv):
    """Found and attended in a captured graph, replayed after forks that change the groups."""
    both, lead = grouped(sv, [(4, 700), (3, 400)], [90], [9, 60], 2, 64, 16, 3)
    g, B = both.g, both.r.batch
    share, group = sv.KVShare(g, 3, 16), i32(lead)
    q, n = queries(both, 3, 8, BF, 1), [3] * B
    nn, out = i32(n), torch.empty_like(queries(both, 3, 8, BF, 1))
    lse = torch.empty(out.shape[:3], device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
        sv.sv_kv_share(g, share, group, stream=st)
        sv.sv_kv_attend_shared(g, 0, q, share, n_new=nn, out=out, lse=lse, stream=st)
    rng = np.random.default_rng(0)
    for k in range(4):
        block(both, 3, k, n)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_attend(both, 0, q, n, got=(out, lse))
        both.same()
        both.commit([int(rng.integers(-1, 3)) for _ in range(B)], 3)
        src = [int(rng.integers(0, B)) for _ in range(B)]
        if k < 2 and all(x == 1 for x in both.fork(src)):
            group.copy_(i32(src))


@needs_cuda
def test_rounds_together(sv):
    """Rounds as a program runs them: prompts appended with rotation, forked into beams, then
    trees of drafted tokens appended with rotation, attended to over the shared pages,
    verified and committed. Against the same rounds with separate rotation, sv_kv_append and
    float64 attention on what the cache holds."""
    H, G, D, T, B = 2, 4, 64, 7, 6
    prompts, rng = [300, 0, 170, 0, 0, 33], np.random.default_rng(1)
    rope = sv.Rope(D, base=500000.0)
    a, b = (Both(sv, 2, 150, 16, H, D, B, 40) for _ in range(2))
    share = sv.KVShare(a.g, T, H * G)

    def write(n, T, par, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        qs = []
        for ly in range(2):
            qkv = torch.randn(B, T, H * (G + 2), D, generator=g, device="cuda").to(BF)
            q, k, v = qkv[:, :, :H * G], qkv[:, :, H * G:-H], qkv[:, :, -H:]
            qs.append(sv.sv_kv_append_rope(a.g, ly, k, v, rope, q=q, n_new=i32(n), parent=par))
            kr = sv.sv_rope(rope, k.float(), start=b.g.len, parent=par, n_new=i32(n))
            b.append(ly, kr, v.float(), n)
        return qs

    for c in (a, b):
        assert all(c.reserve(prompts))
    write(prompts, 300, None, 0)
    src = [0, 0, 2, 2, 0, 5]
    for c in (a, b):
        c.commit([p - 1 for p in prompts], 300)
        assert all(c.fork(src))
    sv.sv_kv_share(a.g, share, i32(src))
    ws = sv.Workspace(B, T, 512)
    for r in range(5):
        n = [T, int(rng.integers(1, T + 1)), T, 3, T, 1]
        par = [tree(rng, T) for _ in range(B)]
        for c in (a, b):
            assert all(c.reserve(n))
        qs = write(n, T, i32(par), 10 + r)
        for ly in range(2):
            got = sv.sv_kv_attend_shared(a.g, ly, qs[ly], share, n_new=i32(n), parent=i32(par),
                                         want_lse=True)
            check_attend(b, ly, qs[ly], n, par, got=got)
        tok = torch.randint(0, 512, (B, T), dtype=torch.int32, device="cuda")
        logits = torch.randn(B, T, 512, device="cuda")
        for row in range(B):  # (the walk takes some of each tree)
            for t in range(1, T):
                if rng.random() < 0.6:
                    logits[row, par[row][t], tok[row, t].long()] = 50.0 + t
        _, acc, path = sv.sv_verify_tree(logits, None, i32(par), tok, i32(n), None, 0.0, ws)
        for c in (a, b):
            c.commit(acc.tolist(), T, path.tolist())
        for f in ("table", "n_pages", "len", "refs", "k_scale", "v_scale"):
            assert torch.equal(getattr(a.g, f), getattr(b.g, f)), f
        b.same()
        if r == 2:
            src = [0, 0, 0, 2, 2, 4]
            for c in (a, b):
                assert all(c.fork(src))
            sv.sv_kv_share(a.g, share, i32(src))
    assert a.g.status() == sv.SV_OK


@needs_cuda
def test_strides_and_another_stream(sv):
    """Queries inside a fused projection, tokens of all rows side by side, and results that the
    binding allocates for another stream: the bits of the dense call."""
    both, q, n, par, share, kw, want = case(sv, [(5, 700), (20, 400)], [90], [9, 60], 9, 2, 8, 64, 16,
                                            trees=True, seed=8)
    B, T, heads, dim = q.shape
    wide = torch.empty(B, T, heads + 6, dim, dtype=BF, device="cuda")
    wide[:, :, 2:heads + 2] = q
    across = q.transpose(0, 1).contiguous().transpose(0, 1)
    for x in (wide[:, :, 2:heads + 2], across):
        got = sv.sv_kv_attend_shared(both.g, 0, x, share, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = sv.sv_kv_attend_shared(both.g, 0, q, share, stream=st, **kw)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@needs_cuda
def test_two_graphs_and_plain_calls(sv):
    """Two captured graphs of other sizes on one cache and one buffer, plain attention between
    them: each gives what it gives alone."""
    both, lead = grouped(sv, [(20, 700), (3, 400)], [90], [9, 60], 2, 64, 16, 9)
    g, B = both.g, both.r.batch
    block(both, 9, 0, [9] * B)
    share = sv.KVShare(g, 9, 16)
    sv.sv_kv_share(g, share, i32(lead))
    runs, nn = [], i32([1] * B)
    for T, n_new in ((9, None), (1, nn)):
        q = queries(both, T, 8, BF, T)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        kw = dict(n_new=n_new if n_new is not None else i32([T] * B))
        check_attend(both, 0, q, [T] * B, got=sv.sv_kv_attend_shared(g, 0, q, share, want_lse=True, **kw))
        first = sv.sv_kv_attend_shared(g, 0, q, share, want_lse=True, **kw)
        plain = sv.sv_kv_attend(g, 0, q, want_lse=True, **kw)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            sv.sv_kv_attend_shared(g, 0, q, share, out=out, lse=lse, **kw)
        runs.append((graph, q, kw, out, lse, first, plain))
    for k in (0, 1, 1, 0, 0, 1):
        graph, q, kw, out, lse, first, plain = runs[k]
        out.fill_(math.nan)
        graph.replay()
        again = sv.sv_kv_attend(g, 0, q, want_lse=True, **kw)
        torch.cuda.synchronize()
        for x, y in zip((out, lse) + tuple(again), tuple(first) + tuple(plain)):
            assert torch.equal(x, y)
    assert g.status() == sv.SV_OK


@needs_cuda
@pytest.mark.parametrize("rows,heads,group", [(4096, 1, 1), (1024, 2, 16)])
def test_largest_batches(sv, rows, heads, group):
    """All rows of the largest batch in one group, and half of them in groups of two: against
    the plain call, both within the bounds that check_attend takes (twice the smaller's)."""
    page, dim, common = 16, 32, 256
    shared, per = common // page, common // page + 1
    g = sv.KVCache(1, shared * (rows // 2 + 1) + rows, page, heads, dim, rows, per)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = 0.5 * torch.randn(g.k.shape, generator=gen, device="cuda")
    g.k.copy_(k.to(torch.float8_e4m3fn))
    g.v.copy_(torch.randn(g.v.shape, generator=gen, device="cuda").to(torch.float8_e4m3fn))
    own = torch.arange(rows, dtype=torch.int32, device="cuda")
    q = torch.randn(rows, 1, heads * group, dim, generator=gen, device="cuda").to(BF)
    share = sv.KVShare(g, 1, heads * group)
    for pairs in (False, True):
        # (Rows b and b ^ 1 are a group in the first half; all are, without pairs.)
        lead = torch.where(own < rows // 2, own // 2, own) if pairs else own * 0
        start = torch.unique(lead, return_inverse=True)[1].int()
        keep = (start < rows // 2) if pairs else (own >= 0)
        pool = start.clamp(max=rows // 2)[:, None] * shared + torch.arange(shared, device="cuda")
        g.table[:, :shared] = pool.int()
        g.table[:, shared] = shared * (rows // 2 + 1) + own
        g.n_pages.fill_(per)
        g.len.fill_(common + 5)
        g.refs.fill_(1)
        group_no = torch.where(keep, lead, -1).int() if pairs else lead
        sv.sv_kv_share(g, share, group_no)
        got = sv.sv_kv_attend_shared(g, 0, q, share, want_lse=True)
        want = sv.sv_kv_attend(g, 0, q, want_lse=True)
        # bf16 results of one sum in two orders: a step of bf16 (2^-7 of the value) and the weights'
        # bound on what the values, up to 4.5, add up to: 2^-9 each way.
        err = (got[0].float() - want[0].float()).abs()
        assert (err <= 2 ** -7 * want[0].float().abs() + 4.5 * 2 ** -8).all()
        assert ((got[1] - want[1]).abs() <= 2 ** -9).all()
    assert g.status() == sv.SV_OK


@needs_cuda
def test_binding_refusals(sv, always):
    both, lead = grouped(sv, [(3, 140)], [9], [9], 2, 64, 16, 2)
    g, B = both.g, both.r.batch
    share, q = sv.KVShare(g, 2, 8), queries(both, 2, 4, BF, 0)
    other = sv.KVCache(1, 8, 16, 2, 64, B, 4)
    for f in (lambda: sv.sv_kv_share(other, share), lambda: sv.sv_kv_share(g, share, i32([0])),
              lambda: sv.sv_kv_share(g, share, torch.zeros(B, device="cuda")),
              lambda: sv.sv_kv_share(g, share, torch.zeros(B, dtype=torch.int32)),
              lambda: sv.sv_kv_attend_shared(other, 0, q, share),
              lambda: sv.sv_kv_attend_shared(g, 0, q[:, :, :, :32], share),
              lambda: sv.sv_kv_attend_shared(g, 0, q[1:], share),
              lambda: sv.sv_kv_attend_shared(g, 0, q.cpu(), share),
              lambda: sv.sv_kv_attend_shared(g, 0, q, share, out=q.float()),
              lambda: sv.sv_kv_attend_shared(g, 0, q, share, lse=torch.empty(B, 2, 7, device="cuda")),
              lambda: sv.sv_kv_attend_shared(g, 0, q, share, n_new=i32([1])),
              lambda: sv.sv_kv_attend_shared(g, 0, q, share, parent=i32([[0]])),
              lambda: sv.KVShare(g, 2, 7), lambda: sv.KVShare(g, -1, 8)):
        with pytest.raises(ValueError):
            f()
    wide = queries(both, 2, 8, BF, 0)
    for f in (lambda: sv.sv_kv_attend_shared(g, 1, q, share),
              lambda: sv.sv_kv_attend_shared(g, 0, q.float(), share),
              lambda: sv.sv_kv_attend_shared(g, 0, wide, share),
              lambda: sv.sv_kv_attend_shared(g, 0, q, share, window=-1)):
        with pytest.raises(sv.SpecVerifyError):
            f()
    assert sv.sv_kv_attend_shared(g, 0, q[:, :0], share).shape == (B, 0, 8, 64)
    assert g.status() == sv.SV_OK


@needs_cuda
@pytest.mark.parametrize("T,heads,group,dim,page,window", [
    (150, 1, 8, 64, 16, 0), (150, 2, 3, 128, 64, 0), (131, 1, 2, 192, 32, 300), (300, 1, 1, 80, 128, 0)])
def test_prompts_behind_common_tokens(sv, T, heads, group, dim, page, window):
    """Questions of many tokens on one document: several query tiles a row, the last ones short."""
    case(sv, [(2, 700), (3, 260)], [90], [40, 3], T, heads, group, dim, page, window=window, seed=T,
         n=[T, 1, T - 1, 129, T, 7])


@needs_cuda
def test_one_row(sv):
    """The smallest batch, alone and named a group of its own."""
    for by_page in (False, True):
        case(sv, [], [300], [9], 3, 2, 4, 64, 16, seed=1, by_page=by_page, n=[3])
    case(sv, [(1, 300)], [], [9], 1, 1, 1, 16, 16, seed=2, n=[1])


@needs_cuda
@pytest.mark.parametrize("dim,window", [(32, 0), (160, 0), (64, 15000)])
def test_some_groups_gain(sv, dim, window):
    """One call in which sharing pays for one group and not for the others, in the kernel for large
    groups, beside the rows, and under a window."""
    case(sv, [(16, 20000), (2, 300), (3, 140)], [77], [3, 130, 60], 1, 8, 8, dim, 128, seed=dim,
         window=window, n=[1] * 22, rows=[0, 1, 2, 3, 7, 20, 21])
