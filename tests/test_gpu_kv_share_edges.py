"""GPU tests of attention over shared pages where its calls, groups and rows meet: launches of
several kinds on one buffer, groups of very different sizes, and rows that no longer hold what
they shared."""
import pytest
import torch

from test_gpu_kv import check_attend, i32, needs_cuda
from test_gpu_kv_shared import BF, block, grouped, queries, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture
def always(sv):  # noqa: F811
    """Every group's common tokens are read once."""
    prev = sv.set_share_always(True)
    yield
    sv.set_share_always(prev)


def flags(share, batch):
    """The words by which CTAs of one launch tell those of the next what they have waited for."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    at = 256 + up(16 * batch) + up(16 * (batch // 2 + 1)) + 2 * up(4 * batch)
    return share.t[at: at + 640].view(torch.int32)


@needs_cuda
def test_flags_between_launches(sv, always):  # noqa: F811
    """Calls with and without a launch for large groups, in turn on one buffer, in a graph too: each
    flag that one launch leaves is taken by the next."""
    both, lead = grouped(sv, [(20, 700), (3, 400)], [90], [9, 60], 2, 64, 16, 9)
    g, B = both.g, both.r.batch
    block(both, 9, 0, [9] * B)
    share, alone = sv.KVShare(g, 9, 16), sv.KVShare(g, 9, 16)
    sv.sv_kv_share(g, share, i32(lead))
    calls = []
    for T, s, window in ((9, share, 0), (1, share, 0), (9, alone, 0), (9, share, 30), (1, alone, 0)):
        q = queries(both, T, 8, BF, T)
        calls.append((q, s, dict(n_new=i32([T] * B), window=window, want_lse=True), T, window))
    seen = set()
    for k in (0, 0, 1, 2, 3, 0, 4, 3, 1, 1):
        q, s, kw, T, window = calls[k]
        got = sv.sv_kv_attend_shared(g, 0, q, s, **kw)
        assert not flags(s, B).any()
        if k not in seen:
            check_attend(both, 0, q, [T] * B, window=window, got=got)
        seen.add(k)
    q, s, kw, T, window = calls[0]
    want = sv.sv_kv_attend_shared(g, 0, q, s, **kw)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    kw = dict(kw, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            sv.sv_kv_attend_shared(g, 0, q, s, **kw)
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert not flags(s, B).any()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and g.status() == sv.SV_OK


@needs_cuda
def test_groups_of_very_different_sizes(sv, always):  # noqa: F811
    """One group of 2,048 rows beside 1,024 of two, with as many queries as the call takes: groups
    times the largest one's query tiles pass 2^31. Rows of each kind against float64."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 95 GB of device memory")
    rows, T, heads, dim, page = 4096, 1024, 128, 16, 128
    g = sv.KVCache(1, 1025 + 8, page, 1, dim, rows, 2)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for pool in (g.k, g.v):
        pool.copy_(torch.randn(pool.shape, generator=gen, device="cuda").to(torch.float8_e4m3fn))
    own = torch.arange(rows, dtype=torch.int32, device="cuda")
    number = torch.where(own < 2048, 0, own // 2 - 1023).int()  # 0, then 1 .. 1024
    live = {0: 3, 2047: 1, 2048: 2, 3071: T, 4094: 5, 4095: 4}
    n_new = torch.zeros(rows, dtype=torch.int32, device="cuda")
    g.table[:, 0], g.table[:, 1] = number, -1
    g.n_pages.fill_(1)
    g.len.fill_(page)
    g.refs.fill_(1)
    for i, (b, n) in enumerate(live.items()):  # (a row of T tokens has room for 128)
        n_new[b] = live[b] = min(n, 128)
        g.table[b, 1], g.n_pages[b] = 1025 + i, 2
    q = torch.randn(1, T, heads, dim, generator=gen, device="cuda").to(BF).expand(rows, -1, -1, -1)
    share = sv.KVShare(g, T, heads)
    sv.sv_kv_share(g, share, number)
    got = sv.sv_kv_attend_shared(g, 0, q, share, n_new=n_new)
    assert g.status() == sv.SV_OK
    for b, n in live.items():
        k, v = (torch.cat([x[0, p, 0] for p in g.table[b].tolist()]).double() for x in (g.k, g.v))
        for t in range(n):
            seen = page + t + 1
            w = torch.softmax(q[b, t].double() @ k[:seen].T * dim ** -0.5, -1)
            want, size = w @ v[:seen], w @ v[:seen].abs()
            # Half a step of bf16, weights off by 2^-11 of themselves or 2^-28 of the largest, and a
            # margin of as much for the scores' and sums' float32.
            err = (got[b, t].double() - want).abs()
            assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * size + 2.0 ** -27 * seen).all()
    del got, share
    torch.cuda.empty_cache()


@needs_cuda
@pytest.mark.parametrize("dim,window", [(32, 0), (160, 0), (32, 300)])
def test_one_large_group_beside_many_small(sv, always, dim, window):  # noqa: F811
    """Groups whose query tiles are found by number, in each kernel that takes groups, against the
    plain call: bf16 results of one sum in two orders, a step of bf16 (2^-7 of the value) and the
    weights' bound on what the values, up to 4.5, add up to, 2^-9 each way."""
    rows, T, group, page, common = 600 + 2 * 150, 3, 8, 16, 256
    shared, per = common // page, common // page + 1
    g = sv.KVCache(1, shared * 151 + rows, page, 1, dim, rows, per)
    gen = torch.Generator(device="cuda").manual_seed(1)
    g.k.copy_((0.5 * torch.randn(g.k.shape, generator=gen, device="cuda")).to(torch.float8_e4m3fn))
    g.v.copy_(torch.randn(g.v.shape, generator=gen, device="cuda").to(torch.float8_e4m3fn))
    own = torch.arange(rows, dtype=torch.int32, device="cuda")
    number = torch.where(own % 3 == 0, own // 6 + 1, 0).int()  # pairs between the others
    g.table[:, :shared] = (number[:, None] * shared + torch.arange(shared, device="cuda")).int()
    g.table[:, shared] = shared * 151 + own
    g.n_pages.fill_(per)
    g.len.copy_(common + own % 10)
    g.refs.fill_(1)
    q = torch.randn(rows, T, group, dim, generator=gen, device="cuda").to(BF)
    n_new = (1 + own % 3).int()
    kw = dict(n_new=n_new, window=window, sinks=5, want_lse=True)
    share = sv.KVShare(g, T, group)
    sv.sv_kv_share(g, share, number)
    got = sv.sv_kv_attend_shared(g, 0, q, share, **kw)
    want = sv.sv_kv_attend(g, 0, q, **kw)
    err = (got[0].float() - want[0].float()).abs()
    assert (err <= 2 ** -7 * want[0].float().abs() + 4.5 * 2 ** -8).all()
    new = torch.arange(T, device="cuda") < n_new[:, None]
    assert ((got[1] - want[1])[new].abs() <= 2 ** -9).all() and (got[1][~new] == want[1][~new]).all()
    assert g.status() == sv.SV_OK


@needs_cuda
@pytest.mark.parametrize("which", ["first", "last"])
@pytest.mark.parametrize("what", ["table", "len", "n_pages", "freed", "longer prompt", "shorter prompt"])
def test_rows_that_change(sv, always, what, which):  # noqa: F811
    """Any row of a group may change, its lowest too: that row is NaN, and the others, which still
    hold the group's pages, are right."""
    T, groups, tails = 6, [(5, 2000), (3, 400), (2, 2600)], [20, 60]
    both, lead = grouped(sv, groups, [90], tails, 2, 64, 16, T)
    g, B = both.g, both.r.batch
    share = sv.KVShare(g, T, 8)
    sv.sv_kv_share(g, share, i32(lead))
    size = {x: lead.count(x) for x in lead}
    mine = next(x for x in lead if size[x] == 5)
    bad = mine if which == "first" else max(b for b in range(B) if lead[b] == mine)
    other = next(x for x in lead if size[x] == (2 if what == "longer prompt" else 3))
    if what in ("freed", "longer prompt", "shorter prompt"):
        src = list(range(B))
        src[bad] = -1 if what == "freed" else other
        assert all(both.fork(src))
    n = [T] * B
    n[bad] = 0 if what == "freed" else T
    block(both, T, 3, n)
    if what == "table":
        g.table[bad, 3] = int(g.table[bad, 126])
    if what == "len":
        g.len[bad] = 30
    if what == "n_pages":
        g.n_pages[bad] = 2
    q = queries(both, T, 4, BF, 8)
    for _ in range(2):
        out, lse = sv.sv_kv_attend_shared(g, 0, q, share, n_new=i32(n), want_lse=True)
        assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
        assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
        check_attend(both, 0, q, n, got=(out, lse), rows=[b for b in range(B) if b != bad])


@needs_cuda
@pytest.mark.parametrize("T,group,live", [(6, 4, 2), (6, 4, 0), (40, 8, 30), (40, 8, 0), (3, 2, 3)])
def test_changed_rows_are_nan_throughout(sv, always, T, group, live):  # noqa: F811
    """A row that changed is NaN in all tokens, new or not, like rows with other wrong data; in calls
    that attend to its group one by one it has its own results."""
    both, lead = grouped(sv, [(5, 2000), (3, 400)], [90], [20, 60], 2, 64, 16, T)
    g, B = both.g, both.r.batch
    share = sv.KVShare(g, T, 2 * group)
    sv.sv_kv_share(g, share, i32(lead))
    bad = max(b for b in range(B) if lead.count(lead[b]) == 5)
    n = [max(1, T - b) for b in range(B)]
    n[bad] = live
    block(both, T, 3, n)
    other = int(g.table[bad, 126])
    old = int(g.table[bad, 3])
    q = queries(both, T, group, BF, 8)
    kw = dict(n_new=i32(n), want_lse=True)
    g.table[bad, 3] = other
    out, lse = sv.sv_kv_attend_shared(g, 0, q, share, **kw)
    assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    check_attend(both, 0, q, n, got=(out, lse), rows=[b for b in range(B) if b != bad])
    g.table[bad, 3] = old
    out, lse = sv.sv_kv_attend_shared(g, 0, q, share, **kw)
    assert torch.isnan(out[bad].float()).all() and torch.isnan(lse[bad]).all()
    # (Numbers of their own: the call reads nobody's tokens once.)
    fresh = sv.KVShare(g, T, 2 * group)
    check_attend(both, 0, q, n, got=sv.sv_kv_attend_shared(g, 0, q, fresh, **kw))
    sv.sv_kv_share(g, share, i32(lead))
    check_attend(both, 0, q, n, got=sv.sv_kv_attend_shared(g, 0, q, share, **kw))
    assert g.status() == sv.SV_OK


@needs_cuda
@pytest.mark.parametrize("groups,T,heads,group,dim,window,once", [
    ([(16, 20000), (2, 300), (3, 140)], 1, 8, 8, 128, 0, [True, False, False]),  # large groups' kernel
    ([(16, 20000), (2, 300)], 1, 8, 8, 160, 0, [True, False]),                   # beside the rows
    ([(4, 20000)], 1, 8, 1, 128, 0, [True]),                                     # a narrow one
    ([(4, 2000)], 1, 1, 1, 128, 0, [False]),           # gains less than a second kind of work costs
    ([(2, 2000), (3, 1500)], 16, 2, 8, 128, 0, [False, False]),  # rows that fill their products
    ([(16, 20000)], 1, 8, 8, 64, 15000, [True]),       # a window that reaches most
    ([(16, 20000)], 1, 8, 8, 64, 200, [False])])       # and one that reaches three tiles
def test_which_groups_are_read_once(sv, groups, T, heads, group, dim, window, once):  # noqa: F811
    """What the rule decides, by groups that clearly gain or lose. Another page in a row's common
    tokens shows it: the row is NaN where they are read once, and has results of its own else."""
    both, lead = grouped(sv, groups, [77], [30, 130], heads, dim, 128, T)
    g, B = both.g, both.r.batch
    block(both, T, 1, [T] * B)
    share, q = sv.KVShare(g, T, heads * group), queries(both, T, group, BF, 1)
    sv.sv_kv_share(g, share, i32(lead))
    kw = dict(window=window, sinks=3 if window else 0)
    before = sv.sv_kv_attend_shared(g, 0, q, share, **kw)
    assert g.status() == sv.SV_OK and torch.isfinite(before.float()).all()
    sizes = [m for m, _ in groups]  # (no two alike)
    changed = [max(b for b in range(B) if lead.count(lead[b]) == m and lead[b] != b) for m in sizes]
    full = int(g.table[changed[0], 1])  # (of the longest group: pages are NaN past what was written)
    for b in changed:
        g.table[b, 0] = full
    out = sv.sv_kv_attend_shared(g, 0, q, share, **kw)
    assert g.status() == (sv.SV_ERR_DEVICE_INPUT if any(once) else sv.SV_OK)
    nan = torch.isnan(out.float()).flatten(1)
    assert [bool(nan[b].all()) for b in changed] == once
    assert not nan[[b for b, x in zip(changed, once) if not x]].any()
    rest = [b for b in range(B) if b not in changed]
    assert torch.equal(out[rest], before[rest])
