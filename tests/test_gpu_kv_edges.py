"""The key/value cache calls on wrong device data, at the ends of their ranges and on streams
and devices other than their own."""
import pytest
import torch

from test_gpu_kv import Both, attend_case, i32, needs_cuda, rand_kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


@needs_cuda
@pytest.mark.parametrize("row", [0, 1, 3])
@pytest.mark.parametrize("held", [-1, -2, -7, -2 ** 31, 5, 2 ** 31 - 1])
def test_reserve_with_wrong_page_counts(sv, row, held):
    """A row whose n_pages is outside [0, max_pages] gets nothing, takes no page from the
    others, and nothing outside the other rows' entries is written."""
    both = Both(sv, 1, 12, 16, 1, 16, 4, 4)
    both.reserve([20, 5, 33, 1])
    both.same()
    g = both.g
    before = g.table.clone()
    guard = torch.full((64 + g.table.numel(),), -7, dtype=torch.int32, device="cuda")
    guard[32: 32 + g.table.numel()] = g.table.flatten()
    g.c.table = guard[32:].data_ptr()  # the same table with entries of nobody around it
    good = int(g.n_pages[row])
    g.n_pages[row] = held
    n = [40, 40, 40, 40]
    ok = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    sv.sv_kv_reserve(g, i32(n), ok)
    torch.cuda.synchronize()
    assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
    n[row] = 0
    want = both.r.reserve(n)
    want[row] = 0
    assert ok.tolist() == want
    assert int(g.n_pages[row]) == held
    g.n_pages[row] = good
    table = guard[32: 32 + g.table.numel()].view_as(before)
    assert (table.cpu().numpy() == both.r.table()).all()
    assert (guard[:32] == -7).all() and (guard[32 + g.table.numel():] == -7).all()
    assert g.n_pages.tolist() == [len(x) for x in both.r.rows]
    assert (g.refs.cpu().numpy() == both.r.refs).all()


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("T,group", [(1, 1), (1, 31), (3, 11), (9, 4), (1, 63), (5, 13), (9, 8),
                                     (1, 97), (1, 127), (3, 43)])
def test_attend_part_filled_warps(sv, T, group, dim, dtype):
    """Query rows that fill a warp's lanes in part, in results that one CTA writes whole and in
    such that are joined: every row's result is its own, and the lanes without a row write
    nothing (the queries past a row's count are zeros)."""
    attend_case(sv, [40, 9000], T, 1, group, dim, 64, dtype, seed=T + group, n_new=[T, T])
    attend_case(sv, [9000, 40], T, 1, group, dim, 64, dtype, seed=T + group, n_new=[T, T - 1])


@needs_cuda
@pytest.mark.parametrize("dim,T,group,lens", [(128, 1, 8, [9000, 300]), (64, 9, 4, [20000, 17]),
                                              (128, 16, 8, [3000, 9000]), (256, 40, 4, [700, 5000])])
def test_attend_gives_up(sv, dim, T, group, lens):
    """Waits with a bound that they pass, at the first of them or later: the call ends, says
    SV_ERR_TIMEOUT, and the next call on the same workspace has the bits it had before."""
    both, q, n, _ = attend_case(sv, lens, T, 2, group, dim, 64, torch.bfloat16, seed=T,
                                n_new=[T, T])
    g = both.g
    want = [t.clone() for t in sv.sv_kv_attend(g, 0, q, n_new=i32(n), want_lse=True)]
    torch.cuda.synchronize()
    for limit in (1, 300, 1000, 3000, 10000, 30000, 1):
        prev = sv.set_wait_limit(limit)
        try:
            sv.sv_kv_attend(g, 0, q, n_new=i32(n))
            torch.cuda.synchronize()
        finally:
            sv.set_wait_limit(prev)
        assert g.status() in ((sv.SV_ERR_TIMEOUT,) if limit == 1 else (sv.SV_OK, sv.SV_ERR_TIMEOUT))
        got = sv.sv_kv_attend(g, 0, q, n_new=i32(n), want_lse=True)
        torch.cuda.synchronize()
        g.status(clear=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), limit


@needs_cuda
@pytest.mark.parametrize("call", ["attend", "read"])
def test_results_of_a_call_on_another_stream(sv, call):
    """Results that the binding allocates for a call on a stream of its own, dropped before the
    call has run: the current stream gets other memory meanwhile."""
    both, q, n, _ = attend_case(sv, [40, 3], 2, 2, 4, 64, 16, torch.bfloat16, seed=1, n_new=[2, 2])
    st, start = torch.cuda.Stream(), i32([0, 0])
    n = i32(n)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    if call == "attend":
        made = sv.sv_kv_attend(both.g, 0, q, n_new=n, want_lse=True, stream=st)
    else:
        made = sv.sv_kv_read(both.g, start, 40, stream=st)
    kinds = [(t.shape, t.dtype, t.data_ptr()) for t in made]
    del made
    again = [torch.empty(s, dtype=d, device="cuda") for s, d, _ in kinds for _ in range(2)]
    assert not st.query()  # (the call has not run yet)
    assert not {t.data_ptr() for t in again} & {p for _, _, p in kinds}
    torch.cuda.synchronize()
    # On the current stream nothing is held back.
    made = sv.sv_kv_read(both.g, start, 40, stream=torch.cuda.current_stream())
    at = made[0].data_ptr()
    del made
    assert torch.empty(1, 2, 40, 2, 64, dtype=torch.bfloat16, device="cuda").data_ptr() == at


@needs_cuda
@pytest.mark.parametrize("T,group", [(1, 4), (3, 8)])
def test_attend_two_rows_of_a_large_batch(sv, T, group):
    """Two rows with new tokens, next to each other and at the ends of 4,096, with a CTA that goes
    from the one to the other: the same results, and rows without any cost next to nothing."""
    B, H, D, lens = sv.SV_MAX_B, 8, 16, [19999, 19990]
    gen = torch.Generator(device="cuda").manual_seed(5)
    kv = torch.randn(2, 1, 20000 + T, H, D, generator=gen, device="cuda").bfloat16()
    kv = kv.expand(2, B, 20000 + T, H, D)  # (every row's source is the same: no stride)
    live = torch.randn(2, T, H * group, D, generator=gen, device="cuda").bfloat16()
    times, results = [], []
    for at in ((0, 1), (0, B - 1), (7, B - 33)):
        c = sv.KVCache(1, 640, 64, H, D, B, 320)
        n0, n = [0] * B, [0] * B
        for b, x in zip(at, lens):
            n0[b], n[b] = x, T
        sv.sv_kv_reserve(c, i32(n0))
        sv.sv_kv_append(c, 0, kv[0, :, :20000], kv[1, :, :20000], n_new=i32(n0))
        sv.sv_kv_commit(c, i32([x - 1 for x in n0]), 20000)
        sv.sv_kv_reserve(c, i32(n))
        sv.sv_kv_append(c, 0, kv[0, :, 20000:], kv[1, :, 20000:], n_new=i32(n))
        q = torch.zeros(B, T, H * group, D, device="cuda", dtype=torch.bfloat16)
        q[list(at)] = live
        nn, out = i32(n), torch.empty_like(q)
        best = []
        for _ in range(30):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                sv.sv_kv_attend(c, 0, q, n_new=nn, out=out)
            b.record()
            b.synchronize()
            best.append(a.elapsed_time(b) * 1e3 / 4)
        times.append(min(best))
        results.append(out[list(at)].clone())
        assert c.status() == 0
        out[list(at)] = 0
        assert (out == 0).all()
    print(f"us a call: {times}")
    assert results[0].abs().max() > 0
    assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])
    assert max(times) < 1.5 * times[0] + 10, times


@needs_cuda
@pytest.mark.parametrize("what", ["", "page", "page_high", "shared", "count", "count_high", "len"])
def test_append_long_rows_with_wrong_data(sv, what):
    """Rows of several hundred pages, one of them wrong at its far end: left as it was, and the
    others (rows without new tokens among them) served."""
    T, page, B = 5000, 16, 4
    both = Both(sv, 1, 960, page, 1, 16, B, 320)
    g, r = both.g, both.r
    n = [T, 4500, 0, 3]
    assert all(both.reserve([3, 9, 5, 0]))
    k, v = rand_kv(r, T, 3)
    both.append(0, k, v, [3, 9, 5, 0])
    both.commit([2, 8, 4, -1], T)
    assert all(both.reserve(n))
    bad = list(n)
    last = (9 + 4500 - 1) // page
    if what.startswith("page"):
        g.table[1, last] = -1 if what == "page" else 960
    elif what == "shared":
        g.refs[int(g.table[1, last])] = 2
    elif what.startswith("count"):
        bad[1] = -1 if what == "count" else T + 1
    elif what == "len":
        g.len[1] = 320 * page - 4499
    mine = r.rows[1]
    before = [t.view(torch.uint8)[:, mine].clone() for t in (g.k, g.v)]
    sv.sv_kv_append(g, 0, k, v, n_new=i32(bad))
    torch.cuda.synchronize()
    assert g.status(clear=True) == (sv.SV_ERR_DEVICE_INPUT if what else sv.SV_OK)
    if what:
        n[1] = 0
        for t, u in zip((g.k, g.v), before):
            assert torch.equal(t.view(torch.uint8)[:, mine], u)
    r.append(0, k.double().cpu().numpy(), v.double().cpu().numpy(), n)
    rows = [b for b in range(B) if b != 1 or not what]
    total = [r.len[b] + n[b] for b in range(B)]
    out = sv.sv_kv_read(g, i32([0] * B), max(total), count=i32(total), dtype=torch.float32)
    for kv in range(2):
        for b in rows:
            assert (out[kv][0, b, : total[b]].double().cpu().numpy()
                    == r.values(kv, 0, b, 0, total[b])).all()


@needs_cuda
def test_append_time_grows_with_the_tokens(sv):
    """Four times the tokens on the smallest pages: about four times the time."""
    times = []
    for T in (16384, 65535):
        c = sv.KVCache(1, T // 16 + 1, 16, 8, 128, 1, T // 16 + 1)
        k = torch.randn(1, T, 8, 128, device="cuda").bfloat16()
        sv.sv_kv_reserve(c, i32([T]))
        best = []
        for _ in range(20):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(3):
                sv.sv_kv_append(c, 0, k, k)
            b.record()
            b.synchronize()
            best.append(a.elapsed_time(b))
        times.append(min(best))
        assert c.status() == 0
    assert times[1] < 5 * times[0], times


@needs_cuda
@pytest.mark.parametrize("with_path", [False, True])
@pytest.mark.parametrize("accepted", [-1, 0, 2])
@pytest.mark.parametrize("what,value", [("n_pages", -5), ("n_pages", -2 ** 31), ("n_pages", 5),
                                        ("n_pages", 2 ** 31 - 1), ("n_pages", 1), ("len", 33),
                                        ("len", 2 ** 31 - 1), ("len", -1)])
def test_commit_with_wrong_counts(sv, what, value, accepted, with_path):
    """A row whose n_pages or len cannot be (33 tokens on two pages of 16): reported and left as
    it was, whether tokens are kept or not; the others are served."""
    both = Both(sv, 1, 20, 16, 1, 16, 3, 4)
    both.fill([20, 20, 20], 5)
    assert all(both.reserve([4, 4, 4]))
    k, v = rand_kv(both.r, 4, 8)
    both.append(0, k, v, [4, 4, 4])
    g, r = both.g, both.r
    getattr(g, what)[1] = value
    state = [t.clone() for t in (g.table, g.n_pages, g.len)]
    path = [[2, 3, -1, -1]] * 3 if with_path else None
    sv.sv_kv_commit(g, i32([1, accepted, 0]), 4, path=None if path is None else i32(path))
    torch.cuda.synchronize()
    assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
    for t, u in zip((g.table, g.n_pages, g.len), state):
        assert torch.equal(t[1], u[1])
    r.commit([1, -1, 0], path)
    assert g.len.tolist()[::2] == r.len[::2]
    assert (g.table.cpu().numpy()[::2] == r.table()[::2]).all()
    # (the wrong row's pages are the ones it had)
    refs = g.refs.cpu().numpy()
    assert all(refs[p] == 1 for b in range(3) for p in r.rows[b])


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_more_layers_than_a_grid_has(sv, dtype):
    """A small cache of 70,000 layers, read at once and from a layer on."""
    L, D = 70000, 16
    c = sv.KVCache(L, 2, 16, 1, D, 1, 2)
    c.table[0] = i32([1, 0])
    c.n_pages.fill_(2)
    c.len.fill_(20)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for pool in (c.k, c.v):
        pool.copy_(torch.randint(-8, 9, pool.shape, generator=gen, device="cuda").float())
    c.k_scale.copy_(2.0 ** torch.randint(-3, 4, c.k_scale.shape, generator=gen, device="cuda"))
    for first in (0, 3000):
        k, v = sv.sv_kv_read(c, i32([14]), 4, layer=first, dtype=dtype)
        pos = [(1, 14), (1, 15), (0, 0), (0, 1)]
        for got, pool, scale in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
            for t, (p, i) in enumerate(pos):
                want = pool[first:, p, 0, i].float() * scale[first:, p, 0][:, None]
                assert torch.equal(got[:, 0, t, 0].float(), want)
    assert c.status() == 0
