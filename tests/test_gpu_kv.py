"""GPU parity of the key/value cache calls with the plain float64 model of kv_ref: tables,
lengths, counts and stored values exactly, attention within bounds derived below."""
import math

import numpy as np
import pytest
import torch

import kv_ref

pytestmark = pytest.mark.gpu

needs_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


class Both:
    """The same cache on the GPU and in the model, driven by the same calls. The pools start
    as NaN bytes, so anything read that was not written shows."""

    def __init__(self, sv, layers, pages, page, heads, dim, batch, max_pages):
        self.sv, a = sv, (layers, pages, page, heads, dim, batch, max_pages)
        self.g, self.r = sv.KVCache(*a), kv_ref.RefCache(*a)
        self.g.k.view(torch.uint8).fill_(0x7F)
        self.g.v.view(torch.uint8).fill_(0xFF)

    def same(self, status=0):
        g, r = self.g, self.r
        torch.cuda.synchronize()
        assert (g.table.cpu().numpy() == r.table()).all()
        assert g.n_pages.tolist() == [len(x) for x in r.rows]
        assert g.len.tolist() == list(r.len)
        assert (g.refs.cpu().numpy() == r.refs).all()
        assert g.status(clear=True) == status

    def reserve(self, n):
        ok = torch.empty(self.r.batch, dtype=torch.int32, device="cuda")
        self.sv.sv_kv_reserve(self.g, i32(n), ok)
        want = self.r.reserve(n)
        assert ok.tolist() == want
        return want

    def append(self, layer, k, v, n):
        self.sv.sv_kv_append(self.g, layer, k, v, n_new=i32(n))
        return self.r.append(layer, f64(k), f64(v), n)

    def fork(self, src):
        ok = torch.empty(self.r.batch, dtype=torch.int32, device="cuda")
        self.sv.sv_kv_fork(self.g, i32(src), ok)
        want = self.r.fork(src)
        assert ok.tolist() == want
        return want

    def commit(self, acc, N, path=None):
        self.sv.sv_kv_commit(self.g, i32(acc), N, path=None if path is None else i32(path))
        self.r.commit(acc, path)

    def same_values(self, extra=None):
        """Every live token (and `extra` new ones) of every layer, exactly."""
        r = self.r
        n = [r.len[b] + (extra[b] if extra else 0) for b in range(r.batch)]
        T = max(n + [1])
        for dt in (torch.bfloat16, torch.float32):
            out = self.sv.sv_kv_read(self.g, i32([0] * r.batch), T, count=i32(n), dtype=dt)
            for kv in range(2):
                got = f64(out[kv])
                for ly in range(r.layers):
                    for b in range(r.batch):
                        assert (got[ly, b, : n[b]] == r.values(kv, ly, b, 0, n[b])).all()
                        assert (got[ly, b, n[b]:] == 0).all()

    def fill(self, lens, seed, sigma=1.0, dtype=torch.bfloat16):
        """Rows of the given lengths, written in two parts."""
        r = self.r
        for part in (0, 1):
            n = [x // 3 if part == 0 else x - x // 3 for x in lens]
            assert all(self.reserve(n))
            for ly in range(r.layers):
                k, v = rand_kv(r, max(n + [1]), seed + 10 * ly + part, sigma, dtype)
                self.append(ly, k, v, n)
            self.commit([x - 1 for x in n], max(n + [1]))


def rand_kv(r, T, seed, sigma=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(2, r.batch, T, r.heads, r.dim, generator=g, device="cuda")
    # Tokens of very different size, so that page scales grow and shrink.
    x *= torch.exp(sigma * torch.randn(2, r.batch, T, r.heads, 1, generator=g, device="cuda"))
    return x.to(dtype)


def tree(rng, T):
    return [-1] + [int(rng.integers(max(0, n - 4), n)) for n in range(1, T)]


def walk(rng, parent, n):
    """A path of accepted nodes of a tree (None: a chain) of n nodes."""
    at, path = 0, []
    while True:
        kids = [i for i in range(1, n) if (parent[i] if parent else i - 1) == at]
        if not kids or rng.random() < 0.25:
            return path
        at = int(rng.choice(kids))
        path.append(at)


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("page,heads,dim", [(16, 1, 16), (16, 3, 80), (32, 2, 64), (64, 2, 128),
                                            (128, 1, 256)])
def test_rounds(sv, page, heads, dim, dtype):
    """Rounds of reserve, append, commit (chains and trees) and forks: everything equal to
    the model after each, values included."""
    rng = np.random.default_rng(page + dim)
    both = Both(sv, 2, 60, page, heads, dim, 5, 9)
    r = both.r
    for step in range(14):
        N = int(rng.integers(1, 20 if step % 4 else 65))
        n = [int(x) for x in rng.integers(0, N + 1, 5)]
        ok = both.reserve(n)
        n = [x if o else 0 for x, o in zip(n, ok)]
        for ly in range(2):
            k, v = rand_kv(r, N, 100 * step + ly, dtype=dtype)
            both.append(ly, k, v, n)
        both.same(0 if all(ok) else sv.SV_ERR_NO_PAGES)
        if step % 5 == 0:
            both.same_values(n)
        trees = [tree(rng, N) for _ in range(5)] if step % 2 else [None] * 5
        paths = [walk(rng, t, m) if m else [] for t, m in zip(trees, n)]
        acc = [len(p) if m else -1 for p, m in zip(paths, n)]
        full = [p + [-1] * (N - len(p)) for p in paths]
        both.commit(acc, N, full if step % 2 else None)
        both.same()
        both.same_values()
        if step % 3 == 2 or max(r.len) > 6 * page:
            ok = both.fork([int(x) for x in rng.integers(-1, 5, 5)])
            both.same(0 if all(ok) else sv.SV_ERR_NO_PAGES)
            both.same_values()


@needs_cuda
def test_reserve_when_pages_run_out(sv):
    """Rows are served in order until the free pages no longer cover one; rows that need
    nothing are served all the same; wrong rows take nothing from the others."""
    both = Both(sv, 1, 6, 16, 1, 16, 5, 4)
    assert both.reserve([16, 0, 33, 0, 16]) == [1, 1, 1, 1, 1]
    both.same()
    assert both.reserve([17, 16, 0, 0, 0]) == [1, 0, 1, 1, 1]
    both.same(sv.SV_ERR_NO_PAGES)
    assert both.reserve([0, 65, 0, 0, 0]) == [1, 0, 1, 1, 1]
    both.same(sv.SV_ERR_DEVICE_INPUT)
    assert both.reserve([0, 0, 0, -1, 0]) == [1, 1, 1, 0, 1]
    both.same(sv.SV_ERR_DEVICE_INPUT)


@needs_cuda
@pytest.mark.parametrize("pages", [4095, 4096, 4097, 70001])
def test_large_pools(sv, pages):
    """More pages than one step of the search for free ones, almost all of them taken."""
    both = Both(sv, 1, pages, 16, 1, 16, 3, 8)
    both.g.refs.fill_(1)
    both.r.refs[:] = 1
    for p in (0, pages // 2, pages - 3, pages - 2, pages - 1):
        both.g.refs[p] = 0
        both.r.refs[p] = 0
    assert both.reserve([16, 33, 1]) == [1, 1, 1]
    both.same()
    assert both.reserve([16, 33, 17]) == [1, 1, 0]
    both.same(sv.SV_ERR_NO_PAGES)


@needs_cuda
def test_large_batches(sv):
    """More rows than threads of the one-block kernels."""
    both = Both(sv, 1, 6000, 16, 1, 16, 2500, 4)
    rng = np.random.default_rng(3)
    n = [int(x) for x in rng.integers(0, 40, 2500)]
    assert all(both.reserve(n))
    k, v = rand_kv(both.r, 40, 1)
    both.append(0, k, v, n)
    both.commit([x - 1 for x in n], 40)
    both.same()
    both.fork([int(x) for x in rng.integers(-1, 2500, 2500)])
    both.same()
    both.same_values()


@needs_cuda
def test_fork_when_pages_run_out(sv):
    """A copy that finds no page holds the full pages of its source."""
    both = Both(sv, 1, 5, 16, 1, 16, 4, 4)
    both.fill([20, 16, 0, 0], 1)
    assert both.fork([0, 1, 0, 0]) == [1, 1, 1, 1]
    both.same()
    both.same_values()
    both = Both(sv, 1, 4, 16, 1, 16, 4, 4)
    both.fill([20, 16, 0, 0], 1)
    assert both.fork([0, 1, 0, 0]) == [1, 1, 1, 0]
    both.same(sv.SV_ERR_NO_PAGES)
    both.same_values()
    # A permutation, and a source out of range (keeps its row).
    g = both.g
    sv.sv_kv_fork(g, i32([1, 0, 7, 3]))
    both.r.fork([1, 0, 2, 3])
    both.same(sv.SV_ERR_DEVICE_INPUT)
    both.same_values()


@needs_cuda
def test_append_out_of_range_values(sv):
    """NaN stays NaN, infinities and values past the largest scale saturate, none of them
    sets the scale, and the status says so; another row is untouched by it."""
    both = Both(sv, 1, 4, 16, 1, 32, 2, 2)
    both.reserve([5, 5])
    k, v = rand_kv(both.r, 5, 3, dtype=torch.float32)
    k[0, 1, 0, 3], k[0, 2, 0, 4], k[0, 3, 0, 5] = math.nan, math.inf, -1e30
    assert both.append(0, k, v, [5, 5])
    both.same(sv.SV_ERR_DEVICE_INPUT)
    got = f64(sv.sv_kv_read(both.g, i32([0, 0]), 5, dtype=torch.float32)[0])[0]
    want = np.stack([both.r.values(0, 0, b, 0, 5) for b in range(2)])
    assert np.isnan(got[0, 1, 0, 3])
    got[0, 1, 0, 3] = want[0, 1, 0, 3] = 0
    assert (got == want).all()
    assert got[0, 2, 0, 4] == 448 * both.r.s[0, 0, both.r.rows[0][0], 0]
    # Zeros, the smallest scale, and the ends of the range.
    k, v = k.fill_(0.0), v.fill_(448.0 * 2.0 ** 64)
    both.reserve([1, 1])
    assert not both.append(0, k, v, [1, 1])
    both.same()
    assert float(both.g.k_scale[0, both.r.rows[0][0], 0]) == 2.0 ** -64
    assert float(both.g.v_scale[0, both.r.rows[0][0], 0]) == 2.0 ** 64


@needs_cuda
def test_append_strides_and_streams(sv):
    """Slices of a fused projection, on another stream than the one they were made on."""
    both = Both(sv, 2, 20, 32, 3, 48, 4, 4)
    qkv = torch.randn(4, 37, 10, 48, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, 2:35, 4:7], qkv[:, 2:35, 7:10]
    st = torch.cuda.Stream()
    n = [33, 1, 0, 17]
    both.reserve(n)
    st.wait_stream(torch.cuda.current_stream())
    sv.sv_kv_append(both.g, 1, k, v, n_new=i32(n), stream=st)
    st.synchronize()
    both.r.append(1, f64(k), f64(v), n)
    sv.sv_kv_append(both.g, 0, k, v, n_new=i32(n))
    both.r.append(0, f64(k), f64(v), n)
    both.same_values(n)
    both.same()


@needs_cuda
def test_rows_with_wrong_data_are_left_alone(sv):
    """Bad counts, lengths, page ids and shared pages: the row stays as it was, the others
    are served, the status reports."""
    def fresh():
        both = Both(sv, 1, 20, 16, 2, 16, 4, 4)
        both.fill([20, 20, 20, 0], 5)
        assert all(both.reserve([14, 14, 14, 0]))
        return both

    k, v = rand_kv(fresh().r, 9, 8)
    for what in ("count", "count_high", "page", "page_high", "shared", "len", "len_neg"):
        both = fresh()
        g, r = both.g, both.r
        n = [9, 9, 9, 0]
        if what == "count":
            n[1] = -2
        elif what == "count_high":
            n[1] = 10
        elif what.startswith("page"):
            g.table[1, 1] = -1 if what == "page" else 20
        elif what == "shared":
            g.refs[int(g.table[1, 1])] = 2
        else:
            g.len[1] = 60 if what == "len" else -5
        before = [t.clone() for t in (g.k, g.v, g.k_scale, g.v_scale)]
        sv.sv_kv_append(g, 0, k, v, n_new=i32(n))
        r.append(0, f64(k), f64(v), [9, 0, 9, 0])
        torch.cuda.synchronize()
        assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT, what
        mine = r.rows[1]
        for t, u in zip((g.k, g.v), before):
            assert torch.equal(t.view(torch.uint8)[:, mine], u.view(torch.uint8)[:, mine])
        # Commit with a path that moves tokens: the same rows, and bad paths.
        path = [[2, 5, 8] + [-1] * 6] * 4
        state = [t.clone() for t in (g.table, g.n_pages, g.len)]
        sv.sv_kv_commit(g, i32([3, 9 if what.startswith("count") else 3, 3, -1]), 9,
                        path=i32(path))
        r.commit([3, -1, 3, -1], path)
        torch.cuda.synchronize()
        assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT, what
        for t, u in zip((g.table, g.n_pages, g.len), state):
            assert torch.equal(t[1], u[1]), what
        for b in (0, 2, 3):
            assert g.table[b].tolist() == r.table()[b].tolist(), what
            assert int(g.len[b]) == r.len[b]
        out = sv.sv_kv_read(g, i32([0] * 4), 24, count=i32([24, 0, 24, 0]))
        for kv in range(2):
            for b in (0, 2):
                assert (f64(out[kv])[0, b] == r.values(kv, 0, b, 0, 24)).all(), what
    for path in ([2, 2, 3], [3, 2, 4], [0, 1, 2], [1, 2, 9], [1, -1, 2]):
        both = fresh()
        sv.sv_kv_append(both.g, 0, k, v, n_new=i32([9, 9, 9, 0]))
        before = [t.clone() for t in (both.g.table, both.g.len, both.g.refs)]
        bytes_ = both.g.k.view(torch.uint8).clone()
        sv.sv_kv_commit(both.g, i32([3, 0, 0, -1]), 9, path=i32([path + [-1] * 6] * 4))
        torch.cuda.synchronize()
        assert both.g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT, path
        assert torch.equal(both.g.table[0], before[0][0]) and int(both.g.len[0]) == 20
        assert torch.equal(both.g.k.view(torch.uint8), bytes_)
        assert both.g.len.tolist() == [20, 21, 21, 0]


# ---------------------------------------------------------------------------------------
# Attention. What the output may be off by, from its parts:
#  - rounding it to the output type: eps/2 |o|;
#  - a score's error d changes each weight by a factor within exp(+-d), the weighted mean by
#    at most 2 d mean|v|. d: the query is carried in at least 8 (bf16) or 11 (fp16) bits,
#    exact above 2^-18 of its largest component: scale * 2^-18 max|q| sum|k|; float32 sums
#    of dim products: scale * 2^-23 * sqrt(dim) * sum|q||k| at most for the orders used,
#    taken as 2^-19; the exponential's argument and function: 2^-20 + 2^-22 |score|;
#  - weights are carried in at least 9 bits with their own exponent: 2^-10 mean|v|, and
#    one that small underflows only below 2^-28 of the largest;
#  - the sum of float32 weights and products: 2^-20.
def bounds(o, lse, av, ab, qk, scale, dtype):
    d = scale * (2.0 ** -18 * qk + 2.0 ** -19 * ab) + 2.0 ** -20 + 2.0 ** -22 * scale * ab
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal
    return (half * np.abs(o) * 1.01 + (2 * d[..., None] + 2.0 ** -10 + 2.0 ** -19) * av * 1.01
            + tiny * half,
            d + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isinf(lse), 0, lse)))


def check_attend(both, layer, q, n, parent=None, scale=None, window=0, sinks=0, rows=None,
                 got=None):
    sv, r = both.sv, both.r
    scale = r.dim ** -0.5 if scale is None else scale
    if got is None:
        got = sv.sv_kv_attend(both.g, layer, q, n_new=i32(n),
                              parent=None if parent is None else i32(parent), scale=scale,
                              window=window, sinks=sinks, want_lse=True)
    out, lse = f64(got[0]), f64(got[1])
    for b in range(r.batch) if rows is None else rows:
        L = r.len[b]
        k = r.values(0, layer, b, 0, L + n[b])
        v = r.values(1, layer, b, 0, L + n[b])
        o, ls, av, ab, qk = kv_ref.attend(f64(q[b]), k, v, L, n[b], scale,
                                          None if parent is None else parent[b], window, sinks)
        bo, bl = bounds(o, ls, av, ab, qk, abs(scale), q.dtype)
        err = np.abs(out[b] - o)
        assert (err <= bo).all(), (b, float((err / bo).max()), np.argwhere(err > bo)[:5])
        assert (np.isinf(ls) == np.isinf(lse[b])).all() and (lse[b][np.isinf(ls)] < 0).all()
        m = ~np.isinf(ls)
        assert (np.abs(lse[b] - ls)[m] <= bl[m]).all(), float((np.abs(lse[b] - ls)[m] / bl[m]).max())


def attend_case(sv, lens, T, heads, group, dim, page, dtype, trees=False, window=0, sinks=0,
                seed=0, n_new=None, fused=False, sigma=0.5, q_sigma=1.0):
    B = len(lens)
    per = -(-(max(lens) + T) // page) + 1
    both = Both(sv, 1, B * per + 2, page, heads, dim, B, per)
    both.fill(lens, seed, sigma)
    rng = np.random.default_rng(seed)
    n = n_new or [int(x) for x in rng.integers(0, T + 1, B)]
    if n_new is None:
        n[0] = T
    assert all(both.reserve(n))
    k, v = rand_kv(both.r, T, seed + 77, sigma)
    both.append(0, k, v, n)
    par = [tree(rng, T) for _ in range(B)] if trees else None
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    q = q_sigma * torch.randn(B, T, heads * group + (2 if fused else 0), dim, generator=g,
                              device="cuda")
    q = q.to(dtype)[:, :, : heads * group]
    check_attend(both, 0, q, n, par, window=window, sinks=sinks)
    both.same()
    return both, q, n, par


ODD = [0, 1, 15, 16, 17, 127, 128, 129, 255, 300]


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,page", [(16, 16), (48, 32), (64, 64), (80, 16), (96, 128),
                                      (128, 64), (144, 32), (192, 16), (256, 128)])
@pytest.mark.parametrize("T,trees", [(1, False), (2, True), (9, False), (16, True)])
def test_attend_sizes(sv, dim, page, T, trees, dtype):
    """Head sizes, page sizes, block lengths and lengths around a tile's and a page's end;
    rows with no new token among them."""
    attend_case(sv, ODD, T, 2, 3, dim, page, dtype, trees, seed=dim + T)


@needs_cuda
@pytest.mark.parametrize("heads,group,T", [(1, 1, 1), (1, 128, 1), (1, 100, 3), (3, 8, 16),
                                           (2, 16, 9), (1, 5, 33), (4, 7, 5), (8, 4, 9),
                                           (1, 71, 2), (2, 1, 64)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_groups(sv, heads, group, T, dim):
    """Query heads per key/value head, up to more rows than one tile holds."""
    for trees in (False, True):
        attend_case(sv, [0, 130, 517], T, heads, group, dim, 32, torch.bfloat16, trees,
                    seed=group + T, fused=trees)


@needs_cuda
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (5, 3), (64, 0), (100, 1),
                                          (100, 130), (128, 4), (1000, 5), (7, 100000)])
@pytest.mark.parametrize("T,trees", [(1, False), (13, False), (16, True)])
def test_attend_window(sv, window, sinks, T, trees):
    """Sliding windows and sinks, smaller and larger than a tile and than the row."""
    attend_case(sv, ODD + [700, 1300], T, 2, 4, 64, 16, torch.bfloat16, trees, window, sinks,
                seed=window + T)


@needs_cuda
@pytest.mark.parametrize("T,lens,window,sinks", [(200, [0, 100, 3], 0, 0), (333, [129, 0], 0, 0),
                                                 (300, [500, 40], 64, 3), (257, [0, 300], 1, 0)])
@pytest.mark.parametrize("dim,group,dtype", [(128, 4, torch.bfloat16), (64, 1, torch.float16),
                                             (256, 8, torch.bfloat16)])
def test_attend_prompts(sv, T, lens, window, sinks, dim, group, dtype):
    """Prompt chunks: many tiles of queries, each with its own causal end."""
    attend_case(sv, lens, T, 1, group, dim, 64, dtype, False, window, sinks, seed=T,
                n_new=[T, T - 7, 1][: len(lens)])


@needs_cuda
@pytest.mark.parametrize("q_sigma", [0.0, 0.01, 30.0])
@pytest.mark.parametrize("sigma", [0.0, 3.0])
def test_attend_score_ranges(sv, q_sigma, sigma):
    """Flat scores (every key counts alike), and scores so far apart that one key takes all;
    tokens of sizes that differ by powers of ten between pages."""
    for dtype in (torch.bfloat16, torch.float16):
        attend_case(sv, [5, 400, 1100], 3, 2, 4, 128, 16, dtype, seed=int(q_sigma), sigma=sigma,
                    q_sigma=q_sigma)


@needs_cuda
def test_attend_scales(sv):
    """Page scales that are no powers of two and lie far apart, as another quantiser may
    write them."""
    rng = np.random.default_rng(1)
    for ex in (2, 20, 60):
        both, q, n, par = attend_case(sv, [300, 77], 4, 2, 4, 64, 32, torch.bfloat16, seed=9)
        ks = np.exp2(rng.uniform(-2, 2, both.r.s[0].shape)).astype(np.float32)
        vs = np.exp2(rng.uniform(-ex, ex, both.r.s[1].shape)).astype(np.float32)
        both.r.s[0], both.r.s[1] = ks, vs
        both.g.k_scale.copy_(torch.from_numpy(ks))
        both.g.v_scale.copy_(torch.from_numpy(vs))
        check_attend(both, 0, q * 0.05, n)
        both.same()


@needs_cuda
@pytest.mark.parametrize("lens,T,group", [([40000], 1, 8), ([25000, 1, 9000], 5, 7),
                                          ([20011], 16, 8)])
def test_attend_long(sv, lens, T, group):
    """Rows long enough to be split over many CTAs and joined; a strong first token over a
    long flat tail, whose many small weights must not be lost."""
    both, q, n, par = attend_case(sv, lens, T, 1, group, 64, 128, torch.bfloat16, seed=3,
                                  sigma=0.0, q_sigma=0.2)
    # The first token's key along the mean query: half the weight on one key.
    r, g = both.r, both.g
    p = r.rows[0][0]
    mean = q[0].float().mean((0, 1)).cpu().numpy()
    target = math.log(lens[0]) / (r.dim ** -0.5 * float(mean @ mean))
    x = kv_ref.e4m3(mean * target / r.s[0, 0, p, 0])
    r.q[0, 0, p, 0, 0] = x
    g.k[0, p, 0, 0] = torch.from_numpy(x).to(torch.float32).cuda().to(torch.float8_e4m3fn)
    check_attend(both, 0, q, n, par)


@needs_cuda
def test_attend_long_sums(sv):
    """120,000 equal keys with values 1: the weighted mean is 1, the sum the count, whatever
    the order of the additions."""
    for dtype in (torch.bfloat16, torch.float16):
        L, D = 120000, 64
        c = sv.KVCache(1, 1000, 128, 1, D, 1, 1000)
        sv.sv_kv_reserve(c, i32([L]))
        c.k.view(torch.uint8).fill_(0)
        c.v.copy_(torch.ones(1, 1, 1, 1, 1, device="cuda").expand_as(c.v))
        c.len.fill_(L - 1)
        q = torch.randn(1, 1, 4, D, device="cuda").to(dtype)
        out, lse = sv.sv_kv_attend(c, 0, q, want_lse=True)
        assert (out.double() - 1).abs().max() <= 2.0 ** -10 + torch.finfo(dtype).eps / 2
        assert (lse.double() - math.log(L)).abs().max() <= 2.0 ** -19 * math.log(L)


@needs_cuda
def test_attend_high_offsets(sv):
    """Pages past 4 GB in the pools (and past 2^31 values), bytes no test initialised
    between them."""
    page, H, D, pages = 128, 4, 128, 70000
    c = sv.KVCache(1, pages, page, H, D, 2, 8)
    assert c.k.numel() > 1 << 32
    r = kv_ref.RefCache(1, 4, page, H, D, 2, 8)
    ids = [pages - 1, 3, 35001, pages - 2]
    r.rows, r.refs[:] = [[0, 1], [2, 3]], 1
    c.table[0, :2], c.table[1, :2] = i32(ids[:2]), i32(ids[2:])
    c.n_pages.fill_(2)
    for p in ids:
        c.refs[p] = 1
    both = Both.__new__(Both)
    both.sv, both.g, both.r = sv, c, r
    k, v = rand_kv(r, 200, 4)
    both.append(0, k, v, [200, 130])
    q = torch.randn(2, 200, 8, D, device="cuda").to(torch.bfloat16)
    check_attend(both, 0, q, [200, 130])
    both.commit([149, 129], 200)
    assert c.len.tolist() == [150, 130]
    both.same_values()
    assert c.status() == 0


@needs_cuda
@pytest.mark.parametrize("what", ["page", "page_high", "len", "len_neg", "count", "count_high",
                                  "parent", "parent_self"])
def test_attend_wrong_data(sv, what):
    """A wrong row becomes NaN and is reported; the others are as without it."""
    both, q, n, par = attend_case(sv, [300, 200, 100], 9, 2, 4, 64, 32, torch.bfloat16, True,
                                  seed=2, n_new=[9, 9, 8])
    g = both.g
    n = list(n)
    if what.startswith("page"):
        g.table[1, 3] = -1 if what == "page" else g.refs.numel()
    elif what.startswith("len"):
        g.len[1] = 10 ** 6 if what == "len" else -1
    elif what.startswith("count"):
        n[1] = -1 if what == "count" else 10
    else:
        par[1][4] = -1 if what == "parent" else 4
    got = sv.sv_kv_attend(g, 0, q, n_new=i32(n), parent=i32(par), want_lse=True)
    torch.cuda.synchronize()
    assert g.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
    assert torch.isnan(got[0][1]).all() and torch.isnan(got[1][1]).all()
    check_attend(both, 0, q, n, par, rows=[0, 2], got=got)


@needs_cuda
def test_attend_graph_and_streams(sv):
    """Captured once, replayed with other lengths, counts and values in the same buffers, and
    the same bits each time; on another stream than the inputs'."""
    both, q, n, _ = attend_case(sv, [300, 4000, 100, 0], 5, 2, 4, 128, 64, torch.bfloat16, seed=4)
    g, st = both.g, torch.cuda.Stream()
    nn = i32(n)
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        sv.sv_kv_attend(g, 0, q, n_new=nn, out=out, lse=lse, stream=st)
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            sv.sv_kv_attend(g, 0, q, n_new=nn, out=out, lse=lse, stream=st)
    first = None
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert first is None or torch.equal(first, out)
        first = out.clone()
    check_attend(both, 0, q, n, got=(out, lse))
    # Fewer tokens and other queries.
    both.commit([n[0] - 1, -1, 1, n[3] - 1], 5)
    n2 = [0, 2, 1, 0]
    both.reserve(n2)
    k, v = rand_kv(both.r, 5, 1234)
    both.append(0, k, v, n2)
    nn.copy_(i32(n2))
    q.copy_(torch.randn(q.shape, device="cuda"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check_attend(both, 0, q, n2, got=(out, lse))
    both.same()


@needs_cuda
def test_round_in_a_graph(sv):
    """A whole round (reserve, append, attend, commit, fork) captured and replayed: the same
    as the calls made one by one."""
    lens, T = [40, 7, 100], 6
    states = []
    for captured in (False, True):
        both = Both(sv, 1, 60, 16, 2, 32, 3, 12)
        both.fill(lens, 11)
        g = both.g
        k, v = rand_kv(both.r, T, 2)
        q = torch.randn(3, T, 4, 32, device="cuda").to(torch.bfloat16)
        torch.manual_seed(0)
        n, acc = i32([6, 3, 0]), i32([2, 1, -1])
        path = i32([[2, 4, -1, -1, -1, -1], [2, -1, -1, -1, -1, -1], [-1] * 6])
        src = i32([0, 0, 2])
        out = torch.empty_like(q)
        st = torch.cuda.Stream()

        def call():
            sv.sv_kv_reserve(g, n, stream=st)
            sv.sv_kv_append(g, 0, k, v, n_new=n, stream=st)
            sv.sv_kv_attend(g, 0, q, n_new=n, out=out, stream=st)
            sv.sv_kv_commit(g, acc, T, path=path, stream=st)
            sv.sv_kv_fork(g, src, stream=st)

        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            if captured:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=st):
                    call()
                graph.replay()
                graph.replay()
            else:
                call()
                call()
        torch.cuda.synchronize()
        assert g.status() == 0
        kr, vr = sv.sv_kv_read(g, i32([0, 0, 0]), 120, count=g.len)
        states.append([t.clone() for t in (g.table, g.n_pages, g.len, g.refs, kr, vr)])
    for a, b in zip(*states):
        assert torch.equal(a, b)


@needs_cuda
def test_binding_refusals(sv):
    """Shapes, dtypes and layouts that the binding rejects before any call."""
    c = sv.KVCache(1, 4, 16, 2, 32, 2, 2)
    q = torch.zeros(2, 3, 4, 32, device="cuda", dtype=torch.bfloat16)
    k = q[:, :, :2]
    good = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sv.KVCache(1, 4, 24, 2, 32, 2, 2)
    for bad in (q[:1], q[..., :16], q.transpose(1, 2), q.cpu()):
        with pytest.raises(ValueError):
            sv.sv_kv_attend(c, 0, bad)
    with pytest.raises(ValueError):
        sv.sv_kv_attend(c, 0, q.to(torch.float64))
    with pytest.raises(sv.SpecVerifyError):
        sv.sv_kv_attend(c, 0, q.float())
    with pytest.raises(sv.SpecVerifyError):
        sv.sv_kv_attend(c, 1, q)
    with pytest.raises(sv.SpecVerifyError):
        sv.sv_kv_attend(c, 0, q[:, :, :3])
    with pytest.raises(ValueError):
        sv.sv_kv_attend(c, 0, q, parent=torch.zeros(2, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        sv.sv_kv_append(c, 0, q, q)
    with pytest.raises(ValueError):
        sv.sv_kv_append(c, 0, k, k.float())
    for n in (good.long(), good[:1], good.cpu()):
        with pytest.raises(ValueError):
            sv.sv_kv_append(c, 0, k, k, n_new=n)
        with pytest.raises(ValueError):
            sv.sv_kv_reserve(c, n)
        with pytest.raises(ValueError):
            sv.sv_kv_fork(c, n)
    with pytest.raises(ValueError):
        sv.sv_kv_commit(c, good, 3, path=torch.zeros(2, 4, dtype=torch.int32, device="cuda"))


@needs_cuda
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("trees,window,sinks,dim,T,lens,at", [
    (False, 0, 0, 64, 9, [130, 300], 134),    # among the new tokens: later queries see it
    (True, 0, 0, 128, 16, [120, 300], 125),   # a node: its descendants
    (False, 40, 0, 128, 20, [250, 300], 222),  # leaves the window during the block
    (False, 40, 3, 192, 20, [250, 300], 4),   # between the sinks and the window
    (False, 40, 3, 64, 20, [250, 300], 2),    # a sink
    (False, 0, 0, 64, 40, [140, 10], 60),     # a tile that every query sees
])
def test_attend_stored_nan(sv, what, trees, window, sinks, dim, T, lens, at):
    """A NaN in the cache reaches the queries that see it and no other."""
    both, q, n, par = attend_case(sv, lens, T, 2, 2, dim, 32, torch.bfloat16, trees, window, sinks,
                                  seed=at, n_new=[T, T])
    g, r = both.g, both.r
    pool = g.k if what == "k" else g.v
    pool.view(torch.uint8)[0, int(g.table[0, at // 32]), 1, at % 32, 5] = 0x7F
    got = sv.sv_kv_attend(g, 0, q, n_new=i32(n), parent=None if par is None else i32(par),
                          window=window, sinks=sinks, want_lse=True)
    out, lse = f64(got[0]), f64(got[1])
    L = r.len[0]
    o, ls, av, ab, qk = kv_ref.attend(f64(q[0]), r.values(0, 0, 0, 0, L + T),
                                      r.values(1, 0, 0, 0, L + T), L, T, dim ** -0.5,
                                      None if par is None else par[0], window, sinks)
    bo, bl = bounds(o, ls, av, ab, qk, dim ** -0.5, q.dtype)
    for t in range(T):
        sees = kv_ref.visible(L, T, t, None if par is None else par[0], window, sinks)[at]
        clean = slice(0, 2) if sees else slice(0, 4)
        if sees:
            assert np.isnan(out[0, t, 2:, 5]).all(), t
            assert what == "v" or np.isnan(lse[0, t, 2:]).all(), t
        assert (np.abs(out[0, t, clean] - o[t, clean]) <= bo[t, clean]).all(), t
        assert (np.abs(lse[0, t, clean] - ls[t, clean]) <= bl[t, clean]).all(), t
    check_attend(both, 0, q, n, par, window=window, sinks=sinks, rows=[1], got=got)


@needs_cuda
def test_attend_without_lse(sv):
    """The log sum left out, output the same bits; whole query tiles and joined ones."""
    for lens in ([50, 7], [30000, 5]):
        both, q, n, _ = attend_case(sv, lens, 3, 2, 4, 64, 64, torch.float16, seed=8, n_new=[3, 2])
        a = sv.sv_kv_attend(both.g, 0, q, n_new=i32(n))
        b, _ = sv.sv_kv_attend(both.g, 0, q, n_new=i32(n), want_lse=True)
        a = a[0] if isinstance(a, tuple) else a
        assert torch.equal(a, b)


@needs_cuda
def test_calls_back_to_back(sv):
    """Rounds on one stream without a pause, each call reading what the one before it wrote:
    the same as with a synchronisation after every call."""
    states = []
    for paused in (False, True):
        both = Both(sv, 1, 80, 16, 2, 64, 4, 18)
        both.fill([40, 0, 33, 100], 21)
        g = both.g
        xs = [rand_kv(both.r, 6, 300 + i) for i in range(12)]
        n, acc = i32([6, 5, 6, 2]), i32([2, 1, 3, 0])
        path = i32([[2, 4] + [-1] * 4, [3] + [-1] * 5, [1, 3, 5] + [-1] * 3, [-1] * 6])
        src = i32([0, 2, 2, 3])
        outs = []
        gap = torch.cuda.synchronize if paused else (lambda: None)
        torch.cuda.synchronize()
        for i, (k, v) in enumerate(xs):
            for call in (lambda: sv.sv_kv_reserve(g, n), lambda: sv.sv_kv_append(g, 0, k, v, n_new=n),
                         lambda: outs.append(sv.sv_kv_attend(g, 0, k, n_new=n, want_lse=True)),
                         lambda: sv.sv_kv_commit(g, acc, 6, path=path),
                         lambda: sv.sv_kv_fork(g, src) if i % 4 == 3 else None,
                         lambda: outs.append(sv.sv_kv_read(g, i32([0] * 4), 120, count=g.len))):
                gap()
                call()
        torch.cuda.synchronize()
        assert g.status() == 0
        states.append([t.clone() for t in (g.table, g.n_pages, g.len, g.refs)] +
                      [t for o in outs for t in o])
    for a, b in zip(*states):
        assert torch.equal(a, b)


@needs_cuda
@pytest.mark.parametrize("B,T,heads,group,window", [(700, 2, 1, 2, 0), (1500, 1, 2, 1, 5),
                                                    (1, 2600, 1, 40, 0), (2, 900, 1, 128, 300)])
def test_attend_many_query_tiles(sv, B, T, heads, group, window):
    """More query tiles than a CTA has threads, one or many to a row, rows without any among
    them."""
    rng = np.random.default_rng(B + T)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    n = [int(x) for x in rng.integers(0, T + 1, B)] if B > 2 else [T] * B
    both = Both(sv, 1, B * (-(-(40 + T) // 16) + 1), 16, heads, 16, B, -(-(40 + T) // 16) + 1)
    both.fill(lens, 3)
    assert all(both.reserve(n))
    k, v = rand_kv(both.r, T, 9)
    both.append(0, k, v, n)
    q = torch.randn(B, T, heads * group, 16, device="cuda").to(torch.bfloat16)
    check_attend(both, 0, q, n, window=window,
                 rows=sorted({0, B - 1, *(int(x) for x in rng.integers(0, B, 60))}))
    both.same()
