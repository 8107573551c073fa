"""GPU parity of the rotary calls with their formula in float64.

Error bound of a rotated component, relative to its pair's length times the gain: the angle is off
by at most pi (2^-25 + 2^-31) (its cut to float32 half turns), cosine and sine by 2 units of 2^-24
(twice the function's documented 1), their product with the gain by 2^-24, and the two products
and their sum by 2^-24 each: less than 14 * 2^-25 in all, below 2^-21. On top of it half a step of
the result's type."""
import math

import numpy as np
import pytest
import torch

import kv_ref

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int64).astype(np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def turned(x, pos, freqs, rot, inter, gain=1.0, sign=1.0):
    """x [B, T, H, D] float64 at positions pos [B, T]; also each component's pair length."""
    # (Angles modulo a turn in extended precision: far positions.)
    ang = np.asarray(pos, dtype=np.longdouble)[..., None] * np.asarray(freqs, dtype=np.longdouble)
    ang = np.mod(ang, 2 * np.longdouble(math.pi) + np.longdouble(2.4492935982947064e-16))
    c, s = np.cos(ang).astype(np.float64)[:, :, None], np.sin(ang).astype(np.float64)[:, :, None]
    y, size = x.copy(), np.zeros_like(x)
    ia = np.arange(rot // 2) * 2 if inter else np.arange(rot // 2)
    ib = ia + (1 if inter else rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = gain * (a * c - sign * b * s), gain * (b * c + sign * a * s)
    size[..., ia] = size[..., ib] = abs(gain) * np.hypot(a, b)
    return y, size


def near(got, y, size, dtype):
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # a subnormal's whole step
    assert (np.abs(got - y) <= size * 2.0 ** -21 + np.abs(y) * half * (1 + 2.0 ** -20) + tiny).all()


def plain_freqs(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def rand(shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def depths(parent):
    d = []
    for t, p in enumerate(parent):
        d.append(0 if t == 0 else d[p] + 1)
    return d


def tree(rng, T):
    return [-1] + [int(rng.integers(max(0, n - 4), n)) for n in range(1, T)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 40), (64, 20), (192, 48), (96, 2), (256, 256),
                                     (16, 16), (512, 30), (112, 104)])
@pytest.mark.parametrize("B,T,heads,how", [(1, 1, 1, "new"), (3, 7, 5, "in place"),
                                           (2, 300, 9, "slice")])
def test_rope(sv, dtype, inter, dim, rot, B, T, heads, how):
    """Both layouts, all or part of a head, dense, in place and sliced, ragged rows."""
    rope = sv.Rope(rot, interleaved=inter, gain=1.25)
    full = rand((B, T, heads + (2 if how == "slice" else 0), dim), B + T + dim, dtype)
    x = full[:, :, 1:-1] if how == "slice" else full
    before, xs = full.clone(), f64(x)
    n = [T] + [max(0, T - 3 * b) for b in range(1, B)]
    start = [5 + 1000 * b for b in range(B)]
    out = sv.sv_rope(rope, x, start=i32(start), n_new=i32(n), out=x if how == "in place" else None)
    assert rope.status() == sv.SV_OK
    pos = np.asarray(start)[:, None] + np.arange(T)
    y, size = turned(xs, pos, plain_freqs(rot), rot, inter, 1.25)
    got = f64(out)
    for b in range(B):
        near(got[b, :n[b]], y[b, :n[b]], size[b, :n[b]], dtype)
        assert (got[b, :n[b], :, rot:] == xs[b, :n[b], :, rot:]).all()
        assert (got[b, n[b]:] == (xs[b, n[b]:] if how == "in place" else 0.0)).all()
    if how != "in place":
        assert torch.equal(full, before)


@pytest.mark.parametrize("at", [0, 1, 131071, 1 << 24, (1 << 24) + 1, 2 ** 31 - 3, -1, -70000,
                                -2 ** 31])
def test_far_positions(sv, at):
    """Angles of far and negative positions are as exact as near ones'."""
    rope = sv.Rope(64, base=500000.0)
    x = rand((1, 2, 3, 64), 1, F32)
    y, size = turned(f64(x), [[at, at + 1]], plain_freqs(64, 500000.0), 64, False)
    # (The table's frequencies are off by 2^-55 of themselves and the model's by 2^-54; at
    # position 2^31 that is 2^-22 radians.)
    slack = size * abs(at) * 2.0 ** -53
    for kw in (dict(pos=i32([[at, at + 1]])), dict(start=i32([at]))):
        got = f64(sv.sv_rope(rope, x, **kw))
        assert (np.abs(got - y) <= size * 2.0 ** -21 + slack + np.abs(y) * 2.0 ** -24 * 1.001).all()


@pytest.mark.parametrize("scaling", ["none", "linear", "turns", "index"])
def test_stretched(sv, scaling):
    """The frequencies of each kind of stretching reach the kernel, and given angles do."""
    kw = dict(base=500000.0, scaling=scaling, stretch=8.0, original=8192.0, low=1.0, high=4.0)
    rope = sv.Rope(128, **kw)
    f = [x % 2 ** 64 / 2.0 ** 64 * 2 * math.pi for x in rope.freq.tolist()]
    x = rand((2, 5, 2, 128), 2, F32)
    y, size = turned(f64(x), [[90000 + i for i in range(5)]] * 2, f, 128, False)
    got = sv.sv_rope(rope, x, start=i32([90000, 90000]))
    near(f64(got), y, size, F32)
    assert torch.equal(got, sv.sv_rope(sv.Rope(128, angles=f), x, start=i32([90000, 90000])))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_trees(sv, dtype):
    """Positions are depths; a wrong link or count makes the row NaN and is reported."""
    rng, T, B = np.random.default_rng(3), 33, 6
    par = [tree(rng, T) for _ in range(B)]
    n = [33, 1, 0, 20, 33, 7]
    rope, x = sv.Rope(64), rand((B, T, 4, 64), 4, dtype)
    start = [100 * b for b in range(B)]
    pos = [[s + d for d in depths(p)] for s, p in zip(start, par)]
    y, size = turned(f64(x), pos, plain_freqs(64), 64, False)
    out = sv.sv_rope(rope, x, start=i32(start), parent=i32(par), n_new=i32(n))
    for b in range(B):
        near(f64(out)[b, :n[b]], y[b, :n[b]], size[b, :n[b]], dtype)
        assert (out[b, n[b]:] == 0).all()
    assert rope.status() == sv.SV_OK
    bad = [list(p) for p in par]
    bad[0][5], bad[3][21], bad[4][32], bad[5][6] = 5, 99, -1, 2 ** 31 - 1  # (row 3: past its 20)
    counts = list(n)
    counts[1], counts[2] = -1, T + 1
    for same in (False, True):
        z = x.clone()
        out = sv.sv_rope(rope, z, start=i32(start), parent=i32(bad), n_new=i32(counts),
                         out=z if same else None)
        for b in (0, 1, 2, 4, 5):
            assert torch.isnan(out[b].float()).all()
        near(f64(out)[3, :20], y[3, :20], size[3, :20], dtype)
        assert rope.status(clear=True) == sv.SV_ERR_DEVICE_INPUT


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(sv, inter):
    """The inverse rotation is the gradient: of the formula, and of differences. Sums of n
    products of values off by 2^-21: their error is below 2^-20 times the sum of sizes."""
    rope = sv.Rope(40, interleaved=inter, gain=1.5)
    x, g = rand((2, 9, 3, 80), 5, F32), rand((2, 9, 3, 80), 6, F32)
    start = i32([3, 7000])
    y, dx = sv.sv_rope(rope, x, start=start), sv.sv_rope(rope, g, start=start, inverse=True)
    a, b = (f64(y) * f64(g)).sum(), (f64(x) * f64(dx)).sum()
    size = 1.5 * (np.abs(f64(x)).sum() + np.abs(f64(g)).sum()) * 4
    assert abs(a - b) <= size * 2.0 ** -20
    pos = np.array([[3 + t for t in range(9)], [7000 + t for t in range(9)]])
    want, s = turned(f64(g), pos, plain_freqs(40), 40, inter, 1.5, -1.0)
    near(f64(dx), want, s, F32)
    # Differences: the map is linear, so (y(x + e) - y(x)) / e is exact but for rounding.
    rng = np.random.default_rng(0)
    for _ in range(8):
        at = tuple(int(rng.integers(k)) for k in x.shape)
        e = x.clone()
        e[at] += 1.0
        step = float(e[at] - x[at])
        d = (f64(sv.sv_rope(rope, e, start=start)) - f64(y)) / step
        err = 2.0 ** -20 * 1.5 * 8  # two rotations of components below 8 in size
        assert abs((d * f64(g)).sum() - f64(dx)[at]) <= err * np.abs(f64(g)[at[0], at[1], at[2]]).sum()


def test_nonfinite_stays_in_its_pair(sv):
    """A NaN or infinity reaches its own pair only."""
    rope = sv.Rope(32)
    x = rand((1, 4, 2, 64), 7, BF)
    clean = sv.sv_rope(rope, x)
    x[0, 1, 0, 3], x[0, 2, 1, 40], x[0, 3, 1, 60] = math.nan, math.inf, -math.inf
    y = sv.sv_rope(rope, x)
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[0, 1, 0, 3] = keep[0, 1, 0, 19] = keep[0, 2, 1, 40] = keep[0, 3, 1, 60] = False
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[0, 1, 0, [3, 19]]).all()
    assert y[0, 2, 1, 40] == math.inf and y[0, 3, 1, 60] == -math.inf


def test_large(sv):
    """Offsets past 2^31 bytes, more tokens than threads, a batch of one-token rows."""
    rope = sv.Rope(128)
    x = torch.empty(3, 65535, 48, 128, dtype=BF, device="cuda")
    x[:] = rand((1, 1, 48, 128), 8, BF)
    sv.sv_rope(rope, x, start=i32([0, 7, 65535]), out=x)
    for b, t in ((0, 0), (0, 65534), (1, 40000), (2, 65534)):
        y, size = turned(f64(rand((1, 1, 48, 128), 8, BF)), [[[0, 7, 65535][b] + t]],
                         plain_freqs(128), 128, False)
        near(f64(x[b:b + 1, t:t + 1]), y, size, BF)
    x = rand((4096, 1, 1, 16), 9, HF)
    y, size = turned(f64(x), np.arange(4096)[:, None], plain_freqs(16), 16, False)
    near(f64(sv.sv_rope(sv.Rope(16), x, start=i32(range(4096)))), y, size, HF)


def test_rope_strides_streams_and_graph(sv):
    """Tokens of all rows side by side, another stream, and a captured call with new data."""
    rope = sv.Rope(64)
    base = rand((6, 3, 2, 64), 10, BF)
    x = base.transpose(0, 1)  # [3 rows, 6 tokens], tokens further apart than rows
    want = sv.sv_rope(rope, x.contiguous(), start=i32([1, 2, 3]))
    out = torch.zeros_like(base).transpose(0, 1)
    assert torch.equal(sv.sv_rope(rope, x, start=i32([1, 2, 3]), out=out), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    st = i32([1, 2, 3])
    torch.cuda.synchronize()
    other = sv.sv_rope(rope, x, start=st, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    st, y = i32([1, 2, 3]), torch.empty_like(want)
    xs = x.contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.sv_rope(rope, xs, start=st, out=y)
    for k in range(3):
        xs.copy_(rand(xs.shape, 20 + k, BF))
        st.fill_(50 * k)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, sv.sv_rope(rope, xs, start=i32([50 * k] * 3)))


# ------------------------------------------------------------------ appending
def caches(sv, n, layers=1, pages=80, page=16, heads=2, dim=64, batch=3, max_pages=20):
    return [sv.KVCache(layers, pages, page, heads, dim, batch, max_pages) for _ in range(n)]


def same_bytes(a, b):
    for f in ("table", "n_pages", "len", "refs"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f
    held = (a.refs > 0).nonzero().flatten()
    for f in ("k", "v"):
        assert torch.equal(getattr(a, f).view(torch.uint8)[:, held],
                           getattr(b, f).view(torch.uint8)[:, held]), f
        assert torch.equal(getattr(a, f + "_scale")[:, held], getattr(b, f + "_scale")[:, held]), f


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("page,heads,dim,rot,inter", [
    (16, 1, 16, 16, False), (32, 3, 80, 40, True), (64, 2, 128, 128, False), (128, 2, 256, 256, True),
    (16, 5, 64, 20, False), (64, 8, 96, 6, True), (128, 1, 192, 48, False)])
@pytest.mark.parametrize("T,trees", [(1, False), (9, True), (150, False)])
def test_append_rope(sv, dtype, page, heads, dim, rot, inter, T, trees):
    """Every byte and scale as rotating to float32 and appending that, over rounds that grow the
    same pages; queries as rotated alone."""
    rng = np.random.default_rng(T + dim)
    B, G, rounds = 3, 3, 4
    most = -(-(rounds * T + 40) // page) + 1
    a, b = (sv.KVCache(2, 3 * most + 2, page, heads, dim, B, most) for _ in range(2))
    for c in (a, b):
        c.k.view(torch.uint8).fill_(0)
        c.v.view(torch.uint8).fill_(0)
    rope = sv.Rope(rot, interleaved=inter, gain=0.75)
    for r in range(rounds):
        n = [T, max(0, T - 2 * r), 1]
        par = i32([tree(rng, T) for _ in range(B)]) if trees else None
        qkv = rand((B, T, heads * (G + 2), dim), 100 * r + T, dtype)
        qkv *= math.exp(r - 1.0)
        q, k, v = qkv[:, :, :heads * G], qkv[:, :, heads * G:-heads], qkv[:, :, -heads:]
        for c in (a, b):
            sv.sv_kv_reserve(c, i32(n))
        for ly in range(2):
            got = sv.sv_kv_append_rope(a, ly, k, v, rope, q=q, n_new=i32(n), parent=par)
            kr = sv.sv_rope(rope, k.float(), start=b.len, parent=par, n_new=i32(n))
            sv.sv_kv_append(b, ly, kr, v.float(), n_new=i32(n))
        assert torch.equal(got, sv.sv_rope(rope, q, start=b.len, parent=par, n_new=i32(n)))
        same_bytes(a, b)
        for c in (a, b):
            sv.sv_kv_commit(c, i32([x - 1 for x in n]), max(T, 1))
    assert a.status() == sv.SV_OK and b.status() == sv.SV_OK


def test_append_rope_formula(sv):
    """Stored keys against the formula: half a step of e4m3 (2^-4 of the value, or 2^-10 of the
    scale), the rotation's 2^-21, and 2^-8 for bf16's copy on the way out."""
    (c,) = caches(sv, 1, page=64, heads=4, dim=128, batch=2, pages=40)
    rope = sv.Rope(128, base=500000.0)
    k, v = rand((2, 200, 4, 128), 1, BF), rand((2, 200, 4, 128), 2, BF)
    sv.sv_kv_reserve(c, i32([200, 200]))
    sv.sv_kv_append_rope(c, 0, k, v, rope)
    y, size = turned(f64(k), [list(range(200))] * 2, plain_freqs(128, 500000.0), 128, False)
    got, _ = sv.sv_kv_read(c, i32([0, 0]), 200, dtype=F32)
    for b in range(2):
        for j in range(4):
            lo, hi = 64 * j, min(200, 64 * j + 64)
            scale = f64(c.k_scale[0, int(c.table[b, j])])
            for h in range(4):
                yy, ss = y[b, lo:hi, h], size[b, lo:hi, h]
                assert scale[h] == kv_ref.scale_for(np.abs(yy).max())  # (not next to a border)
                step = np.maximum(2.0 ** -4 * np.abs(yy), 2.0 ** -10 * scale[h])
                assert (np.abs(f64(got)[0, b, lo:hi, h] - yy) <= step * (1 + 2.0 ** -20)
                        + ss * 2.0 ** -21).all()


@pytest.mark.parametrize("what", ["page", "page_high", "shared", "count", "count_high", "len",
                                  "tree", "tree_high", "pages"])
def test_append_rope_leaves_wrong_rows_alone(sv, what):
    """A row with wrong data keeps its bytes; the others' are written."""
    a, b = caches(sv, 2)
    rng, T = np.random.default_rng(1), 9
    par = [tree(rng, T) for _ in range(3)]
    n = [9, 9, 9]
    rope, k, v = sv.Rope(64), rand((3, T, 2, 64), 1, BF), rand((3, T, 2, 64), 2, BF)
    q = rand((3, T, 4, 64), 3, BF)
    for c in (a, b):
        c.k.view(torch.uint8).fill_(0)
        c.v.view(torch.uint8).fill_(0)
        sv.sv_kv_reserve(c, i32([30, 30, 30]))
        sv.sv_kv_append(c, 0, rand((3, 21, 2, 64), 4, BF), rand((3, 21, 2, 64), 5, BF))
        sv.sv_kv_commit(c, i32([20, 20, 20]), 21)
        sv.sv_kv_reserve(c, i32([9, 9, 9]))
    page = int(a.table[1, 1])
    for c in (a, b):
        if what == "page":
            c.table[1, 1] = -1
        elif what == "page_high":
            c.table[1, 1] = 1 << 20
        elif what == "shared":
            c.refs[page] = 2
        elif what == "len":
            c.len[1] = -1
        elif what == "pages":
            c.n_pages[1] = 1
    if what == "count":
        n[1] = -1
    if what == "count_high":
        n[1] = T + 1
    if what == "tree":
        par[1][4] = 4
    if what == "tree_high":
        par[1][8] = 2 ** 30
    out = sv.sv_kv_append_rope(a, 0, k, v, rope, q=q, n_new=i32(n), parent=i32(par))
    good = [9, 0, 9]
    good_par = [p if i != 1 else tree(np.random.default_rng(0), T) for i, p in enumerate(par)]
    want = sv.sv_kv_append_rope(b, 0, k, v, rope, q=q, n_new=i32(good), parent=i32(good_par))
    same_bytes(a, b)
    assert torch.equal(out[[0, 2]], want[[0, 2]])
    if what in ("count", "count_high", "len", "tree", "tree_high"):
        assert torch.isnan(out[1].float()).all()
    assert a.status(clear=True) == sv.SV_ERR_DEVICE_INPUT


def test_append_rope_odd_values(sv):
    """NaN and infinite components do not count towards the scale, are stored as NaN or
    saturated, and are reported; another quantiser's scale is kept."""
    a, b = caches(sv, 2)
    rope, v = sv.Rope(64), rand((3, 5, 2, 64), 2, BF)
    k = rand((3, 5, 2, 64), 1, BF)
    k[0, 1, 0, 5], k[1, 2, 1, 9], k[2, 0, 0, 0] = math.nan, math.inf, -math.inf
    for c in (a, b):
        c.k.view(torch.uint8).fill_(0)
        c.v.view(torch.uint8).fill_(0)
        sv.sv_kv_reserve(c, i32([5, 5, 5]))
    sv.sv_kv_append_rope(a, 0, k, v, rope)
    sv.sv_kv_append(b, 0, sv.sv_rope(rope, k.float()), v.float())
    same_bytes(a, b)
    assert a.status(clear=True) == b.status(clear=True) == sv.SV_ERR_DEVICE_INPUT
    # Pages with older tokens at a scale of 0.3, then new tokens that fit, and that do not.
    for c in (a, b):
        sv.sv_kv_commit(c, i32([4, 4, 4]), 5)
        c.k_scale.fill_(0.3)
        c.v_scale.fill_(0.3)
    for size in (0.01, 400.0):
        x = rand((3, 6, 2, 64), 3, BF) * size
        for c in (a, b):
            sv.sv_kv_reserve(c, i32([6, 6, 6]))
        sv.sv_kv_append_rope(a, 0, x, x, rope)
        sv.sv_kv_append(b, 0, sv.sv_rope(rope, x.float(), start=b.len), x.float())
        same_bytes(a, b)
        for c in (a, b):
            sv.sv_kv_commit(c, i32([5, 5, 5]), 6)


def test_append_rope_long_row(sv):
    """More pages than a block checks itself, and the same with a page that is not the row's."""
    a, b = (sv.KVCache(1, 620, 16, 2, 64, 2, 310) for _ in range(2))
    rope, T = sv.Rope(64), 4801
    k, v = rand((2, T, 2, 64), 1, BF), rand((2, T, 2, 64), 2, BF)
    for c in (a, b):
        c.k.view(torch.uint8).fill_(0)
        c.v.view(torch.uint8).fill_(0)
        sv.sv_kv_reserve(c, i32([T, T]))
    for shared in (False, True):
        for c in (a, b):
            if shared:
                c.refs[c.table[1, 300].long()] = 2
        sv.sv_kv_append_rope(a, 0, k, v, rope)
        sv.sv_kv_append(b, 0, sv.sv_rope(rope, k.float()), v.float())
        same_bytes(a, b)
        want = sv.SV_ERR_DEVICE_INPUT if shared else sv.SV_OK
        assert a.status(clear=True) == b.status(clear=True) == want
        k, v = -k, -v


def test_append_rope_without_queries_and_in_place(sv):
    a, b = caches(sv, 2)
    rope = sv.Rope(64)
    k, v, q = rand((3, 7, 2, 64), 1, BF), rand((3, 7, 2, 64), 2, BF), rand((3, 7, 6, 64), 3, BF)
    for c in (a, b):
        c.k.view(torch.uint8).fill_(0)
        c.v.view(torch.uint8).fill_(0)
        sv.sv_kv_reserve(c, i32([7, 7, 7]))
    want = sv.sv_kv_append_rope(a, 0, k, v, rope, q=q)
    assert sv.sv_kv_append_rope(b, 0, k, v, rope) is None
    same_bytes(a, b)
    n = i32([7, 2, 0])
    before = q.clone()
    assert sv.sv_kv_append_rope(b, 0, k, v, rope, q=q, q_out=q, n_new=n) is q
    for i, m in enumerate((7, 2, 0)):
        assert torch.equal(q[i, :m], want[i, :m]) and torch.equal(q[i, m:], before[i, m:])


def test_binding_refusals(sv):
    (c,) = caches(sv, 1)
    rope, big = sv.Rope(64), sv.Rope(128)
    k = rand((3, 7, 2, 64), 1, BF)
    q = rand((3, 7, 6, 64), 1, BF)
    bad = [
        lambda: sv.sv_rope(rope, k.cpu()), lambda: sv.sv_rope(rope, k[0]),
        lambda: sv.sv_rope(rope, k.transpose(2, 3)), lambda: sv.sv_rope(rope, k.to(torch.int32)),
        lambda: sv.sv_rope(rope, k, pos=i32([0])), lambda: sv.sv_rope(rope, k, start=i32([0])),
        lambda: sv.sv_rope(rope, k, start=torch.zeros(3, device="cuda")),
        lambda: sv.sv_rope(rope, k, parent=i32([[0] * 7])), lambda: sv.sv_rope(rope, k, out=q),
        lambda: sv.sv_rope(rope, k, out=k.float()), lambda: sv.sv_rope(rope, k, n_new=i32([1, 2])),
        lambda: sv.sv_kv_append_rope(c, 0, k, k.float(), rope),
        lambda: sv.sv_kv_append_rope(c, 0, k, k[:, :3], rope),
        lambda: sv.sv_kv_append_rope(c, 0, k, k, rope, q=q[:, :3]),
        lambda: sv.sv_kv_append_rope(c, 0, k, k, rope, q=q.float()),
        lambda: sv.sv_kv_append_rope(c, 0, k, k, rope, q_out=q),
        lambda: sv.sv_kv_append_rope(c, 0, k, k, rope, q=q, q_out=k),
        lambda: sv.sv_kv_append_rope(c, 0, k, k, rope, parent=i32([[0] * 7]))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: sv.sv_rope(big, k), lambda: sv.sv_kv_append_rope(c, 0, k, k, big),
              lambda: sv.sv_kv_append_rope(c, 1, k, k, rope),
              lambda: sv.sv_rope(rope, k, pos=i32([[0] * 7] * 3), start=i32([0, 0, 0]))):
        with pytest.raises(sv.SpecVerifyError):
            f()
    assert sv.sv_rope(rope, k[:, :0]).shape == (3, 0, 2, 64)
    assert sv.sv_rope(rope, k[:0]).shape == (0, 7, 2, 64)


@pytest.mark.parametrize("T", [1, 17, 1300])
def test_append_rope_many_heads(sv, T):
    """More heads than a block takes, with few blocks and with many; older tokens whose scale
    grows, or stays, head by head."""
    B, H = 8, 70
    a, b = (sv.KVCache(1, B * 85, 16, H, 16, B, 85) for _ in range(2))
    for c in (a, b):  # (bytes that no call writes are compared too)
        c.k.view(torch.uint8).fill_(0)
        c.v.view(torch.uint8).fill_(0)
    rope = sv.Rope(16)
    size = torch.exp2(torch.arange(H, device="cuda") % 7 - 3.0)[None, None, :, None]
    for r, n in enumerate((5, T, 3)):
        for c in (a, b):
            sv.sv_kv_reserve(c, i32([n] * B))
        k, v = rand((B, n, H, 16), r, F32) * size, rand((B, n, H, 16), r + 9, F32) / size
        sv.sv_kv_append_rope(a, 0, k, v, rope)
        sv.sv_kv_append(b, 0, sv.sv_rope(rope, k, start=b.len), v)
        same_bytes(a, b)
        for c in (a, b):
            sv.sv_kv_commit(c, i32([n - 1] * B), n)
        size = size.flip(2)
    assert a.status() == sv.SV_OK


@pytest.mark.parametrize("old", [0.3, 2.0 ** -20, 2.0 ** 60, 2.0 ** 126, 2.0 ** 127])
@pytest.mark.parametrize("page,dim", [(16, 16), (64, 128), (128, 256)])
def test_append_rope_other_scales(sv, old, page, dim):
    """Pages whose older tokens have another quantiser's scale, in some heads, with new tokens that
    fit a block's registers, and that do not."""
    a, b = caches(sv, 2, page=page, heads=3, dim=dim, pages=12, max_pages=4)
    rope = sv.Rope(dim, interleaved=True)
    for c in (a, b):
        c.k.view(torch.uint8).fill_(0x31)
        c.v.view(torch.uint8).fill_(0x31)
        sv.sv_kv_reserve(c, i32([5, 0, 1]))
        c.k_scale[:, :, 1] = old
        c.v_scale[:, :, 0] = old
        c.v_scale[:, :, 2] = old
        sv.sv_kv_commit(c, i32([4, -1, 0]), 5)
    n = page + 7
    for c in (a, b):
        sv.sv_kv_reserve(c, i32([n] * 3))
    k, v = rand((3, n, 3, dim), 1, BF), rand((3, n, 3, dim), 2, BF) * 900.0
    sv.sv_kv_append_rope(a, 0, k, v, rope)
    sv.sv_kv_append(b, 0, sv.sv_rope(rope, k.float(), start=b.len), v.float())
    same_bytes(a, b)
    assert a.status() == b.status()
