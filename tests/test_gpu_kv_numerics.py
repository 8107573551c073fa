"""What the cache attention's numbers may be off by, on inputs where each part of that shows:
weights, queries, keys of very different size, and scales of another quantiser."""

import numpy as np
import pytest
import torch

import kv_ref
from test_gpu_kv import Both, f64, i32, needs_cuda, rand_kv, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


# A weight: fp16's rounding, 2^-11 of itself, and the end of its terms, 2^-28 of the row's
# largest weight times value scale. A query's result: the weighted mean over keys of that, its
# float32 sums (2^-19), and rounding to the output's type.
W_REL, W_ABS, SUM = 2.0 ** -11, 2.0 ** -28, 2.0 ** -19


# A query component: exact, or this much of the row's largest.
Q_ABS = {torch.bfloat16: 2.0 ** -21, torch.float16: 2.0 ** -24}


def per_key(q, k, v, L, n, scale, dtype, vs=None, **mask):
    """One row: the result in float64 (o [n, q_heads, dim], lse) and what a call's may be off by,
    vs [tokens, heads] being the scales of the values (None: all the same), from an error of its
    own for each key's score:
      d_j = scale (Q_ABS max|q| sum|k_j| + 2^-19 sum|q k_j|)     query terms, float32 sums
            + 2^-20 + 2^-20 max|s|        the power; a score, the reference and its moves as
                                          float32 numbers: 16 roundings of 2^-24
    With weights w'_j = w_j e^(e_j), |e_j| <= d_j, the result moves by
    sum w_j (e^(e_j) - 1)(v_j - o) / sum w'_j. A weight times its value's scale is off by W_ABS of
    the largest such product, its value by that many times its code v_j / vs_j."""
    vs = np.ones(k.shape[:2]) if vs is None else vs
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, bo = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, bl = np.zeros((n, Hq)), np.zeros((n, Hq))
    for t in range(n):
        see = kv_ref.visible(L, n, t, **mask)
        for h in range(Hq):
            kk, vv, u, x = k[see, h // G], v[see, h // G], vs[see, h // G], q[t, h]
            s = kk @ x * scale
            m = s.max()
            w = np.exp(s - m)
            w /= w.sum()
            d = abs(scale) * (Q_ABS[dtype] * np.abs(x).max() * np.abs(kk).sum(1)
                              + 2.0 ** -19 * (np.abs(kk) @ np.abs(x)))
            d += 2.0 ** -20 + 2.0 ** -20 * np.abs(s).max()
            o[t, h] = w @ vv
            lse[t, h] = np.log(np.exp(s - m).sum()) + m
            move = (w * np.expm1(d)) @ np.abs(vv - o[t, h]) / (w @ np.exp(-d))
            bo[t, h] = (torch.finfo(dtype).eps / 2 * (np.abs(o[t, h]) + move) + move
                        + (W_REL + SUM) * (w @ np.abs(vv))
                        + W_ABS * (w * u).max() * (np.abs(vv) / u[:, None]).sum(0)
                        + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps)
            bl[t, h] = np.log(w @ np.exp(d)) + SUM + 2.0 ** -22 * abs(lse[t, h])
    return o, lse, bo * 1.01, bl * 1.01


def store(both, k, v):
    """One row's cache made of k, v [tokens, heads, dim] (numbers that e4m3 holds at the scales
    that append gives them)."""
    n = k.shape[0]
    assert all(both.reserve([n]))
    x = [torch.from_numpy(y[None]).cuda().float() for y in (k, v)]
    both.append(0, x[0], x[1], [n])
    for kv, y in enumerate((k, v)):
        assert (both.r.values(kv, 0, 0, 0, n) == y).all(), "inputs must be exact in the cache"


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,group", [(2, 8), (8, 7), (16, 8), (60, 16)])
def test_weights(sv, T, group, dtype):
    """Keys of weight 1 between keys that share a weight below it, with values of opposite sign:
    where they nearly cancel, what the shared weight is off by is all that is left. (The weight
    at the row's reference is a power of two and has no rounding.)"""
    L, D = 200, 64
    both = Both(sv, 1, 8, 64, 1, D, 1, 8)
    k, v = np.zeros((L + T, 1, D)), np.ones((L + T, 1, D))
    k[1::2, 0, 0] = 1.0
    v[::2, 0] = -np.ldexp(1 + np.arange(D) % 8 / 8, np.arange(D) // 8 - 8)  # 2^-8 .. 1.875
    store(both, k, v)
    both.commit([L - 1], L)
    assert all(both.reserve([T]))
    rng = np.random.default_rng(T)
    q = torch.zeros(1, T, group, D)
    q[..., 0] = torch.from_numpy(-rng.uniform(0.5, 5.0, (1, T, group)))
    q = q.to(dtype).cuda()
    out = f64(sv.sv_kv_attend(both.g, 0, q, n_new=i32([T]), scale=1.0))[0]
    o, _, av, ab, _ = kv_ref.attend(f64(q[0]), k, v, L, T, 1.0)
    _, _, weak, _, _ = kv_ref.attend(f64(q[0]), k, v * k[:, :, :1], L, T, 1.0)
    # Scores are exact (one product); the power's argument and the power, 2^-20 + 2^-22 |score|.
    d = 2.0 ** -20 + 2.0 ** -22 * ab
    bound = (torch.finfo(dtype).eps / 2 * np.abs(o) + W_REL * weak
             + (SUM + 2 * d[..., None]) * av + W_ABS * 2 * (L + T)) * 1.01
    err = np.abs(out - o)
    assert (np.abs(o) < av / 32).sum() > T * group  # (cancellations there are)
    assert (err <= bound).all(), float((err / bound).max())
    assert both.g.status() == 0


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,T,group", [(64, 1, 8), (128, 5, 7), (256, 3, 16), (128, 16, 8)])
@pytest.mark.parametrize("ratio", [8, 10, 12, 15])
def test_queries_with_one_large_channel(sv, ratio, dim, T, group, dtype):
    """One channel of the queries 2^8 to 2^15 times the others, and keys that are zero there:
    the scores come from the small ones alone, which keep their bits."""
    L = 150
    both = Both(sv, 1, 6, 64, 1, dim, 1, 6)
    rng = np.random.default_rng(ratio + dim)
    k = np.ldexp(rng.integers(8, 16, (L + T, 1, dim)), -3).astype(float)
    k *= np.ldexp(rng.choice([-1.0, 1.0], (L + T, 1, dim)), rng.integers(0, 5, (L + T, 1, 1)))
    k[..., 0] = 0.0
    v = np.ldexp(rng.integers(-15, 16, (L + T, 1, dim)), -3).astype(float)
    store(both, k, v)
    both.commit([L - 1], L)
    assert all(both.reserve([T]))
    # Small channels of about 1 / 32, aligned with a few of the keys, so that these stand out.
    q = 0.02 * rng.standard_normal((1, T, group, dim))
    some = rng.integers(0, L, (T, group))
    q[0] += 0.02 * np.sign(k[some, 0])
    q[..., 0] = 2.0 ** (ratio - 5) * rng.uniform(1, 1.9, (1, T, group))
    q = torch.from_numpy(q).to(dtype).cuda()
    scale = 4 * dim ** -0.5
    got = sv.sv_kv_attend(both.g, 0, q, n_new=i32([T]), scale=scale, want_lse=True)
    o, lse, bo, bl = per_key(f64(q[0]), k, v, L, T, scale, dtype)
    err, erl = np.abs(f64(got[0])[0] - o), np.abs(f64(got[1])[0] - lse)
    assert (bo < np.abs(o)).mean() > 0.4  # a zero output would not pass
    assert (err <= bo).all(), float((err / bo).max())
    assert (erl <= bl).all(), float((erl / bl).max())
    assert both.g.status() == 0


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_small_channels_together(sv, dim, dtype):
    """Small channels that all have one value, at and below where a term of 8 bits ends, and
    keys that add them up: what is lost of one is lost of all."""
    L, T, group = 100, 8, 5
    both = Both(sv, 1, 4, 64, 1, dim, 1, 4)
    k, v = np.zeros((L + T, 1, dim)), np.zeros((L + T, 1, dim))
    k[::2, 0, 1:] = 4.0
    v[::2, 0], v[1::2, 0] = 1.0, -1.0
    store(both, k, v)
    both.commit([L - 1], L)
    assert all(both.reserve([T]))
    c = 0.998 * 2.0 ** -(np.arange(T * group) % 4) * np.linspace(1, 0.6, T * group)
    q = np.zeros((1, T, group, dim))
    q[0, ..., 1:] = (2.0 ** -4 * c).reshape(T, group, 1)
    q[..., 0] = 448 * 2.0 ** 6
    q = torch.from_numpy(q).to(dtype).cuda()
    scale = 32 / dim
    got = sv.sv_kv_attend(both.g, 0, q, n_new=i32([T]), scale=scale, want_lse=True)
    o, lse, bo, bl = per_key(f64(q[0]), k, v, L, T, scale, dtype)
    err, erl = np.abs(f64(got[0])[0] - o), np.abs(f64(got[1])[0] - lse)
    assert (err <= bo).all(), float((err / bo).max())
    assert (erl <= bl).all(), float((erl / bl).max())


def near(x):
    """float32 x and its neighbours on both sides."""
    x = np.float32(x)
    return [np.nextafter(x, np.float32(0)), x, np.nextafter(x, np.float32(np.inf))]


def halfway(rng, n, lo, hi):
    """Numbers halfway between two e4m3 values: 17/16, 19/16 .. times a power of two."""
    return (rng.integers(8, 16, n) * 2 + 1) * np.ldexp(1.0 / 16, rng.integers(lo, hi, n))


def odd_pages(sv, heads, dim, layers=1):
    """One row of 5 cached tokens of random codes, in a page of 16 whose scales are set after."""
    both = Both(sv, layers, 4, 16, heads, dim, 1, 4)
    rng = np.random.default_rng(heads)
    codes = kv_ref.e4m3(np.ldexp(rng.uniform(-1, 1, (5, heads, dim)), rng.integers(-10, 9, dim)))
    codes[0, :, 0] = 448.0
    store(both, codes, codes)
    both.commit([4], 5)
    return both, rng, codes


def codes_of(g, p):
    return [f64(x.float()[0, p]) for x in (g.k, g.v)]  # [heads, page, dim]


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_at_a_scale_that_stays(sv, dtype):
    """New values on a page whose scale is no power of two and stays: each is the nearest e4m3
    of the exact quotient, also next to the points halfway between two."""
    H, D, T = 48, 96, 7
    both, rng, codes = odd_pages(sv, H, D)
    g = both.g
    s = np.exp2(rng.uniform(-9, 9, H)).astype(np.float32)
    g.k_scale[0, 0] = g.v_scale[0, 0] = torch.from_numpy(s).cuda()
    x = np.zeros((1, T, H, D), dtype=np.float32)
    for h in range(H):
        at = halfway(rng, T * D // 3, -8, 7)
        x[0, :, h] = np.array([near(m * float(s[h])) for m in at]).reshape(T, D) \
            * rng.choice([-1, 1], (T, D))
    k = torch.from_numpy(x).to(dtype)
    assert all(both.reserve([T]))
    sv.sv_kv_append(g, 0, k.cuda(), -k.cuda(), n_new=i32([T]))
    want = kv_ref.e4m3(f64(k)[0] / s.astype(np.float64)[None, :, None])
    for got, sign in zip(codes_of(g, 0), (1, -1)):
        assert (got[:, :5].transpose(1, 0, 2) == codes).all()
        assert (got[:, 5:5 + T].transpose(1, 0, 2) == sign * want).all()
    assert (g.k_scale[0, 0].cpu().numpy() == s).all() and g.status() == 0


@needs_cuda
@pytest.mark.parametrize("call", ["append", "commit"])
def test_rescale_from_a_scale_that_is_no_power_of_two(sv, call):
    """Tokens of a page whose scale grows, from one that is no power of two, chosen so that an
    old value lands next to a point halfway between two e4m3 values (append); and tokens that a
    path moves between pages of such scales (commit)."""
    H, D = 144, 96
    both, rng, codes = odd_pages(sv, H, D)
    g = both.g
    u = np.abs(codes[1, np.arange(H), np.arange(H) % D])
    u = np.where(u > 0, u, 448.0)
    s = np.ldexp(1.0, rng.integers(-5, 6, H))
    m = halfway(rng, H, -6, 0)
    m *= np.ldexp(1.0, np.minimum(0, np.floor(np.log2(u / m)).astype(int)))  # (the scale grows)
    old = np.array([near(s[h] * m[h] / u[h])[h % 3] for h in range(H)], dtype=np.float32)
    if call == "append":
        x = torch.zeros(1, 3, H, D)
        x[0, 1, :, 0] = torch.from_numpy(448 * s)
        g.k_scale[0, 0] = g.v_scale[0, 0] = torch.from_numpy(old).cuda()
        assert all(both.reserve([3]))
        sv.sv_kv_append(g, 0, x.cuda(), x.cuda(), n_new=i32([3]))
        want = kv_ref.e4m3(codes * old.astype(float)[None, :, None] / s[None, :, None])
        for got in codes_of(g, 0):
            assert (got[:, :5].transpose(1, 0, 2) == want).all()
            assert (got[:, 6, 0] == 448).all()
        assert (f64(g.k_scale[0, 0]) == s).all() and g.status() == 0
        return
    # Path 0, 14: the second token comes from the next page, whose scale is larger and no power
    # of two either; the page's older ones are rounded to it.
    T = 15
    big = (s * rng.uniform(1, 2, H)).astype(np.float32)
    # (Its ratio to the first page's is what lands next to the halfway points.)
    old = np.array([near(float(big[h]) * m[h] / u[h])[h % 3] for h in range(H)], dtype=np.float32)
    assert all(both.reserve([T]))
    new = kv_ref.e4m3(np.ldexp(rng.uniform(-1, 1, (1, T, H, D)), rng.integers(-10, 9, D)))
    new[0, :, :, 0] = 448.0
    sv.sv_kv_append(g, 0, torch.from_numpy(new).float().cuda(), torch.from_numpy(new).float().cuda(),
                    n_new=i32([T]))
    for sc in (g.k_scale, g.v_scale):
        sc[0, 0], sc[0, 1] = torch.from_numpy(old).cuda(), torch.from_numpy(big).cuda()
    path = [[14] + [-1] * (T - 1)]
    sv.sv_kv_commit(g, i32([1]), T, path=i32(path))
    stay = np.concatenate([codes, new[0, :1]])
    want = kv_ref.e4m3(stay * old.astype(float)[None, :, None] / big.astype(float)[None, :, None])
    for got in codes_of(g, 0):
        assert (got[:, :6].transpose(1, 0, 2) == want).all()
        assert (got[:, 6] == new[0, 14]).all()
    assert (f64(g.k_scale[0, 0]) == big).all() and g.len.tolist() == [7] and g.status() == 0


def check_rows(both, q, n, got, scale, informative, **mask):
    """Every row's results against per_key; `informative`: the share of the components that a
    zero output would have to fail."""
    r = both.r
    told = []
    for b in range(r.batch):
        if not n[b]:
            continue
        L = r.len[b]
        k, v = (r.values(kv, 0, b, 0, L + n[b]) for kv in (0, 1))
        one = {m: (x[b] if m == "parent" and x is not None else x) for m, x in mask.items()}
        vs = np.array([r.s[1, 0, r.rows[b][j // r.page]] for j in range(L + n[b])])
        o, lse, bo, bl = per_key(f64(q[b]), k, v, L, n[b], scale, q.dtype, vs, **one)
        out, top = f64(got[0])[b, :n[b]], torch.finfo(q.dtype).max
        # Past the type's range a result is infinite.
        past = np.isinf(out) & (np.sign(out) == np.sign(o)) & (np.abs(o) + bo > top)
        err = np.where(past, 0.0, np.abs(out - o))
        erl = np.abs(f64(got[1])[b, :n[b]] - lse)
        assert (err <= bo).all(), (b, float((err / bo).max()), np.argwhere(err > bo)[:5])
        assert (erl <= bl).all(), (b, float((erl / bl).max()))
        told.append((bo < np.abs(o)).ravel())
    assert np.concatenate(told).mean() > informative


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_sigma,sigma", [(0.0, 3.0), (0.01, 0.0), (0.01, 3.0), (1.0, 0.0),
                                           (1.0, 3.0), (5.0, 1.0), (30.0, 0.0), (30.0, 3.0)])
@pytest.mark.parametrize("dim,T,heads,group,trees,window", [
    (128, 3, 2, 4, False, 0), (64, 16, 1, 8, True, 0), (256, 9, 1, 4, False, 200),
    (80, 33, 1, 3, False, 0)])
def test_score_ranges(sv, q_sigma, sigma, dim, T, heads, group, trees, window, dtype):
    """Flat scores, and scores so far apart that one key takes all, with tokens whose sizes
    differ by powers of ten: each key has the error of its own score, so that what is certain
    in the result has to be right."""
    lens, n = [5, 400, 1100], [T, T, max(1, T - 2)]
    per = -(-(max(lens) + T) // 16) + 1
    both = Both(sv, 1, 3 * per, 16, heads, dim, 3, per)
    seed = int(q_sigma) + dim
    both.fill(lens, seed, sigma)
    assert all(both.reserve(n))
    k, v = rand_kv(both.r, T, seed + 77, sigma)
    both.append(0, k, v, n)
    rng = np.random.default_rng(seed)
    par = [tree(rng, T) for _ in lens] if trees else None
    gen = torch.Generator(device="cuda").manual_seed(seed + 5)
    q = q_sigma * torch.randn(3, T, heads * group, dim, generator=gen, device="cuda")
    q = q.to(dtype)
    got = sv.sv_kv_attend(both.g, 0, q, n_new=i32(n), parent=None if par is None else i32(par),
                          window=window, want_lse=True)
    check_rows(both, q, n, got, dim ** -0.5, 0.75, parent=par, window=window)
    assert both.g.status() == 0


@needs_cuda
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,group", [(1, 8), (5, 7), (16, 8), (40, 4)])
def test_one_key_takes_all(sv, T, group, dtype):
    """A key in each row whose score is 40 above the others': the result is its value, the log
    sum its score, wherever the key is."""
    dim, L, page = 128, 700, 32
    scale = dim ** -0.5
    both = Both(sv, 1, 60, page, 1, dim, 2, 30)
    r = both.r
    rng = np.random.default_rng(T)
    tot = L + T
    k = kv_ref.e4m3(rng.standard_normal((2, tot, 1, dim)))
    v = kv_ref.e4m3(4 * rng.standard_normal((2, tot, 1, dim)))
    mean = kv_ref.e4m3(rng.standard_normal(dim))
    top = (3, L - 1)
    for b in range(2):  # (one key along the queries, all others without a part along them)
        k[b, :, 0, :] -= (k[b, :, 0] @ mean)[:, None] * mean / (mean @ mean)
        k[b, top[b], 0] = mean * 4
    k = kv_ref.e4m3(np.clip(k, -100, 100))
    assert all(both.reserve([tot, tot]))
    x = [torch.from_numpy(y).cuda().float() for y in (k, v)]
    both.append(0, x[0], x[1], [tot, tot])
    both.commit([L - 1, L - 1], L)
    assert all(both.reserve([T, T]))
    a = 48 / (scale * 4 * (mean @ mean))
    q = torch.from_numpy(a * mean * np.ones((2, T, group, 1))).to(dtype).cuda()
    got = sv.sv_kv_attend(both.g, 0, q, n_new=i32([T, T]), want_lse=True)
    check_rows(both, q, [T, T], got, scale, 0.99)
    for b in range(2):
        want = r.values(1, 0, b, top[b], top[b] + 1)[0, 0]
        lse = scale * (f64(q)[b] @ r.values(0, 0, b, top[b], top[b] + 1)[0, 0])
        # The other keys together: 740 e^-40, less than 2^-48 of the value's largest.
        half = torch.finfo(dtype).eps / 2
        assert (np.abs(f64(got[0])[b] - want) <= (half + SUM) * np.abs(want) + 2.0 ** -27 * 32).all()
        assert (np.abs(f64(got[1])[b] - lse) <= 2.0 ** -17 * 48).all()


@needs_cuda
@pytest.mark.parametrize("with_path", [False, True])
@pytest.mark.parametrize("factor", [6, 15])
def test_a_rejected_outlier_keeps_its_scale(sv, factor, with_path):
    """A rejected token 2^6 or 2^15 times the others of its page: the page's older tokens stay
    rounded to the scale it needed, exactly as the formula says, which costs them bits only in
    the latter case; pages without older tokens start anew."""
    D = 32
    both = Both(sv, 2, 4, 16, 1, D, 1, 4)
    rng = np.random.default_rng(1)
    x = rng.uniform(1, 1.9, (13, 1, D))
    x[0, 0, 0] = 448.0 / 256  # the first page's scale is 2^-8

    def append(y):
        z = torch.from_numpy(y[None]).float().cuda()
        for layer in range(2):
            sv.sv_kv_append(both.g, layer, z, -z)
        both.r.append(0, f64(z), -f64(z), [len(y)])
        both.r.append(1, f64(z), -f64(z), [len(y)])

    assert all(both.reserve([13]))
    append(x)
    both.commit([12], 13)
    before = both.r.values(0, 0, 0, 0, 13)
    assert both.r.s[0, 0, 0, 0] == 2.0 ** -7  # (1.9 > 448 / 256)
    y = rng.uniform(1, 1.7, (6, 1, D))
    y[1] *= 2.0 ** factor  # position 14, on the first page
    y[4] *= 2.0 ** factor  # position 17, on the next
    assert all(both.reserve([6]))
    append(y)
    both.commit([0], 6, [[2, 3, -1, -1, -1, -1]] if with_path else None)
    both.same()
    both.same_values()
    after = both.r.values(0, 0, 0, 0, 13)
    s = both.r.s[0, 0, 0, 0]
    assert s == 2.0 ** (factor - 8) and (after == kv_ref.e4m3(before / s) * s).all()
    assert (after != before).any() == (factor > 14)
    assert (np.abs(after - before) <= 2.0 ** -10 * s).all()  # half of e4m3's smallest step
    # The next round overwrites the outlier; the first page keeps the scale, the next has its own.
    assert all(both.reserve([6]))
    append(rng.uniform(1, 1.7, (6, 1, D)))
    both.commit([5], 6)
    both.same()
    both.same_values()
    assert both.r.s[0, 0, 0, 0] == s and both.r.s[0, 0, 1, 0] == 2.0 ** -8
    for got in (both.g.k_scale, both.g.v_scale):
        assert got[:, :2, 0].tolist() == [[s, 2.0 ** -8]] * 2
