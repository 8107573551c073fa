"""CPU checks of the key/value cache: host-side refusals of its calls, and the plain host
model that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import kv_ref


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


FAKE = 1 << 20  # never dereferenced: every call below fails its checks first
DIMS = dict(layers=2, pages=40, page=64, heads=2, dim=128, batch=3, max_pages=8)


def cache(sv, **over):
    c = sv._CacheStruct(**{**DIMS, **{k: v for k, v in over.items() if k in DIMS}})
    for n in ("k", "v", "k_scale", "v_scale", "table", "n_pages", "len", "refs"):
        setattr(c, n, over.get("p_" + n, FAKE))
    return c


def need(sv, c):
    return sv.load().sv_kv_workspace_bytes(ctypes.byref(c))


def calls(sv, c, ws=FAKE, nb=None, **a):
    """Every cache call on cache c with valid arguments except those in a."""
    lib, p = sv.load(), ctypes.byref(c) if c is not None else None
    nb = (need(sv, c) if c is not None else 1 << 30) if nb is None else nb
    g = lambda k, d: a.get(k, d)  # noqa: E731
    w = c.heads * c.dim if c is not None else 256
    dt = g("dtype", 1)
    return {
        "reserve": lambda: lib.sv_kv_reserve(p, g("n_new", FAKE), g("ok", None), ws, nb, None),
        "append": lambda: lib.sv_kv_append(p, g("layer", 0), g("k", FAKE), g("v", FAKE), dt,
                                           g("row", 5 * w), g("tok", w), 5 * w, w, g("T", 5),
                                           g("n", None), ws, nb, None),
        "read": lambda: lib.sv_kv_read(p, g("layer", 0), g("n_layers", 1), g("start", FAKE), None,
                                       g("T", 5), g("k", FAKE), g("v", FAKE), dt, ws, nb, None),
        "attend": lambda: lib.sv_kv_attend(p, g("layer", 0), g("q", FAKE), dt, g("row", 20 * w),
                                           g("tok", 4 * w), g("T", 5), g("q_heads", 8), None,
                                           g("parent", None), g("scale", 0.1), g("window", 0),
                                           g("sinks", 0), g("out", FAKE), g("lse", None), ws, nb,
                                           None),
        "commit": lambda: lib.sv_kv_commit(p, g("accepted", FAKE), g("path", None), g("N", 5), ws,
                                           nb, None),
        "fork": lambda: lib.sv_kv_fork(p, g("src", FAKE), g("ok", None), ws, nb, None),
    }


@pytest.mark.parametrize("over", [dict(page=8), dict(page=48), dict(page=256), dict(dim=0),
                                  dict(dim=24), dict(dim=272), dict(heads=0), dict(heads=1025),
                                  dict(batch=0), dict(batch=5000), dict(layers=0), dict(pages=0),
                                  dict(max_pages=0), dict(pages=1 << 24),
                                  dict(max_pages=1 << 25)])
def test_sizes(sv, over):
    c = cache(sv, **over)
    assert need(sv, c) == 0
    for name, f in calls(sv, c).items():
        assert f() == sv.SV_ERR_SHAPE, name


def test_cache_and_workspace_pointers(sv):
    for name, f in calls(sv, None).items():
        assert f() == sv.SV_ERR_ARG, name
    for n in ("k", "v", "k_scale", "v_scale", "table", "n_pages", "len", "refs"):
        for bad in (None, FAKE + 2):
            for name, f in calls(sv, cache(sv, **{"p_" + n: bad})).items():
                assert f() == sv.SV_ERR_ARG, (n, name)
    c = cache(sv)
    for kw in (dict(ws=None), dict(ws=FAKE + 16), dict(nb=need(sv, c) - 1)):
        for name, f in calls(sv, c, **kw).items():
            assert f() == sv.SV_ERR_WORKSPACE, (kw, name)


@pytest.mark.parametrize("name,arg,code", [
    ("reserve", dict(n_new=None), "ARG"), ("reserve", dict(n_new=FAKE + 1), "ARG"),
    ("reserve", dict(ok=FAKE + 2), "ARG"),
    ("append", dict(dtype=3), "DTYPE"), ("append", dict(T=-1), "SHAPE"),
    ("append", dict(T=65536), "SHAPE"), ("append", dict(layer=2), "ARG"),
    ("append", dict(layer=-1), "ARG"), ("append", dict(k=None), "ARG"),
    ("append", dict(v=FAKE + 8), "ARG"), ("append", dict(tok=255), "ARG"),
    ("append", dict(tok=260), "ARG"), ("append", dict(row=-8), "ARG"),
    ("append", dict(n=FAKE + 1), "ARG"),
    ("read", dict(dtype=2), "DTYPE"), ("read", dict(T=-1), "SHAPE"),
    ("read", dict(n_layers=3), "ARG"), ("read", dict(layer=1, n_layers=2), "ARG"),
    ("read", dict(start=None), "ARG"), ("read", dict(k=FAKE + 4), "ARG"),
    ("attend", dict(dtype=0), "DTYPE"), ("attend", dict(T=65536), "SHAPE"),
    ("attend", dict(T=65, parent=FAKE), "SHAPE"), ("attend", dict(q_heads=7), "SHAPE"),
    ("attend", dict(q_heads=1), "SHAPE"), ("attend", dict(q_heads=258), "SHAPE"),
    ("attend", dict(layer=5), "ARG"), ("attend", dict(scale=float("nan")), "ARG"),
    ("attend", dict(scale=float("inf")), "ARG"), ("attend", dict(window=-1), "ARG"),
    ("attend", dict(sinks=-1), "ARG"), ("attend", dict(q=None), "ARG"),
    ("attend", dict(q=FAKE + 2), "ARG"), ("attend", dict(tok=1020), "ARG"),
    ("attend", dict(out=None), "ARG"), ("attend", dict(lse=FAKE + 2), "ARG"),
    ("attend", dict(parent=FAKE + 2), "ARG"),
    ("commit", dict(N=0), "SHAPE"), ("commit", dict(N=65, path=FAKE), "SHAPE"),
    ("commit", dict(accepted=None), "ARG"), ("commit", dict(path=FAKE + 2), "ARG"),
    ("fork", dict(src=None), "ARG"), ("fork", dict(ok=FAKE + 2), "ARG"),
])
def test_refusals(sv, name, arg, code):
    assert calls(sv, cache(sv), **arg)[name]() == getattr(sv, "SV_ERR_" + code)


def test_nothing_to_do(sv):
    """No new tokens, or no layers to read: accepted without any device work."""
    c = cache(sv)
    assert calls(sv, c, T=0)["append"]() == sv.SV_OK
    assert calls(sv, c, T=0)["attend"]() == sv.SV_OK
    assert calls(sv, c, T=0)["read"]() == sv.SV_OK
    assert calls(sv, c, n_layers=0)["read"]() == sv.SV_OK
    assert sv.status_string(sv.SV_ERR_NO_PAGES) == "not enough free cache pages"


def test_model_e4m3():
    """The 8-bit grid of the host model: ends, ties to even, subnormals."""
    x = np.array([0.0, 448, 449, 1e9, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -17.0])
    y = np.array([0.0, 448, 448, 448, 1.0, 1.25, 2.0 ** -9, 0.0, 2.0 ** -8, -16.0])
    assert (kv_ref.e4m3(x) == y).all()
    assert kv_ref.scale_for(448.0) == 1.0 and kv_ref.scale_for(448.1) == 2.0
    assert kv_ref.scale_for(0.0) == 2.0 ** -64


def test_model_invariants():
    """Whatever the calls, refs counts the rows that hold each page, and a row's tokens stay
    readable at the precision of their page."""
    rng = np.random.default_rng(0)
    c = kv_ref.RefCache(1, 40, 16, 1, 16, 4, 8)
    for step in range(60):
        n = rng.integers(0, 6, 4)
        ok = c.reserve(n)
        n = np.where(ok, n, 0)
        x = rng.standard_normal((4, 6, 1, 16))
        before = list(c.len)
        c.append(0, x, x, n)
        for b in range(4):
            if n[b]:
                got = c.values(0, 0, b, before[b], before[b] + n[b])
                assert np.abs(got - x[b, : n[b]]).max() <= 2.0 ** -4 * np.abs(x[b]).max() * 1.01
        c.commit([int(rng.integers(-1, m)) for m in n])
        if step % 7 == 3:
            c.fork(rng.integers(-1, 4, 4))
        count = np.zeros(40, dtype=int)
        for r in c.rows:
            for p in r:
                count[p] += 1
        assert (count == c.refs).all()


def test_attend_limits(sv):
    """Work units and positions that pass 31 bits are refused, by attend only."""
    c = cache(sv, max_pages=1 << 24)
    assert calls(sv, c, T=65535, tok=1024)["attend"]() == sv.SV_ERR_SHAPE
    c = cache(sv, page=16, max_pages=(1 << 27) - 1, batch=1)
    assert calls(sv, c)["attend"]() == sv.SV_ERR_SHAPE
    assert calls(sv, c, T=0)["append"]() == sv.SV_OK
