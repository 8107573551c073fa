"""CPU checks of the rotary calls: frequencies, and host-side refusals."""
import ctypes
import decimal
import math

import pytest
import torch

FAKE = 1 << 20  # never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


def fixed(sv, angles):
    out = (ctypes.c_int64 * max(len(angles), 1))()
    rc = sv.load().sv_rope_fixed((ctypes.c_double * max(len(angles), 1))(*angles), len(angles), out)
    return rc, [x % 2 ** 64 for x in out][:len(angles)]


def freqs(sv, rot, base=10000.0, scaling=0, stretch=1.0, original=0.0, low=0.0, high=0.0):
    out = (ctypes.c_int64 * max(rot // 2, 1))()
    rc = sv.load().sv_rope_freqs(rot, base, scaling, stretch, original, low, high, out)
    return rc, [x % 2 ** 64 / 2.0 ** 64 * 2 * math.pi for x in out][:rot // 2]


def test_fixed_point(sv):
    """Radians as a fraction of a turn in 64 bits; whole turns and signs wrap."""
    rc, f = fixed(sv, [math.pi, 0.0, math.pi / 2, -math.pi / 2, 2 * math.pi + math.pi / 4, -1e-300])
    assert rc == sv.SV_OK
    near = lambda a, b: min((a - b) % 2 ** 64, (b - a) % 2 ** 64) <= 2 ** 12  # noqa: E731
    want = [2 ** 63, 0, 2 ** 62, 3 * 2 ** 62, 2 ** 61, 0]
    assert all(near(a, b) for a, b in zip(f, want)), f
    for bad in (math.nan, math.inf):
        assert fixed(sv, [0.1, bad])[0] == sv.SV_ERR_ARG
    assert fixed(sv, [])[0] == sv.SV_OK
    assert sv.load().sv_rope_fixed(None, 2, None) == sv.SV_ERR_ARG
    assert sv.load().sv_rope_fixed(None, 257, None) == sv.SV_ERR_SHAPE


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (20, 500000.0), (128, 10000.0), (512, 1e6)])
def test_frequencies(sv, rot, base):
    """Plain, and every kind of stretching, against their formulas."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    same = lambda a, b: all(abs(x - y) <= 1e-14 * y + 1e-17 for x, y in zip(a, b))  # noqa: E731
    rc, got = freqs(sv, rot, base)
    assert rc == sv.SV_OK and same(got, f)
    rc, got = freqs(sv, rot, base, 1, 8.0)
    assert rc == sv.SV_OK and same(got, [x / 8 for x in f])
    rc, got = freqs(sv, rot, base, 2, 8.0, 8192.0, 1.0, 4.0)
    w = [min(1, max(0, (8192 * x / (2 * math.pi) - 1) / 3)) for x in f]
    assert rc == sv.SV_OK and same(got, [x * (k + (1 - k) / 8) for x, k in zip(f, w)])
    rc, got = freqs(sv, rot, base, 3, 16.0, 4096.0, 1.0, 32.0)
    at = lambda n: rot * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
    w = [1 - min(1, max(0, (i - a) / max(b - a, 1e-3))) for i in range(rot // 2)]
    assert rc == sv.SV_OK and same(got, [x * (k + (1 - k) / 16) for x, k in zip(f, w)])


def test_frequency_refusals(sv):
    for rot in (0, 1, 3, -2, 514):
        assert freqs(sv, rot)[0] == sv.SV_ERR_SHAPE
    for kw in (dict(scaling=4), dict(scaling=-1), dict(base=1.0), dict(base=math.nan),
               dict(base=math.inf), dict(stretch=0.0), dict(stretch=math.inf),
               dict(scaling=2, original=0.0, low=1.0, high=4.0),
               dict(scaling=2, original=100.0, low=4.0, high=4.0),
               dict(scaling=3, original=100.0, low=0.0, high=4.0),
               dict(scaling=3, original=math.nan, low=1.0, high=4.0),
               dict(scaling=3, original=100.0, low=1.0, high=math.inf)):
        assert freqs(sv, 64, **kw)[0] == sv.SV_ERR_ARG, kw
    assert sv.load().sv_rope_freqs(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None) == sv.SV_ERR_ARG


def spec(sv, freq=FAKE, rot=64, interleaved=0, gain=1.0):
    return sv._RopeStruct(freq, rot, interleaved, gain)


def rope(sv, s=None, **a):
    g = lambda k, d: a.get(k, d)  # noqa: E731
    h, d = g("heads", 4), g("dim", 128)
    return sv.load().sv_rope(
        ctypes.byref(s or spec(sv)), g("x", FAKE), g("dtype", 1), g("row", 8 * h * d),
        g("tok", h * d), g("batch", 3), g("T", 8), h, d, g("pos", None), g("start", None),
        g("parent", None), g("n", None), 0, g("out", 2 * FAKE), g("out_row", 8 * h * d),
        g("out_tok", h * d), g("ws", FAKE), g("nb", 256), None)


@pytest.mark.parametrize("arg,code", [
    (dict(dtype=3), "DTYPE"), (dict(batch=-1), "SHAPE"), (dict(batch=4097), "SHAPE"),
    (dict(T=-1), "SHAPE"), (dict(T=65536), "SHAPE"), (dict(heads=0), "SHAPE"),
    (dict(heads=1025), "SHAPE"), (dict(dim=0), "SHAPE"), (dict(dim=136), "SHAPE"),
    (dict(dim=528), "SHAPE"), (dict(T=65, parent=FAKE), "SHAPE"), (dict(dim=48), "ARG"),
    (dict(pos=FAKE, start=FAKE), "ARG"), (dict(pos=FAKE, parent=FAKE), "ARG"),
    (dict(ws=None), "WORKSPACE"), (dict(ws=FAKE + 8), "WORKSPACE"), (dict(nb=255), "WORKSPACE"),
    (dict(x=None), "ARG"), (dict(x=FAKE + 8), "ARG"), (dict(tok=511), "ARG"),
    (dict(tok=516), "ARG"), (dict(row=-8), "ARG"), (dict(out=None), "ARG"),
    (dict(out=FAKE + 4), "ARG"), (dict(out_tok=504), "ARG"), (dict(out_row=0), "ARG"),
    (dict(out_row=512), "ARG"), (dict(out=FAKE, out_tok=1024, out_row=8192), "ARG"),
    (dict(pos=FAKE + 1), "ARG"), (dict(start=FAKE + 2), "ARG"), (dict(parent=FAKE + 2), "ARG"),
    (dict(n=FAKE + 1), "ARG"), (dict(batch=0), "OK"), (dict(T=0), "OK"),
])
def test_rope_refusals(sv, arg, code):
    assert rope(sv, **arg) == (sv.SV_OK if code == "OK" else getattr(sv, "SV_ERR_" + code))


@pytest.mark.parametrize("bad", [dict(freq=None), dict(freq=FAKE + 4), dict(rot=0), dict(rot=63),
                                 dict(rot=130), dict(gain=math.nan), dict(gain=math.inf)])
def test_spec_refusals(sv, bad):
    assert rope(sv, spec(sv, **bad)) == sv.SV_ERR_ARG
    assert append(sv, s=spec(sv, **bad)) == sv.SV_ERR_ARG


def append(sv, s=None, **a):
    c = sv._CacheStruct(layers=2, pages=40, page=64, heads=2, dim=128, batch=3, max_pages=8)
    for n in ("k", "v", "k_scale", "v_scale", "table", "n_pages", "len", "refs"):
        setattr(c, n, FAKE)
    g, lib = lambda k, d: a.get(k, d), sv.load()  # noqa: E731
    nb = lib.sv_kv_workspace_bytes(ctypes.byref(c))
    return lib.sv_kv_append_rope(
        ctypes.byref(c), g("layer", 0), g("k", FAKE), g("v", FAKE), g("dtype", 1), g("row", 1280),
        g("tok", 256), 1280, 256, g("T", 5), g("n", None), g("parent", None),
        ctypes.byref(s or spec(sv)), g("q", FAKE), g("q_row", 5120), g("q_tok", 1024),
        g("q_heads", 8), g("q_out", FAKE), g("q_out_row", 5120), 1024, g("ws", FAKE), g("nb", nb),
        None)


@pytest.mark.parametrize("arg,code", [
    (dict(dtype=5), "DTYPE"), (dict(T=-1), "SHAPE"), (dict(T=65536), "SHAPE"),
    (dict(T=65, parent=FAKE), "SHAPE"), (dict(layer=2), "ARG"), (dict(layer=-1), "ARG"),
    (dict(k=None), "ARG"), (dict(v=FAKE + 8), "ARG"), (dict(tok=255), "ARG"),
    (dict(n=FAKE + 1), "ARG"), (dict(parent=FAKE + 2), "ARG"), (dict(q=None), "ARG"),
    (dict(q_heads=0), "ARG"), (dict(q_heads=-1), "SHAPE"), (dict(q_heads=1 << 18), "SHAPE"),
    (dict(q=FAKE + 2), "ARG"), (dict(q_tok=1000), "ARG"), (dict(q_out=None), "ARG"),
    (dict(q_out_row=10240), "ARG"), (dict(q_out=2 * FAKE, q_out_row=1024), "ARG"),
    (dict(ws=None), "WORKSPACE"), (dict(nb=512), "WORKSPACE"), (dict(T=0), "OK"),
])
def test_append_rope_refusals(sv, arg, code):
    assert append(sv, **arg) == (sv.SV_OK if code == "OK" else getattr(sv, "SV_ERR_" + code))


def test_table_refusals(sv):
    for kw in (dict(rot=7), dict(rot=0), dict(rot=514), dict(rot=64, scaling="other"),
               dict(rot=64, gain=math.nan), dict(rot=64, gain=1e39), dict(rot=64, angles=[0.1])):
        with pytest.raises(ValueError):
            sv.Rope(device="cpu", **kw)
    with pytest.raises(sv.SpecVerifyError):
        sv.Rope(64, base=0.5, device="cpu")
    with pytest.raises(sv.SpecVerifyError):
        sv.Rope(4, angles=[0.1, math.inf], device="cpu")


TAU = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257242")


def units(turns):
    """A fraction of a turn in units of 2^-64, not rounded."""
    return (turns % 1) * 2 ** 64


def off(got, want):
    """How far, in units of 2^-64, whole turns left out."""
    d = (got - want) % 2 ** 64
    return float(min(d, 2 ** 64 - d))


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (20, 500000.0), (128, 10000.0), (128, 500000.0),
                                      (512, 1e6), (64, 1.0000001), (256, 1e200), (96, 10000.3)])
def test_frequencies_to_the_last_unit(sv, rot, base):
    """Every frequency is its formula's, rounded once to 2^-64 of a turn (half a unit, and 2^-9 of one
    for sums of two doubles), so that at position 2^31 an angle is off by 2^-34 of a turn."""
    with decimal.localcontext() as c:
        c.prec = 70
        D = decimal.Decimal
        f = [(-(D(2 * i) / rot) * D(base).ln()).exp() for i in range(rot // 2)]

        def exactly(scaling, want, **kw):
            out = (ctypes.c_int64 * (rot // 2))()
            args = dict(dict(stretch=1.0, original=0.0, low=0.0, high=0.0), **kw)
            rc = sv.load().sv_rope_freqs(rot, base, scaling, *args.values(), out)
            assert rc == sv.SV_OK
            assert max(off(D(x % 2 ** 64), units(y / TAU)) for x, y in zip(out, want)) <= 0.5 + 2 ** -9

        exactly(0, f)
        exactly(1, [x / D(7.3) for x in f], stretch=7.3)
        w = [min(D(1), max(D(0), (8192 * x / TAU - 1) / 3)) for x in f]
        exactly(2, [x * (k + (1 - k) / 8) for x, k in zip(f, w)], stretch=8.0, original=8192.0, low=1.0,
                high=4.0)
        at = lambda n: rot * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        a, b = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
        w = [1 - min(D(1), max(D(0), D(i - a) / D(max(b - a, 1e-3)))) for i in range(rot // 2)]
        exactly(3, [x * (k + (1 - k) / 16) for x, k in zip(f, w)], stretch=16.0, original=4096.0,
                low=1.0, high=32.0)


def test_given_angles_to_the_last_unit(sv):
    """Angles as the doubles they are, up to a million turns and signs; larger ones wrap somehow."""
    a = [1.0, -1.0, 0.1, -0.1, 1e-3, 3.0, -3.0, 6.0, 6.283185307179586, -6.283185307179586, 1e-17,
         -1e-17, 1e-300, -1e-300, 0.0, 12345.678, -98765.4321, 5e6, -5e6, 2.0 ** -40, -(2.0 ** -40)]
    rc, got = fixed(sv, a)
    assert rc == sv.SV_OK
    with decimal.localcontext() as c:
        c.prec = 70
        want = [units(decimal.Decimal(x) / TAU) for x in a]
        for x, g, w in zip(a, got, want):
            assert off(decimal.Decimal(g), w) <= 0.5 + 2 ** -9, x
    big = [s * 10.0 ** e for e in (10, 17, 20, 40, 300) for s in (1, -1)]
    assert fixed(sv, big)[0] == sv.SV_OK


def test_out_of_a_tensor_that_requires_grad(sv):
    """A result written to out would lose x's graph without a word: refused, as torch does."""
    x, out = (torch.zeros(1, 1, 1, 16, requires_grad=g) for g in (True, False))
    for o in (out, x):
        with pytest.raises(ValueError, match="requires grad"):
            sv.sv_rope(object(), x, out=o)
