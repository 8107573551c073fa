"""CPU checks of the shared-prefix attention's host side: buffer sizes and refusals."""
import ctypes

import pytest
import torch

from test_kv_device import Stream, Tensor, bind  # noqa: F401
from test_kv_host import FAKE, cache, need


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_79_gb300 as m

    m.load()
    return m


def size(sv, c, T=5, heads=8):
    return sv.load().sv_kv_share_bytes(ctypes.byref(c), T, heads)


def calls(sv, c, **a):
    lib, p = sv.load(), ctypes.byref(c)
    g = lambda k, d: a.get(k, d)  # noqa: E731
    w, nb = c.heads * c.dim, need(sv, c)
    share = g("share", FAKE), g("share_bytes", size(sv, c))
    ws = g("ws", FAKE), g("nb", nb)
    return {
        "share": lambda: lib.sv_kv_share(p, g("group", None), *share, *ws, None),
        "attend": lambda: lib.sv_kv_attend_shared(
            p, g("layer", 0), g("q", FAKE), g("dtype", 1), g("row", 20 * w), g("tok", 4 * w),
            g("T", 5), g("q_heads", 8), g("n", None), g("parent", None), g("scale", 0.1),
            g("window", 0), g("sinks", 0), g("out", FAKE), g("lse", None), *share, *ws, None)}


def test_sizes(sv):
    """Bytes grow with T and heads, and are 0 for what is not supported."""
    c = cache(sv)
    assert 0 < size(sv, c, 1, 2) <= size(sv, c, 1, 8) < size(sv, c, 64, 8) < size(sv, c, 600, 8)
    for T, heads in ((0, 8), (-1, 8), (65536, 8), (5, 7), (5, 1), (5, 258), (5, 0)):
        assert size(sv, c, T, heads) == 0
    assert size(sv, cache(sv, page=48)) == 0
    assert size(sv, cache(sv, batch=4096, heads=1024, pages=8, max_pages=1), 65535, 1024 * 128) == 0


@pytest.mark.parametrize("call,arg,code", [
    ("share", dict(share=None), "WORKSPACE"), ("share", dict(share=FAKE + 16), "WORKSPACE"),
    ("share", dict(share_bytes=256), "WORKSPACE"), ("share", dict(ws=None), "WORKSPACE"),
    ("share", dict(nb=0), "WORKSPACE"), ("share", dict(group=FAKE + 2), "ARG"),
    ("attend", dict(share=None), "WORKSPACE"), ("attend", dict(share=FAKE + 16), "WORKSPACE"),
    ("attend", dict(ws=None), "WORKSPACE"), ("attend", dict(dtype=0), "DTYPE"),
    ("attend", dict(T=65536), "SHAPE"), ("attend", dict(T=65, parent=FAKE), "SHAPE"),
    ("attend", dict(q_heads=7), "SHAPE"), ("attend", dict(q_heads=258), "SHAPE"),
    ("attend", dict(layer=5), "ARG"), ("attend", dict(scale=float("nan")), "ARG"),
    ("attend", dict(window=-1), "ARG"), ("attend", dict(sinks=-1), "ARG"),
    ("attend", dict(q=None), "ARG"), ("attend", dict(tok=1020), "ARG"),
    ("attend", dict(out=None), "ARG"), ("attend", dict(lse=FAKE + 2), "ARG"),
    ("attend", dict(parent=FAKE + 2), "ARG"), ("attend", dict(n=FAKE + 1), "ARG"),
    ("attend", dict(T=0), "OK")])
def test_refusals(sv, call, arg, code):
    got = calls(sv, cache(sv), **arg)[call]()
    assert got == (sv.SV_OK if code == "OK" else getattr(sv, "SV_ERR_" + code))


def test_buffers_for_fewer_tokens(sv):
    """A buffer made for fewer tokens or heads than a call has is refused."""
    c = cache(sv)
    small = size(sv, c, 1, 2)
    assert calls(sv, c, share_bytes=small)["attend"]() == sv.SV_ERR_WORKSPACE
    assert calls(sv, c, share_bytes=size(sv, c) - 1)["attend"]() == sv.SV_ERR_WORKSPACE


def test_binding(bind):  # noqa: F811
    """Devices, streams, shapes, and the cache that the groups belong to."""
    sv, cache, lib = bind
    share = type("Share", (), dict(cache=cache, ptr=1 << 21, nbytes=999, index=0))()
    q, n = Tensor((2, 3, 4, 32), torch.bfloat16), Tensor((2,), torch.int32)
    sv.sv_kv_share(cache, share, n)
    sv.sv_kv_attend_shared(cache, 0, q, share, n_new=n, out=q, stream=Stream())
    assert [c[0] for c in lib.calls] == ["sv_kv_share", "sv_kv_attend_shared"]
    assert lib.calls[0][1][2:4] == (1 << 21, 999) and lib.calls[1][1][-5:-3] == (1 << 21, 999)
    assert lib.calls[0][1][-1] == 55 and lib.calls[1][1][-1] == 77
    for f in (lambda: sv.sv_kv_share(cache, share, Tensor((3,), torch.int32)),
              lambda: sv.sv_kv_share(cache, share, Tensor((2,), torch.int64)),
              lambda: sv.sv_kv_share(cache, share, Tensor((2,), torch.int32, 1)),
              lambda: sv.sv_kv_share(cache, share, stream=Stream(1)),
              lambda: sv.sv_kv_attend_shared(cache, 0, q, share, stream=Stream(1)),
              lambda: sv.sv_kv_attend_shared(cache, 0, Tensor((2, 3, 4, 32), torch.int8), share),
              lambda: sv.sv_kv_share(object(), share), ):
        with pytest.raises((ValueError, AttributeError)):
            f()
    other = type("Share", (), dict(cache=object(), ptr=1, nbytes=1, index=0))()
    for f in (lambda: sv.sv_kv_share(cache, other),
              lambda: sv.sv_kv_attend_shared(cache, 0, q, other)):
        with pytest.raises(ValueError, match="another cache"):
            f()
