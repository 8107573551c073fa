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
