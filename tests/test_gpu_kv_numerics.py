"""What the cache attention's numbers may be off by, on inputs where each part of that shows:
weights, queries, keys of very different size, and scales of another quantiser."""
import math

import numpy as np
import pytest
import torch

import kv_ref
from test_gpu_kv import Both, f64, i32, needs_cuda

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
