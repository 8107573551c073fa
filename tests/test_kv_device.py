"""CPU checks of how the cache calls keep devices, streams and integer ranges apart."""
import os
import subprocess
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_79_gb300", "csrc")


def test_set_up_runs_once_per_device(tmp_path):
    """A device's set-up runs once, another device's too, and one that failed again."""
    src = tmp_path / "once.cpp"
    src.write_text("""
#include "sv_device.cuh"
#include <cstdio>
int main() {
  static sv::OncePerDevice once;
  int ran[70] = {}, fail = 1;
  auto call = [&](int dev) { return once.run(dev, [&] { ++ran[dev]; return fail; }); };
  if (call(0) != 1 || call(0) != 1 || ran[0] != 2) return 1;  // failed: tried again
  fail = 0;
  if (call(0) || call(0) || ran[0] != 3) return 2;            // took: not again
  if (call(1) || call(1) || ran[1] != 1) return 3;            // another device
  if (call(69) || call(69) || ran[69] != 2) return 4;         // past the table: every time
  return 0;
}
""")
    exe = tmp_path / "once"
    # (Headers of the library end in .cuh whether they hold device code or not.)
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_attention_sizes_its_shared_memory_per_device():
    """The opt-in to large shared memory goes through that set-up, not once per process."""
    src = open(os.path.join(CSRC, "sv_kv_attend.cu")).read()
    assert "call_once" not in src and "OncePerDevice" in src


# ---------------------------------------------------------------------------------------
# The binding, with stand-ins for tensors, streams and the library: what reaches the C calls.
class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index

    def stride(self):
        out, n = [], 1
        for x in reversed(self.shape):
            out.insert(0, n)
            n *= x
        return tuple(out)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def new_empty(self, shape, dtype=None):
        return Tensor(shape, dtype or self.dtype, self.index)


class Stream:
    def __init__(self, index=0):
        self.device, self.cuda_stream = torch.device("cuda", index), 77


class Lib:
    """Every C call succeeds and is kept with its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def bind(monkeypatch):
    import speculative_decoding_verification_79_gb300 as sv

    lib = Lib()
    monkeypatch.setattr(sv, "load", lambda: lib)
    monkeypatch.setattr(sv, "_raw_stream", lambda index: 55 + index)
    monkeypatch.setattr(sv, "_current_device", lambda: 0)
    cache = types.SimpleNamespace(
        batch=2, dim=32, heads=2, rows=(2,), index=0, ref=None, ws=1 << 20, nbytes=1 << 20,
        t=types.SimpleNamespace(device=torch.device("cuda", 0)),
        c=types.SimpleNamespace(layers=3, batch=2, heads=2, dim=32))
    return sv, cache, lib


def kv_calls(sv, cache, dev=None, stream=None, **over):
    """Every cache call of the binding; `dev` names one tensor that is on another device."""
    at = lambda name, shape, dtype: Tensor(shape, dtype, 1 if name == dev else 0)  # noqa: E731
    i32, bf, f32 = torch.int32, torch.bfloat16, torch.float32
    n = lambda name: at(name, (2,), i32)  # noqa: E731
    return {
        "reserve": lambda: sv.sv_kv_reserve(cache, n("n_new"), n("ok"), stream=stream),
        "append": lambda: sv.sv_kv_append(cache, over.get("layer", 0), at("k", (2, 3, 2, 32), bf),
                                          at("v", (2, 3, 2, 32), bf), n_new=n("n_new"),
                                          stream=stream),
        "read": lambda: sv.sv_kv_read(cache, n("start"), 3, count=n("count"),
                                      layer=over.get("layer", 0), n_layers=over.get("n_layers", 1),
                                      k_out=at("k_out", (1, 2, 3, 2, 32), bf),
                                      v_out=at("v_out", (1, 2, 3, 2, 32), bf), stream=stream),
        "attend": lambda: sv.sv_kv_attend(
            cache, over.get("layer", 0), at("q", (2, 3, 4, 32), bf), n_new=n("n_new"),
            parent=at("parent", (2, 3), i32), window=over.get("window", 0),
            sinks=over.get("sinks", 0), out=at("out", (2, 3, 4, 32), bf),
            lse=at("lse", (2, 3, 4), f32), stream=stream),
        "commit": lambda: sv.sv_kv_commit(cache, n("accepted"), over.get("N", 3),
                                          path=at("path", (2, 3), i32), stream=stream),
        "fork": lambda: sv.sv_kv_fork(cache, n("src"), n("ok"), stream=stream),
    }


@pytest.mark.parametrize("call,name", [
    ("reserve", "n_new"), ("reserve", "ok"), ("append", "k"), ("append", "v"),
    ("append", "n_new"), ("read", "start"), ("read", "count"), ("read", "k_out"),
    ("read", "v_out"), ("attend", "q"), ("attend", "n_new"), ("attend", "parent"),
    ("attend", "out"), ("attend", "lse"), ("commit", "accepted"), ("commit", "path"),
    ("fork", "src"), ("fork", "ok")])
def test_tensors_of_another_device_are_refused(bind, call, name):
    sv, cache, lib = bind
    kv_calls(sv, cache)[call]()
    assert len(lib.calls) == 1
    with pytest.raises(ValueError, match=name + " must be on cuda:0"):
        kv_calls(sv, cache, dev=name)[call]()
    assert len(lib.calls) == 1


def test_calls_run_on_the_caches_device(bind, monkeypatch):
    """On its current stream or the one given; another current device or a stream of another
    device is refused."""
    sv, cache, lib = bind
    for call in kv_calls(sv, cache).values():
        call()
    assert len(lib.calls) == 6 and all(args[-1] == 55 for _, args in lib.calls)
    for call in kv_calls(sv, cache, stream=Stream()).values():
        call()
    assert all(args[-1] == 77 for _, args in lib.calls[6:])
    for call in kv_calls(sv, cache, stream=Stream(1)).values():
        with pytest.raises(ValueError, match="the stream on cuda:1"):
            call()
    monkeypatch.setattr(sv, "_current_device", lambda: 1)
    for call in (*kv_calls(sv, cache).values(), lambda: sv.KVCache.status(cache)):
        with pytest.raises(ValueError, match="not the current device"):
            call()
    assert len(lib.calls) == 12


@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32, 2 ** 40 + 5, -2 ** 31 - 1, -2 ** 32])
def test_integers_past_32_bits(bind, x):
    """Arguments of C ints never wrap into other values: the nearest end of the range, or a
    refusal of sizes."""
    sv, cache, lib = bind
    end = 2 ** 31 - 1 if x > 0 else -2 ** 31
    kv_calls(sv, cache, window=x, sinks=x, layer=x)["attend"]()
    args = lib.calls[-1][1]
    assert args[1] == end and args[11:13] == (end, end)
    kv_calls(sv, cache, layer=x)["append"]()
    assert lib.calls[-1][1][1] == end
    kv_calls(sv, cache, layer=x)["read"]()
    assert lib.calls[-1][1][1] == end
    sv.sv_kv_commit(cache, Tensor((2,), torch.int32), x)
    assert lib.calls[-1][1][3] == end


@pytest.mark.parametrize("name", ["layers", "pages", "page", "heads", "dim", "batch", "max_pages"])
def test_cache_sizes_past_32_bits(name):
    """A size that C would wrap to a supported one."""
    import speculative_decoding_verification_79_gb300 as sv

    sizes = dict(layers=1, pages=4, page=16, heads=1, dim=16, batch=1, max_pages=4)
    for wrap in (2 ** 32, -2 ** 32):
        with pytest.raises(ValueError, match="unsupported cache sizes"):
            sv.KVCache(**{**sizes, name: sizes[name] + wrap}, device="cpu")
