"""CPU checks of how the cache calls keep devices, streams and integer ranges apart."""
import os
import subprocess

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
