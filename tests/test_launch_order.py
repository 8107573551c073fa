"""Every kernel of the cache may be brought up while the one before it in the stream still runs, so
it reads nothing of the call before it has waited for that one, or has taken over what that one
waited for (kv_enter_behind). Checked in the sources: on a GPU such a mistake shows by chance."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_79_gb300", "csrc")
READS = r"kv_ld\(|__ldcg\(|\bat_count\b|\bat_large\(|\bat_row\b|\bA\.S\.|\bA\.H\.|\bC\.(len|np|table|refs)\b"


def body(text, at):
    """The block that opens at or after `at`, with its braces."""
    start = at = text.index("{", at)
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        at += 1
        if depth == 0:
            return text[start:at]


def kernels():
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "sv_kv*")) + glob.glob(os.path.join(CSRC, "sv_rope*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            name = re.search(r"\b(\w*kernel)\(", text[m.end():]).group(1)
            out.append(pytest.param(body(text, text.index(name + "(", m.end())), id=name))
    return out


@pytest.mark.parametrize("code", kernels())
def test_kernels_wait_before_they_read(code):
    enter, read = re.search(r"\bkv_enter\w*\(", code), re.search(READS, code)
    assert enter, "never waits for the launch before it"
    # (An argument of the entry itself is an address, not a read.)
    assert read is None or enter.start() < read.start()
    if "kv_enter_behind" in enter.group():
        assert code.rstrip("} \n").endswith('asm volatile("griddepcontrol.wait;" ::: "memory");')
        for m in re.finditer(r"\breturn;", code):
            assert code[:m.start()].rstrip().endswith('asm volatile("griddepcontrol.wait;" ::: "memory");')


def test_entries():
    common = open(os.path.join(CSRC, "sv_kv.cuh")).read()
    share = open(os.path.join(CSRC, "sv_kv_share.cuh")).read()
    wait = "griddepcontrol.wait"
    for text, name in ((common, "kv_enter("), (share, "kv_enter_ready(")):
        code = body(text, text.index(" " + name))
        assert wait in code and code.index(wait) < code.index("launch_dependents")
    code = body(share, share.index(" kv_enter_ready("))
    assert code.index(wait) < code.index("st.release.gpu") < code.index("launch_dependents")
    code = body(share, share.index(" kv_enter_behind("))
    assert code.index("atom.exch.acq_rel.gpu") < code.index("if (!take())") < code.index(wait)
