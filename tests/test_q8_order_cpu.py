"""What the kernels over the 8-bit cache do before and after they have waited
for the launch ahead (they may begin before it has ended), from their source:
a wrong order could only be seen on a GPU as a hang."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_kv_block_gb300", "csrc")


def kernels(name):
    """(kernel name, body without comments) of each __global__ function of a file."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    out = []
    for m in re.finditer(r"__global__.*?\b(\w+)\s*\(\s*const \w+Args", text, re.S):
        body = text.index("{", m.end())
        depth, at = 1, body + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        out.append((m.group(1), text[body:at]))
    return out


def test_every_kernel_waits_for_the_launch_ahead():
    seen = []
    for f in ("q8.cu", "q8_attn.cu", "prefix.cu", "verify.cu"):
        for name, body in kernels(f):
            seen.append(name)
            assert "previous_done()" in body and "next_may_begin()" in body, (f, name)
            assert body.index("previous_done()") < body.index("next_may_begin()"), (f, name)
    assert sorted(seen) == ["attn_kernel", "join_kernel", "join_parts", "prefix_kernel", "read_kernel",
                            "verify_kernel", "write_kernel"]


@pytest.mark.parametrize("call", ["tmem_alloc(", "mbar_init(", "load(", "a.q"])
def test_prefix_takes_nothing_before_it_has_waited(call):
    """Tensor memory least of all: a kernel ahead that lets its dependents begin and takes its own
    afterwards would wait for this one, which waits for it."""
    body = dict(kernels("prefix.cu"))["prefix_kernel"]
    body = re.sub(r"auto load = .*?\};", "", body, flags=re.S)
    assert body.index("previous_done()") < body.index(call)
