"""What the kernels of a tree step do before and after they have waited for the
launch ahead, from their source: a wrong order could only be seen on a GPU as a
hang."""
import re

from tests.test_q8_order_cpu import kernels


def test_every_kernel_waits_for_the_launch_ahead():
    seen = []
    for f in ("append.cu", "tree.cu", "logprobs.cu"):
        for name, body in kernels(f):
            seen.append(name)
            assert "previous_done()" in body and "next_may_begin()" in body, (f, name)
            assert body.index("previous_done()") < body.index("next_may_begin()"), (f, name)
            first = re.search(r"a\.\w+", body)
            assert first is None or "previous_done()" in body[:first.start()], (f, name)
    assert sorted(seen) == ["append_kernel", "keep_kernel", "logprobs_kernel", "tree_join", "tree_kernel"]


def test_tensor_memory_is_taken_between_the_two():
    """A kernel ahead that lets its dependents begin and takes its own afterwards would wait for
    this one, which waits for it; and so would this one for the kernel behind."""
    body = dict(kernels("tree.cu"))["tree_kernel"]
    assert body.index("previous_done()") < body.index("tmem_alloc(") < body.index("next_may_begin()")
    assert body.index("tmem_free(") > body.rindex("mbar_wait(")
