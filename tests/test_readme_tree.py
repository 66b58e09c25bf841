"""The example of a tree step in README.md runs as written."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_tree_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    text = open(os.path.join(ROOT, "README.md")).read()
    m = re.search(r"## Decoding trees of drafted tokens.*?```python\n(.*?)```", text, re.S)
    assert m, "example block not found"
    scope = {}
    exec(compile(m.group(1), "README.md", "exec"), scope)
    assert torch.isfinite(scope["out"].float()).all() and scope["out"].abs().sum() > 0
    assert all(p[:2] == [0, 1] for p in scope["paths"])
    assert scope["lens"].tolist() == [len(p) for p in scope["paths"]]
    # The kept tokens are the path's nodes: read back, they are the appended values, rounded to codes.
    units = torch.empty(scope["R"], scope["Hkv"], 1, 2, 16, 128, device="cuda")
    scope["cache"].oasis_q8_read(scope["table"], scope["lens"], units)
    v = scope["v"].view(scope["R"], scope["N"], scope["Hkv"], 128).float()
    for r, path in enumerate(scope["paths"]):
        for i, n in enumerate(path):
            off = (units[r, :, 0, 1, i] - v[r, n]).abs()
            top = v[r, n].abs().amax(-1, keepdim=True)
            assert (off <= torch.maximum(v[r, n].abs() * 2 ** -4, top * 2 ** -17)).all()
