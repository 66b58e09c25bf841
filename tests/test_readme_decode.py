"""The 8-bit decode example in README.md runs as written."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_decode_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    text = open(os.path.join(ROOT, "README.md")).read()
    m = re.search(r"## Decoding over an 8-bit cache.*?```python\n(.*?)```", text, re.S)
    assert m, "example block not found"
    scope = {}
    exec(compile(m.group(1), "README.md", "exec"), scope)
    acc, tok, n = scope["accepted"].cpu(), scope["tokens"].cpu(), scope["n"]
    assert ((acc >= 0) & (acc <= n)).all()
    assert torch.equal(scope["lens"].cpu(), 5 + 1 + acc)
    assert torch.isfinite(scope["out"].float()).all() and scope["out"].abs().sum() > 0
    for r in range(scope["R"]):
        k = int(acc[r])
        assert (tok[r, :k + 1] >= 0).all() and (tok[r, k + 1:] == -1).all()
        assert torch.equal(tok[r, :k], scope["drafted"][r, :k].cpu())
