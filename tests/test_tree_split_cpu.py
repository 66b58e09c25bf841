"""What is left of a query row that the tree attention splits into e4m3 rows
times a power of two, over every entry that a row can have."""
import math
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype,terms,bits,exact", [(torch.bfloat16, 2, 8, 9), (torch.float16, 3, 11, 6)])
def test_what_the_split_loses(dtype, terms, bits, exact):
    """A row is scaled so that its largest entry is in (224, 448]; an entry is any significand times
    a power of two up to that."""
    significands = 1 + torch.arange(1 << (bits - 1), dtype=torch.float64) / (1 << (bits - 1))
    assert torch.equal(significands.to(dtype).double(), significands)
    x = torch.cat([significands * 2.0 ** e for e in range(-24, 9)])
    x = x[x <= 448]
    left = x.clone()
    for _ in range(terms):
        left = left - left.to(torch.float8_e4m3fn).double()
    # The least largest entry that goes with x: x itself, or the first number above 224.
    top = torch.maximum(x, torch.tensor(224 * (1 + 2.0 ** (1 - bits) / 1.75), dtype=torch.float64))
    worst = (left.abs() / top).max().item()
    assert worst <= 2.0 ** -17.8 < 1.02 * worst
    inexact = x[left != 0]
    # An entry within 2^-exact of any largest one is exact (and not all within half of that are).
    assert inexact.max() < 224 * 2.0 ** -exact and inexact.max() > 224 * 2.0 ** -(exact + 1)


def test_the_header_says_so():
    text = " ".join(open(os.path.join(ROOT, "include", "oasis.h")).read().replace("\n *", "\n").split())
    assert "a query's entries count to 2^-17.8 of its row's largest (exactly those within 2^-9 of it in bf16, 2^-6 in fp16)" in text
    assert math.log2(2.0 ** -10 / 224) < -17.8
