"""The arithmetic of the tree attention's ceil_div: rounding down (x + y - 1/2) / y in fp32 gives ceil(x / y) over its
stated range, for every quotient that is off by up to 2 ulp. Needs no GPU."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_flash_gqa_gb300", "csrc", "tree_paged.cu")


def wrong(x, y):
    """Whether 2 ulp of error either way can give another result than ceil(x / y)."""
    n = (x + y).astype(np.float32) - np.float32(0.5)
    assert np.array_equal(n.astype(np.float64), x + y - 0.5)
    q = n.astype(np.float64) / y
    near = q.astype(np.float32)
    ulp = np.spacing(near).astype(np.float64)
    want = -(-x // y)
    # the results that lie within 2 ulp of the exact quotient
    return (np.floor(q - 2 * ulp) != want) | (np.floor(q + 2 * ulp) != want)


def bound():
    m = re.search(r"kCeilDivSum = 1 << (\d+);", open(SOURCE).read())
    assert m, "the range is stated in the source"
    return 1 << int(m.group(1))


@pytest.mark.parametrize("y", [1, 2, 3, 5, 7, 12, 31, 76, 100, 152, 191, 255, 4097, 16384, 65535, 1 << 20])
def test_whole_range(y):
    top = bound() - y
    x = np.arange(0, top, max(1, top // 400_000), dtype=np.int64)
    k = np.arange(0, top // y + 1, max(1, top // y // 100_000), dtype=np.int64) * y  # around multiples of y
    x = np.concatenate([x, k, k + 1, k - 1, [top - 1, top - 2]])
    x = x[(x >= 0) & (x < top)]
    assert not wrong(x, y).any(), x[wrong(x, y)][:5]


def test_range_is_not_wider_than_the_margin():
    """Up to twice the stated range there are wrong results: the bound is not one to be stretched."""
    y = 3
    x = np.arange(3 * bound() // 2, 2 * bound() - y, dtype=np.int64)
    assert wrong(x, y).any()
