"""The 64-bit definition of windowed attention with sinks against automatic differentiation, differences and its
special cases. Needs no GPU."""
import math

import pytest
import torch

import sink_ref as ref


def inputs(n, Hq, Hkv, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h: torch.randn(n, h, D, generator=g, dtype=torch.float64)  # noqa: E731
    return r(Hq), r(Hkv), r(Hkv), r(Hq)


def loss(q, k, v, do, scale, window, sink):
    G = q.shape[1] // k.shape[1]
    see = ref.visible(len(q), len(q), window, sink)
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(G, 1)) * scale
    return (torch.einsum("hij,jhd->ihd", s.masked_fill(~see, -math.inf).softmax(-1), v.repeat_interleave(G, 1)) * do).sum()


def test_visible_by_hand():
    assert ref.visible(5, 5, 2, 1).int().tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert ref.visible(2, 5, 1, 2).int().tolist() == [[1, 1, 0, 1, 0], [1, 1, 0, 0, 1]]
    assert torch.equal(ref.visible(9, 9, 0, 4), ref.visible(9, 9, 9, 0)) and torch.equal(ref.visible(9, 9, 3, 9), ref.visible(9, 9, 0, 0))


@pytest.mark.parametrize("n,window,sink", [(1, 1, 1), (12, 3, 2), (12, 1, 4), (9, 20, 3), (12, 4, 0), (12, 0, 5)])
def test_gradient(n, window, sink):
    x = inputs(n, 4, 2, 8)
    scale = 0.3
    got = ref.backward(*x, scale, window, sink)[::2]
    leaves = [t.clone().requires_grad_() for t in x[:3]]
    loss(*leaves, x[3], scale, window, sink).backward()
    for a, b in zip(got, leaves):
        assert (a - b.grad).abs().max() < 1e-12
    g = torch.Generator().manual_seed(1)
    d = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in x[:3]]
    h = 1e-5
    up, down = (loss(*(t + w * h * e for t, e in zip(x[:3], d)), x[3], scale, window, sink) for w in (1, -1))
    assert abs((up - down) / (2 * h) - sum((a * e).sum() for a, e in zip(got, d))) < 1e-7
