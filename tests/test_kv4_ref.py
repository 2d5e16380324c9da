"""The 4-bit cache's plain code: the rounding by hand, its bounds, the layout as a bijection. Needs no GPU."""
import math

import pytest
import torch

import kv4_ref as ref


def test_by_hand():
    x = torch.zeros(32, dtype=torch.float64)
    x[0], x[1], x[2], x[3] = 8, -7, 3.5, 2.5  # s = -1
    n, s = ref.quantise(x)
    assert s.item() == -1 and n[:4].tolist() == [-8, 7, -4, -2]  # -3.5 and -2.5 go to the even neighbour
    x[0] = -8
    n, s = ref.quantise(x)
    assert s.item() == 1 and n[:4].tolist() == [-8, -7, 4, 2]
    x[1] = 8
    n, s = ref.quantise(x)
    assert s.item() == 1 and n[:2].tolist() == [-8, 7]  # of the two the negative one counts
    x[:] = 0
    x[5] = -8.25  # 33 / 32: between 32 and 34 of 32, to the even one
    assert ref.quantise(x)[1].item() == 1
    x[5] = -8.75
    assert ref.quantise(x)[1].item() == 1.125  # 35 / 32: between 34 and 36
    x[5] = math.inf
    assert ref.values(x).isnan().all()
    x[5] = 1e-40
    assert (ref.values(x) == 0).all()


def test_half_a_step():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(500, 128, generator=g) * torch.exp(4 * torch.randn(500, 1, generator=g))).bfloat16()
    n, s = ref.quantise(x)
    v = n * s.repeat_interleave(32, -1)
    assert torch.equal(v.bfloat16().double(), v)  # bf16 numbers
    # half a step, but the largest value, which s rounds away from by up to 1 / 32 of 8 steps, and values above 7.5 steps
    assert ((v - x.double()).abs() <= (0.5 * s.abs()).repeat_interleave(32, -1) * (1 + 1e-12) + ((n == 7) | (n == -8)) * s.abs().repeat_interleave(32, -1) * 0.8).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout(D):
    key, value, sk, sv = ref.places(D)
    assert sorted(torch.cat([key.flatten(), value.flatten()]).tolist()) == list(range(32 * D))
    assert sorted(torch.cat([sk.flatten(), sv.flatten()]).tolist()) == list(range(16 * D, 18 * D, 2))
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(20, 2, D, generator=g).bfloat16() for _ in range(2))
    slots = torch.randperm(48, generator=g)[:20]
    K, V = ref.get(ref.put(torch.zeros(3, 2, 18, D, dtype=torch.uint8), slots, k, v))
    assert torch.equal(K.flatten(0, 1)[slots], ref.values(k)) and torch.equal(V.flatten(0, 1)[slots], ref.values(v))
