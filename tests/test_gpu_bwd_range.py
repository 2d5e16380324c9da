"""Range of the gradient: keys whose probability is far below that of the others, and dO near the ends of what fp32 sums hold."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import sink_ref as ref
from operator_ref import close

pytestmark = pytest.mark.gpu
SHAPES = [(64, 3, 1), (128, 4, 2), (256, 2, 1), (512, 2, 1), (512, 3, 1)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def rows(T, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv, Hq)]


@pytest.mark.parametrize("D,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 0), (100, 4), (30, 20)])
def test_keys_of_small_probability(D, Hq, Hkv, window, sink):
    """Every other key's scores are 10 to 80 nats below the rest, give or take a few: its dK and dV are right to the same relative bounds as
    those of the others, down to where fp32 ends.

    There (e^-87) the bounds get an absolute part: a P, or a product with one, below 2^-126 may count as zero, so a P is off by that besides, a
    dS by that times |dP - Delta| <= |dO| (|v| + |o|) and once more itself, and so are the terms of their sums over the queries that see the key."""
    S, scale = 400, 1 / math.sqrt(D)
    q, k, v, do = rows(S, Hq, Hkv, D, D + window)
    below = torch.linspace(10, 80, S)
    below[0::2] = 0
    q[..., 0], k[..., 0] = 4.0, (-below / (4 * scale))[:, None].bfloat16()
    want = ref.backward(q, k, v, do, scale, window, sink)
    a, b, c, d = (t.view(1, S, -1, D).cuda() for t in (q, k, v, do))
    o, lse = attn.attn_fwd(a, b, c, window=window, sink=sink, scale=scale)
    got = attn.attn_bwd(a, b, c, o, lse, d, window=window, sink=sink, scale=scale)
    assert attn.attn_get_device_status() == 0
    G, see = Hq // Hkv, ref.visible(S, S, window, sink).double()
    heads = lambda x: x.double().abs().transpose(0, 1).unflatten(0, (Hkv, G))  # noqa: E731  [Hkv, G, S, D]
    aq, ao, ad, av = heads(q), heads(o[0].cpu()), heads(do), v.double().abs().transpose(0, 1)[:, None]
    least = (see * (1 + (ad * ao).sum(3, keepdim=True) + ad @ av.transpose(2, 3))).transpose(2, 3) @ (1 + aq) * scale
    tiny = (0, 2.0 ** -126 * least.sum(1).transpose(0, 1), 2.0 ** -126 * (see.T @ (1 + ad)).sum(1).transpose(0, 1))
    for i, name in enumerate(("dq", "dk", "dv")):
        close(name, got[i].flatten(0, 1), want[2 * i], want[2 * i + 1] + tiny[i])
    # the bounds tell enough of these gradients from zero (one of 14 at least: over 512 dims the error of Delta takes up most of them)
    assert all((want[2 * i][1::2].abs() > want[2 * i + 1][1::2]).float().mean() > 0.05 for i in (1, 2))


@pytest.mark.parametrize("D,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 0), (100, 4), (1, 100)])
@pytest.mark.parametrize("power", [108, -70])
def test_scaled_dO(D, Hq, Hkv, window, sink, power):
    """The gradient is linear in dO, and a power of two changes no rounding: dK and dV are the same bits times it."""
    S = 700
    q, k, v, do = (t.view(1, S, -1, D).cuda() for t in rows(S, Hq, Hkv, D, 5))
    how = dict(window=window, sink=sink)
    o, lse = attn.attn_fwd(q, k, v, **how)
    want = attn.attn_bwd(q, k, v, o, lse, do, **how)
    got = attn.attn_bwd(q, k, v, o, lse, do * 2.0 ** power, **how)
    assert attn.attn_get_device_status() == 0
    assert torch.equal(got[1], want[1] * 2.0 ** power) and torch.equal(got[2], want[2] * 2.0 ** power)
    # (dQ's fp32 sums are in no fixed order)
    assert ((got[0].double() * 2.0 ** -power - want[0].double()).abs() <= 2.0 ** -7 * want[0].double().abs().max()).all()
