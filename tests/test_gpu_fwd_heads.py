"""Forward calls of many tiles, where a block takes several query heads one after the other: the bits of calls of few tiles, where it
takes one, and the 64-bit definition."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import sink_ref as ref
from operator_ref import close

pytestmark = pytest.mark.gpu
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def rows(T, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, D, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]


def tiles(Hq, n, S):
    return Hq * n * -(-S // 128)


# (D, Hq, Hkv, B, S, window, sink): one, two and more key tiles a query tile; heads that no number of heads a block divides, groups
# that begin inside a block; two and four heads a block
DENSE = [(64, 95, 5, 20, 97, 0, 0), (64, 95, 19, 40, 128, 0, 0), (64, 61, 61, 12, 700, 100, 4), (64, 96, 8, 6, 900, 0, 0),
         (128, 95, 5, 20, 1, 0, 0), (128, 96, 6, 20, 129, 0, 0), (128, 95, 19, 14, 300, 100, 17), (128, 33, 11, 15, 1000, 300, 0),
         (256, 97, 1, 40, 50, 0, 0), (256, 33, 11, 40, 200, 50, 3), (256, 62, 31, 10, 400, 130, 4), (256, 47, 47, 8, 1100, 0, 0)]


@pytest.mark.parametrize("D,Hq,Hkv,B,S,window,sink", DENSE)
def test_dense(D, Hq, Hkv, B, S, window, sink):
    assert tiles(Hq, B, S) >= 12 * SMS > tiles(Hq, 1, S)
    scale = 1 / math.sqrt(D)
    q, k, v = (x.view(B, S, -1, D) for x in rows(B * S, Hq, Hkv, D, S + D))
    how = dict(window=window, sink=sink, scale=scale)
    o, lse = attn.attn_fwd(q, k, v, **how)
    for b in range(B):
        one = attn.attn_fwd(q[b:b + 1].contiguous(), k[b:b + 1].contiguous(), v[b:b + 1].contiguous(), **how)
        assert torch.equal(o[b], one[0][0]) and torch.equal(lse[b], one[1][0]), b
    with torch.device("cuda"):
        want = ref.forward(q[B - 1], k[B - 1], v[B - 1], scale, window, sink)
    close("o", o[B - 1].cpu(), want[0].cpu(), want[1].cpu())
    close("lse", lse[B - 1].cpu(), want[2].cpu(), want[3].cpu())
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 41, 41), (128, 40, 8), (128, 42, 3), (256, 39, 13)])
@pytest.mark.parametrize("window,sink", [(0, 0), (1, 1), (100, 30)])
def test_packed(D, Hq, Hkv, window, sink):
    lens = [1, 0, 129, 400, 64, 128, 300, 2, 257, 390] * 3
    assert tiles(Hq, len(lens), 400) >= 24 * SMS
    T, scale = sum(lens), 1 / math.sqrt(D)
    q, k, v = rows(T + 5, Hq, Hkv, D, 7)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    how = dict(window=window, sink=sink, scale=scale)
    o = torch.full_like(q, 7.0)
    lse = torch.full((Hq, T + 5), 7.0, device="cuda")
    attn.attn_fwd_varlen(q, k, v, cu, 400, o, lse, **how)
    assert bool((o[T:] == 7.0).all()) and bool((lse[:, T:] == 7.0).all())
    at = 0
    for n in lens:
        if n:
            one = attn.attn_fwd(*(x[at:at + n].unsqueeze(0).contiguous() for x in (q, k, v)), **how)
            assert torch.equal(o[at:at + n], one[0][0]) and torch.equal(lse[:, at:at + n], one[1][0])
        at += n
    assert attn.attn_get_device_status() == 0


def test_bad_slices_are_reported():
    """One report each, nothing of them touched, the others computed: by blocks of several heads too."""
    D, Hq, lens = 128, 96, [129] * 30
    q, k, v = rows(sum(lens), Hq, 3, D, 3)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    want, _ = attn.attn_fwd_varlen(q, k, v, cu, 129)
    bad = cu.clone()
    bad[-1] += 1
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, sum(lens)), 7.0, device="cuda")
    attn.attn_fwd_varlen(q, k, v, bad, 129, o, lse)
    assert attn.attn_get_device_status() == 7
    at = sum(lens[:-1])
    assert torch.equal(o[:at], want[:at]) and bool((o[at:] == 7.0).all()) and bool((lse[:, at:] == 7.0).all())


def test_captured_and_on_two_streams():
    q, k, v = (x.view(20, 300, -1, 128) for x in rows(6000, 96, 6, 128, 9))
    want = attn.attn_fwd(q, k, v, window=130)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [attn.attn_fwd(q, k, v, window=130, stream=s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn.attn_fwd(q, k, v, window=130)
    for _ in range(2):
        got[0].zero_(), got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert attn.attn_get_device_status() == 0
