"""4-bit decode of many requests, whose pieces are joined by the pages that the decode kernel counted."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
from test_gpu_kv4 import check, gen, i32, problem, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


# around the number up to which the lengths are summed; more than the first kernel has threads; several KV heads; empty ones between all others
@pytest.mark.parametrize("D,Hkv,G", [(64, 3, 2), (128, 1, 8), (256, 2, 1)])
@pytest.mark.parametrize("B", [127, 128, 129, 257, 511, 513, 1500])
@pytest.mark.parametrize("window,sink", [(0, 0), (20, 3)])
def test_lengths(D, Hkv, G, B, window, sink):
    lens = torch.randint(0, 45, (B,), generator=gen(B + D))
    lens[::3] = 0
    lens[5] = 700
    check(*problem(lens.tolist(), Hkv, G, D, 23, window, sink), window, sink)


@pytest.mark.parametrize("D,B,Hkv", [(64, 129, 1), (128, 600, 4), (256, 4096, 2)])
def test_one_long_request_among_empty_ones(D, B, Hkv):
    """Every block has a piece of it; and no request has a key."""
    lens = [0] * B
    lens[B // 2] = 9000
    q, cache, table, n = problem(lens, Hkv, 2, D, 24)
    check(q, cache, table, n)
    o, lse = attn.attn_decode_kv4(q.cuda(), cache.cuda(), table.cuda(), i32([0] * B))
    assert not o.any() and (lse == -math.inf).all() and attn.attn_get_device_status() == 0


def test_more_segments_than_a_block_looks_at():
    """4096 requests of 60 KV heads: 246 thousand segments, more than a thread of the join's blocks has one of each."""
    B, Hkv, D = 4096, 60, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = torch.randint(0, 256, (300, Hkv, 18, D), generator=g, device="cuda", dtype=torch.uint8)
    cache.view(300, Hkv, 18 * D)[..., 16 * D:].view(torch.bfloat16).fill_(0.125)
    lens = torch.randint(0, 70, (B,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.randint(0, 300, (B, 5), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(B, 2 * Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
    o, lse = attn.attn_decode_kv4(q, cache, table, lens, scale=0.05)
    k, v = (x.transpose(1, 2) for x in attn.attn_kv4_unpack(cache, torch.arange(300, dtype=torch.int32, device="cuda")))  # [page, head, 16, D]
    for b in range(0, B, 97):
        n = int(lens[b])
        if n == 0:
            assert not o[b].any() and (lse[b] == -math.inf).all()
            continue
        kk, vv = (x[table[b].long()].transpose(0, 1).flatten(1, 2)[:, :n].double() for x in (k, v))
        s = torch.einsum("hgd,hnd->hgn", q[b].double().view(Hkv, 2, D), kk) * 0.05
        want = (s.softmax(-1) @ vv).view(-1, D)
        # P and the result round to bf16 (2^-8 each); scores of 64 products are off by 2^-24 of some hundreds
        assert ((o[b].double() - want).abs() <= 2.0 ** -8 * (want.abs() + (s.softmax(-1) @ vv.abs()).view(-1, D)) + 2.0 ** -12).all(), b
        assert ((lse[b].double() - s.logsumexp(-1).view(-1)).abs() <= 2.0 ** -12).all()
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("B", [300, 700])  # (up to 512 the layout is first made on a guess)
def test_workspace_and_chains(B):
    """In exactly the bytes that are named, whatever they hold; calls of different lengths one after the other in one workspace, and in a
    graph, lengths made by the kernel in front."""
    Hkv, G, D = 2, 2, 128
    lens = torch.randint(0, 60, (B,), generator=gen(1))
    q, cache, table, _ = problem([60] * B, Hkv, G, D, 25)
    q, cache, table = q.cuda(), cache.cuda(), table.cuda()
    need = attn.attn_workspace_size(attn.ATTN_OP_DECODE_KV4, B, Hkv * G, Hkv, 0, D)
    assert need >= attn.attn_workspace_size(attn.ATTN_OP_DECODE_KV4, 128, Hkv * G, Hkv, 0, D) + 4 * (B + 1)
    room = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    both = [i32(lens), i32(60 - lens)]
    want = [[t.clone() for t in attn.attn_decode_kv4(q, cache, table, n)] for n in both]
    torch.cuda.synchronize()
    n = both[0].clone()

    def run():
        out = []
        for x in both:
            n.copy_(x)
            out.append(attn.attn_decode_kv4(q, cache, table, n, workspace=room[:need]))
        n.zero_()
        return out

    for _ in range(3):
        assert all(same(a, b) for x, y in zip(run(), want) for a, b in zip(x, y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    assert bool((room[need:] == 255).all()) and attn.attn_get_device_status() == 0
    with pytest.raises(attn.AttnError):
        attn.attn_decode_kv4(q, cache, table, n, workspace=room[:need - 1])
