"""Forward and gradient read what the kernels in front of them write, and what follows them reads theirs: in a stream without
synchronisation and in a graph (they are launched with programmatic serialisation)."""
import pytest
import torch

import attention_flash_gqa_gb300 as attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


# short calls and calls of many tiles; with sinks' parts; pages. 512: the kernels in clusters between them
CASES = [(64, 3, 1, 1, 200, 100, 1), (128, 4, 2, 2, 700, 60, 4), (128, 96, 6, 20, 129, 0, 0), (256, 2, 1, 1, 400, 30, 20),
         (256, 32, 16, 1, 4200, 300, 4), (512, 4, 2, 1, 300, 50, 4), (512, 3, 1, 1, 300, 0, 0)]


@pytest.mark.parametrize("D,Hq,Hkv,B,S,window,sink", CASES)
@pytest.mark.parametrize("captured", [False, True])
def test_chain(D, Hq, Hkv, B, S, window, sink, captured):
    """q, k, v and dO are written, the cu_seqlens too, a step runs, and its results are copied and cleared: again and again."""
    T, rounds = B * S, 6
    g = torch.Generator(device="cuda").manual_seed(D + S)
    data = [[torch.randn(T, h, D, generator=g, device="cuda", dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq)] for _ in range(rounds)]
    at = dict(window=window, sink=sink)
    cu = torch.arange(0, T + 1, S, dtype=torch.int32, device="cuda")

    def step(q, k, v, do, cu):
        o, lse = attn.attn_fwd_varlen(q, k, v, cu, S, **at)
        return [o, lse, *attn.attn_bwd(q, k, v, o, lse, do, cu_seqlens=cu, max_seqlen=S, **at)]

    want = []
    for x in data:
        want.append([t.clone() for t in step(*x, cu)])
        torch.cuda.synchronize()
    q, k, v, do, given = (torch.zeros_like(t) for t in (*data[0], cu))
    src = [torch.empty_like(t) for t in data[0]]

    def chained():
        given.copy_(cu)
        for a, b in zip((q, k, v, do), src):
            a.copy_(b)
        out = step(q, k, v, do, given)
        kept = [t.clone() for t in out]
        for t in (*out, q, k, v, do, given):
            t.zero_()
        return kept

    graph = None
    if captured:
        for a, b in zip(src, data[0]):
            a.copy_(b)
        chained()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = chained()
    got = []
    for x in data:
        for a, b in zip(src, x):
            a.copy_(b)
        if graph is not None:
            graph.replay()
        else:
            kept = chained()
        got.append([t.clone() for t in kept])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for i in (0, 1, 3, 4):
            assert torch.equal(a[i], b[i])
        # dQ's fp32 sums are in no fixed order
        assert (a[2].float() - b[2].float()).abs().max() <= 2.0 ** -7 * b[2].float().abs().max()
    assert attn.attn_get_device_status() == 0


def test_plan_then_chunk_then_decode():
    """The step plan's outputs are read by the chunk's forward and the decode behind it, in one graph replayed over changing lengths."""
    D, Hkv, Hq = 128, 2, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    kc, vc = (torch.randn(64, 16, Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.randperm(60, generator=g, device="cuda").to(torch.int32).view(3, 20)
    q = torch.randn(96, Hq, D, generator=g, device="cuda", dtype=torch.bfloat16)
    lens, cu = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    new, n = torch.tensor([32, 32, 32], dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")

    def step():
        lens.copy_(n + new)
        cu[1:].copy_(new.cumsum(0))
        o, lse = attn.attn_fwd_paged(q, kc, vc, table, lens, cu, 32, window=50, sink=3)
        return o, lse, *attn.attn_decode_paged(q[:3].contiguous(), kc, vc, table, lens, window=50, sink=3)

    n.copy_(torch.tensor([5, 100, 200], dtype=torch.int32))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for now in ([0, 0, 0], [17, 250, 3], [288, 1, 90]):
        n.copy_(torch.tensor(now, dtype=torch.int32))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("D", [64, 256, 512])
def test_captured_with_two_streams(D):
    """Inputs made on two streams that join in front of the call, and its results used on both."""
    g = torch.Generator(device="cuda").manual_seed(D)
    src = [torch.randn(1, 500, h, D, generator=g, device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2, 4)]
    q, k, v, do = (torch.zeros_like(t) for t in src)
    how = dict(window=70, sink=4)

    def step(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q.copy_(src[0]), do.copy_(src[3])
        k.copy_(src[1]), v.copy_(src[2])
        main.wait_stream(side)
        o, lse = attn.attn_fwd(q, k, v, **how)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            twice = o * 2
        grads = attn.attn_bwd(q, k, v, o, lse, do, **how)
        main.wait_stream(side)
        return [twice, lse, *grads[1:]]

    side = torch.cuda.Stream()
    want = [t.clone() for t in step(side)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(side)
    for _ in range(3):
        for t in (q, k, v, do, *got):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert attn.attn_get_device_status() == 0
