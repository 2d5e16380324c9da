"""Scratch and results of the calls belong to the call: gradients and decode steps on two streams and in two threads at once, in a
captured graph that is replayed after larger calls, and on a stream that is given."""
import threading

import pytest
import torch

import attention_flash_gqa_gb300 as attn


@pytest.fixture(scope="module")
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def gradient(D, S, seed, **how):
    """A gradient call of its own data: f(stream), and the indices of its results that are the same bits every time."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn(1, S, h, D, generator=g, device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2, 4))
    o, lse = attn.attn_fwd(q, k, v, **how)
    return lambda stream=None: attn.attn_bwd(q, k, v, o, lse, do, stream=stream, **how)


def decode(D, B, L, seed, **how):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-L // 16)
    kc, vc = (torch.randn(B * pages, 16, 2, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(B, 8, D, generator=g, device="cuda", dtype=torch.bfloat16)
    table = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    return lambda stream=None: attn.attn_decode_paged(q, kc, vc, table, lens, stream=stream, **how)


def same(got, want):
    if len(got) == 3:  # dQ's fp32 sums are in no fixed order
        return torch.equal(got[1], want[1]) and torch.equal(got[2], want[2]) and bool(
            (got[0].float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max())
    return all(torch.equal(a, b) for a, b in zip(got, want))


CALLS = {
    "gradient 64": lambda s: gradient(64, 3000, s), "gradient 128 window": lambda s: gradient(128, 2500, s, window=300),
    "gradient 256": lambda s: gradient(256, 1500, s), "gradient 512": lambda s: gradient(512, 900, s),
    "gradient sinks": lambda s: gradient(128, 2500, s, window=300, sink=4), "decode 128": lambda s: decode(128, 3, 20000, s),
    "decode 256 window": lambda s: decode(256, 5, 9000, s, window=3000), "decode sinks": lambda s: decode(128, 3, 9000, s, window=3000, sink=4),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_two_streams(_built, name):
    calls = [CALLS[name](s) for s in (1, 2)]
    want = [[t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = [[f(s) for f, s in zip(calls, streams)] for _ in range(3)]
        torch.cuda.synchronize()
        assert all(same(a, b) for g in got for a, b in zip(g, want))
    assert attn.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["gradient 128 window", "decode 128"])
def test_two_threads(_built, name):
    calls = [CALLS[name](s) for s in (3, 4)]
    want = [[t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    found = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [calls[i]() for _ in range(20)]
        s.synchronize()
        found[i] = all(same(g, want[i]) for g in got)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert found == [True, True] and attn.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("small,large", [(lambda: gradient(128, 500, 5), lambda: gradient(128, 9000, 6)),
                                         (lambda: gradient(512, 300, 5, window=100), lambda: gradient(512, 2000, 6)),
                                         (lambda: decode(128, 2, 700, 5), lambda: decode(128, 200, 900, 6))])
def test_replay_after_larger_calls(_built, small, large):
    """A captured call keeps its scratch, whatever is allocated and freed after it."""
    f, big = small(), large()
    want = [t.clone() for t in f()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    for _ in range(3):
        big()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 21, 1 << 25, 1 << 28)]
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want) and all(bool((t == 255).all()) for t in held)
        del held
    assert attn.attn_get_device_status() == 0


def large(stream):
    """Calls with results of several MB (the allocator keeps blocks of that size apart): {name: results}."""
    x = [torch.zeros(1, 4096, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    flat, parts = [t[0] for t in x], torch.zeros(2, 1, 4096, 16, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 4096], dtype=torch.int32, device="cuda")
    kc = x[0].view(256, 16, 16, 128)
    table, lens = torch.arange(256, dtype=torch.int32, device="cuda")[None], torch.tensor([4096], dtype=torch.int32, device="cuda")
    many = table.expand(4096, 256)[:, :1].contiguous(), torch.ones(4096, dtype=torch.int32, device="cuda")
    lse_parts = torch.zeros(2, 1, 16, 4096, device="cuda")
    torch.cuda.synchronize()
    o, lse = attn.attn_fwd(*x[:3])
    torch.cuda.synchronize()
    yield "fwd", lambda: attn.attn_fwd(*x[:3], stream=stream)
    yield "fwd sinks", lambda: attn.attn_fwd(*x[:3], window=99, sink=4, stream=stream)
    yield "bwd", lambda: attn.attn_bwd(*x[:3], o, lse, x[3], stream=stream)
    yield "bwd sinks", lambda: attn.attn_bwd(*x[:3], o, lse, x[3], window=99, sink=4, stream=stream)
    yield "varlen", lambda: attn.attn_fwd_varlen(*flat[:3], cu, 4096, stream=stream)
    yield "paged", lambda: attn.attn_fwd_paged(flat[0], kc, kc, table, lens, cu, 4096, stream=stream)
    yield "decode", lambda: attn.attn_decode_paged(flat[0], kc, kc, *many, stream=stream)
    yield "merge", lambda: attn.attn_merge_lse(parts, lse_parts, stream=stream)


@pytest.mark.gpu
@pytest.mark.parametrize("external", [False, True])
def test_results_belong_to_the_given_stream(_built, external):
    """What a call allocates is of the stream that it runs on: freed, it is not handed out again on the caller's current stream (where
    nothing waits for the call's kernels)."""
    s = torch.cuda.Stream()
    if external:
        class Other:  # what only has the handle
            cuda_stream = s.cuda_stream
    for name, call in large(Other() if external else s):
        got = call()
        old = {t.data_ptr() for t in got if t.nbytes > 1 << 20}
        shapes = [t.shape for t in got if t.nbytes > 1 << 20]
        assert old, name
        del got
        new = [torch.empty(x, dtype=torch.bfloat16, device="cuda") for x in shapes for _ in range(8)]
        assert not old & {t.data_ptr() for t in new}, name
        torch.cuda.synchronize()
    assert attn.attn_get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sink", [0, 4])
def test_buffers_of_a_larger_batch(_built, sink):
    """Results and lengths may be contiguous buffers of another shape or with room for more; what does not hold the call is refused."""
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v, do = (torch.randn(2, 300, h, 128, generator=g, device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2, 4))
    how = dict(window=100, sink=sink)
    want = attn.attn_fwd(q, k, v, **how)
    room, few = torch.zeros(3, 300, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 300, 511, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(5000, device="cuda")
    o, got = attn.attn_fwd(q, k, v, room, lse, **how)
    assert o is room and got is lse and torch.equal(room[:2].view_as(q), want[0]) and not room[2].any()
    assert torch.equal(lse[:2400].view(2, 4, 300), want[1]) and not lse[2400:].any()
    a = attn.attn_bwd(q, k, v, room, lse, do.flatten(2), **how)
    b = attn.attn_bwd(q, k, v, *want, do, **how)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    for bad in (dict(o=few), dict(lse=lse[:2399]), dict(o=room.float()), dict(o=room.transpose(0, 1))):
        with pytest.raises(ValueError):
            attn.attn_fwd(q, k, v, **bad, **how)
    kc = k.reshape(-1)[:2 * 16 * 16 * 2 * 128].view(32, 16, 2, 128)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(5, 8) % 32
    lens = torch.tensor([100, 128, 3, 7, 9], dtype=torch.int32, device="cuda")
    qd = q[0, :2].contiguous()
    want = attn.attn_decode_paged(qd, kc, kc, table[:2].contiguous(), lens[:2].contiguous(), **how)
    o = torch.zeros(5, 512, dtype=torch.bfloat16, device="cuda")
    got = attn.attn_decode_paged(qd, kc, kc, table, lens, o, torch.zeros(9, device="cuda"), **how)
    assert torch.equal(o[:2].view_as(qd), want[0]) and torch.equal(got[1][:8].view(2, 4), want[1]) and not o[2:].any()
    for bad in (dict(block_table=table[:1]), dict(seq_lens=lens[:1]), dict(seq_lens=lens.long())):
        with pytest.raises(ValueError):
            attn.attn_decode_paged(qd, kc, kc, **{"block_table": table, "seq_lens": lens, **bad}, **how)
    assert attn.attn_get_device_status() == 0


@pytest.mark.gpu
def test_without_the_native_part(_built, monkeypatch):
    """Calls without sinks go to the C library where the binding's native part is missing, with the same results."""
    f, d = gradient(128, 500, 8), decode(128, 3, 400, 8)
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = (torch.randn(1, 300, h, 64, generator=g, device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2))
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    calls = [f, d, lambda stream=None: attn.attn_fwd(q, k, v, window=50, stream=stream),
             lambda stream=None: attn.attn_fwd_varlen(q[0], k[0], v[0], cu, 200, stream=stream)]
    want = [c() for c in calls]

    def missing():
        raise RuntimeError("missing")

    monkeypatch.setattr(attn, "_bound", None)
    monkeypatch.setattr(attn, "_unbound", False)
    monkeypatch.setattr(attn, "_native", missing)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        a, b = c(), c(s)
        torch.cuda.synchronize()
        assert same(a, w) and same(b, w)
    with pytest.raises(RuntimeError, match="missing"):
        attn.attn_fwd(q, k, v, window=50, sink=4)
    assert attn.attn_get_device_status() == 0


def test_stream_of_another_device_is_refused(monkeypatch):
    """(Without a GPU: the kernels would run on the stream's device, over the tensors of another.)"""
    class Fake:
        device = torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "Stream", Fake)
    with pytest.raises(ValueError):
        attn._on(Fake(), torch.device("cuda", 0))
