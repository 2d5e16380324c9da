"""Decode over the 4-bit cache directly behind the calls that write what it reads: lengths, block table and records may be their
results, and what stood there before does not count, also where the call in front lets it start early."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import kv4_ref as ref
from operator_ref import close
from test_gpu_decode_order import i32, written_by_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("what", ["lengths", "table", "records", "all"])
@pytest.mark.parametrize("Hq,Hkv,D,window,sink", [(8, 2, 128, 0, 0), (4, 4, 256, 0, 0), (16, 8, 64, 50, 4)])
def test_inputs_written_by_the_call_in_front(Hq, Hkv, D, window, sink, what, captured):
    R, cap, pages = 6, 10, 64
    g = torch.Generator().manual_seed(Hq + D)
    lens = [37, 0, 160, 5, 64, 1]
    ids = torch.randperm(pages, generator=g)[: R * cap].tolist()
    words = -(-max(R, R * cap) // 512)
    call_l, o_l = written_by_decode(lens, words)
    call_t, o_t = written_by_decode(ids, words)
    halves = pages * Hkv * 9 * D
    bits = torch.randint(0, 1 << 11, (halves,), generator=g, dtype=torch.int16) << 3  # bf16 values below 2, of 5 significant bits
    call_c, o_c = written_by_decode(bits.view(torch.int32).tolist(), -(-halves // 1024))
    old = torch.randint(0, 256, (pages, Hkv, 18, D), generator=g, dtype=torch.uint8).cuda()
    old.view(pages, Hkv, -1)[..., 16 * D:].view(torch.int16)[:] &= 0x3FF8
    q = torch.randn(R, Hq, D, generator=g).bfloat16().cuda()
    front = {"lengths": [call_l], "table": [call_t], "records": [call_c], "all": [call_t, call_c, call_l]}[what]
    lengths = o_l.flatten().view(torch.int32)[:R] if what in ("lengths", "all") else i32(lens)
    table = (o_t.flatten().view(torch.int32)[: R * cap] if what in ("table", "all") else i32(ids)).view(R, cap)
    cache = o_c.flatten().view(torch.uint8)[: 2 * halves].view(pages, Hkv, 18, D) if what in ("records", "all") else old
    o, lse = torch.empty_like(q), torch.empty(R, Hq, device="cuda")
    ws = torch.empty(attn.attn_workspace_size(attn.ATTN_OP_DECODE_KV4, R, Hq, Hkv, 0, D), dtype=torch.uint8, device="cuda")

    def run():
        for f in front:
            f()
        attn.attn_decode_kv4(q, cache, table, lengths, o, lse, scale=0.1, window=window, sink=sink, workspace=ws)

    run()
    torch.cuda.synchronize()
    assert attn.attn_get_device_status() == 0
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    assert lengths.tolist() == lens and table.flatten().tolist() == ids
    if cache is not old:
        assert torch.equal(cache.cpu().flatten().view(torch.int16), bits)
    want = ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens, 0.1, window, sink)
    for before in (0, 3, 160, -1, 2 ** 30, 7):  # as a length, and as a page id
        if what in ("lengths", "all"):
            lengths.fill_(before)
        if what in ("table", "all"):
            table.fill_(before)
        if what in ("records", "all"):
            cache.fill_(255)  # NaN scales
        o.fill_(5.0), lse.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay() if captured else run()
        assert attn.attn_get_device_status() == 0, before
        close("o", o, want[0], want[1])
        close("lse", lse, want[2], want[3])
        assert (o[1] == 0).all() and (lse[1] == -math.inf).all()


def test_steps_in_one_graph():
    """12 steps of one token each: plan in place, append, decode; replayed on other lengths, pages and tokens."""
    R, Hq, Hkv, D, steps, top = 37, 8, 2, 128, 12, 100
    cap = -(-(top + steps) // 16)
    pages = R * cap + 5
    g = torch.Generator().manual_seed(4)
    cache = torch.empty(pages, Hkv, 18, D, dtype=torch.uint8, device="cuda")
    lens, held, used, table = i32([0] * R), i32([0] * R), i32([0]), i32([[-1] * cap] * R)
    free, one = i32(list(range(pages))), i32([1] * R)
    rows = [[torch.empty(R, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)] for _ in range(steps)]
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = attn.PagedPlan(lens, e(R + 1), e(R), e(R), held, used, e(1))
    got = []

    def loop():
        del got[:]
        for q, k, v in rows:
            attn.attn_paged_plan(lens, one, free, table, held, used, R, num_pages=pages, out=out)
            attn.attn_kv4_append(k, v, out.slots, cache)
            got.append(attn.attn_decode_kv4(q, cache, table, lens, scale=0.1))

    def start(seed):
        g.manual_seed(seed)
        n = torch.randint(1, top, (R,), generator=g).tolist()
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        free.copy_(perm)
        ids, at = [], 0
        for x in n:
            need = -(-x // 16)
            ids.append(perm[at: at + need].tolist() + [-1] * (cap - need))
            at += need
        lens.copy_(i32(n)), held.copy_(i32([-(-x // 16) for x in n])), used.fill_(at), table.copy_(i32(ids))
        new = torch.randint(0, 256, cache.shape, generator=g, dtype=torch.uint8)
        new.view(pages, Hkv, -1)[..., 16 * D:].view(torch.int16)[:] &= 0x3FF8
        cache.copy_(new)
        for t in rows:
            for x in t:
                x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        return n, new

    start(1)
    loop()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    for seed in (2, 3):
        n, state = start(seed)
        torch.cuda.synchronize()
        graph.replay()
        assert attn.attn_get_device_status() == 0
        assert lens.tolist() == [x + steps for x in n]
        ids = table.cpu()
        for s, (q, k, v) in enumerate(rows):
            at = [int(ids[b, (x + s) // 16]) * 16 + (x + s) % 16 for b, x in enumerate(n)]
            ref.put(state, at, k.cpu(), v.cpu())
            want = ref.decode(q.cpu(), state, ids, [x + s + 1 for x in n], 0.1)
            close(f"o {s}", got[s][0], want[0], want[1])
            close(f"lse {s}", got[s][1], want[2], want[3])
        assert torch.equal(cache.cpu(), state)


def test_threads_on_their_own_streams():
    """Threads that call with different numbers of requests and heads at the same time: the kernel's settings are every call's."""
    import threading

    def one(k, D, G):
        try:
            torch.cuda.set_device(0)
            g = torch.Generator().manual_seed(k)
            R, Hkv = 3 + 40 * k, 2
            cache = ref.put(torch.zeros(R * 2, Hkv, 18, D, dtype=torch.uint8), torch.arange(R * 32), *(torch.randn(R * 32, Hkv, D, generator=g).bfloat16() for _ in range(2)))
            q, table, lens = torch.randn(R, G * Hkv, D, generator=g).bfloat16(), torch.arange(2 * R, dtype=torch.int32).view(R, 2), [1 + (7 * b) % 32 for b in range(R)]
            want = ref.decode(q, cache, table, lens, 0.1)
            dev = [x.cuda() for x in (q, cache, table)] + [i32(lens)]
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.default_stream())
            for _ in range(60):
                got = attn.attn_decode_kv4(*dev, scale=0.1, stream=s)
            s.synchronize()
            close("o", got[0], want[0], want[1])
            close("lse", got[1], want[2], want[3])
        except BaseException as e:  # noqa: BLE001
            failed.append(repr(e))

    failed = []
    torch.cuda.synchronize()
    jobs = [threading.Thread(target=one, args=(k, D, G)) for k, (D, G) in enumerate([(128, 8), (128, 1), (64, 3), (256, 2), (128, 4)])]
    [j.start() for j in jobs], [j.join() for j in jobs]
    assert not failed and attn.attn_get_device_status() == 0
