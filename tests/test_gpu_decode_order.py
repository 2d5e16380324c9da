"""Decode directly behind the calls that write what it reads: every step of a captured loop (plan in place, head norm
into the pages, decode) sees that step's lengths, block table and pages, and a decode call without work does not let
the kernel behind it run before the one in front of it has finished. Where a call in front lets decode start early, what
decode reads before that call's end does not count."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import operator_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("R,Hq,Hkv,D,window", [(5, 8, 2, 128, 0), (37, 4, 2, 256, 60), (70, 8, 8, 128, 0), (256, 4, 1, 128, 0), (257, 4, 1, 128, 0)])
def test_steps_in_one_graph(R, Hq, Hkv, D, window):
    """18 steps of one token each in a graph, replayed on other lengths, pages and tokens: unwritten slots hold NaN and
    the block table -1, so a step that saw an older state would show it."""
    steps, top, rot = 18, 150, 64
    pages = R * (-(-(top + steps) // 16)) + 9
    g = torch.Generator().manual_seed(R + D)
    cs = ref.table(256, rot).cuda()
    kc, vc = (torch.empty(pages, 16, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cap = -(-(top + steps) // 16)
    lens, held, used, table = i32([0] * R), i32([0] * R), i32([0]), i32([[-1] * cap] * R)
    free, one = i32(list(range(pages))), i32([1] * R)
    qkv = [[torch.empty(R, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)] for _ in range(steps)]
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = attn.PagedPlan(lens, e(R + 1), e(R), e(R), held, used, e(1))
    before = e(R)
    got = []

    def loop():
        del got[:]
        for q, k, v in qkv:
            attn.attn_paged_plan(lens, one, free, table, held, used, R, num_pages=pages, out=out)
            qo = attn.attn_qk_norm_rope_paged(q, k, v, None, None, out.positions, out.slots, cs, kc, vc, eps=EPS)
            now = attn.attn_decode_paged(qo, kc, vc, table, lens, window=window, scale=0.1)
            torch.sub(lens, 1, out=before)  # lengths written by a kernel directly in front
            got.append((qo, now, attn.attn_decode_paged(qo, kc, vc, table, before, window=window, scale=0.1)))

    def start(seed):
        g.manual_seed(seed)
        n = torch.randint(1, top, (R,), generator=g).tolist()
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        free.copy_(perm)
        rows, at = [], 0
        for x in n:
            need = -(-x // 16)
            rows.append(perm[at: at + need].tolist() + [-1] * (cap - need))
            at += need
        lens.copy_(i32(n)), held.copy_(i32([-(-x // 16) for x in n])), used.fill_(at), table.copy_(i32(rows))
        kc.fill_(math.nan), vc.fill_(math.nan)
        for r, x in zip(rows, n):
            for p in range(-(-x // 16)):
                m = min(16, x - 16 * p)
                kc[r[p], :m], vc[r[p], :m] = (torch.randn(m, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
        for t in qkv:
            for x in t:
                x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        return n

    start(1)
    loop()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    for seed in (2, 3, 4):
        n = start(seed)
        torch.cuda.synchronize()
        graph.replay()
        assert attn.attn_get_device_status() == 0
        assert lens.tolist() == [x + steps for x in n]
        k, v, ids = kc.cpu(), vc.cpu(), table.cpu()
        mask, cu = torch.ones(R, 1, dtype=torch.int32), list(range(R + 1))
        for s in ([0, 3, 17] if R > 100 else range(steps)):  # a step sees the keys up to its own
            qo, *results = got[s]
            y, tol = ref.norm_rope(qkv[s][0].cpu(), None, cs.cpu()[[x + s for x in n]], EPS, 0.0, False)
            ref.close("q", qo, y, tol)
            for (o, lse), more in zip(results, (s + 1, s)):
                L = [x + more for x in n]
                ro, to, rl, tl = ref.tree(qo.cpu(), k, v, ids, L, cu, mask, 0.1, window, torch.tensor(L) - 1)
                ref.close(f"o {s}", o, ro, to)
                ref.close(f"lse {s}", lse, rl.t(), tl.t())
        y, tol = ref.norm_rope(qkv[5][1].cpu(), None, cs.cpu()[[x + 5 for x in n]], EPS, 0.0, False)
        at = [int(ids[b, (x + 5) // 16]) * 16 + (x + 5) % 16 for b, x in enumerate(n)]
        ref.close("k", k.view(-1, Hkv, D)[at], y, tol)


def test_empty_decode_keeps_the_order():
    """Tree attention, a decode call whose requests are all empty, then a head norm over the trees' result."""
    R, Hq, Hkv, D = 6, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    pages = 600
    kc, vc = r(R * pages, 16, Hkv, D), r(R * pages, 16, Hkv, D)
    table = torch.randperm(R * pages, generator=g, device="cuda").to(torch.int32).view(R, pages)
    n = 20
    q, mask = r(R * n, Hq, D), i32([[(1 << (i % n + 1)) - 1] for i in range(R * n)])
    lens, cu, none = i32([9000 + 7 * b for b in range(R)]), i32([n * b for b in range(R + 1)]), i32([0] * R)
    o = torch.empty_like(q)
    lse = torch.empty(Hq, R * n, device="cuda")
    k = r(R * n, Hkv, D)

    def run():
        attn.attn_tree_paged(q, kc, vc, table, lens, cu, mask, n, o, lse, scale=0.1)
        do, dl = attn.attn_decode_paged(q[:R].contiguous(), kc, vc, table, none, scale=0.1)
        y, _ = attn.attn_qk_norm_rope(o, k, None, None, None, None, eps=EPS)
        return do, dl, y

    run()
    torch.cuda.synchronize()
    want, _ = attn.attn_qk_norm_rope(o.clone(), k, None, None, None, None, eps=EPS)
    keep = o.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        do, dl, y = run()
    for _ in range(20):
        o.fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, keep) and torch.equal(y, want)
        assert (do == 0).all() and (dl == -math.inf).all()
    assert attn.attn_get_device_status() == 0


def written_by_decode(ints, rows):
    """A decode call (head_dim 256, one key a request) whose result is, bit for bit, these small int32 values, and the buffer
    of its result. Its merge lets the kernel behind it start before it has written anything."""
    flat = torch.zeros(rows * 4 * 128, dtype=torch.int32)
    flat[: len(ints)] = torch.tensor(ints, dtype=torch.int32)
    vc = torch.zeros(rows, 16, 4, 256, dtype=torch.bfloat16, device="cuda")
    vc[:, 0] = flat.view(torch.bfloat16).view(rows, 4, 256).cuda()
    kc, q = torch.ones_like(vc), torch.ones(rows, 4, 256, dtype=torch.bfloat16, device="cuda")
    table = i32([[b] for b in range(rows)])
    o, lse, one = torch.empty_like(q), torch.empty(rows, 4, device="cuda"), i32([1] * rows)
    ws = torch.empty(attn.attn_workspace_size(attn.ATTN_OP_DECODE_PAGED, rows, 4, 4, 0, 256), dtype=torch.uint8, device="cuda")
    return (lambda: attn.attn_decode_paged(q, kc, vc, table, one, o, lse, scale=0.1, workspace=ws)), o


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("what", ["lengths", "table", "pages", "all"])
@pytest.mark.parametrize("Hq,Hkv,D,window", [(8, 2, 128, 0), (4, 4, 256, 0), (16, 8, 256, 50), (32, 8, 128, 30)])
def test_inputs_written_by_the_call_in_front(Hq, Hkv, D, window, what, captured):
    """Lengths, block table or pages are the result of a decode call directly in front, and what stood there before is
    something else, valid or not: nothing of it reaches the result or the device status."""
    R, cap, pages = 6, 10, 64
    g = torch.Generator().manual_seed(Hq + D)
    lens = [37, 0, 160, 5, 64, 1]
    ids = torch.randperm(pages, generator=g)[: R * cap].tolist()
    words = -(-max(R, R * cap) // 512)
    call_l, o_l = written_by_decode(lens, words)
    call_t, o_t = written_by_decode(ids, words)
    bits = torch.randint(0, 1 << 14, (pages * 16 * Hkv * D,), generator=g, dtype=torch.int16)  # bf16 values below 2
    call_k, o_k = written_by_decode(bits.view(torch.int32).tolist(), pages * 16 * Hkv * D // 1024)
    kc, vc = (torch.randn(pages, 16, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(R, Hq, D, generator=g).bfloat16().cuda()
    front = {"lengths": [call_l], "table": [call_t], "pages": [call_k], "all": [call_t, call_k, call_l]}[what]
    lengths = o_l.flatten().view(torch.int32)[:R] if what in ("lengths", "all") else i32(lens)
    table = (o_t.flatten().view(torch.int32)[: R * cap] if what in ("table", "all") else i32(ids)).view(R, cap)
    keys = o_k.view(pages, 16, Hkv, D) if what in ("pages", "all") else kc
    o, lse = torch.empty_like(q), torch.empty(R, Hq, device="cuda")
    ws = torch.empty(attn.attn_workspace_size(attn.ATTN_OP_DECODE_PAGED, R, Hq, Hkv, 0, D), dtype=torch.uint8, device="cuda")

    def run():
        for f in front:
            f()
        attn.attn_decode_paged(q, keys, vc, table, lengths, o, lse, scale=0.1, window=window, workspace=ws)

    run()
    torch.cuda.synchronize()
    assert attn.attn_get_device_status() == 0
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    now = keys.cpu()
    assert torch.equal(lengths.cpu(), torch.tensor(lens, dtype=torch.int32)) and table.flatten().tolist() == ids
    if keys is not kc:
        assert torch.equal(now.view(torch.int16).flatten(), bits)
    live = [b for b in range(R) if lens[b]]
    ro, to, rl, tl = ref.tree(q.cpu()[live], now, vc.cpu(), table.cpu()[live], [lens[b] for b in live], list(range(len(live) + 1)),
                              torch.ones(len(live), 1, dtype=torch.int32), 0.1, window, torch.tensor([lens[b] - 1 for b in live]))
    for before in (0, 3, 160, -1, 2 ** 30, 7):  # as a length, and as a page id
        if what in ("lengths", "all"):
            lengths.fill_(before)
        if what in ("table", "all"):
            table.fill_(before)
        if what in ("pages", "all"):
            keys.fill_(math.nan)
        o.fill_(5.0), lse.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay() if captured else run()
        assert attn.attn_get_device_status() == 0, before
        ref.close("o", o[live], ro, to)
        ref.close("lse", lse[live], rl.t(), tl.t())
        assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
