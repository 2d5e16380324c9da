"""Windows with sinks and the 4-bit cache together, as a program uses them: prompts, decode steps and a later chunk over one
4-bit cache (plan, head norm, append, decode; pages back as bf16 for the chunk and for drafted trees), and a training step with sinks
through the head norm. Each stage against its 64-bit definition on its actual inputs."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import kv4_ref
import operator_ref
import sink_ref
from operator_ref import close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("Hq,Hkv,D,window,sink", [(8, 2, 128, 40, 4), (6, 2, 64, 0, 0), (4, 4, 256, 33, 20)])
def test_serving(Hq, Hkv, D, window, sink):
    R, pages, scale = 4, 60, 1 / math.sqrt(D)
    g = torch.Generator().manual_seed(1)
    cache = torch.randint(0, 256, (pages, Hkv, 18, D), generator=g, dtype=torch.uint8).cuda()
    free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    table = torch.full((R, 14), -1, dtype=torch.int32, device="cuda")
    lens, held, used = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (R, R, 1))
    cs = operator_ref.table(256, D).cuda()
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2))

    def step(new):
        """Plan, norm, append; the step's queries, its keys and values as the cache holds them."""
        T = sum(new)
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        plan = attn.attn_paged_plan(lens, i32(new), free, table, held, used, T, num_pages=pages,
                                    out=attn.PagedPlan(lens, e(R + 1), e(T), e(T), held, used, e(1)))
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).bfloat16().cuda()
        q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        q, k = attn.attn_qk_norm_rope(q, k, qw, kw, plan.positions, cs)
        attn.attn_kv4_append(k, v, plan.slots, cache)
        K, V = kv4_ref.get(cache.cpu())
        at = plan.slots.cpu().long()
        for have, rows in ((K, k), (V, v)):
            assert torch.equal(have.flatten(0, 1)[at], kv4_ref.values(rows.cpu()))
        return plan, q, k, v.contiguous()

    prompts = [50, 1, 17, 130]
    plan, q, k, v = step(prompts)
    o, lse = attn.attn_fwd_varlen(q, k, v, plan.cu_q, 130, window=window, sink=sink, scale=scale)  # prompts see their own bf16 rows
    want = sink_ref.packed(lambda *x: sink_ref.forward(*x, scale, window, sink), prompts, q.cpu(), k.cpu(), v.cpu())
    close("prompt o", o, want[0], want[1])
    close("prompt lse", lse, want[2], want[3])
    for _ in range(3):
        plan, q, k, v = step([1] * R)
        got = attn.attn_decode_kv4(q, cache, table, lens, window=window, sink=sink, scale=scale)
        want = kv4_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens.tolist(), scale, window, sink)
        close("decode o", got[0], want[0], want[1])
        close("decode lse", got[1], want[2], want[3])
    # a chunk: its requests' pages back as bf16, and the calls that read such a cache over them
    new = [20, 3, 1, 40]
    plan, q, k, v = step(new)
    total = lens.tolist()
    at = torch.full_like(table, -1)
    listed = torch.cat([table[b, : held[b]] for b in range(R)])
    first = 0
    for b in range(R):
        at[b, : held[b]] = torch.arange(first, first + int(held[b]), dtype=torch.int32)
        first += int(held[b])
    kc, vc = attn.attn_kv4_unpack(cache, listed)
    # slots past the requests' ends hold anything: the tree call wants finite ones up to each page's end only where they are used
    o, lse = attn.attn_fwd_paged(q, kc, vc, at, lens, plan.cu_q, max(new), window=window, sink=sink, scale=scale)
    K, V = (x.bfloat16() for x in kv4_ref.get(cache.cpu()))
    row = 0
    for b in range(R):
        ids = table[b].cpu().long()[: int(held[b])]
        kk, vv = (x[ids].flatten(0, 1)[: total[b]] for x in (K, V))
        ro, to, rl, tl = sink_ref.forward(q[row: row + new[b]].cpu(), kk, vv, scale, window, sink)
        close("chunk o", o[row: row + new[b]], ro, to)
        close("chunk lse", lse[:, row: row + new[b]], rl, tl)
        row += new[b]
    if window == 0:
        words = [[(1 << (i + 1)) - 1 if i < 31 else -1, (1 << (i - 31)) - 1 if i > 31 else 0] for n in new for i in range(n)]
        to_, tl_ = attn.attn_tree_paged(q, kc, vc, at, lens, plan.cu_q, i32(words), max(new), scale=scale)
        ro, to, rl, tl = operator_ref.tree(q.cpu(), kc.cpu(), vc.cpu(), at.cpu(), total, plan.cu_q.tolist(), torch.tensor(words), scale)
        close("tree o", to_, ro, to)
        close("tree lse", tl_, rl, tl)
    # the same decode over the cache in bf16 and in 4 bits
    plan, q, k, v = step([1] * R)
    if D != 64 and Hq // Hkv in (1, 2, 4):
        kc, vc = attn.attn_kv4_unpack(cache, torch.arange(pages, dtype=torch.int32, device="cuda"))
        a = attn.attn_decode_kv4(q, cache, table, lens, window=window, sink=sink, scale=scale)
        b = attn.attn_decode_paged(q, kc, vc, table, lens, window=window, sink=sink, scale=scale)
        want = kv4_ref.decode(q.cpu(), cache.cpu(), table.cpu(), lens.tolist(), scale, window, sink)
        for x in (a, b):
            close("o", x[0], want[0], want[1])
            close("lse", x[1], want[2], want[3])
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_training(D):
    """Gradients through head norm, windowed attention with sinks, and back, against automatic differentiation in 64 bits."""
    S, Hq, Hkv, window, sink, scale = 200, 4, 2, 30, 3, 1 / math.sqrt(D)
    g = torch.Generator().manual_seed(D)
    q, k, v, do = (torch.randn(S, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv, Hq))
    qw, kw = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2))
    cs, pos = operator_ref.table(S, 64), torch.arange(S, dtype=torch.int32)
    dev = [t.cuda() for t in (q, k, v, do, qw, kw, cs, pos)]
    qn, kn = attn.attn_qk_norm_rope(dev[0], dev[1], dev[4], dev[5], dev[7], dev[6])
    how = dict(window=window, sink=sink, scale=scale)
    o, lse = attn.attn_fwd(qn[None], kn[None], dev[2][None], **how)
    dqn, dkn, dv = attn.attn_bwd(qn[None], kn[None], dev[2][None], o, lse, dev[3][None], **how)
    # the attention stage on its actual inputs
    want = sink_ref.backward(qn.cpu(), kn.cpu(), v, do, scale, window, sink)
    for name, got, i in (("dqn", dqn, 0), ("dkn", dkn, 2), ("dv", dv, 4)):
        close(name, got[0], want[i], want[i + 1])
    dq, dk, dqw, dkw = attn.attn_qk_norm_rope_bwd(dqn[0], dkn[0], dev[0], dev[1], dev[4], dev[5], dev[7], dev[6])
    for x, dy, w, got, gw in ((q, dqn, qw, dq, dqw), (k, dkn, kw, dk, dkw)):
        dx, tol, dw, wtol = operator_ref.norm_rope_bwd(dy[0].cpu(), x, w, cs, 1e-6, 0.0, False)
        close("dx", got, dx, tol)
        close("dw", gw, dw, wtol)
    assert attn.attn_get_device_status() == 0
