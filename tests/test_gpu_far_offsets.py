"""Head norm and tree attention where element offsets pass 32 bits: long packed batches and large caches. The
rows compared lie at both ends."""
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
    yield
    torch.cuda.empty_cache()


def test_head_norm_and_gradient():
    """2.15e9 query elements (4.3 GB) and their gradients."""
    T, Hq, Hkv, D, rot = 140001, 30, 1, 512, 128
    assert (T - 1) * Hq * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, gq, gk = (torch.empty(T, h, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for h in (Hq, Hkv, Hq, Hkv))
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2))
    cs = ref.table(300, rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 300
    y, _ = attn.attn_qk_norm_rope(q, k, qw, kw, pos, cs.cuda(), eps=EPS)
    dq, _, dqw, _ = attn.attn_qk_norm_rope_bwd(gq, gk, q, k, qw, kw, pos, cs.cuda(), eps=EPS)
    assert attn.attn_get_device_status() == 0
    rows = torch.tensor([0, 1, T - 3, T - 2, T - 1])
    at = cs[pos[rows.cuda()].cpu().long()]
    want, tol = ref.norm_rope(q[rows].cpu(), qw.cpu(), at, EPS, 0.0, False)
    ref.close("q_out", y[rows], want, tol)
    dx, tol, _, _ = ref.norm_rope_bwd(gq[rows].cpu(), q[rows].cpu(), qw.cpu(), at, EPS, 0.0, False)
    ref.close("dq", dq[rows], dx, tol)
    assert torch.isfinite(dqw).all()


def test_large_cache():
    """Caches of 9.2 GB: K and V written at far slots, then read by trees whose pages lie at both ends."""
    pages, Hq, Hkv, D, rot = 140000, 8, 4, 512, 64
    assert (pages - 10) * 16 * Hkv * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(6)
    kc, vc = (torch.empty(pages, 16, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = [70, 150, 33]
    ids = torch.tensor([list(range(pages - 5, pages)) + [-1] * 5, [3, pages - 6, 70000, 1, pages - 9, 2, 69999, pages - 7, 0, 80001],
                        [5, pages - 11, 90000] + [-1] * 7], dtype=torch.int32)
    slots = [int(ids[b, i // 16]) * 16 + i % 16 for b, L in enumerate(lens) for i in range(L)]
    T = len(slots)
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    cs = ref.table(200, rot)
    pos = torch.tensor([i for L in lens for i in range(L)], dtype=torch.int32)
    qo = attn.attn_qk_norm_rope_paged(q, k, v, None, None, pos.cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), cs.cuda(), kc, vc,
                                      eps=EPS)
    want, tol = ref.norm_rope(k.cpu(), None, cs[pos.long()], EPS, 0.0, False)
    at = torch.tensor(slots).cuda()
    ref.close("k_cache", kc.view(-1, Hkv, D)[at], want, tol)
    assert torch.equal(vc.view(-1, Hkv, D)[at], v)
    # the last tokens of each request as a tree over the rest
    n = [6, 20, 1]
    starts = [sum(lens[:b]) for b in range(3)]
    qt = torch.cat([qo[starts[b] + lens[b] - n[b]: starts[b] + lens[b]] for b in range(3)])
    cg = torch.Generator().manual_seed(7)
    mask = torch.tensor([m for x in n for m in ref.random_tree(x, 1, cg)[0]], dtype=torch.int32).reshape(-1, 1)
    cu = [0, 6, 26, 27]
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    o, lse = attn.attn_tree_paged(qt, kc, vc, ids.cuda(), i32(lens), i32(cu), mask.cuda(), 20, scale=1 / math.sqrt(D))
    assert attn.attn_get_device_status() == 0
    used = sorted({int(x) for x in ids.flatten() if x >= 0})
    back = {p: i for i, p in enumerate(used)}
    small = torch.tensor([[back.get(int(x), -1) for x in row] for row in ids], dtype=torch.int32)
    sub = torch.tensor(used).cuda()
    ro, to, rl, tl = ref.tree(qt.cpu(), kc[sub].cpu(), vc[sub].cpu(), small, lens, cu, mask, 1 / math.sqrt(D))
    ref.close("o", o, ro, to)
    ref.close("lse", lse, rl, tl)
