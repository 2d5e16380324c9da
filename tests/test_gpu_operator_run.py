"""The operators together, as a program uses them: a speculative decoding step over a paged cache
(plan, head norm into the pages, tree attention; then single-token decode and a chunk over the same cache)
and a training step (head norm, attention forward and backward, gradient of the norm), each stage against
its 64-bit definition on the actual inputs of that stage."""
import math

import numpy as np
import pytest
import torch

import attention_flash_gqa_gb300 as attn
import operator_ref as ref
from gpu_util import check, check_lse, to_np

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


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Cache:
    """The state that a serving program keeps."""

    def __init__(self, R, Hkv, D, pages, max_pages, seed):
        g = torch.Generator().manual_seed(seed)
        self.kc, self.vc = (torch.full((pages, 16, Hkv, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
        self.table = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens, self.held, self.used = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (R, R, 1))


@pytest.mark.parametrize("Hq,Hkv,D,rot,window", [(8, 2, 128, 128, 0), (8, 4, 256, 64, 40), (4, 2, 512, 128, 0)])
def test_serving_steps(orc, Hq, Hkv, D, rot, window):
    R, pages = 5, 120
    s = Cache(R, Hkv, D, pages, 24, 5)
    g = torch.Generator().manual_seed(7)
    cs = ref.table(512, rot).cuda()
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2))
    scale = 1 / math.sqrt(D)
    shadow = [[torch.zeros(0, Hkv, D).bfloat16(), torch.zeros(0, Hkv, D).bfloat16()] for _ in range(R)]

    def step(new, tree):
        T = sum(new)
        # the accepted lengths stay in s.lens: a plan writes its step's lengths elsewhere, pages in place
        e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        out = attn.PagedPlan(e(R), e(R + 1), e(T), e(T), s.held, s.used, e(1))
        p = attn.attn_paged_plan(s.lens, i32(new), s.free, s.table, s.held, s.used, T, num_pages=pages, out=out)
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).bfloat16().cuda()
        q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        pos, mask = p.positions, None
        if tree:
            mask, depth = [], []
            for x in new:
                m, d = ref.random_tree(x, 1, g)
                mask, depth = mask + m, depth + d
            first = p.positions - torch.cat([torch.arange(x, dtype=torch.int32) for x in new]).cuda()
            pos = first + i32(depth)  # a drafted token's position is its depth's, its slot its own
            mask = torch.tensor(mask, dtype=torch.int32).reshape(T, 1).cuda()
        qo = attn.attn_qk_norm_rope_paged(q, k, v, qw, kw, pos, p.slots, cs, s.kc, s.vc, eps=EPS)
        if tree:
            o, lse = attn.attn_tree_paged(qo, s.kc, s.vc, s.table, p.seq_lens, p.cu_q, mask, max(new), positions=pos,
                                          window=window, scale=scale)
        else:
            o, lse = attn.attn_fwd_paged(qo, s.kc, s.vc, s.table, p.seq_lens, p.cu_q, max(new), window=window, scale=scale)
        assert attn.attn_get_device_status() == 0
        # the stages against their definitions
        y, tol = ref.norm_rope(q.cpu(), qw.cpu(), cs.cpu()[pos.cpu().long()], EPS, 0.0, False)
        ref.close("q", qo, y, tol)
        y, tol = ref.norm_rope(k.cpu(), kw.cpu(), cs.cpu()[pos.cpu().long()], EPS, 0.0, False)
        rows = p.slots.cpu().long()
        ref.close("k", s.kc.view(-1, Hkv, D).cpu()[rows], y, tol)
        assert torch.equal(s.vc.view(-1, Hkv, D)[rows.cuda()], v)
        cu = p.cu_q.tolist()
        assert cu[-1] == T and p.seq_lens.tolist() == [a + b for a, b in zip(s.lens.tolist(), new)]
        for b in range(R):  # what earlier steps left in the pages is still there
            ids = s.table[b, : s.held[b]].long()
            n = len(shadow[b][0])
            for c, old in zip((s.kc, s.vc), shadow[b]):
                assert torch.equal(c[ids].flatten(0, 1)[:n].cpu(), old)
        if tree:
            ro, to, rl, tl = ref.tree(qo.cpu(), s.kc.cpu(), s.vc.cpu(), s.table.cpu(), p.seq_lens.tolist(), cu, mask.cpu(), scale,
                                      window, pos.cpu())
            ref.close("o", o, ro, to)
            ref.close("lse", lse, rl, tl)
        else:
            ro, rl = orc.prefill_paged(bits(qo), bits(s.kc), bits(s.vc), s.table.cpu().numpy(), p.seq_lens.cpu().numpy(),
                                       p.cu_q.cpu().numpy(), scale, window)
            check("o", to_np(o), ro)
            check_lse("lse", to_np(lse), rl)
        return p

    def accept(keep):
        s.lens += i32(keep)
        for b in range(R):
            ids = s.table[b, : s.held[b]].long()
            n = int(s.lens[b])
            shadow[b] = [c[ids].flatten(0, 1)[:n].cpu() for c in (s.kc, s.vc)]

    step([33, 16, 1, 70, 47], tree=False)  # prompts
    accept([33, 16, 1, 70, 47])
    held = s.held.tolist()
    assert held == [3, 1, 1, 5, 3]
    step([8, 3, 5, 20, 2], tree=True)       # drafts; some requests take a page
    assert s.held.tolist() == [3, 2, 1, 6, 4]
    accept([2, 0, 5, 1, 1])                  # rejected tokens' pages stay held
    step([9, 14, 11, 30, 1], tree=True)
    accept([1, 1, 1, 1, 1])
    step([1, 1, 1, 1, 1], tree=False)        # plain decode as a chunk of one token
    accept([1, 1, 1, 1, 1])
    if D == 512:
        return
    # single-token decode over the same cache: the plan's outputs feed the decode call directly
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    qd = torch.randn(R, Hq, D, generator=g).bfloat16().cuda()
    kd, vd = (torch.randn(R, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    out = attn.PagedPlan(s.lens, e(R + 1), e(R), e(R), s.held, s.used, e(1))
    p = attn.attn_paged_plan(s.lens, i32([1] * R), s.free, s.table, s.held, s.used, R, num_pages=pages, out=out)
    qo = attn.attn_qk_norm_rope_paged(qd, kd, vd, qw, kw, p.positions, p.slots, cs, s.kc, s.vc, eps=EPS)
    o, lse = attn.attn_decode_paged(qo, s.kc, s.vc, s.table, s.lens, window=window, scale=scale)
    assert attn.attn_get_device_status() == 0
    ro, rl = orc.decode_paged(bits(qo), bits(s.kc), bits(s.vc), s.table.cpu().numpy(), s.lens.cpu().numpy(), scale, window)
    check("decode o", to_np(o), ro)
    check_lse("decode lse", to_np(lse), rl)


@pytest.mark.parametrize("D,rot,window", [(128, 128, 0), (256, 64, 50), (512, 128, 0)])
def test_training_step(D, rot, window):
    """Gradients of the fused projection and of the norm weights through norm, attention and back."""
    B, S, Hq, Hkv = 2, 150, 4, 2
    T, g = B * S, torch.Generator().manual_seed(D)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).bfloat16()
    q, k, v = (x.view(B, S, -1, D) for x in qkv.cuda().split([Hq * D, Hkv * D, Hkv * D], 1))
    qw, kw = (0.3 * torch.randn(D, generator=g) for _ in range(2))
    cs = ref.table(S, rot)
    pos = torch.arange(S, dtype=torch.int32).repeat(B)
    do = torch.randn(B, S, Hq, D, generator=g).bfloat16()
    scale = 1 / math.sqrt(D)
    opt = dict(eps=EPS, weight_offset=1.0)

    qn, kn = attn.attn_qk_norm_rope(q, k, qw.cuda(), kw.cuda(), pos.cuda(), cs.cuda(), **opt)
    o, lse = attn.attn_fwd(qn, kn, v.contiguous(), window=window, scale=scale)
    dqkv = torch.empty_like(qkv, device="cuda")
    dq, dk, dv = (x.view(B, S, -1, D) for x in dqkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    dqn, dkn, dvn = attn.attn_bwd(qn, kn, v.contiguous(), o, lse, do.cuda(), window=window, scale=scale)
    dv.copy_(dvn)
    _, _, dqw, dkw = attn.attn_qk_norm_rope_bwd(dqn, dkn, q, k, qw.cuda(), kw.cuda(), pos.cuda(), cs.cuda(), dq, dk, **opt)
    assert attn.attn_get_device_status() == 0

    # the gradient stage on its actual inputs, within its derived bounds
    at = cs[pos.long()]
    for x, dy, w, got, gw in ((q, dqn, qw, dq, dqw), (k, dkn, kw, dk, dkw)):
        x, dy, got = (y.flatten(0, 1).cpu() for y in (x, dy, got))
        dx, tol, dw, wtol = ref.norm_rope_bwd(dy, x, w, at, EPS, 1.0, False)
        ref.close("dx", got, dx, tol)
        ref.close("dw", gw, dw, wtol)

    # the whole chain in 64 bits by automatic differentiation, at the attention's own tolerance
    x64 = qkv.double().requires_grad_()
    w64 = [w.double().requires_grad_() for w in (qw, kw)]
    qx, kx, vx = (y.view(T, -1, D) for y in x64.split([Hq * D, Hkv * D, Hkv * D], 1))
    a, b = ref._pairs(rot, False)
    c, sn = at.double()[:, None, : rot // 2], at.double()[:, None, rot // 2:]

    def normed(x, w):
        n = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * (1 + w)
        return torch.cat([n[..., a] * c - n[..., b] * sn, n[..., b] * c + n[..., a] * sn, n[..., rot:]], -1)

    qy, ky = (normed(x, w).view(B, S, -1, D).transpose(1, 2) for x, w in ((qx, w64[0]), (kx, w64[1])))
    vy = vx.view(B, S, -1, D).transpose(1, 2)
    ky, vy = (y.repeat_interleave(Hq // Hkv, 1) for y in (ky, vy))
    i = torch.arange(S)
    d = i[:, None] - i[None, :]
    see = (d >= 0) & ((d < window) if window else torch.ones_like(d, dtype=torch.bool))
    out = ((qy @ ky.transpose(-1, -2) * scale).masked_fill(~see, -math.inf)).softmax(-1) @ vy
    (out.transpose(1, 2) * do.double()).sum().backward()
    check("o", to_np(o), out.transpose(1, 2).detach().numpy())
    for name, got, want in (("dq", dq, x64.grad[:, : Hq * D]), ("dk", dk, x64.grad[:, Hq * D: (Hq + Hkv) * D]),
                            ("dv", dv, x64.grad[:, (Hq + Hkv) * D:])):
        check(name, to_np(got.reshape(T, -1)), want.numpy())
    check("dqw", to_np(dqw), w64[0].grad.numpy())
    check("dkw", to_np(dkw), w64[1].grad.numpy())


def test_fork_and_join_in_a_graph():
    """Plan on one captured stream, a head norm on another, joined before the cache write, the trees and a decode step."""
    R, Hq, Hkv, D, rot, pages = 5, 8, 2, 128, 64, 60
    s = Cache(R, Hkv, D, pages, 10, 3)
    g = torch.Generator().manual_seed(11)
    s.kc.normal_(), s.vc.normal_()
    n = [4, 1, 7, 2, 3]
    T = sum(n)
    s.held += 2
    s.table[:, :2] = torch.arange(2 * R, dtype=torch.int32, device="cuda").view(R, 2)
    s.free = torch.arange(2 * R, pages, dtype=torch.int32, device="cuda")
    ctx, new = i32([20, 3, 31, 0, 17]), i32(n)
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    cs = ref.table(100, rot).cuda()
    words = [ref.random_tree(x, 1, g)[0] for x in n]
    mask = torch.tensor([m for w in words for m in w], dtype=torch.int32).reshape(T, 1).cuda()
    table = s.table.clone()

    def run(side=None):
        main = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(main)
        p = attn.attn_paged_plan(ctx, new, s.free, table, s.held, s.used, T, num_pages=pages)
        with torch.cuda.stream(side if side is not None else main):
            extra = attn.attn_qk_norm_rope(q, k, None, None, torch.arange(T, dtype=torch.int32, device="cuda"), cs, eps=EPS)
        if side is not None:
            main.wait_stream(side)
        qo = attn.attn_qk_norm_rope_paged(q, k, v, None, None, p.positions, p.slots, cs, s.kc, s.vc, eps=EPS)
        o, lse = attn.attn_tree_paged(qo, s.kc, s.vc, table, p.seq_lens, p.cu_q, mask, max(n), scale=0.1)
        do, dl = attn.attn_decode_paged(qo[:R].contiguous(), s.kc, s.vc, table, p.seq_lens, scale=0.1)
        return [*p, *extra, qo, o, lse, do, dl]

    want = run()
    torch.cuda.synchronize()
    keep = s.kc.clone(), s.vc.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        got = run(side)
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(s.kc, keep[0]) and torch.equal(s.vc, keep[1])
    assert attn.attn_get_device_status() == 0
