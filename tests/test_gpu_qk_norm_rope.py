"""Head norm with rotary position encoding (attn_qk_norm_rope, its gradient, its paged form) against a
64-bit implementation; the tolerances are derived in operator_ref."""
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


def problem(T, Hq, Hkv, D, rot, fused=False, w32=False, rows=500, seed=0, scale=1.5):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + D + rot)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wt = torch.float32 if w32 else torch.bfloat16
    p = dict(qw=(1 + 0.3 * n(D)).to(wt), kw=(1 + 0.3 * n(D)).to(wt), cs=ref.table(rows, rot) if rot else None,
             pos=torch.randint(0, rows, (T,), generator=g).to(torch.int32))
    qkv = (scale * n(T, (Hq + 2 * Hkv) * D)).bfloat16()
    p["q"], p["k"], p["v"] = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    d = {k: None if v is None else v.cuda() for k, v in p.items() if k not in "qkv"}
    if fused:
        qkv = qkv.cuda()
        d["q"], d["k"], d["v"] = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        d["q"], d["k"], d["v"] = (p[k].contiguous().cuda() for k in "qkv")
    p["gq"], p["gk"] = n(T, Hq, D).bfloat16(), n(T, Hkv, D).bfloat16()
    d["gq"], d["gk"] = p["gq"].cuda(), p["gk"].cuda()
    return p, d


def angles(p):
    T = p["pos"].numel()
    return p["cs"][p["pos"].long()] if p["cs"] is not None else torch.zeros(T, 0)


SHAPES = [  # T, Hq, Hkv, D, rot, interleaved, fused, fp32 weights, weight offset
    (1, 1, 1, 64, 64, False, False, False, 0.0), (1, 32, 8, 128, 128, False, True, False, 0.0),
    (7, 2, 1, 512, 512, False, False, True, 1.0), (33, 5, 3, 64, 16, True, True, True, 0.0),
    (65, 12, 3, 128, 96, False, True, False, 1.0), (130, 32, 16, 256, 256, False, True, False, 0.0),
    (257, 32, 4, 512, 128, False, True, True, 0.0), (64, 7, 7, 256, 32, True, False, False, 0.0),
    (19, 40, 10, 128, 0, False, True, False, 0.0), (3000, 3, 1, 64, 32, False, False, True, 0.0),
    (50, 100, 1, 128, 64, True, False, False, 0.0), (40, 6, 2, 512, 512, True, True, False, 1.0),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,fused,w32,off", SHAPES)
def test_forward(T, Hq, Hkv, D, rot, inter, fused, w32, off):
    p, d = problem(T, Hq, Hkv, D, rot, fused, w32)
    q, k = attn.attn_qk_norm_rope(d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["cs"], eps=EPS, weight_offset=off,
                                  interleaved=inter)
    assert attn.attn_get_device_status() == 0
    for name, got, x, w in (("q", q, p["q"], p["qw"]), ("k", k, p["k"], p["kw"])):
        y, tol = ref.norm_rope(x, w, angles(p), EPS, off, inter)
        ref.close(name, got, y, tol)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,fused,w32,off", SHAPES)
def test_gradient(T, Hq, Hkv, D, rot, inter, fused, w32, off):
    p, d = problem(T, Hq, Hkv, D, rot, fused, w32)
    dq = dk = None
    if fused:  # into slices of a fused gradient
        dqkv = torch.full((T, (Hq + 2 * Hkv) * D), 3.0, dtype=torch.bfloat16, device="cuda")
        dq, dk, dv = (x.view(T, -1, D) for x in dqkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    args = (d["gq"], d["gk"], d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["cs"], dq, dk)
    kw = dict(eps=EPS, weight_offset=off, interleaved=inter)
    got = attn.attn_qk_norm_rope_bwd(*args, **kw)
    assert attn.attn_get_device_status() == 0
    for i, (x, dy, w) in enumerate(((p["q"], p["gq"], p["qw"]), (p["k"], p["gk"], p["kw"]))):
        dx, tol, dw, wtol = ref.norm_rope_bwd(dy, x, w, angles(p), EPS, off, inter)
        ref.close("dx%d" % i, got[i], dx, tol)
        ref.close("dw%d" % i, got[2 + i], dw, wtol)
    if fused:
        assert (dv == 3.0).all()  # the value slice is left alone
    again = attn.attn_qk_norm_rope_bwd(*args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits


def test_gradient_against_differences():
    """The 64-bit gradient that the kernel is held to, against central differences of the 64-bit forward
    (no GPU arithmetic: the formula itself)."""
    for inter, off, rot in ((False, 0.0, 32), (True, 1.0, 64)):
        p, _ = problem(3, 2, 1, 64, rot, w32=True)
        x, w, dy, cs = p["q"].double(), p["qw"].double(), p["gq"].double(), angles(p)
        f = lambda x, w: (ref.norm_rope(x, w, cs, EPS, off, inter)[0] * dy).sum()  # noqa: E731
        dx, _, dw, _ = ref.norm_rope_bwd(dy, x, w, cs, EPS, off, inter)
        h = 1e-5
        for i in ((0, 0, 0), (1, 1, 33), (2, 0, 63)):
            e = torch.zeros_like(x)
            e[i] = h
            assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-6
            e = torch.zeros_like(w)
            e[i[2]] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i[2]]) < 1e-6


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,fused,w32,off", SHAPES)
def test_paged(T, Hq, Hkv, D, rot, inter, fused, w32, off):
    p, d = problem(T, Hq, Hkv, D, rot, fused, w32)
    pages = T // 8 + 3
    slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    if T > 5:
        slots[2] = slots[5] = -1  # padding
    caches = [torch.full((pages, 16, Hkv, D), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q_out = torch.full((T, Hq, D), 4.0, dtype=torch.bfloat16, device="cuda")
    pos = p["pos"].clone()
    pos[slots == -1] = -9  # a padding row's position is not looked at
    attn.attn_qk_norm_rope_paged(d["q"], d["k"], d["v"], d["qw"], d["kw"], pos.cuda(), slots.cuda(), d["cs"], *caches, q_out,
                                 eps=EPS, weight_offset=off, interleaved=inter)
    assert attn.attn_get_device_status() == 0
    live = slots >= 0
    y, tol = ref.norm_rope(p["q"], p["qw"], angles(p), EPS, off, inter)
    y[~live], tol[~live] = 4.0, 0.0
    ref.close("q", q_out, y, tol)
    y, tol = ref.norm_rope(p["k"], p["kw"], angles(p), EPS, off, inter)
    want, wtol = torch.full((pages * 16, Hkv, D), 2.0, dtype=torch.float64), torch.zeros(pages * 16, Hkv, D, dtype=torch.float64)
    want[slots[live].long()], wtol[slots[live].long()] = y[live], tol[live]
    ref.close("k cache", caches[0].view(-1, Hkv, D), want, wtol)
    want[slots[live].long()] = p["v"].double()[live]
    assert torch.equal(caches[1].view(-1, Hkv, D).double().cpu(), want)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,fused,w32,off", [(2500, 5, 5, 512, 128, False, True, False, 0.0),
                                                                (2503, 12, 4, 256, 256, False, False, True, 1.0),
                                                                (2600, 30, 15, 64, 32, True, True, False, 0.0),
                                                                (2500, 14, 14, 128, 0, False, True, False, 0.0)])
def test_paged_long(T, Hq, Hkv, D, rot, inter, fused, w32, off):
    """Several tasks for each warp of the GPU: the rows come through rings."""
    test_paged(T, Hq, Hkv, D, rot, inter, fused, w32, off)


def test_paged_long_in_place_with_bad_tokens():
    T, Hq, Hkv, D = 3000, 20, 5, 128
    p, d = problem(T, Hq, Hkv, D, 64)
    slots, pos = torch.arange(T, dtype=torch.int32), p["pos"].clone()
    slots[1000], slots[1001], slots[5] = -7, T + 40, -1
    pos[2000], pos[7] = 500, -1
    dead = torch.zeros(T, dtype=torch.bool)
    dead[[1000, 1001, 5, 2000, 7]] = True
    caches = [torch.full((-(-T // 16), 16, Hkv, D), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = d["q"]
    out = attn.attn_qk_norm_rope_paged(q, d["k"], d["v"], d["qw"], d["kw"], pos.cuda(), slots.cuda(), d["cs"], *caches, q, eps=EPS)
    assert out is q and attn.attn_get_device_status() == 7
    y, tol = ref.norm_rope(p["q"], p["qw"], angles(p), EPS, 0.0, False)
    y[dead], tol[dead] = p["q"].double()[dead], 0.0
    ref.close("q", q, y, tol)
    y, tol = ref.norm_rope(p["k"], p["kw"], angles(p), EPS, 0.0, False)
    y[dead], tol[dead] = 2.0, 0.0
    ref.close("k cache", caches[0].view(-1, Hkv, D)[:T], y, tol)
    want = p["v"].clone()
    want[dead] = 2.0
    assert torch.equal(caches[1].view(-1, Hkv, D)[:T].cpu(), want)


def test_no_weights_batch_layout_and_in_place():
    p, d = problem(60, 4, 2, 128, 64)
    want = attn.attn_qk_norm_rope(d["q"], d["k"], None, None, d["pos"], d["cs"])
    y, tol = ref.norm_rope(p["q"], None, angles(p), EPS, 0.0, False)
    ref.close("q", want[0], y, tol)
    # a weight offset does not matter without weights
    off = attn.attn_qk_norm_rope(d["q"], d["k"], None, None, d["pos"], d["cs"], weight_offset=1.0)
    assert torch.equal(off[0], want[0])
    # [B, S, H, D], positions too
    b = attn.attn_qk_norm_rope(d["q"].view(3, 20, 4, 128), d["k"].view(3, 20, 2, 128), None, None, d["pos"].view(3, 20), d["cs"])
    assert b[0].shape == (3, 20, 4, 128) and torch.equal(b[0].flatten(0, 1), want[0]) and torch.equal(b[1].flatten(0, 1), want[1])
    q, k = d["q"].clone(), d["k"].clone()
    attn.attn_qk_norm_rope(q, k, None, None, d["pos"], d["cs"], q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # the gradient over its own inputs
    ref_g = attn.attn_qk_norm_rope_bwd(d["gq"], d["gk"], d["q"], d["k"], None, None, d["pos"], d["cs"])
    gq, gk = d["gq"].clone(), d["gk"].clone()
    got = attn.attn_qk_norm_rope_bwd(gq, gk, d["q"], d["k"], None, None, d["pos"], d["cs"], gq, gk)
    assert all(torch.equal(a, b) for a, b in zip(got, ref_g))


def test_extreme_rows():
    """Rows of zeros, of one large value, and large and tiny magnitudes stay finite and right."""
    p, d = problem(8, 2, 2, 128, 128)
    q = p["q"].clone()
    q[0] = 0
    q[1] = 0
    q[1, :, 5] = 3e4
    q[2] *= 1e15
    q[3] *= 1e-20
    qd = q.cuda()
    got = attn.attn_qk_norm_rope(qd, d["k"], d["qw"], d["kw"], d["pos"], d["cs"], eps=EPS)
    y, tol = ref.norm_rope(q, p["qw"], angles(p), EPS, 0.0, False)
    ref.close("q", got[0], y, tol + 1e-38)
    g = attn.attn_qk_norm_rope_bwd(d["gq"], d["gk"], qd, d["k"], d["qw"], d["kw"], d["pos"], d["cs"], eps=EPS)
    dx, tol, dw, wtol = ref.norm_rope_bwd(p["gq"], q, p["qw"], angles(p), EPS, 0.0, False)
    ref.close("dq", g[0], dx, tol + 1e-38)
    ref.close("dqw", g[2], dw, wtol)


def test_bad_positions_and_slots_are_reported_and_skipped():
    p, d = problem(40, 4, 2, 128, 128)
    pos = p["pos"].clone()
    pos[3], pos[30] = -1, 500
    bad = torch.zeros(40, dtype=torch.bool)
    bad[3] = bad[30] = True
    out = [torch.full_like(d[k], 5.0) for k in ("q", "k")]
    attn.attn_qk_norm_rope(d["q"], d["k"], d["qw"], d["kw"], pos.cuda(), d["cs"], *out, eps=EPS)
    assert attn.attn_get_device_status() == 7
    y, tol = ref.norm_rope(p["q"], p["qw"], angles(p), EPS, 0.0, False)
    y[bad], tol[bad] = 5.0, 0.0
    ref.close("q", out[0], y, tol)
    # in the gradient they add nothing, whatever they hold
    gq = d["gq"].clone()
    gq[3] = float("nan")
    grads = [torch.full_like(d[k], 5.0) for k in ("q", "k")]
    got = attn.attn_qk_norm_rope_bwd(gq, d["gk"], d["q"], d["k"], d["qw"], d["kw"], pos.cuda(), d["cs"], *grads, eps=EPS)
    assert attn.attn_get_device_status() == 7
    ok = ~bad
    dx, tol, dw, wtol = ref.norm_rope_bwd(p["gq"][ok], p["q"][ok], p["qw"], angles(p)[ok], EPS, 0.0, False)
    ref.close("dq", got[0].cpu()[ok], dx, tol)
    ref.close("dqw", got[2], dw, wtol)
    assert (got[0].cpu()[bad] == 5.0).all()
    # slots outside the cache
    slots = torch.arange(40, dtype=torch.int32)
    slots[7], slots[8] = -2, 64
    caches = [torch.full((4, 16, 2, 128), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qo = torch.full_like(d["q"], 5.0)
    attn.attn_qk_norm_rope_paged(d["q"], d["k"], d["v"], d["qw"], d["kw"], d["pos"], slots.cuda(), d["cs"], *caches, qo, eps=EPS)
    assert attn.attn_get_device_status() == 7
    assert (qo[7:9] == 5.0).all() and (caches[0].view(64, 2, 128)[[7, 8, 40, 63]] == 2.0).all()
    assert torch.equal(caches[1].view(64, 2, 128)[9:40], d["v"][9:40])


def test_empty():
    _, d = problem(4, 2, 1, 64, 64)
    e = lambda x: x[:0]  # noqa: E731
    q, k = attn.attn_qk_norm_rope(e(d["q"]), e(d["k"]), d["qw"], d["kw"], e(d["pos"]), d["cs"])
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    g = attn.attn_qk_norm_rope_bwd(e(d["gq"]), e(d["gk"]), e(d["q"]), e(d["k"]), d["qw"], d["kw"], e(d["pos"]), d["cs"])
    assert (g[2] == 0).all() and (g[3] == 0).all()


def test_captured_gradient():
    """Forward and gradient captured once, replayed on other inputs; an eager gradient of the same leaves lives."""
    p, d = problem(300, 8, 2, 256, 64, fused=True)
    eager = attn.attn_qk_norm_rope_bwd(d["gq"], d["gk"], d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["cs"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = attn.attn_qk_norm_rope(d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["cs"])
        got = attn.attn_qk_norm_rope_bwd(d["gq"], d["gk"], d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["cs"])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    d["gq"].mul_(-2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[2], -2 * eager[2]) and torch.equal(got[3], eager[3])
    want = attn.attn_qk_norm_rope(d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["cs"])
    assert torch.equal(y[0], want[0])
