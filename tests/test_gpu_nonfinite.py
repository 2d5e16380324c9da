"""Non-finite inputs in places that count: a row whose scores hold a NaN comes out as NaN, whichever of its keys
are NaN and however they are split over the GPU, and no other row is touched."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import operator_ref as ref
from test_gpu_tree_paged import i32, problem, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def definition(p, window=0, **other):
    p = dict(p, **other)
    return ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"], window, p["pos"])


def rows_but(nan, got, want, tol, what):
    """NaN where `nan` [T, Hq] says so, within the tolerance elsewhere."""
    assert torch.isnan(got.cpu()[nan]).all(), what
    ref.close(what, got.cpu()[~nan], want[~nan], tol[~nan])


# one key tile (a single CTA writes the row), many tiles (partial results are merged), a batch of both
CONTEXTS = [([40], [5]), ([9000], [5]), ([0, 700, 30, 2500], [3, 9, 1, 33])]


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("ctx,n", CONTEXTS)
def test_tree_query_rows(D, ctx, n):
    p = problem(ctx, n, 4, 2, D, seed=51)
    T = sum(n)
    nan = torch.zeros(T, 4, dtype=torch.bool)
    nan[0, 1] = nan[T - 1, 3] = nan[T // 2, 0] = True
    q = p["q"].clone()
    q[nan] = math.nan
    q[0, 1] = p["q"][0, 1]
    q[0, 1, 7] = math.nan  # one value is enough
    ro, to, rl, tl = definition(p)
    o, lse = run(dict(p, q=q))
    assert attn.attn_get_device_status() == 0
    rows_but(nan, o, ro, to, "o")
    rows_but(nan, lse.t(), rl.t(), tl.t(), "lse")


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("window", [0, 4000])
@pytest.mark.parametrize("first,count", [(0, 2000), (5500, 1), (5100, 300), (8990, 10)])
def test_tree_visible_keys(D, window, first, count):
    """K of one head is NaN for a stretch of the context (as long as several CTAs' shares, or a single key):
    every row of that head's group is NaN, unless the window hides all of the stretch."""
    p = problem([9000], [6], 4, 2, D, seed=52)
    ro, to, rl, tl = definition(p, window)
    kc = p["kc"].clone()
    for j in range(first, first + count):
        kc[p["table"][0, j // 16], j % 16, 1] = math.nan
    o, lse = run(dict(p, kc=kc), window)
    assert attn.attn_get_device_status() == 0
    nan = torch.zeros(6, 4, dtype=torch.bool)
    start = (torch.maximum(p["pos"], torch.tensor(9000)) - window + 1) if window else torch.zeros(6)
    nan[:, 2:] = (start < first + count)[:, None]
    rows_but(nan, o, ro, to, "o")
    rows_but(nan, lse.t(), rl.t(), tl.t(), "lse")


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("ctx", [20, 3000])
def test_tree_infinite_scores(D, ctx):
    """A score of +inf leaves no finite result, one of -inf counts as a key with probability zero."""
    p = problem([ctx], [8], 4, 2, D, seed=53)
    p["mask"][:] = -1  # every row sees every drafted token
    j = ctx + 5
    kc = p["kc"].clone()
    kc[p["table"][0, j // 16], j % 16, 0, 3] = math.inf
    up = torch.zeros(8, 4, dtype=torch.bool)
    up[:, :2] = p["q"][:, :2, 3] > 0
    assert up.any() and not up[:, :2].all() and (p["q"][:, :, 3] != 0).all()
    mask = p["mask"].clone()
    mask &= ~(1 << 5)
    ro, to, rl, tl = definition(p, mask=mask)  # heads 0 and 1: without the key
    so, st, sl, sm = definition(p)
    ro[:, 2:], to[:, 2:], rl[2:], tl[2:] = so[:, 2:], st[:, 2:], sl[2:], sm[2:]
    o, lse = run(dict(p, kc=kc))
    assert attn.attn_get_device_status() == 0
    o, lse = o.cpu(), lse.t().cpu()
    assert not torch.isfinite(o[up]).any() and not torch.isfinite(lse[up]).any() and (lse[up] != -math.inf).all()
    ref.close("o", o[~up], ro[~up], to[~up])
    ref.close("lse", lse[~up], rl.t()[~up], tl.t()[~up])


@pytest.mark.parametrize("window", [0, 4000])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 128), (4, 2, 128), (8, 2, 128), (32, 8, 128), (16, 2, 128), (2, 2, 256), (8, 4, 256), (16, 4, 256)])
def test_decode(Hq, Hkv, D, window):
    """A decode step is a tree of one token: NaN query rows, and NaN keys of one head in some of a request's pages."""
    G = Hq // Hkv
    p = problem([8999, 4, 699], [1, 1, 1], Hq, Hkv, D, seed=54)
    ro, to, rl, tl = definition(p, window)

    def check(nan, **other):
        d = dict(p, **other)
        o, lse = attn.attn_decode_paged(d["q"].cuda(), d["kc"].cuda(), d["vc"].cuda(), d["table"].cuda(), i32(d["lens"]),
                                        scale=d["scale"], window=window)
        assert attn.attn_get_device_status() == 0
        rows_but(nan, o, ro, to, "o")
        rows_but(nan, lse, rl.t(), tl.t(), "lse")

    nan = torch.zeros(3, Hq, dtype=torch.bool)
    check(nan)
    q = p["q"].clone()
    nan[0, 1] = nan[1, 0] = nan[2, Hq - 1] = True
    q[nan] = math.nan
    check(nan, q=q)
    for first, count in ((0, 2000), (5500, 1), (8000, 999)):
        kc = p["kc"].clone()
        for j in range(first, first + count):
            kc[p["table"][0, j // 16], j % 16, 1] = math.nan
        nan = torch.zeros(3, Hq, dtype=torch.bool)
        nan[0, G: 2 * G] = not window or first + count > 5000
        check(nan, kc=kc)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 4, 2), (256, 4, 2), (512, 4, 2), (512, 3, 3)])
@pytest.mark.parametrize("window", [0, 300])
def test_forward(D, Hq, Hkv, window):
    """The same of the causal forward, dense and over a paged cache: NaN query rows, a NaN key."""
    n, j = 700, 150
    p = problem([0], [n], Hq, Hkv, D, seed=55)
    g = torch.Generator().manual_seed(56)
    q, kc = p["q"].clone(), p["kc"].clone()
    q[300, 1, 5] = q[699, 0, 0] = math.nan
    kc[p["table"][0, j // 16], j % 16, Hkv - 1] = math.nan
    k, v = (c[p["table"][0, : -(-n // 16)].long()].flatten(0, 1)[:n][None].cuda() for c in (kc, p["vc"]))
    i = torch.arange(n)
    nan = torch.zeros(n, Hq, dtype=torch.bool)
    nan[300, 1] = nan[699, 0] = True
    nan[:, Hq - Hq // Hkv:] |= ((i >= j) & (i - j < window if window else i >= 0))[:, None]
    for o, lse in (attn.attn_fwd(q[None].cuda(), k.contiguous(), v.contiguous(), window=window, scale=p["scale"]),
                   attn.attn_fwd_paged(q.cuda(), kc.cuda(), p["vc"].cuda(), p["table"].cuda(), i32([n]), i32([0, n]), n, window=window,
                                       scale=p["scale"])):
        assert attn.attn_get_device_status() == 0
        o, lse = o.view(n, Hq, D).cpu(), lse.view(Hq, n).t().cpu()
        for x in (o, lse):
            assert torch.isnan(x[nan]).all() and torch.isfinite(x[~nan]).all()
        rows = i[torch.randperm(n, generator=g)[:20]]
        for r in rows.tolist():  # the others are the definition's
            lo = max(0, r - window + 1) if window else 0
            for h in range(Hq):
                if nan[r, h]:
                    continue
                kk, vv = (c[0, lo: r + 1, h // (Hq // Hkv)].double().cpu() for c in (k, v))
                s = kk @ q[r, h].double() * p["scale"]
                a = kk.abs() @ q[r, h].double().abs() * p["scale"]
                x = torch.logsumexp(s, 0)
                w = (s - x).exp()
                e = ((2 * D + 8) * ref.U * a + 4 * ref.U * s.abs() + 2.0 ** -21).amax()  # as in operator_ref.tree
                tol = (ref.BF + 2 * e + len(s) * ref.U) * (w @ vv.abs()) + ref.BF * (w @ vv).abs()
                ref.close("o", o[r, h], w @ vv, tol)
                ref.close("lse", lse[r, h][None], x[None], (e + len(s) * ref.U + 2.0 ** -21 * (1 + x.abs()))[None])


@pytest.mark.parametrize("P", [1, 2, 3, 8])
@pytest.mark.parametrize("D", [64, 512])
def test_merge(P, D):
    """A part whose lse is NaN makes the row NaN, beside finite parts and beside empty ones; empty parts still hide theirs."""
    S, H = 40, 3
    g = torch.Generator().manual_seed(57 + P)
    op, lp = torch.randn(P, 1, S, H, D, generator=g).bfloat16(), torch.randn(P, 1, H, S, generator=g)
    lp[:, 0, 1, 5:9] = -math.inf  # no key in any part
    if P > 1:
        lp[P - 1, 0, :, 20:24] = -math.inf
        op[P - 1, 0, 20:24] = math.nan  # of an empty part: not looked at
    w = lp.double().softmax(0).nan_to_num(0.0).transpose(2, 3)[..., None]
    want = (w * op.double().nan_to_num(0.0)).sum(0)
    # fp32 over P parts: P + 8 roundings and the exponentials' (2 ulp, arguments up to 8), then bf16
    tol = ref.BF * want.abs() + (P + 32) * ref.U * (w * op.double().nan_to_num(0.0).abs()).sum(0)
    x = lp.double().logsumexp(0)
    nan = torch.zeros(1, S, H, dtype=torch.bool)
    for p, s, h in ((0, 3, 0), (P - 1, 9, 2), (P // 2, 6, 1), (0, 21, 1)):  # (6, 1): every other part is empty
        lp[p, 0, h, s] = math.nan
        nan[0, s, h] = True
    o, lse = attn.attn_merge_lse(op.cuda(), lp.cuda())
    assert attn.attn_get_device_status() == 0
    rows_but(nan, o, want, tol, "o")
    rows_but(nan, lse.transpose(1, 2), x.transpose(1, 2), torch.full((1, S, H), (P + 32) * ref.U * 8, dtype=torch.float64), "lse")
