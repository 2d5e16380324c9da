"""Attention of drafted token trees over a paged cache (attn_tree_paged) against a 64-bit
implementation; the tolerances are derived in operator_ref."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import operator_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def problem(ctx, n, Hq, Hkv, D, seed=0, words=None, spare=3, poison=True):
    """Random trees behind contexts of these lengths; unused slots and pages hold NaN."""
    g = torch.Generator().manual_seed(seed * 101 + Hq * 7 + D)
    L = [a + b for a, b in zip(ctx, n)]
    npg = [-(-x // 16) for x in L]
    pages = sum(npg) + spare
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(L), max(npg + [1]) + 1), -1, dtype=torch.int32)
    kc, vc = (torch.randn(pages, 16, Hkv, D, generator=g).bfloat16() for _ in range(2))
    at = 0
    for b, x in enumerate(npg):
        table[b, :x] = perm[at: at + x]
        at += x
        if poison and L[b] % 16:
            kc[table[b, x - 1], L[b] % 16:] = math.nan
            vc[table[b, x - 1], L[b] % 16:] = math.nan
    if poison:
        kc[perm[at:].long()] = math.nan
        vc[perm[at:].long()] = math.nan
    words = words or -(-max(n + [1]) // 32)
    mask, pos, cu = [], [], [0]
    for b, x in enumerate(n):
        m, d = ref.random_tree(x, words, g)
        mask += m
        pos += [ctx[b] + i for i in d]
        cu.append(cu[-1] + x)
    T = cu[-1]
    return dict(q=torch.randn(T, Hq, D, generator=g).bfloat16(), kc=kc, vc=vc, table=table, lens=L, cu=cu, n=n, ctx=ctx,
                mask=torch.tensor(mask, dtype=torch.int32).reshape(T, words), pos=torch.tensor(pos, dtype=torch.int32),
                scale=1 / math.sqrt(D))


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def run(p, window=0, max_q=None, **kw):
    return attn.attn_tree_paged(p["q"].cuda(), p["kc"].cuda(), p["vc"].cuda(), p["table"].cuda(), i32(p["lens"]), i32(p["cu"]),
                                p["mask"].cuda(), max(p["n"]) if max_q is None else max_q, scale=p["scale"], window=window,
                                positions=p["pos"].cuda() if window else None, **kw)


def compare(p, window=0, **kw):
    o, lse = run(p, window, **kw)
    assert attn.attn_get_device_status() == 0
    ro, to, rl, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"], window, p["pos"])
    ref.close("o", o, ro, to)
    ref.close("lse", lse, rl, tl)
    return o, lse


# contexts and drafted tokens: nothing cached, one token, borders of pages and of 128-key tiles, no drafts
CTX = [0, 1, 15, 16, 17, 120, 127, 128, 129, 300, 0, 611]
N = [1, 1, 2, 16, 15, 8, 1, 1, 33, 20, 7, 0]


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 3), (3, 1), (4, 2), (5, 1), (8, 1)])
def test_tree(D, G, Hkv):
    compare(problem(CTX, N, G * Hkv, Hkv, D))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("window", [1, 2, 17, 100, 128, 5000])
def test_tree_window(D, window):
    compare(problem(CTX, N, 4, 2, D, seed=window), window)


@pytest.mark.parametrize("D,G", [(64, 7), (128, 1), (128, 4), (128, 16), (128, 100), (256, 6), (512, 2)])
def test_wide_trees(D, G):
    """More rows than one tile, up to the largest tree, and words that no tree fills."""
    compare(problem([200, 0, 40], [256, 130, 65], G, 1, D, words=8))


@pytest.mark.parametrize("D", [128, 256, 512])
def test_long_context(D):
    """A context that many CTAs share, beside short ones."""
    compare(problem([9000, 30, 2500], [5, 3, 9], 8, 2, D))
    compare(problem([9000, 30, 2500], [5, 3, 9], 8, 2, D, seed=1), window=4000)


def test_many_requests():
    ctx = [(37 * i) % 90 for i in range(700)]
    compare(problem(ctx, [1 + i % 3 for i in range(700)], 4, 2, 64))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_rows_that_see_nothing(D):
    """Rows whose mask is empty: with no context (or a window that leaves none) o = 0 and lse = -inf."""
    p = problem([0, 0, 50], [3, 20, 4], 4, 2, D)
    p["mask"][1] = 0
    p["mask"][5] = 0
    p["mask"][24] = 0  # of the third request: its context is still seen
    o, lse = compare(p)
    assert (o[[1, 5]] == 0).all() and (lse[:, [1, 5]] == -math.inf).all() and (lse[:, 24] > -math.inf).all()
    o, lse = compare(p, window=1)
    assert (lse[:, 24] == -math.inf).all()


def test_masks_are_taken_as_they_are():
    """Any pattern: later tokens, all of them, none but one; bits past the drafted tokens are ignored."""
    p = problem([130, 5, 40], [40, 33, 1], 2, 1, 128, words=3)
    g = torch.Generator().manual_seed(3)
    p["mask"] = torch.randint(-2 ** 31, 2 ** 31, p["mask"].shape, generator=g).to(torch.int32)
    p["mask"][0] = -1
    compare(p)


def test_hidden_keys_may_hold_anything():
    """K of a key that no row sees: NaN and infinities in drafted tokens and before the window."""
    for D in (64, 128, 256, 512):
        p = problem([300], [12], 4, 2, D)
        p["mask"] &= ~(1 << 5)  # nobody sees drafted token 5, not even itself
        ref_k = p["kc"].clone()
        at = 305
        p["kc"][p["table"][0, at // 16], at % 16] = math.nan
        first = 300 - 100 + 1  # of the window
        for j in (first - 1, first - first % 16):
            p["kc"][p["table"][0, j // 16], j % 16] = math.inf
        o, lse = run(p, window=100)
        assert attn.attn_get_device_status() == 0
        p["kc"] = ref_k
        ro, to, rl, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"], 100, p["pos"])
        ref.close("o", o, ro, to)
        ref.close("lse", lse, rl, tl)


def test_nothing_to_do():
    p = problem([40], [3], 4, 2, 128)
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for top in (0, 3):
        o, lse = attn.attn_tree_paged(p["q"].cuda()[:0], p["kc"].cuda(), p["vc"].cuda(), e(0, 4), e(0), i32([0]), e(0, 1), top)
        assert o.shape == (0, 4, 128) and lse.shape == (4, 0)
    # requests without drafted tokens only: nothing is written
    o = torch.full((2, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    attn.attn_tree_paged(torch.zeros_like(o), p["kc"].cuda(), p["vc"].cuda(), p["table"].cuda(), i32(p["lens"]), i32([0, 0]),
                         e(2, 1), 3, o)
    assert attn.attn_get_device_status() == 0 and (o == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_single_tiles_and_pairs_in_turn(D):
    """Requests of one, two and three row tiles after one another, short enough that a CTA meets several."""
    n = [3, 40, 1, 70, 90, 2, 33, 64, 5, 6] * 6
    ctx = [(53 * i) % 300 for i in range(len(n))]
    compare(problem(ctx, n, 8, 2, D))


def test_causal_chain_is_chunked_prefill():
    """A tree that is a chain is the causal chunk of attn_fwd_paged."""
    p = problem([100, 0, 513], [31, 20, 1], 8, 2, 256, poison=False)
    rows = []
    for x in p["n"]:
        rows += [[(2 << i) - 1 if i < 31 else -1] for i in range(x)]
    p["mask"] = torch.tensor([[r[0] - (1 << 32) if r[0] >> 31 and r[0] > 0 else r[0]] for r in rows], dtype=torch.int32)
    o, lse = compare(p)
    po, pl = attn.attn_fwd_paged(p["q"].cuda(), p["kc"].cuda(), p["vc"].cuda(), p["table"].cuda(), i32(p["lens"]), i32(p["cu"]),
                                 max(p["n"]), scale=p["scale"])
    assert attn.attn_get_device_status() == 0
    ro, to, rl, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"])
    ref.close("o against the chunk", o, po.double().cpu(), 2 * to)
    ref.close("lse against the chunk", lse, pl.double().cpu(), 2 * tl)


def test_large_scores():
    """Scores that grow along the context (the running maximum moves on every tile) and large magnitudes."""
    for D in (128, 512):
        p = problem([700], [6], 4, 1, D)
        pages = -(-706 // 16)
        p["kc"][p["table"][0, :pages].long()] *= torch.linspace(0.1, 6, pages)[:, None, None, None].bfloat16()
        compare(p)


def test_rows_behind_the_last_request_and_empty_ones():
    """q may hold more rows than cu_q ends with: they are left as they were."""
    p = problem([40, 0, 77], [3, 0, 6], 4, 2, 128)
    q = torch.cat([p["q"], torch.full((4, 4, 128), math.nan).bfloat16()])
    o = torch.full((13, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 13), 7.0, device="cuda")
    mask = torch.cat([p["mask"], torch.zeros(4, 1, dtype=torch.int32)])
    attn.attn_tree_paged(q.cuda(), p["kc"].cuda(), p["vc"].cuda(), p["table"].cuda(), i32(p["lens"]), i32(p["cu"]), mask.cuda(), 6,
                         o, lse, scale=p["scale"])
    assert attn.attn_get_device_status() == 0
    ro, to, rl, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"])
    ref.close("o", o[:9], ro, to)
    ref.close("lse", lse[:, :9], rl, tl)
    assert (o[9:] == 7.0).all() and (lse[:, 9:] == 7.0).all()


@pytest.mark.parametrize("D", [128, 512])
def test_inconsistent_requests_are_reported_and_skipped(D):
    base = problem([40, 30, 77, 20], [3, 5, 6, 4], 4, 2, D)
    ro, to, rl, tl = ref.tree(base["q"], base["kc"], base["vc"], base["table"], base["lens"], base["cu"], base["mask"], base["scale"])
    cap = base["table"].shape[1] * 16

    def check(lens, cu, max_q, bad_rows):
        o = torch.full((18, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, 18), 7.0, device="cuda")
        attn.attn_tree_paged(base["q"].cuda(), base["kc"].cuda(), base["vc"].cuda(), base["table"].cuda(), i32(lens), i32(cu),
                             base["mask"].cuda(), max_q, o, lse, scale=base["scale"])
        assert attn.attn_get_device_status() == 7
        good = torch.ones(18, dtype=torch.bool)
        good[bad_rows] = False
        ref.close("o", o.cpu()[good], ro[good], to[good])
        ref.close("lse", lse.cpu()[:, good], rl[:, good], tl[:, good])
        assert (o.cpu()[~good] == 7.0).all() and (lse.cpu()[:, ~good] == 7.0).all()

    L, cu = base["lens"], base["cu"]
    rows = [range(a, b) for a, b in zip(cu, cu[1:])]
    check([L[0], 2, L[2], L[3]], cu, 6, rows[1])             # more drafted than cached
    check([L[0], L[1], cap + 1, L[3]], cu, 6, rows[2])       # longer than its block-table row
    check([L[0], -4, L[2], L[3]], cu, 6, rows[1])
    check(L, cu, 5, rows[2])                                  # more drafted than max_q_len
    check(L, cu[:4] + [19], 6, rows[3])                       # past the rows
    check(L, [-1] + cu[1:], 6, rows[0])
    check(L, [0, 3, 2, 14, 18], 6, list(rows[1]) + list(rows[2]))  # decreasing, then more than max_q_len


@pytest.mark.parametrize("D", [64, 128, 512])
@pytest.mark.parametrize("R", [1, 31, 32, 33, 64, 65])
def test_numbers_of_requests(D, R):
    """Up to 32 requests each warp finds its share alone, beyond that the CTA does; the one in the middle is skipped."""
    p = problem([(61 * i) % 200 for i in range(R)], [i % 4 if i else 2 for i in range(R)], 4, 2, D)
    bad = R // 2 if R > 1 else None
    lens = list(p["lens"])
    if bad is not None:
        lens[bad] = -1
    T = p["cu"][-1]
    o = torch.full((T, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, T), 7.0, device="cuda")
    attn.attn_tree_paged(p["q"].cuda(), p["kc"].cuda(), p["vc"].cuda(), p["table"].cuda(), i32(lens), i32(p["cu"]), p["mask"].cuda(),
                         3, o, lse, scale=p["scale"])
    assert attn.attn_get_device_status() == (0 if bad is None else 7)
    ro, to, rl, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"])
    good = torch.ones(T, dtype=torch.bool)
    if bad is not None:
        good[p["cu"][bad]: p["cu"][bad + 1]] = False
    ref.close("o", o.cpu()[good], ro[good], to[good])
    ref.close("lse", lse.cpu()[:, good], rl[:, good], tl[:, good])
    assert (o.cpu()[~good] == 7.0).all() and (lse.cpu()[:, ~good] == 7.0).all()


@pytest.mark.parametrize("D,Hkv,G,n,window", [(256, 5, 6, [37, 5, 20], 1024), (256, 1, 4, [58, 3, 30], 0), (128, 3, 4, [41, 33, 37], 0),
                                               (512, 4, 4, [4, 6, 1], 0), (64, 11, 2, [28, 12, 3], 0), (128, 4, 1, [6, 6, 6], 0)])
def test_shares_within_segments(D, Hkv, G, n, window):
    """Few units: every CTA's share lies in one segment, and segments of different lengths are cut evenly."""
    for seed, ctx in enumerate(([1500, 300, 2300], [129, 127, 120], [640, 0, 9])):
        compare(problem(ctx, n, Hkv * G, Hkv, D, seed=seed), window)


def test_bad_page_ids_are_reported():
    """A page id outside the pool stands for page 0; other requests are not touched."""
    p = problem([40, 30], [3, 5], 4, 2, 128, poison=False)
    p["table"][0, 1] = 10 ** 6
    o, lse = run(p)
    assert attn.attn_get_device_status() == 7
    p["table"][0, 1] = 0
    ro, to, rl, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"])
    ref.close("o", o, ro, to)
    ref.close("lse", lse, rl, tl)


def test_same_bits_every_time_and_on_dirty_workspaces():
    for D in (128, 256):
        p = problem([3000, 500, 0, 90], [9, 4, 20, 1], 8, 2, D)
        o, lse = run(p)
        need = attn.attn_workspace_size(attn.ATTN_OP_TREE_PAGED, Hq=8, Hkv=2, S=20, D=D)
        for fill in (0, 255):
            ws = torch.full((max(need, 256),), fill, dtype=torch.uint8, device="cuda")
            o2, l2 = run(p, workspace=ws)
            assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_two_streams_at_once():
    """Two calls that may overlap on the GPU: each has a workspace of its own."""
    ps = [problem([5000, 800], [6, 9], 8, 2, 128, seed=s) for s in (1, 2)]
    want = [run(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    dev = [[p[k].cuda() for k in ("q", "kc", "vc", "table")] + [i32(p["lens"]), i32(p["cu"]), p["mask"].cuda()] for p in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [attn.attn_tree_paged(*d, 9, scale=p["scale"], stream=s) for p, d, s in zip(ps, dev, streams)]
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_captured_with_a_padded_batch():
    """Captured for four requests of up to 9 tokens and replayed for a smaller step: the lengths are read on the device."""
    big = problem([500, 60, 33, 90], [9, 4, 8, 1], 8, 2, 128)
    small = problem([400, 60, 0, 20], [3, 4, 0, 1], 8, 2, 128, seed=4, words=1)
    d = dict(q=big["q"].cuda(), kc=big["kc"].cuda(), vc=big["vc"].cuda(), table=big["table"].cuda(), lens=i32(big["lens"]),
             cu=i32(big["cu"]), mask=big["mask"].cuda())
    o, lse = torch.zeros_like(d["q"]), torch.zeros(8, 22, device="cuda")
    call = lambda: attn.attn_tree_paged(d["q"], d["kc"], d["vc"], d["table"], d["lens"], d["cu"], d["mask"], 9, o, lse,  # noqa: E731
                                        scale=big["scale"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize()
    ro, to, rl, tl = ref.tree(big["q"], big["kc"], big["vc"], big["table"], big["lens"], big["cu"], big["mask"], big["scale"])
    ref.close("o", o, ro, to)
    ref.close("lse", lse, rl, tl)
    T = small["cu"][-1]
    pages = small["kc"].shape[0]
    d["q"][:T].copy_(small["q"])
    d["mask"][:T].copy_(small["mask"])
    d["kc"][:pages].copy_(small["kc"])
    d["vc"][:pages].copy_(small["vc"])
    d["table"].fill_(-1)
    d["table"][:, : small["table"].shape[1]].copy_(small["table"])
    d["lens"].copy_(i32(small["lens"]))
    d["cu"].copy_(i32(small["cu"]))
    o.fill_(7.0)
    g.replay()
    assert attn.attn_get_device_status() == 0
    ro, to, rl, tl = ref.tree(small["q"], small["kc"], small["vc"], small["table"], small["lens"], small["cu"], small["mask"],
                              small["scale"])
    ref.close("o", o[:T], ro, to)
    ref.close("lse", lse[:, :T], rl, tl)
    assert (o[T:] == 7.0).all()
