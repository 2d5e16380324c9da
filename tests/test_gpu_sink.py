"""Windows with sinks on the GPU: forward (dense, packed, over a paged cache), gradient and single-token decode
against the 64-bit definition, and the calls that must agree with those without sinks bit by bit."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import sink_ref as ref
from operator_ref import close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def rows(T, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv, Hq)]


def cu_of(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


# lengths around the tile of 128 and the window's edge; sinks of one key, of a whole tile, of more than the sequence
SHAPES = [(1, 1, 1), (130, 1, 1), (257, 64, 4), (300, 128, 128), (513, 100, 17), (700, 129, 64), (385, 256, 127), (200, 1000, 4), (60, 5, 128)]


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (128, 4, 2), (256, 2, 2), (256, 6, 3), (512, 4, 2), (512, 3, 1)])
@pytest.mark.parametrize("S,window,sink", SHAPES)
def test_forward(D, Hq, Hkv, S, window, sink):
    scale = 1 / math.sqrt(D)
    q, k, v, _ = rows(2 * S, Hq, Hkv, D, S + D)
    want = ref.packed(lambda *x: ref.forward(*x, scale, window, sink), [S, S], q, k, v)
    a, b, c = (x.view(2, S, -1, D).cuda() for x in (q, k, v))
    o, lse = attn.attn_fwd(a, b, c, window=window, sink=sink, scale=scale)
    close("o", o.flatten(0, 1), want[0], want[1])
    close("lse", lse.transpose(0, 1).flatten(1), want[2], want[3])
    po, plse = attn.attn_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cu_of([S, S]), S, window=window, sink=sink, scale=scale)
    assert torch.equal(po, o.flatten(0, 1)) and torch.equal(plse, lse.transpose(0, 1).flatten(1))
    assert attn.attn_get_device_status() == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 4, 2), (256, 2, 1), (512, 4, 2)])
@pytest.mark.parametrize("window,sink", [(1, 1), (100, 4), (128, 30)])
def test_packed(D, Hq, Hkv, window, sink):
    lens = [1, 0, 129, 400, 64, 128, 300, 2]
    scale = 0.2
    q, k, v, do = rows(sum(lens), Hq, Hkv, D, 3)
    want = ref.packed(lambda *x: ref.forward(*x, scale, window, sink), lens, q, k, v)
    grad = ref.packed(lambda *x: ref.backward(*x, scale, window, sink), lens, q, k, v, do)
    q, k, v, do = (x.cuda() for x in (q, k, v, do))
    o, lse = attn.attn_fwd_varlen(q, k, v, cu_of(lens), 401, window=window, sink=sink, scale=scale)
    close("o", o, want[0], want[1])
    close("lse", lse, want[2], want[3])
    got = attn.attn_bwd(q, k, v, o, lse, do, window=window, sink=sink, scale=scale, cu_seqlens=cu_of(lens), max_seqlen=401)
    assert attn.attn_get_device_status() == 0
    for i, name in enumerate(("dq", "dk", "dv")):
        close(name, got[i], grad[2 * i], grad[2 * i + 1])


# the longer ones have far queries in one, two and several slices; 2600: the last slice is shorter
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (128, 4, 2), (256, 2, 1), (512, 2, 1)])
@pytest.mark.parametrize("S,window,sink", SHAPES + [(1300, 130, 4), (2600, 5, 3), (2305, 1, 128)])
def test_gradient(D, Hq, Hkv, S, window, sink):
    scale = 1 / math.sqrt(D)
    B = 2 if S < 1000 else 1
    x = rows(B * S, Hq, Hkv, D, S + D)
    want = ref.packed(lambda *t: ref.backward(*t, scale, window, sink), [S] * B, *x)
    q, k, v, do = (t.view(B, S, -1, D).cuda() for t in x)
    o, lse = attn.attn_fwd(q, k, v, window=window, sink=sink, scale=scale)
    got = attn.attn_bwd(q, k, v, o, lse, do, window=window, sink=sink, scale=scale)
    assert attn.attn_get_device_status() == 0
    for i, name in enumerate(("dq", "dk", "dv")):
        close(name, got[i].flatten(0, 1), want[2 * i], want[2 * i + 1])
    again = attn.attn_bwd(q, k, v, o, lse, do, window=window, sink=sink, scale=scale)
    assert torch.equal(got[1], again[1]) and torch.equal(got[2], again[2])


# queries past the first tile's windows in many sequences, with empty ones and some without such queries between them
MANY = [([130, 0, 129, 257, 5, 0, 300, 193] * 5, 1), ([700, 1, 1100], 60), ([4] * 1100 + [260, 40, 280], 3)]


def check_gradient_packed(D, Hq, Hkv, sink, lens, window, device="cpu"):
    scale, T = 1 / math.sqrt(D), sum(lens)
    q, k, v, do = (x.to(device) for x in rows(T + 3, Hq, Hkv, D, sink + D))  # three rows behind the last sequence
    with torch.device(device):
        want = ref.packed(lambda *x: ref.backward(*x, scale, window, sink), lens, *(x[:T] for x in (q, k, v, do)))
    q, k, v, do = (x.cuda() for x in (q, k, v, do))
    o, lse = attn.attn_fwd_varlen(q, k, v, cu_of(lens), max(lens), window=window, sink=sink, scale=scale)
    dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
    attn.attn_bwd(q, k, v, o, lse, do, dq, dk, dv, window=window, sink=sink, scale=scale, cu_seqlens=cu_of(lens), max_seqlen=max(lens))
    assert attn.attn_get_device_status() == 0
    assert bool((dk[T:] == 7.0).all()) and bool((dv[T:] == 7.0).all())
    for i, (name, got) in enumerate((("dq", dq), ("dk", dk), ("dv", dv))):
        close(name, got[:T].cpu(), want[2 * i].cpu(), want[2 * i + 1].cpu())
    return q, k, v, o, lse, do, dk, dv


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (128, 4, 2), (256, 2, 1), (512, 2, 2)])
@pytest.mark.parametrize("sink", [2, 16, 17])
@pytest.mark.parametrize("lens,window", MANY)
def test_gradient_packed(D, Hq, Hkv, sink, lens, window):
    check_gradient_packed(D, Hq, Hkv, sink, lens, window)


# 2^25 elements of q and more, with few sinks: the far queries are a kernel's own. (The 64-bit side on the GPU as well.)
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 64, 64), (64, 96, 2), (128, 40, 8), (128, 64, 1), (256, 32, 16), (256, 33, 11)])
@pytest.mark.parametrize("sink", [1, 16])
@pytest.mark.parametrize("lens,window", [(x * (9000 // sum(x) + 1), w) for x, w in MANY[:2]] + [([40] * 200 + [261] * 5, 3)])
def test_gradient_packed_of_large_calls(D, Hq, Hkv, sink, lens, window):
    assert (sum(lens) + 3) * Hq * D >= 2 ** 25
    q, k, v, o, lse, do, dk, dv = check_gradient_packed(D, Hq, Hkv, sink, lens, window, "cuda")
    again = attn.attn_bwd(q, k, v, o, lse, do, window=window, sink=sink, scale=1 / math.sqrt(D), cu_seqlens=cu_of(lens), max_seqlen=max(lens))
    T = sum(lens)
    assert torch.equal(again[1][:T], dk[:T]) and torch.equal(again[2][:T], dv[:T])


@pytest.mark.parametrize("D,Hq,Hkv,B,S,window,sink", [(64, 64, 8, 33, 257, 1, 16), (128, 32, 16, 3, 2777, 130, 5), (256, 24, 4, 8, 700, 300, 3)])
def test_gradient_of_large_calls(D, Hq, Hkv, B, S, window, sink):
    assert B * S * Hq * D >= 2 ** 25
    scale = 1 / math.sqrt(D)
    x = [t.cuda() for t in rows(B * S, Hq, Hkv, D, S + D)]
    with torch.device("cuda"):
        want = ref.packed(lambda *t: ref.backward(*t, scale, window, sink), [S] * B, *x)
    q, k, v, do = (t.view(B, S, -1, D) for t in x)
    o, lse = attn.attn_fwd(q, k, v, window=window, sink=sink, scale=scale)
    got = attn.attn_bwd(q, k, v, o, lse, do, window=window, sink=sink, scale=scale)
    assert attn.attn_get_device_status() == 0
    for i, name in enumerate(("dq", "dk", "dv")):
        close(name, got[i].flatten(0, 1).cpu(), want[2 * i].cpu(), want[2 * i + 1].cpu())


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_gradient_against_differences(D):
    """The GPU's gradient along a direction against the difference of the 64-bit loss on both sides."""
    S, window, sink, scale = 1200, 40, 3, 1 / math.sqrt(D)
    x = rows(S, 2, 1, D, 9)
    want = ref.backward(*x, scale, window, sink)
    q, k, v, do = (t.view(1, S, -1, D).cuda() for t in x)
    o, lse = attn.attn_fwd(q, k, v, window=window, sink=sink, scale=scale)
    got = attn.attn_bwd(q, k, v, o, lse, do, window=window, sink=sink, scale=scale)
    d = rows(S, 2, 1, D, 10)[:3]
    h = 1e-4

    def loss(w):
        y = [t.double() + w * h * e.double() for t, e in zip(x[:3], d)]
        return (ref.forward(*y, scale, window, sink)[0] * x[3].double()).sum()

    got = sum((a[0].double().cpu() * e.double()).sum() for a, e in zip(got, d))
    # a value's bound counts once; the difference itself is off by the loss's third derivative, of its own size times h^2
    tol = sum((t * e.double().abs()).sum() for t, e in zip(want[1::2], d)) + 1e-6 * sum((a * e.double()).abs().sum() for a, e in zip(want[::2], d))
    assert abs((loss(1) - loss(-1)) / (2 * h) - got) <= tol


@pytest.mark.parametrize("D,G", [(64, 1), (128, 2), (256, 2), (512, 2), (512, 1)])
def test_agrees_with_calls_without_sinks(D, G):
    """No sink, no window, a window that is never left, sinks that the window always covers: the same bits."""
    S = 400
    q, k, v, do = (t.view(1, S, -1, D).cuda() for t in rows(S, 2 * G, 2, D, 4))
    for a, b in [(dict(window=70, sink=0), dict(window=70)), (dict(window=0, sink=9), {}), (dict(window=S, sink=9), {}), (dict(window=S + 50, sink=9), {}),
                 (dict(window=S - 1, sink=0), dict(window=S - 1))]:
        (o, lse), (po, plse) = attn.attn_fwd(q, k, v, **a), attn.attn_fwd(q, k, v, **b)
        assert torch.equal(o, po) and torch.equal(lse, plse), a
        x, y = attn.attn_bwd(q, k, v, o, lse, do, **a), attn.attn_bwd(q, k, v, o, lse, do, **b)
        assert torch.equal(x[1], y[1]) and torch.equal(x[2], y[2]), a
    assert attn.attn_get_device_status() == 0


def paged(lens, Hkv, D, seed, window, sink, new=None):
    """A cache whose pages that no query sees, and slots past the end, hold NaN, and stale table entries for such pages."""
    g = torch.Generator().manual_seed(seed)
    npg = [-(-n // 16) for n in lens]
    pages = sum(npg) + 3
    ids = torch.randperm(pages, generator=g)[: sum(npg)].tolist()
    kc, vc = (torch.full((pages, 16, Hkv, D), math.nan).bfloat16() for _ in range(2))
    table = torch.full((len(lens), max(npg) + 2), -7, dtype=torch.int32)
    seqs = []
    for b, n in enumerate(lens):
        k, v = (torch.randn(n, Hkv, D, generator=g).bfloat16() for _ in range(2))
        seqs.append((k, v))
        first = max(0, n - (new[b] if new else 1) - window + 1) if window else 0
        for p in range(npg[b]):
            page = ids.pop()
            if p * 16 >= sink and p < first // 16:
                continue  # given back
            table[b, p] = page
            m = min(16, n - 16 * p)
            kc[page, :m], vc[page, :m] = k[16 * p: 16 * p + m], v[16 * p: 16 * p + m]
    return kc, vc, table, seqs


@pytest.mark.parametrize("D,G", [(64, 2), (128, 4), (256, 2), (512, 1), (512, 2)])
@pytest.mark.parametrize("window,sink", [(1, 1), (50, 4), (100, 40), (16, 128), (129, 16)])
def test_chunk_over_pages(D, G, window, sink):
    lens, new = [700, 33, 300, 1, 900, 17], [130, 33, 1, 1, 300, 2]
    Hkv, scale = 2, 0.15
    kc, vc, table, seqs = paged(lens, Hkv, D, 6, window, sink, new)
    g = torch.Generator().manual_seed(7)
    q = torch.randn(sum(new), G * Hkv, D, generator=g).bfloat16()
    o, lse = attn.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu_of(new), 300,
                                 window=window, sink=sink, scale=scale)
    assert attn.attn_get_device_status() == 0
    at = 0
    for (k, v), n in zip(seqs, new):
        ro, to, rl, tl = ref.forward(q[at: at + n], k, v, scale, window, sink)
        close("o", o[at: at + n], ro, to)
        close("lse", lse[:, at: at + n], rl, tl)
        at += n


@pytest.mark.parametrize("D,G", [(128, 1), (128, 2), (128, 4), (128, 8), (256, 1), (256, 2), (256, 4)])
@pytest.mark.parametrize("window,sink", [(1, 1), (50, 4), (33, 40), (16, 128), (100, 17), (128, 16), (5000, 4), (0, 4)])
@pytest.mark.parametrize("lens", [[1, 16, 17, 700, 0, 100, 33, 129, 51], [3000]])
def test_decode(D, G, window, sink, lens):
    Hkv, scale = 2, 0.15
    kc, vc, table, seqs = paged(lens, Hkv, D, 8, window, sink)
    q = torch.randn(len(lens), G * Hkv, D, generator=torch.Generator().manual_seed(9)).bfloat16()
    o, lse = attn.attn_decode_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), window=window,
                                    sink=sink, scale=scale)
    assert attn.attn_get_device_status() == 0
    for b, (k, v) in enumerate(seqs):
        if lens[b] == 0:
            assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        ro, to, rl, tl = ref.forward(q[b: b + 1], k, v, scale, window, sink)
        close("o", o[b: b + 1], ro, to)
        close("lse", lse[b][:, None], rl, tl)


@pytest.mark.parametrize("D", [128, 256])
def test_captured(D):
    """Training step and decode in a graph; the eager calls between two replays leave the replays as they are."""
    S, how = 1500, dict(window=60, sink=4)
    q, k, v, do = (t.view(1, S, -1, D).cuda() for t in rows(S, 4, 2, D, 5))
    kc, vc, table, _ = (t.cuda() if torch.is_tensor(t) else t for t in paged([500, 90], 2, D, 6, 60, 4))
    lens = torch.tensor([500, 90], dtype=torch.int32).cuda()
    qd = q[0, :2].contiguous()

    def step():
        o, lse = attn.attn_fwd(q, k, v, **how)
        _, dk, dv = attn.attn_bwd(q, k, v, o, lse, do, **how)
        return [o, lse, dk, dv, *attn.attn_decode_paged(qd, kc, vc, table, lens, **how)]

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        step()
    assert attn.attn_get_device_status() == 0


def test_bad_slices_are_reported():
    """Packed sequences whose prefix sums are bad are left alone, with their sinks; the others are computed."""
    D, how = 128, dict(window=30, sink=4, scale=0.1)
    lens = [1300, 1400, 300]
    x = rows(sum(lens), 2, 1, D, 12)
    want = ref.packed(lambda *t: ref.backward(*t, 0.1, 30, 4), [1300], *(t[:1300] for t in x))
    q, k, v, do = (t.cuda() for t in x)
    cu = torch.tensor([0, 1300, 2700, 3100], dtype=torch.int32).cuda()  # the last one is too long
    good = cu_of(lens)
    o, lse = attn.attn_fwd_varlen(q, k, v, good, 1400, **how)
    dq, dk, dv = (torch.full_like(t, 7) for t in (q, k, v))
    attn.attn_bwd(q, k, v, o, lse, do, dq, dk, dv, cu_seqlens=cu, max_seqlen=1350, **how)  # and the second one longer than it says
    assert attn.attn_get_device_status() == 7
    for i, t in enumerate((dq, dk, dv)):
        close("first", t[:1300], want[2 * i], want[2 * i + 1])
    assert (dk[1300:] == 7).all() and (dv[1300:] == 7).all() and (dq[1300:] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_gradient_of_scores_that_fp32_holds_coarsely(D):
    """Scores of 2^27 and more: their logsumexp is off by whole numbers, P by powers of two, but nothing overflows."""
    S = 200
    q, k, v, do = (t.view(1, S, -1, D) for t in rows(S, 2, 1, D, 27))
    q[..., 0] = 2.0 ** 13 * (1 + q[..., 0].abs() / 8)
    k[..., 0] = 2.0 ** 14 * (1 + k[..., 0].abs() / 8)
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    for window, sink in ((0, 0), (70, 4)):
        o, lse = attn.attn_fwd(q, k, v, window=window, sink=sink, scale=1.0)
        got = attn.attn_bwd(q, k, v, o, lse, do, window=window, sink=sink, scale=1.0)
        assert attn.attn_get_device_status() == 0
        assert all(bool(t.isfinite().all()) for t in (o, lse, *got))


@pytest.mark.parametrize("D,Hq,Hkv,sink,lens,window", [
    (128, 4, 2, 100, [700, 1, 0, 1100, 130, 129], 1), (512, 4, 1, 4, [900, 640, 3], 100), (64, 3, 3, 16, [2000, 129, 128], 5),
    (128, 40, 8, 16, [300, 150, 129, 700] * 6, 20), (256, 33, 11, 3, [129] * 40, 1), (64, 96, 2, 7, [5999], 1)])
def test_gradient_in_a_given_workspace(D, Hq, Hkv, sink, lens, window):
    """Exactly the bytes that attn_bwd_sink_workspace_size names, whatever they hold, and none behind them."""
    T, scale = sum(lens), 1 / math.sqrt(D)
    q, k, v, do = (x.cuda() for x in rows(T, Hq, Hkv, D, 31))
    at = dict(window=window, sink=sink, scale=scale, cu_seqlens=cu_of(lens), max_seqlen=max(lens))
    o, lse = attn.attn_fwd_varlen(q, k, v, at["cu_seqlens"], max(lens), window=window, sink=sink, scale=scale)
    want = attn.attn_bwd(q, k, v, o, lse, do, **at)
    n = attn.attn_bwd_sink_workspace_size(1, Hq, Hkv, T, D, len(lens), window, sink)
    room = torch.full((n + (64 << 20),), 255, dtype=torch.uint8, device="cuda")  # (NaN, were it read)
    given = [torch.empty_like(x) for x in (q, k, v)]
    got = attn.attn_bwd(q, k, v, o, lse, do, *given, workspace=room[:n], **at)
    assert all(a is b for a, b in zip(got, given)) and attn.attn_get_device_status() == 0
    assert bool((room[n:] == 255).all())
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2]) and bool(got[0].isfinite().all())
    with pytest.raises(attn.AttnError):
        attn.attn_bwd(q, k, v, o, lse, do, *given, workspace=room[:n - 1], **at)


def test_bad_slices_of_a_large_call():
    """As above, where the far queries are a kernel's own."""
    D, Hq, how = 128, 96, dict(window=30, sink=4, scale=0.1)
    lens = [1300, 1400, 300]
    assert sum(lens) * Hq * D >= 2 ** 25
    x = [t.cuda() for t in rows(sum(lens), Hq, 3, D, 12)]
    with torch.device("cuda"):
        want = ref.packed(lambda *t: ref.backward(*t, 0.1, 30, 4), [1300], *(t[:1300] for t in x))
    q, k, v, do = x
    o, lse = attn.attn_fwd_varlen(q, k, v, cu_of(lens), 1400, **how)
    dq, dk, dv = (torch.full_like(t, 7) for t in (q, k, v))
    cu = torch.tensor([0, 1300, 2700, 3100], dtype=torch.int32).cuda()
    attn.attn_bwd(q, k, v, o, lse, do, dq, dk, dv, cu_seqlens=cu, max_seqlen=1350, **how)
    assert attn.attn_get_device_status() == 7
    for i, t in enumerate((dq, dk, dv)):
        close("first", t[:1300].cpu(), want[2 * i].cpu(), want[2 * i + 1].cpu())
    assert (dk[1300:] == 7).all() and (dv[1300:] == 7).all() and (dq[1300:] == 0).all()


def test_large_gradient_captured_and_on_two_streams():
    S, D, how = 4200, 256, dict(window=500, sink=16)
    q, k, v, do = (t.view(1, S, -1, D).cuda() for t in rows(S, 32, 16, D, 8))
    assert q.numel() >= 2 ** 25
    o, lse = attn.attn_fwd(q, k, v, **how)
    want = attn.attn_bwd(q, k, v, o, lse, do, **how)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [attn.attn_bwd(q, k, v, o, lse, do, stream=s, **how) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g in got for x, y in zip(g[1:], want[1:]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn.attn_bwd(q, k, v, o, lse, do, **how)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        assert (got[0].float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()  # (fp32 sums in no fixed order)
    assert attn.attn_get_device_status() == 0
