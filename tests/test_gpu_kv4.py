"""The 4-bit paged cache on the GPU: what append writes, byte by byte, what unpack reads, and decode over it against the
64-bit definition."""
import math

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import kv4_ref as ref
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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def noise(P, H, D, seed):
    """A cache that holds anything: random bytes."""
    return torch.randint(0, 256, (P, H, 18, D), generator=gen(seed), dtype=torch.uint8)


def same(a, b):
    """Equal values, NaN where the other has NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0), b.nan_to_num(0))


# ---- append and unpack -------------------------------------------------------------------------

def odd_rows(T, H, D, seed):
    """Rows with all that a group may hold: zeros, subnormals, the largest numbers, ties, infinities, NaN, any bit pattern."""
    g = gen(seed)
    x = (torch.randn(T, H, D, generator=g) * torch.exp(3 * torch.randn(T, H, 1, generator=g))).bfloat16()
    if T >= 8:
        x[0] = 0
        x[1] = 1e-39
        x[2, :, :40] = 3e38
        x[3] = (torch.randint(-16, 17, (H, D), generator=g) / 4).bfloat16()  # many exact ties
        x[4, 0, 5], x[5, 0, 33] = math.inf, math.nan
        x[6] = torch.randint(-32768, 32768, (H, D), generator=g).to(torch.int16).view(torch.bfloat16)
        x[7, :, 0], x[7, :, 1] = 9, -9
    return x


@pytest.mark.parametrize("D,H", [(64, 1), (64, 5), (128, 8), (128, 3), (256, 1), (256, 16)])
@pytest.mark.parametrize("T", [1, 9, 100, 1000])
def test_append(D, H, T):
    P = T // 8 + 3
    g = gen(T + D)
    k, v = odd_rows(T, H, D, 1), odd_rows(T, H, D, 2)
    slots = torch.randperm(16 * P, generator=g)[:T].to(torch.int32)
    if T > 20:
        slots[11] = slots[17] = -1
    cache = noise(P, H, D, 3)
    got = cache.cuda()
    assert attn.attn_kv4_append(k.cuda(), v.cuda(), slots.cuda(), got) is None
    want = ref.put(cache.clone(), slots, k, v)
    got = got.cpu()
    half = [x.view(P, H, -1).view(torch.bfloat16)[..., 8 * D:] for x in (got, want)]
    assert same(*half)
    codes = [x.view(P, H, -1)[..., : 16 * D] for x in (got, want)]
    assert torch.equal(*codes)
    assert attn.attn_get_device_status() == 0


def test_every_value_against_every_scale():
    """All bf16 numbers next to a largest one of each of the 128 mantissas, whose scale takes each of its 16 values."""
    D, H = 64, 1
    top = torch.arange(128, 256).repeat_interleave(32) / 128.0  # in [1, 2)
    x = torch.zeros(128 * 32, 1, 64)
    mant = torch.arange(128, 256).repeat(32)[: 128 * 31].view(128, 31)  # 31 others a group, every mantissa within 5 rows
    for sign in (1, -1):
        for e in range(-8, 1):
            rows = x.view(128, 32, 64)
            rows[:, :, 0] = sign * top.view(128, 32)
            for r in range(32):
                others = ((mant + 31 * r - 128) % 128 + 128) / 128.0 * 2.0 ** e
                rows[:, r, 1:32] = torch.minimum(others, torch.full_like(others, 0.0) + top.view(128, 32)[:, r: r + 1])
                rows[:, r, 32:] = -rows[:, r, :32]
            b = x.bfloat16()
            cache = torch.zeros(256, 1, 18, D, dtype=torch.uint8, device="cuda")
            attn.attn_kv4_append(b.cuda(), (-b).cuda(), i32(torch.arange(4096)), cache)
            k, v = attn.attn_kv4_unpack(cache, i32(torch.arange(256)))
            assert torch.equal(k.view(4096, 1, 64).cpu().double(), ref.values(b)) and torch.equal(v.view(4096, 1, 64).cpu().double(), ref.values(-b))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_strided_rows(D):
    T, H = 37, 3
    qkv = torch.randn(T, 5 * H * D, generator=gen(4)).bfloat16()
    k, v = qkv[:, 2 * H * D: 3 * H * D].view(T, H, D), qkv[:, 4 * H * D:].view(T, H, D)
    slots = torch.randperm(48, generator=gen(5))[:T]
    dev = qkv.cuda()
    cache = torch.zeros(3, H, 18, D, dtype=torch.uint8, device="cuda")
    attn.attn_kv4_append(dev[:, 2 * H * D: 3 * H * D].view(T, H, D), dev[:, 4 * H * D:].view(T, H, D), i32(slots), cache)
    assert torch.equal(cache.cpu(), ref.put(torch.zeros(3, H, 18, D, dtype=torch.uint8), slots, k, v))
    # [B, S, H, D] with slots [B, S]
    cache.zero_()
    attn.attn_kv4_append(k[:36].view(4, 9, H, D).cuda(), v[:36].reshape(4, 9, H, D).cuda(), i32(slots[:36]).view(4, 9), cache)
    assert torch.equal(cache.cpu(), ref.put(torch.zeros(3, H, 18, D, dtype=torch.uint8), slots[:36], k[:36], v[:36]))


def test_bad_slots_and_pages():
    D, H, P = 128, 2, 4
    k, v = (torch.randn(6, H, D, generator=gen(s)).bfloat16() for s in (6, 7))
    slots = torch.tensor([3, 64, -1, 40, -2, 2 ** 31 - 1])
    cache = noise(P, H, D, 8)
    cache.view(P, H, -1)[..., 16 * D:] = 0
    got = cache.cuda()
    attn.attn_kv4_append(k.cuda(), v.cuda(), i32(slots), got)
    assert attn.attn_get_device_status() == 7
    want = ref.put(cache.clone(), slots, k, v)
    assert torch.equal(got.cpu(), want)
    out = [torch.full((5, 16, H, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    attn.attn_kv4_unpack(got, i32([2, -1, 4, 0, 2]), *out)
    assert attn.attn_get_device_status() == 7
    for x, y in zip(out, ref.get(want)):
        assert (x[1:3] == 3).all() and torch.equal(x[[0, 3, 4]].cpu().double(), y[[2, 0, 2]])
    attn.attn_kv4_unpack(got, i32([-1, 1]))
    attn.attn_kv4_append(k[:1].cuda(), v[:1].cuda(), i32([-1]), got)
    assert attn.attn_get_device_status() == 0 and torch.equal(got.cpu(), want)


@pytest.mark.parametrize("D,H", [(64, 7), (128, 8), (256, 3)])
@pytest.mark.parametrize("n", [1, 33, 300])
def test_unpack(D, H, n):
    P = 40
    cache = noise(P, H, D, n)
    half = cache.view(P, H, -1).view(torch.bfloat16)[..., 8 * D:]
    s = torch.randn(half.shape, generator=gen(9)).bfloat16().view(torch.int16) & ~7  # 5 significant bits
    half.copy_(s.view(torch.bfloat16))
    pages = torch.randint(0, P, (n,), generator=gen(10))
    k, v = attn.attn_kv4_unpack(cache.cuda(), i32(pages))
    rk, rv = ref.get(cache)
    assert torch.equal(k.cpu().double(), rk[pages]) and torch.equal(v.cpu().double(), rv[pages])
    assert attn.attn_get_device_status() == 0


def test_nothing_to_do():
    D, H = 128, 2
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    cache = e(0, H, 18, D, t=torch.uint8)
    attn.attn_kv4_append(e(0, H, D), e(0, H, D), i32([]), cache)
    k, v = attn.attn_kv4_unpack(cache, i32([]))
    assert k.shape == v.shape == (0, 16, H, D)
    o, lse = attn.attn_decode_kv4(e(0, 4, D), cache, e(0, 3, t=torch.int32), i32([]))
    assert o.shape == (0, 4, D) and lse.shape == (0, 4)
    o, lse = attn.attn_decode_kv4(e(2, 4, D), cache, e(2, 0, t=torch.int32), i32([0, 0]))
    assert (o == 0).all() and (lse == -math.inf).all()
    assert attn.attn_get_device_status() == 0


# ---- decode ------------------------------------------------------------------------------------

def problem(lens, Hkv, G, D, seed, window=0, sink=0):
    """A pool with random records, the requests' pages anywhere in it. Pages of no request, and table entries of pages that no
    query sees, hold what must not be used (NaN scales, ids outside the pool)."""
    g = gen(seed)
    npg = [-(-n // 16) for n in lens]
    P = sum(npg) + 4
    K, V = (torch.randn(P * 16, Hkv, D, generator=g).bfloat16() for _ in range(2))
    K[:, :, ::17] *= 4
    cache = ref.put(noise(P, Hkv, D, seed), torch.arange(P * 16), K, V)
    ids = torch.randperm(P, generator=g)[: sum(npg)].tolist()
    table = torch.full((len(lens), max(npg + [0]) + 1), -5, dtype=torch.int32)
    _, _, sk, sv = ref.places(D)
    flat = cache.view(P, Hkv, 18 * D)
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        for p in range(npg[b]):
            page = ids.pop()
            hidden = [t for t in range(16) if not (16 * p + t < n and (16 * p + t >= first or 16 * p + t < sink))]
            for t in hidden:
                for at in (sk, sv):  # infinities and NaN
                    flat[page, :, at[t]], flat[page, :, at[t] + 1] = 0xC0 if t % 2 else 0x80, 0x7F
            if len(hidden) < 16:
                table[b, p] = page
    q = torch.randn(len(lens), G * Hkv, D, generator=g).bfloat16()
    return q, cache, table, torch.tensor(lens, dtype=torch.int32)


def check(q, cache, table, lens, window=0, sink=0, scale=0.1, got=None):
    if got is None:
        got = attn.attn_decode_kv4(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), window=window, sink=sink, scale=scale)
        assert attn.attn_get_device_status() == 0
    ro, to, rl, tl = ref.decode(q, cache, table, lens, scale, window, sink)
    close("o", got[0], ro, to)
    close("lse", got[1], rl, tl)


LENS = [[1], [16], [17], [0, 5, 0, 33, 700, 16, 0], [3000], [1, 1, 1, 1], list(range(0, 90, 3)), [257, 1023, 640, 31]]


@pytest.mark.parametrize("D,Hkv,G", [(64, 1, 1), (64, 3, 5), (128, 8, 4), (128, 1, 8), (128, 2, 3), (256, 1, 2), (256, 4, 7), (256, 2, 8)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_decode(D, Hkv, G, lens):
    check(*problem(lens, Hkv, G, D, 11))


@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 4), (128, 3, 2), (256, 2, 1)])
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (50, 4), (33, 40), (16, 128), (100, 17), (128, 16), (5000, 4), (640, 0)])
def test_window_and_sinks(D, Hkv, G, window, sink):
    check(*problem([1, 16, 17, 700, 0, 100, 33, 129, 51, 2000], Hkv, G, D, 12, window, sink), window, sink)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B", [300, 1000])
def test_many_requests(D, B):
    """More requests than threads, most of them short, some empty."""
    lens = torch.randint(0, 40, (B,), generator=gen(B)).tolist()
    lens[7] = 500
    check(*problem(lens, 2, 2, D, 13))


@pytest.mark.parametrize("D,G", [(64, 8), (128, 8), (256, 8), (256, 1)])
def test_most_requests(D, G):
    """As many as a call takes: with a group of 8 their lengths no longer fit in shared memory beside the rings."""
    lens = torch.randint(0, 20, (4096,), generator=gen(D + G)).tolist()
    lens[4095] = 300
    check(*problem(lens, 1, G, D, 17, 0, 0))


@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 1), (256, 1), (128, 4)])
def test_one_long_request(D, Hkv):
    """Every block of the GPU has a piece of it."""
    check(*problem([40000], Hkv, 2, D, 14))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 8.0])
def test_scales(D, scale):
    """Flat and sharp softmax: with the large scale one key has all of the weight."""
    check(*problem([300, 2000], 2, 4, D, 15), scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_and_small_values(D):
    """Scales of 2^-100 and 2^100 in K and V of different tokens and groups."""
    q, cache, table, lens = problem([100, 300], 2, 2, D, 16)
    _, _, sk, sv = ref.places(D)
    half = cache.view(cache.shape[0], 2, -1).view(torch.bfloat16)
    tiny, big = torch.tensor([2.0 ** -100, 2.0 ** 100]).bfloat16()
    half[:, :, sk[::3, 0] // 2] = tiny
    half[:, 0, sv[:, 1] // 2] = tiny
    half[:, 1, sv[:, 0] // 2] = big
    check(q, cache, table, lens)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("length", [40, 9000])
def test_nan(D, length):
    """A NaN in q, in a visible key or in a visible value is in its rows, and in no others."""
    q, cache, table, lens = problem([length, 50], 2, 2, D, 17)
    ro, to, rl, tl = ref.decode(q, cache, table, lens, 0.1)
    page, t = int(table[0, (length - 1) // 16]), (length - 1) % 16
    flat, (_, _, sk, sv) = cache.view(cache.shape[0], 2, 18 * D), ref.places(D)
    bad = cache.clone().view_as(flat)
    bad[page, 1, sk[t, 1]], bad[page, 1, sk[t, 1] + 1] = 0xC0, 0x7F
    o, lse = (x.cpu() for x in attn.attn_decode_kv4(q.cuda(), bad.view_as(cache).cuda(), table.cuda(), lens.cuda(), scale=0.1))
    assert o[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    close("o", o[0, :2], ro[0, :2], to[0, :2])
    close("o", o[1], ro[1], to[1])
    bad = cache.clone().view_as(flat)
    bad[page, 1, sv[t, 1]], bad[page, 1, sv[t, 1] + 1] = 0xC0, 0x7F
    o, lse = (x.cpu() for x in attn.attn_decode_kv4(q.cuda(), bad.view_as(cache).cuda(), table.cuda(), lens.cuda(), scale=0.1))
    assert o[0, 2:, 32: 64].isnan().all() and not o[0, 2:, :32].isnan().any() and not o[0, :2].isnan().any()
    close("lse", lse, rl, tl)
    q[0, 1, 3] = math.nan
    o, lse = (x.cpu() for x in attn.attn_decode_kv4(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), scale=0.1))
    assert o[0, 1].isnan().all() and lse[0, 1].isnan() and not o[0, [0, 2, 3]].isnan().any() and not lse[0, [0, 2, 3]].isnan().any()
    assert attn.attn_get_device_status() == 0


def test_bad_pages_and_lengths():
    """Pages outside the pool are skipped, lengths outside the table row cut, both reported."""
    q, cache, table, lens = problem([100, 64, 40], 2, 2, 128, 18)
    broken = table.clone()
    broken[0, 2], broken[1, :] = cache.shape[0], -1
    o, lse = attn.attn_decode_kv4(q.cuda(), cache.cuda(), broken.cuda(), lens.cuda(), scale=0.1)
    assert attn.attn_get_device_status() == 7
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
    whole = ref.decode(q, cache, table, lens, 0.1)
    close("o", o[2], whole[0][2], whole[1][2])
    # request 0 without its third page: a request of 84 tokens that has the others
    short, n = table.clone(), lens.clone()
    short[0, 2: 6], n[0] = table[0, 3: 7], 84
    ro, to, rl, tl = ref.decode(q, cache, short, n, 0.1)
    close("o", o[0], ro[0], to[0])
    close("lse", lse[0], rl[0], tl[0])
    o, lse = attn.attn_decode_kv4(q.cuda(), cache.cuda(), table[:, :2].contiguous().cuda(), i32([32, 33, -4]), scale=0.1)
    assert attn.attn_get_device_status() == 7
    ro, to, rl, tl = ref.decode(q, cache, table, [32, 32, 0], 0.1)
    close("o", o, ro, to)
    close("lse", lse, rl, tl)


def test_outputs_and_workspace_given():
    q, cache, table, lens = (x.cuda() for x in problem([300, 20], 2, 4, 128, 19))
    want = attn.attn_decode_kv4(q, cache, table, lens)
    o, lse = torch.full_like(q, 9), torch.full((2, 8), 9.0, device="cuda")
    ws = torch.randint(0, 256, (attn.attn_workspace_size(attn.ATTN_OP_DECODE_KV4, 2, 8, 2, 0, 128),), dtype=torch.uint8, device="cuda")
    got = attn.attn_decode_kv4(q, cache, table, lens, o, lse, workspace=ws)
    assert got[0] is o and got[1] is lse and torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_streams_and_graphs():
    """The same bits every time: repeated, on two streams at once, in two graphs replayed in turn."""
    a, b = (tuple(x.cuda() for x in problem([900, 20, 3, 400], 2, 4, D, 20)) for D in (128, 256))
    want = [attn.attn_decode_kv4(*x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [attn.attn_decode_kv4(*x, stream=s) for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
    graphs = []
    for x in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = attn.attn_decode_kv4(*x)
        graphs.append((graph, out))
    for _ in range(3):
        for (graph, out), w in zip(graphs, want):
            out[0].zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for (_, g), w in zip(graphs, want) for x, y in zip(g, w))
    assert attn.attn_get_device_status() == 0


def test_far_offsets():
    """Records past 2^31 bytes of the cache."""
    D, H = 256, 8
    P = 2 ** 32 // (18 * D * H) + 3
    cache = torch.empty(P, H, 18, D, dtype=torch.uint8, device="cuda")
    k, v = (torch.randn(40, H, D, generator=gen(s)).bfloat16() for s in (21, 22))
    pages = [P - 1, 2, P - 2]
    slots = torch.tensor([16 * p + t for p in pages for t in range(16)][:40], dtype=torch.int32)
    attn.attn_kv4_append(k.cuda(), v.cuda(), slots.cuda(), cache)
    uk, uv = attn.attn_kv4_unpack(cache, i32(pages))
    assert torch.equal(uk.flatten(0, 1)[:40].cpu().double(), ref.values(k)) and torch.equal(uv.flatten(0, 1)[:40].cpu().double(), ref.values(v))
    q = torch.randn(1, 16, D, generator=gen(23)).bfloat16()
    got = attn.attn_decode_kv4(q.cuda(), cache, i32([pages]), i32([40]), scale=0.1)
    small = torch.zeros(3, H, 18, D, dtype=torch.uint8)
    ref.put(small, torch.arange(40), k, v)
    check(q, small, torch.tensor([[0, 1, 2]]), [40], got=got)
    assert attn.attn_get_device_status() == 0
