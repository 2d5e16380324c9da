"""The gradient of the head norm where every ring of copies goes round several times: all of dq, dk and both weight
gradients against the 64-bit definition, evaluated on the GPU in pieces."""
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


def blocks(H, rows):
    """Heads of the blocks that a token's heads of one kind are cut into."""
    n = -(-H // rows)
    each = -(-H // n)
    return [min(each, H - i * each) for i in range(n)]


def tokens_per_warp(T, Hq, Hkv, D):
    """Tokens that a warp walks at most (three CTAs of four warps an SM, a warp keeping one block of heads)."""
    warps = 12 * torch.cuda.get_device_properties(0).multi_processor_count
    return -(-T // (warps // len(blocks(Hq, 2048 // D) + blocks(Hkv, 2048 // D))))


def inputs(T, Hq, Hkv, D, rot, w32, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    q, k, gq, gk = n(T, Hq, D), n(T, Hkv, D), n(T, Hq, D), n(T, Hkv, D)
    wt = torch.float32 if w32 else torch.bfloat16
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(wt) for _ in range(2))
    pos = torch.randint(0, 300, (T,), generator=g, device="cuda", dtype=torch.int32)
    return q, k, gq, gk, qw, kw, pos, ref.table(300, rot).cuda()


def compare(x, dy, w, pos, cs, off, inter, dx, dw, chain):
    """dx within its tolerance, piece by piece; dw within the roundings of its own order of summation: `chain`
    terms one after the other at most, each of 20 u."""
    T, H, D = x.shape
    want, terms = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, 20_000_000 // (H * D))
    for a in range(0, T, step):
        s = slice(a, a + step)
        at = cs[pos[s].long()]
        y, tol, part, mag = ref.norm_rope_bwd(dy[s], x[s], w, at, EPS, off, inter)
        over = (dx[s].double() - y).abs() - tol
        assert torch.isfinite(dx[s]).all() and over.max() <= 0, (a, int((over > 0).sum()), float(over.max()))
        want += part
        terms += mag / ((2 * x[s].shape[0] + 148) * ref.U)  # the sum of the terms' magnitudes
    over = (dw.double() - want).abs() - (chain + 20) * ref.U * terms
    assert torch.isfinite(dw).all() and over.max() <= 0, (int((over > 0).sum()), float(over.max()))


def run(T, Hq, Hkv, D, rot, inter, w32, off, seed):
    q, k, gq, gk, qw, kw, pos, cs = inputs(T, Hq, Hkv, D, rot, w32, seed)
    dq, dk, dqw, dkw = attn.attn_qk_norm_rope_bwd(gq, gk, q, k, qw, kw, pos, cs, eps=EPS, weight_offset=off, interleaved=inter)
    assert attn.attn_get_device_status() == 0
    # a warp's rows, its row groups, a CTA's four warps, every 16th of up to 1024 CTAs, 16 of those
    chain = 4 * tokens_per_warp(T, Hq, Hkv, D) + 5 + 4 + 64 + 16
    compare(q, gq, qw, pos, cs, off, inter, dq, dqw, chain)
    compare(k, gk, kw, pos, cs, off, inter, dk, dkw, chain)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,w32,off", [
    (4001, 24, 4, 128, 128, False, False, 0.0),   # blocks of 12, 12 and 4 heads
    (4507, 17, 3, 128, 64, True, True, 1.0),      # 9, 8 and 3
    (4001, 10, 3, 256, 256, False, True, 0.0),    # 5, 5 and 3
    (6007, 9, 8, 256, 32, True, False, 0.0),      # 5, 4 and 8
    (22501, 1, 1, 512, 128, False, False, 0.0),   # one row a task: rings of eight stages
    (23003, 2, 1, 512, 512, True, True, 1.0),     # of four and of eight
    (5801, 5, 5, 512, 128, False, True, 0.0),     # blocks of 3 and 2 rows: rings of two and of four
    (4507, 6, 3, 512, 0, False, False, 0.0),      # of 3 rows
    (4201, 4, 8, 512, 64, False, False, 1.0),     # of 4 rows
    (9001, 40, 13, 64, 32, False, True, 0.0)])
def test_gradient_rings(T, Hq, Hkv, D, rot, inter, w32, off):
    rows = 2048 // D
    depth = max(min(8, 16384 // (r * D * 4)) if D == 512 else 2 for r in blocks(Hq, rows) + blocks(Hkv, rows))
    assert tokens_per_warp(T, Hq, Hkv, D) >= 3 * depth  # every stage is filled three times
    run(T, Hq, Hkv, D, rot, inter, w32, off, T + D)


def test_gradient_past_32_bits():
    """2.15e9 query elements: every gradient, not the rows at the ends alone."""
    run(140001, 30, 1, 512, 128, False, False, 0.0, 5)
