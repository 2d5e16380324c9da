"""Packed prompts of uneven lengths and of a max_seqlen that says too much, where a block takes one, two and four query heads: the bits of each
sequence's own call."""
import pytest
import torch

import attention_flash_gqa_gb300 as attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


# (Hq, Hkv, lens, max_seqlen, window, sink): one head a block; two; four; four for the empty blocks' sake
CASES = [(8, 2, [1000], 32768, 0, 0), (8, 2, [3000] + [16] * 63, 4096, 0, 0), (37, 37, [700, 1, 0, 130, 2500, 3000], 3000, 300, 4),
         (96, 8, [129, 500, 7, 128, 4000, 0, 300], 4100, 0, 0), (95, 5, [129, 500, 7, 128, 4000, 0, 300], 4100, 1, 1),
         (8, 4, [4000] + [16, 3, 0] * 120, 4100, 0, 0), (6, 3, [257] + [1, 2] * 300, 8192, 100, 20)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,lens,top,window,sink", CASES)
def test_bits(D, Hq, Hkv, lens, top, window, sink):
    g = torch.Generator(device="cuda").manual_seed(D + Hq)
    T = sum(lens)
    q, k, v = (torch.randn(T + 3, h, D, generator=g, device="cuda", dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    how = dict(window=window, sink=sink)
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, T + 3), 7.0, device="cuda")
    attn.attn_fwd_varlen(q, k, v, cu, top, o, lse, **how)
    assert bool((o[T:] == 7.0).all()) and bool((lse[:, T:] == 7.0).all())
    at = 0
    for n in lens:
        if n:
            rows = slice(at, at + n)
            for h in (0, Hq // 2, Hq - 1):  # (one head alone: one a block)
                x = h * Hkv // Hq
                one = attn.attn_fwd(q[None, rows, h:h + 1].contiguous(), k[None, rows, x:x + 1].contiguous(), v[None, rows, x:x + 1].contiguous(), **how)
                assert torch.equal(o[rows, h], one[0][0, :, 0]) and torch.equal(lse[h, rows], one[1][0, 0]), (n, h)
        at += n
    assert attn.attn_get_device_status() == 0
