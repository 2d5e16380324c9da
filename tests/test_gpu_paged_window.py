"""Chunked prefill with windows that no request reaches, up to the largest number there is: the bits of the call without a window."""
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


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 4, 2), (256, 2, 1), (512, 4, 2), (512, 1, 1)])
def test_windows_past_the_table(D, Hq, Hkv):
    g = torch.Generator(device="cuda").manual_seed(D)
    lens, new = [300, 17, 640, 1], [200, 17, 3, 1]
    kc, vc = (torch.randn(160, 16, Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.arange(160, dtype=torch.int32, device="cuda").view(4, 40)
    q = torch.randn(sum(new), Hq, D, generator=g, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    want = attn.attn_fwd_paged(q, kc, vc, table, seq, cu, 200)
    for window in (640, 641, 2 ** 31 - 200, 2 ** 31 - 1):
        for sink in (0, 5, 128):
            got = attn.attn_fwd_paged(q, kc, vc, table, seq, cu, 200, window=window, sink=sink)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (window, sink)
    got = attn.attn_fwd_paged(q, kc, vc, table, seq, cu, 200, window=639)  # the last token of the third request misses one key
    assert torch.equal(got[0][:217], want[0][:217]) and not torch.equal(got[0][219], want[0][219])
    assert attn.attn_get_device_status() == 0
