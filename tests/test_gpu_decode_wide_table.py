"""Decode with block-table rows so wide that their tokens pass 32 bits."""
import pytest
import torch

import attention_flash_gqa_gb300 as attn
import operator_ref as ref
from test_gpu_tree_paged import i32, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("R,width", [(1, 1 << 27), (3, (1 << 27) + 5), (20, 1 << 27)])
def test_wide_rows(R, width):
    """2^27 pages a row are 2^31 tokens; 20 such rows have more pages than 32 bits count."""
    p = problem([17 * b + 30 for b in range(R)], [1] * R, 8, 2, 128, seed=71)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    table[:, : p["table"].shape[1]] = p["table"].cuda()
    ro, to, rl, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"])
    for _ in range(3):
        o, lse = attn.attn_decode_paged(p["q"].cuda(), p["kc"].cuda(), p["vc"].cuda(), table, i32(p["lens"]), scale=p["scale"])
        assert attn.attn_get_device_status() == 0
        ref.close("o", o, ro, to)
        ref.close("lse", lse, rl.t(), tl.t())
