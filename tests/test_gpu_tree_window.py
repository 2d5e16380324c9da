"""Trees deeper than the window: with the bits of ancestors out of the window cleared, the tree attention is the windowed
attention of the framework's other calls; with the bits set they stay visible."""
import pytest
import torch

import attention_flash_gqa_gb300 as attn
import operator_ref as ref
from test_gpu_tree_paged import compare, i32, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def chain(n, window, words):
    """Mask rows of a chain: row i sees tokens i - window + 1 .. i (all of 0 .. i without a window)."""
    rows = []
    for i in range(n):
        bits = sum(1 << d for d in range(n) if d <= i and (not window or i - d < window))
        w = [bits >> 32 * k & 0xFFFFFFFF for k in range(words)]
        rows.append([x - (1 << 32) if x >> 31 else x for x in w])
    return rows


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("window", [1, 7, 40])
def test_chain_deeper_than_the_window(D, window):
    p = problem([200, 0, 33], [100, 64, 41], 4, 2, D, seed=61, poison=False)
    words = p["mask"].shape[1]
    p["pos"] = torch.tensor([c + i for c, n in zip(p["ctx"], p["n"]) for i in range(n)], dtype=torch.int32)
    p["mask"] = torch.tensor([r for n in p["n"] for r in chain(n, window, words)], dtype=torch.int32)
    o, lse = compare(p, window)
    po, pl = attn.attn_fwd_paged(p["q"].cuda(), p["kc"].cuda(), p["vc"].cuda(), p["table"].cuda(), i32(p["lens"]), i32(p["cu"]),
                                 max(p["n"]), window=window, scale=p["scale"])
    assert attn.attn_get_device_status() == 0
    _, to, _, tl = ref.tree(p["q"], p["kc"], p["vc"], p["table"], p["lens"], p["cu"], p["mask"], p["scale"], window, p["pos"])
    ref.close("o against the chunk", o, po.double().cpu(), 2 * to)
    ref.close("lse against the chunk", lse, pl.double().cpu(), 2 * tl)
    # with every ancestor's bit set the window limits the context alone
    p["mask"] = torch.tensor([r for n in p["n"] for r in chain(n, 0, words)], dtype=torch.int32)
    full, _ = compare(p, window)
    assert not torch.equal(full, o)
