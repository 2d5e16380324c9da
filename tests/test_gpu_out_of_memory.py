"""Outputs and workspaces that do not fit the GPU: the calls raise torch's own error, launch nothing, and work afterwards."""
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


def calls():
    """Inputs of one row, repeated by a stride of zero: their outputs would take 2 TB."""
    T, H, D = 1 << 24, 128, 512
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k = z(1, H, D).expand(T, H, D), z(1, 1, D).expand(T, 1, D)
    small, one = z(2, 2, D), z(2, 1, D)
    cache = z(4, 16, 1, D)
    return {
        "norm_rope": lambda: attn.attn_qk_norm_rope(q, k, None, None, None, None),
        "norm_rope_paged": lambda: attn.attn_qk_norm_rope_paged(q, k, k, None, None, None, torch.full((T,), -1, dtype=torch.int32, device="cuda"),
                                                                None, cache, cache.clone()),
        "fwd": lambda: attn.attn_fwd(*(z(1, 1, 1, D).expand(1, T, H, D) for _ in range(3))),
    }, lambda: attn.attn_qk_norm_rope(small, one, None, None, None, None)


@pytest.mark.parametrize("name", ["norm_rope", "norm_rope_paged", "fwd"])
def test_out_of_memory_is_torch_s_error(name):
    big, after = calls()
    before = attn.attn_launch_count()
    with pytest.raises(torch.OutOfMemoryError):
        big[name]()
    assert attn.attn_launch_count() == before
    after()
    torch.cuda.synchronize()
    assert attn.attn_launch_count() == before + 1 and attn.attn_get_device_status() == 0


def test_plan_out_of_memory(monkeypatch):
    """The largest step there is needs 8.6 GB of rows: with the process held to less it raises too."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    kv, free, table, held, used = i(4), i(4), i(4, 4), i(4), i(1)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.01)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            attn.attn_paged_plan(kv, kv.clone(), free, table, held, used, 1 << 30, num_pages=4)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    p = attn.attn_paged_plan(kv, kv.clone(), free, table, held, used, 5, num_pages=4)
    assert p.slots.tolist() == [-1] * 5 and attn.attn_get_device_status() == 0
