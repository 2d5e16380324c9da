"""Decode calls with different numbers of KV heads from several host threads at once, through the C ABI."""
import ctypes
import threading

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


@pytest.mark.parametrize("D", [128, 256])
def test_decodes_from_several_threads(D):
    """Shared memory of a decode call grows with its KV heads: one thread's call must not take away what another's needs."""
    lib = attn.load_library()
    heads = [8, 1, 4, 2] if D == 128 else [4, 1, 2, 3]
    first = threading.Lock()
    start = threading.Barrier(len(heads), timeout=60)
    bad, results = [], {}

    def work(Hkv):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g = torch.Generator(device="cuda").manual_seed(Hkv)
            r = lambda *n: torch.randn(*n, generator=g, device="cuda").bfloat16()  # noqa: E731
            B, Hq = 3, 4 * Hkv
            q, kc, vc = r(B, Hq, D), r(12, 16, Hkv, D), r(12, 16, Hkv, D)
            table = torch.arange(12, dtype=torch.int32, device="cuda").view(B, 4)
            lens = torch.tensor([40, 1, 64], dtype=torch.int32, device="cuda")
            o, lse = torch.zeros_like(q), torch.zeros(B, Hq, device="cuda")
            n = attn.attn_workspace_size(attn.ATTN_OP_DECODE_PAGED, B, Hq, Hkv, 0, D)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            with first:  # one at a time
                want = [t.clone() for t in attn.attn_decode_paged(q, kc, vc, table, lens, scale=0.1, workspace=ws)]
            s.synchronize()
            p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
            start.wait()
            for _ in range(1500):
                rc = lib.attn_decode_paged(p(q), p(kc), p(vc), p(table), p(lens), p(o), p(lse), B, Hq, Hkv, D, 16, 4, 12, 0.1, 0, p(ws), n,
                                           ctypes.c_void_p(s.cuda_stream))
                if rc:
                    bad.append((Hkv, rc))
            s.synchronize()
            results[Hkv] = torch.equal(o, want[0]) and torch.equal(lse, want[1])

    threads = [threading.Thread(target=work, args=(h,)) for h in heads]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, (len(bad), bad[0])
    assert results == {h: True for h in heads}
    assert attn.attn_get_device_status() == 0
