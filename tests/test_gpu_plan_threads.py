"""Step plans of large batches of different sizes from several host threads at once, through the C ABI."""
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


@pytest.mark.parametrize("in_place", [False, True])
def test_plans_from_several_threads(in_place):
    """Shared memory of a plan grows with its requests (over 48 KB from 6 thousand on): one thread's call must not take
    away what another's needs."""
    lib = attn.load_library()
    sizes = [16384, 6500, 12000, 9000]
    start = threading.Barrier(len(sizes), timeout=60)
    bad, results = [], {}

    def work(R):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            i32 = lambda n, v: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
            kv, new, held, used, table = i32(R, 16), i32(R, 0), i32(R, 1), i32(1, 0), i32(2 * R, 5)
            seq, cu, adm = (kv if in_place else i32(R, -1)), i32(R + 1, -1), i32(1, -1)
            ho, uo = (held, used) if in_place else (i32(R, -1), i32(1, -1))
            s.synchronize()
            p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
            start.wait()
            for _ in range(1500):
                rc = lib.attn_paged_plan(p(kv), p(new), p(held), None, p(used), p(table), p(seq), p(cu), None, None, p(ho), p(uo),
                                         p(adm), R, 0, 0, 16, 2, 8, ctypes.c_void_p(s.cuda_stream))
                if rc:
                    bad.append((R, rc))
            s.synchronize()
            results[R] = adm.item(), seq.unique().tolist(), ho.unique().tolist(), cu.unique().tolist()

    threads = [threading.Thread(target=work, args=(R,)) for R in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, (len(bad), bad[0])
    assert results == {R: (R, [16], [1], [0]) for R in sizes}
    assert attn.attn_get_device_status() == 0
