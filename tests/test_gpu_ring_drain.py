"""What a warp waits for when it leaves a ring of copies early (ring_drain): every copy on its way, each at its own phase."""
import ctypes
import os
import subprocess

import pytest
import torch

from attention_flash_gqa_gb300 import _build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("ring") / "ring_drain_check.so")
    subprocess.run([_build.nvcc(), _build.GENCODE, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", _build.CSRC,
                    os.path.join(HERE, "ring_drain_check.cu"), "-o", so], check=True, capture_output=True)
    f = ctypes.CDLL(so).ring_drain_check
    f.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int] * 4
    return f


@pytest.mark.parametrize("depth,bytes", [(1, 65536), (2, 8192), (2, 65536), (4, 32768), (8, 1024), (8, 16384)])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 40])
def test_every_copy_has_landed(check, depth, bytes, tokens):
    g = torch.Generator(device="cuda").manual_seed(depth * 100 + tokens)
    flush = torch.empty(200 << 20, dtype=torch.uint8, device="cuda")
    for stop in sorted({0, 1, depth - 1, depth, depth + 1, 2 * depth, tokens - depth, tokens - 1, tokens}):
        if not 0 <= stop <= tokens:
            continue
        src = torch.randint(0, 255, (tokens, bytes), dtype=torch.uint8, device="cuda", generator=g)  # 255: what the ring starts with
        out = torch.full_like(src, 254)
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        flush.fill_(1)  # the copies come from memory, not from L2
        torch.cuda.synchronize()
        assert check(src.data_ptr(), out.data_ptr(), status.data_ptr(), tokens, bytes, depth, stop) == 0
        torch.cuda.synchronize()
        n = min(tokens, stop + depth)
        assert status.tolist() == [0, 0]
        assert torch.equal(out[:n], src[:n]) and (out[n:] == 254).all(), (stop, n)
