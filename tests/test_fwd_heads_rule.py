"""How many query heads a block of the forward takes: the rule's own code, compiled for the host, against the sides that were measured. Needs
no GPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 152


@pytest.fixture(scope="module")
def heads(tmp_path_factory):
    """f(Hq, nseq, S, rows, packed, window) -> heads a block."""
    from attention_flash_gqa_gb300 import _build

    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text('#include <cstdio>\n#include "attn_internal.h"\nint main() { int h, n, s, r, p, w;\n'
                                'while (std::scanf("%d %d %d %d %d %d", &h, &n, &s, &r, &p, &w) == 6)\n'
                                f'std::printf("%d\\n", attn::fwd_heads(h, n, s, r, p != 0, w, {SMS})); }}\n')
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", cuda, "-I", os.path.join(ROOT, "attention_flash_gqa_gb300", "csrc"),
                    str(d / "rule.cpp"), "-o", str(d / "rule")], check=True)

    def run(*cases):
        out = subprocess.run([str(d / "rule")], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True, check=True)
        return [int(x) for x in out.stdout.split()]

    return run


def dense(Hq, B, S, window=0):
    return Hq, B, S, B * S, 0, window


def packed(Hq, lens, top, window=0):
    return Hq, len(lens), top, sum(lens), 1, window


def test_measured_sides(heads):
    many = [packed(8, [4096] + [16] * 300, 4096), packed(32, [16] * 512, 16), packed(32, [64] * 200 + [1500] * 4, 1500),
            packed(32, [3700, 128, 1500, 2900, 4096, 17, 2200, 2000], 4096, 500), dense(32, 2, 8192, 1024), dense(32, 2, 8192)]
    assert heads(*many) == [4] * len(many)
    # few tiles in fact, whatever max_seqlen says
    few = [packed(16, [1000], 32768), packed(16, [1000], 1000), packed(8, [4096] + [16] * 63, 4096), packed(8, [1], 4096), dense(8, 1, 16000, 700)]
    assert heads(*few) == [1] * len(few)
    assert heads(dense(12, 1, 128 * SMS), dense(12, 1, 128 * SMS - 128), dense(24, 1, 128 * SMS), dense(24, 1, 128 * SMS - 128)) == [2, 1, 4, 2]


def test_no_more_heads_than_there_are(heads):
    assert heads(dense(1, 1, 1 << 20, 300), dense(2, 1, 1 << 20, 300), dense(3, 1, 1 << 20, 300), dense(4, 1, 1 << 20, 300)) == [1, 2, 2, 4]


def test_packed_like_dense(heads):
    """Packed sequences of one length, a multiple of 128 or no longer than that, count as the dense call does."""
    for S in (1, 16, 100, 128, 256, 1024):
        for B in (1, 3, 40, 500, 3000):
            for Hq in (1, 5, 32):
                assert heads(dense(Hq, B, S)) == heads(packed(Hq, [S] * B, S)), (S, B, Hq)


def test_largest_sizes(heads):
    top = 65535 * 128
    assert heads((1 << 20, 65535, top, 2 ** 31 - 1, 1, 0), (1 << 20, 65535, top, 2 ** 31 - 1, 1, 2 ** 31 - 1), (64, 0, 0, 0, 1, 0), (64, 5, top, 0, 1, 1)) == [4, 4, 1, 4]
