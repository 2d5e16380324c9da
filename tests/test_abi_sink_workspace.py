"""Size of the sinks' gradient workspace over windows and sequences. Needs no GPU."""
import os
import subprocess

import pytest

import attention_flash_gqa_gb300 as attn
from attention_flash_gqa_gb300 import _build
from test_abi_operators import A, MISALIGNED, WORKSPACE
from test_abi_sink_kv4 import call_of


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return attn.load_library()


@pytest.mark.parametrize("S", [1, 300, 3000, 200000])
def test_windows_that_hide_nothing(lib, S):
    """From the length on, up to the largest number there is, a window needs what the plain gradient does."""
    plain = attn.attn_workspace_size(attn.ATTN_OP_BWD, 1, 8, 2, S, 128)
    for window in (S, S + 1, 2 ** 31 - 385, 2 ** 31 - 129, 2 ** 31 - 1):
        assert lib.attn_bwd_sink_workspace_size(1, 8, 2, S, 128, 0, window, 4) == plain, window
        assert lib.attn_bwd_sink_workspace_size(1, 8, 2, S, 128, 9, window, 128) == plain, window


def test_call_and_size_agree(lib):
    """The call wants the bytes that the size function names, also where max_seqlen is beyond all rows."""
    _, call = call_of(lib, "attn_bwd_sink")
    for top in (50, 700, 701, 5000, 1 << 22):
        for window in (1, 40, 699, 700, 4000, 2 ** 31 - 1):
            need = lib.attn_bwd_sink_workspace_size(1, 8, 2, 700, 128, 3, window, 4)
            packed = dict(B=1, S=700, cun=A, ns=3, top=top, window=window)
            assert call(**packed, wsb=attn.attn_workspace_size(attn.ATTN_OP_BWD, 1, 8, 2, 700, 128) - 1) == WORKSPACE
            # (so many bytes are enough: what is refused then is where they start)
            assert call(**packed, wsb=need, ws=A + 16) == MISALIGNED, (top, window)


def test_sizes_that_no_call_takes(lib):
    """The size is host arithmetic over any numbers: two parts of one sequence's sinks at least, for the longest too."""
    for S in (65535 * 128, 2 ** 31 - 1):
        for window in (1, 65535 * 128 - 1, S - 1):
            parts = lib.attn_bwd_sink_workspace_size(1, 8, 2, S, 128, 0, window, 4) - attn.attn_workspace_size(attn.ATTN_OP_BWD, 1, 8, 2, S, 128)
            assert parts >= 2 * 2 * 2 * 4 * 128 * 4, (S, window)


def test_short_sequences_need_no_room(lib):
    """Sequences that the window covers have no parts: 16384 tokens hold 14 at most that are longer than a window of 1000, whatever they are cut into."""
    def parts(nseq, window, T=16384):
        plain = attn.attn_workspace_size(attn.ATTN_OP_BWD, 1, 32, 8, T, 128)
        return (lib.attn_bwd_sink_workspace_size(1, 32, 8, T, 128, nseq, window, 128) - plain) / (8 * 2 * 128 * 128 * 4)

    assert parts(1024, 1000) == parts(16384, 1000) == parts(14, 1000) <= 16384 // 1024 + 2 * 14
    assert parts(3, 1000) < parts(5, 1000) < parts(14, 1000)
    assert parts(16384, 1) <= 16384 // 1024 + 2 * 16384 // 128


def test_parts_of_sequences_lie_apart(tmp_path):
    """The kernels' own arithmetic, compiled for the host: parts of sequences with far queries never overlap and stay below the bound, wherever the
    sequences begin; parts of bad slices stay below it too."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "parts.cpp").write_text(r"""
#include <cstdio>
#include <random>
#include <vector>
#include "attn_internal.h"
int main() {
    std::mt19937 g(1);
    auto upto = [&](int n) { return (int)(g() % (unsigned)(n + 1)); };
    for (int round = 0; round < 20000; ++round) {
        attn::SinkSplit s = {};
        const int window = 1 + upto(round % 3 ? 300 : 3000);
        s.rows = 64 * (1 + upto(30)), s.shares = 1 + upto(7), s.reach = window + 127, s.sink = 1;
        const int nseq = 1 + upto(60);
        std::vector<int> cu(1, 0);
        for (int i = 0; i < nseq; ++i) {  // short ones, ones around the first far query, long ones
            const int kind = upto(3), n = kind == 0 ? upto(3) : kind == 1 ? upto(window + 400) : kind == 2 ? window + 120 + upto(16) : upto(3 * window + 3000);
            cu.push_back(cu.back() + n);
        }
        const int T = cu.back() + upto(5);
        const long long most = s.parts(T, nseq);
        std::vector<char> taken(most + 1);
        auto count = [&](int L) { const int far = attn::far_from(L, window); return far < L ? 1 + (L - far + s.rows - 1) / s.rows * s.shares : 0; };
        for (int i = 0; i < nseq; ++i) {
            const long long at = s.first_part(i, cu[i]);
            const int n = count(cu[i + 1] - cu[i]);
            if (at < 0 || (n && at + n > most)) return std::printf("out of room: round %d\n", round), 1;
            for (int p = 0; p < n; ++p)
                if (taken[at + p]++) return std::printf("overlap: round %d\n", round), 1;
        }
        for (int i = 0; i < 20; ++i) {  // any slice of the rows, under any number
            const int start = upto(T), L = upto(T - start), n = count(L);
            if (n && s.first_part(upto(nseq - 1), start) + n > most) return std::printf("slice out of room: round %d\n", round), 1;
        }
    }
    return std::printf("ok\n"), 0;
}
""")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", cuda, "-I", os.path.join(root, "attention_flash_gqa_gb300", "csrc"),
                    str(tmp_path / "parts.cpp"), "-o", str(tmp_path / "parts")], check=True)
    r = subprocess.run([str(tmp_path / "parts")], capture_output=True, text=True)
    assert r.stdout == "ok\n", r.stdout + r.stderr
