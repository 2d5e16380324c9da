"""Size of the sinks' gradient workspace over windows and sequences. Needs no GPU."""
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
