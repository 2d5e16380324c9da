"""Argument checks of the calls with sinks and of the 4-bit cache: every refusal returns its documented code (or raises in the
binding) before anything is launched. Needs no GPU."""
import pytest
import torch

import attention_flash_gqa_gb300 as attn
from attention_flash_gqa_gb300 import _build
from test_abi_operators import A, INF, INVALID, MISALIGNED, NAN, OK, UNSUPPORTED, WORKSPACE, caller


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return attn.load_library()


def p(s):
    return s.split()


BASE = dict(B=2, Hq=8, Hkv=2, S=300, D=128, T=300, ns=2, top=200, R=2, maxp=8, np=64, ps=16, scale=0.1, causal=1, window=40, sink=4, ws=A,
            wsb=1 << 40, stream=None, cu=A)
CALLS = {
    "attn_fwd_sink": p("q k v o lse B Hq Hkv S D scale causal window sink ws wsb stream"),
    "attn_fwd_varlen_sink": p("q k v o lse cu ns T top Hq Hkv D scale causal window sink ws wsb stream"),
    "attn_fwd_paged_sink": p("q k v table lens cu o lse R T top Hq Hkv D ps maxp np scale causal window sink stream"),
    "attn_bwd_sink": p("q k v o lse do dq dk dv B Hq Hkv S D scale causal window sink cun ns top ws wsb stream"),
    "attn_decode_paged_sink": p("q k v table lens o lse B Hq Hkv D ps maxp np scale window sink ws wsb stream"),
    "attn_decode_kv4": p("q kv table lens o lse B Hq Hkv D ps maxp np scale window sink ws wsb stream"),
}


def call_of(lib, name):
    n = CALLS[name]
    return n, caller(getattr(lib, name), n, dict({x: A for x in n}, **{k: v for k, v in BASE.items() if k in n}, **({"cun": None} if "cun" in n else {})))


@pytest.mark.parametrize("name", CALLS)
def test_refusals(lib, name):
    names, call = call_of(lib, name)
    assert call(sink=-1) == INVALID and call(sink=129) == UNSUPPORTED
    assert call(window=-1) == INVALID and call(Hq=7) == INVALID and call(Hkv=0) == INVALID
    for bad in (0.0, -1.0, NAN, INF):
        assert call(scale=bad) == INVALID
    assert call(D=96) == UNSUPPORTED
    for n in ("q", "k", "v", "kv", "o", "lse", "do", "dq", "dk", "dv", "table", "lens", "cu"):
        if n in names:
            assert call(**{n: None}) == INVALID, n
            if n != "cu" or "paged" in name:
                assert call(**{n: A + 2}) == MISALIGNED, n
    if "causal" in names:
        assert call(causal=0) == UNSUPPORTED
    if "ps" in names:
        assert call(ps=0) == INVALID and call(ps=32) == UNSUPPORTED
    if "ws" in names and "fwd" not in name:
        assert call(ws=None) == WORKSPACE and call(wsb=10) == WORKSPACE and call(ws=A + 16) == MISALIGNED
    if "kv4" in name:
        assert call(D=512) == UNSUPPORTED and call(Hq=18) == UNSUPPORTED and call(Hkv=300, Hq=300) == UNSUPPORTED
        assert call(B=4097) == UNSUPPORTED and call(np=(1 << 26) + 1) == UNSUPPORTED and call(maxp=1 << 30) == UNSUPPORTED
        assert call(B=-1) == INVALID and call(maxp=-1) == INVALID and call(np=-1) == INVALID
        assert call(B=0, q=None, ws=None) == OK


def test_bwd_workspace(lib):
    """The sinks' parts need their bytes on top of the plain backward's, and no call takes less."""
    plain = attn.attn_workspace_size(attn.ATTN_OP_BWD, 2, 8, 2, 300, 128)
    size = lib.attn_bwd_sink_workspace_size
    assert size(2, 8, 2, 300, 128, 0, 0, 4) == size(2, 8, 2, 300, 128, 0, 40, 0) == plain
    with_sinks = size(2, 8, 2, 300, 128, 0, 40, 4)
    assert with_sinks >= plain + 4 * 2 * 2 * 4 * 128 * 4
    _, call = call_of(lib, "attn_bwd_sink")
    assert call(wsb=with_sinks - 1) == WORKSPACE
    assert call(window=0, wsb=plain - 1) == WORKSPACE and call(window=300, wsb=plain - 1) == WORKSPACE
    assert size(-1, 8, 2, 300, 128, 0, 40, 4) == 0 and size(1, 8, 2, 300, 128, -1, 40, 4) == 0
    assert size(1, 8, 2, 3000, 128, 9, 40, 4) > size(1, 8, 2, 3000, 128, 1, 40, 4)


def test_append_and_unpack_refusals(lib):
    n = p("k v slots kv T Hkv D ps np ks vs stream")
    call = caller(lib.attn_kv4_append, n, dict({x: A for x in n}, T=7, Hkv=2, D=128, ps=16, np=64, ks=256, vs=256, stream=None))
    for x in ("k", "v", "slots", "kv"):
        assert call(**{x: None}) == INVALID and call(**{x: A + 2}) == MISALIGNED, x
    assert call(T=-1) == INVALID and call(Hkv=0) == INVALID and call(ps=0) == INVALID and call(np=-1) == INVALID
    assert call(ks=-8) == INVALID and call(vs=260) == MISALIGNED
    assert call(D=512) == UNSUPPORTED and call(D=32) == UNSUPPORTED and call(Hkv=257) == UNSUPPORTED and call(ps=32) == UNSUPPORTED
    assert call(np=(1 << 26) + 1) == UNSUPPORTED and call(T=1 << 30) == UNSUPPORTED
    assert call(T=0, k=None, kv=None) == OK
    n = p("kv pages ko vo n Hkv D ps np stream")
    call = caller(lib.attn_kv4_unpack, n, dict({x: A for x in n}, n=7, Hkv=2, D=128, ps=16, np=64, stream=None))
    for x in ("kv", "pages", "ko", "vo"):
        assert call(**{x: None}) == INVALID and call(**{x: A + 2}) == MISALIGNED, x
    assert call(n=-1) == INVALID and call(Hkv=0) == INVALID and call(ps=0) == INVALID and call(np=-1) == INVALID
    assert call(D=512) == UNSUPPORTED and call(Hkv=257) == UNSUPPORTED and call(ps=8) == UNSUPPORTED and call(n=1 << 28) == UNSUPPORTED
    assert call(n=0, kv=None) == OK


def test_workspace_size(lib):
    size = lambda *a: attn.attn_workspace_size(attn.ATTN_OP_DECODE_KV4, *a)  # noqa: E731
    assert size(4, 8, 2, 0, 128) % 256 == 0 and size(4, 8, 2, 0, 128) > 256 * 2 * 4 * 130 * 4
    for bad in ((4, 8, 3, 0, 128), (4, 18, 2, 0, 128), (4, 8, 2, 0, 512), (5000, 8, 2, 0, 128), (-1, 8, 2, 0, 128)):
        assert size(*bad) == 0


def test_binding_refuses_cpu_tensors(lib):
    x, c = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 18, 128, dtype=torch.uint8)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_kv4_append(x, x, i, c)
    with pytest.raises(ValueError):
        attn.attn_kv4_unpack(c, i)
    with pytest.raises(ValueError):
        attn.attn_decode_kv4(x, c, i.view(4, 1), i)
    with pytest.raises(TypeError):
        attn.attn_kv4_append(None, x, i, c)


def test_bwd_workspace_of_the_largest_window(lib):
    size = lib.attn_bwd_sink_workspace_size
    assert size(1, 8, 2, 3000, 128, 0, 2 ** 31 - 1, 4) >= attn.attn_workspace_size(attn.ATTN_OP_BWD, 1, 8, 2, 3000, 128)
