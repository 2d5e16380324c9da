"""Argument checks of the step plan, the head norm and the tree attention: every refusal returns its documented
code (or raises in the binding) before anything is launched. Needs no GPU."""
import ctypes

import pytest
import torch

import attention_flash_gqa_gb300 as attn
from attention_flash_gqa_gb300 import _build

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
A = 1 << 20  # a fake, aligned "device" address: never dereferenced on these paths
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return attn.load_library()


def caller(fn, names, defaults):
    def call(**kw):
        args = dict(defaults, **kw)
        return fn(*[args[n] for n in names])
    return call


def test_plan_refusals(lib):
    names = ("kv new held free used table seq cu pos slots held_out used_out adm R T F ps maxp np stream").split()
    call = caller(lib.attn_paged_plan, names, dict({n: A for n in names}, R=4, T=9, F=5, ps=16, maxp=8, np=64, stream=None))
    for n in ("kv", "new", "held", "free", "used", "table", "seq", "cu", "pos", "slots", "held_out", "used_out", "adm"):
        assert call(**{n: None}) == INVALID, n
        assert call(**{n: A + 2}) == MISALIGNED, n
    for n in ("R", "T", "F", "maxp", "np"):
        assert call(**{n: -1}) == INVALID, n
    assert call(ps=0) == INVALID and call(ps=32) == UNSUPPORTED
    assert call(R=16385) == UNSUPPORTED and call(np=(1 << 26) + 1) == UNSUPPORTED and call(T=(1 << 30) + 1) == UNSUPPORTED


NORM = "T Hq Hkv D rot maxp".split()
TAIL = "eps off w32 inter".split()
BASE = dict(T=7, Hq=8, Hkv=2, D=128, rot=128, maxp=100, qs=1024, ks=256, vs=256, dqs=1024, dks=256, eps=1e-6, off=0.0, w32=0,
            inter=0, ps=16, np=64, wsb=1 << 40, stream=None)


def norm_callers(lib):
    p = lambda s: s.split()  # noqa: E731
    sig = {
        "fwd": (lib.attn_qk_norm_rope, p("q k qo ko qw kw pos cs") + NORM + p("qs ks") + TAIL + p("stream")),
        "bwd": (lib.attn_qk_norm_rope_bwd, p("dqo dko q k dq dk dqw dkw qw kw pos cs") + NORM + p("qs ks dqs dks") + TAIL + p("ws wsb stream")),
        "paged": (lib.attn_qk_norm_rope_paged, p("q k v qo kc vc qw kw pos slots cs") + NORM + p("ps np qs ks vs") + TAIL + p("stream")),
    }
    # distinct fake addresses: equal ones would mean an update in place
    return {k: caller(f, n, dict({x: A * (i + 1) for i, x in enumerate(n)}, **BASE)) for k, (f, n) in sig.items()}


def test_norm_rope_refusals(lib):
    calls = norm_callers(lib)
    for kind, call in calls.items():
        for kw, code in ((dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(rot=-16), INVALID),
                         (dict(maxp=-1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
                         (dict(eps=INF), INVALID), (dict(off=NAN), INVALID), (dict(D=96, rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
                         (dict(rot=144), UNSUPPORTED), (dict(Hq=2049), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED),
                         (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(pos=None), INVALID), (dict(cs=None), INVALID),
                         (dict(q=A + 8), MISALIGNED), (dict(cs=A + 4), MISALIGNED), (dict(pos=A + 1), MISALIGNED),
                         (dict(qw=A + 2), MISALIGNED), (dict(qs=-8), INVALID), (dict(qs=1025), MISALIGNED), (dict(ks=4), MISALIGNED)):
            assert call(**kw) == code, (kind, kw)
    for kw, code in ((dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(ko=A + 2), MISALIGNED), (dict(T=0), OK),
                     (dict(T=0, q=None, k=None, pos=None, cs=None, qo=None, ko=None), OK),
                     (dict(q=A, qo=A, qs=2048), INVALID)):  # in place over rows that are not the output's
        assert calls["fwd"](**kw) == code, kw
    for kw, code in ((dict(dqo=None), INVALID), (dict(dk=None), INVALID), (dict(dq=A + 8), MISALIGNED), (dict(dqw=A + 2), MISALIGNED),
                     (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=A + 16), MISALIGNED),
                     (dict(dqs=512), INVALID), (dict(dks=260), MISALIGNED),  # overlapping rows; not 16-byte multiples
                     (dict(dqo=A, dq=A, dqs=2048), INVALID)):
        assert calls["bwd"](**kw) == code, kw
    for kw, code in ((dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(kc=None), INVALID), (dict(vc=A + 8), MISALIGNED),
                     (dict(slots=A + 1), MISALIGNED), (dict(ps=0), INVALID), (dict(ps=64), UNSUPPORTED), (dict(np=-1), INVALID),
                     (dict(np=1 << 27), UNSUPPORTED), (dict(vs=7), MISALIGNED), (dict(T=0), OK)):
        assert calls["paged"](**kw) == code, kw


def test_tree_refusals(lib):
    names = ("q kc vc bt sl cu mask pos o lse R T maxq words Hq Hkv D ps maxp np scale window ws wsb stream").split()
    call = caller(lib.attn_tree_paged, names, dict({n: A for n in names}, R=3, T=20, maxq=9, words=1, Hq=8, Hkv=2, D=128, ps=16,
                                                   maxp=8, np=64, scale=0.1, window=0, wsb=1 << 40, stream=None))
    for n in ("q", "kc", "vc", "bt", "sl", "cu", "mask", "o", "lse"):
        assert call(**{n: None}) == INVALID, n
        assert call(**{n: A + 2}) == MISALIGNED, n
    for kw, code in ((dict(R=-1), INVALID), (dict(T=-1), INVALID), (dict(maxq=-1), INVALID), (dict(words=-1), INVALID),
                     (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=NAN), INVALID),
                     (dict(window=-1), INVALID), (dict(window=5, pos=None), INVALID), (dict(maxq=33), INVALID), (dict(np=0), INVALID),
                     (dict(maxp=0), INVALID), (dict(ps=0), INVALID), (dict(ps=32), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
                     (dict(maxq=257, words=9), UNSUPPORTED), (dict(words=9), UNSUPPORTED), (dict(R=4097), UNSUPPORTED),
                     (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(Hq=257, Hkv=257), UNSUPPORTED), (dict(np=1 << 27), UNSUPPORTED),
                     (dict(pos=A + 1, window=3), MISALIGNED), (dict(ws=A + 16), MISALIGNED),
                     (dict(R=0), OK), (dict(T=0), OK), (dict(maxq=0, words=0), OK),
                     (dict(T=0, q=None, kc=None, vc=None, bt=None, sl=None, cu=None, mask=None, o=None, lse=None), OK)):
        assert call(**kw) == code, kw
    need = attn.attn_workspace_size(attn.ATTN_OP_TREE_PAGED, Hq=8, Hkv=2, S=9, D=128)
    if need:
        assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE


def test_workspace_sizes(lib):
    size = attn.attn_workspace_size
    assert size(attn.ATTN_OP_QK_NORM_ROPE_BWD, D=256) % 256 == 0 and size(attn.ATTN_OP_QK_NORM_ROPE_BWD, D=100) == 0
    assert size(attn.ATTN_OP_TREE_PAGED, Hq=8, Hkv=2, S=9, D=96) == 0 and size(attn.ATTN_OP_TREE_PAGED, Hq=8, Hkv=3, S=9, D=128) == 0


def test_binding_refuses_cpu_tensors(lib):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        attn.attn_qk_norm_rope(z(2, 2, 64), z(2, 1, 64), None, None, None, None)
    with pytest.raises(ValueError):
        attn.attn_qk_norm_rope_paged(z(2, 2, 64), z(2, 1, 64), z(2, 1, 64), None, None, None, i(2), None, z(1, 16, 1, 64), z(1, 16, 1, 64))
    with pytest.raises(ValueError):
        attn.attn_paged_plan(i(2), i(2), i(2), i(2, 2), i(2), i(1), 2, num_pages=2)
    with pytest.raises(ValueError):
        attn.attn_tree_paged(z(2, 2, 64), z(1, 16, 1, 64), z(1, 16, 1, 64), i(1, 1), i(1), i(2), i(2, 1), 2)


def test_launch_pointers_are_not_read_on_refusals(lib):
    """A refused call leaves the launch counter alone."""
    before = attn.attn_launch_count()
    norm_callers(lib)["fwd"](D=100)
    assert attn.attn_launch_count() == before and isinstance(before, int) and ctypes.sizeof(ctypes.c_longlong) == 8
