"""The plan of a serving step (attn_paged_plan) against a plain integer implementation."""
import random

import pytest
import torch

import attention_flash_gqa_gb300 as attn
import operator_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_flash_gqa_gb300 import _build

    _build.build()
    attn.load_library()
    torch.cuda.set_device(0)
    attn.attn_get_device_status()


def i32(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32, device="cuda")
    return t if shape is None else t.reshape(shape)


def problem(R, lo, hi, new_lo, new_hi, seed, extra=1, spare=8, pad=0):
    r = random.Random(seed)
    kv = [r.randint(lo, hi) for _ in range(R)]
    new = [r.randint(new_lo, new_hi) for _ in range(R)]
    held = [-(-a // 16) + r.randint(0, extra) for a in kv]
    cap = max([-(-(a + b) // 16) for a, b in zip(kv, new)] + held + [1]) + 1
    need = sum(max(0, -(-(a + b) // 16) - h) for a, b, h in zip(kv, new, held))
    num_pages = sum(held) + need + spare + 3
    ids = list(range(num_pages))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at: at + h] + [-1] * (cap - h))
        at += h
    free = [7] * 3 + ids[at: at + need + spare]  # three of them already taken
    return dict(kv=kv, new=new, held=held, free=free, used=3, table=table, T=sum(new) + pad, num_pages=num_pages)


def run(p, in_place=False):
    R = len(p["kv"])
    kv, new, held, used = i32(p["kv"]), i32(p["new"]), i32(p["held"]), i32([p["used"]])
    table = i32(p["table"], (R, -1 if R else 4))
    out = None
    if in_place:
        e = lambda n: torch.full((n,), 99, dtype=torch.int32, device="cuda")  # noqa: E731
        out = attn.PagedPlan(kv, e(R + 1), e(p["T"]), e(p["T"]), held, used, e(1))
    got = attn.attn_paged_plan(kv, new, i32(p["free"]), table, held, used, p["T"], num_pages=p["num_pages"], out=out)
    status = attn.attn_get_device_status()
    return got, table, status


def compare(p, in_place=False):
    got, table, status = run(p, in_place)
    want = ref.plan(p["kv"], p["new"], p["held"], p["free"], p["used"], p["table"], p["T"], p["num_pages"])
    for name in attn.PagedPlan._fields:
        assert getattr(got, name).tolist() == want[name], name
    assert table.tolist() == want["table"]
    assert status == (7 if want["bad"] else 0)
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,lo,hi,new_lo,new_hi", [(1, 0, 0, 1, 1), (1, 15, 17, 1, 1), (3, 0, 40, 0, 3), (64, 256, 1024, 1, 1),
                                                   (33, 0, 100, 0, 700), (700, 0, 50, 0, 2), (2000, 0, 33, 0, 40)])
def test_plan(R, lo, hi, new_lo, new_hi, in_place):
    for seed in range(3):
        compare(problem(R, lo, hi, new_lo, new_hi, 100 * R + seed, pad=seed * 5), in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_many_rows(in_place):
    """More rows than four for each thread of the GPU, ending inside a thread's run."""
    p = problem(300, 0, 100, 500, 2700, 21, pad=3)
    assert p["T"] > 400000
    compare(p, in_place)


def test_plan_largest_batch():
    """16384 requests, two of them with everything: the prefix sums fill 128 KB of shared memory."""
    p = problem(16384, 0, 20, 0, 2, 5)
    compare(p)
    compare(p, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_out_of_pages_and_rows(in_place):
    """Requests are admitted in order up to the first that does not fit; the others keep their state."""
    p = problem(40, 0, 60, 1, 30, 11, spare=0)
    for cut in (1, 5, len(p["free"]) - 4):
        want = compare(dict(p, free=p["free"][: len(p["free"]) - cut]), in_place)
        assert want["admitted"][0] < 40
    want = compare(dict(p, T=p["T"] - 1), in_place)
    assert want["admitted"] == [39]
    want = compare(dict(p, T=3), in_place)
    assert want["bad"]
    compare(dict(p, free=[], used=0), in_place)


def test_plan_refuses_inconsistent_requests():
    """A request with impossible lengths gets nothing and is reported; the others are served."""
    for key, b, value in (("kv", 4, -1), ("new", 5, -7), ("held", 6, -1), ("held", 7, 10000), ("kv", 8, 5000),
                          ("new", 9, 2 ** 31 - 1), ("kv", 10, 2 ** 31 - 1)):
        p = problem(20, 0, 60, 1, 30, 13)
        p[key][b] = value
        want = compare(p)
        assert want["bad"] and want["admitted"] == [20]
        compare(p, in_place=True)


def test_plan_refuses_bad_ids_and_cursors():
    p = problem(20, 0, 60, 1, 30, 17)
    p["free"][6] = p["num_pages"]  # handed out
    p["free"][9] = -5
    assert compare(p)["bad"]
    p = problem(20, 20, 60, 1, 1, 19, extra=0)
    b = next(i for i in range(20) if p["kv"][i] % 16)
    p["table"][b][p["kv"][b] // 16] = -3  # the page that the new token falls into
    assert compare(p)["bad"]
    for used in (-1, 10 ** 6):
        assert compare(dict(problem(5, 0, 60, 1, 30, 23), used=used))["bad"]


def test_plan_nothing_to_do():
    got, _, status = run(dict(kv=[], new=[], held=[], free=[4], used=1, table=[], T=3, num_pages=8))
    assert status == 0 and got.cu_q.tolist() == [0] and got.slots.tolist() == [-1] * 3 and got.positions.tolist() == [0] * 3
    assert got.free_used.tolist() == [1] and got.admitted.tolist() == [0]
    compare(problem(9, 0, 60, 0, 0, 29))


def test_plan_long_request():
    """One prompt longer than many: rows and pages of one request spread over the whole grid."""
    compare(problem(2, 70000, 70001, 130000, 130001, 31))


def test_plan_state_kept_in_place_over_captured_steps():
    """A captured step replayed: the state advances on the device as the plain implementation's does."""
    p = problem(12, 0, 100, 1, 20, 37, spare=400)
    for row in p["table"]:
        row += [-1] * 40
    T = p["T"]
    kv, new, held, used = i32(p["kv"]), i32(p["new"]), i32(p["held"]), i32([p["used"]])
    table, free = i32(p["table"]), i32(p["free"])
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = attn.PagedPlan(kv, e(13), e(T), e(T), held, used, e(1))
    step = lambda: attn.attn_paged_plan(kv, new, free, table, held, used, T, num_pages=p["num_pages"], out=out)  # noqa: E731
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    want = None
    for k in range(6):
        g.replay()
        if k == 2:  # a smaller step: fewer rows than the capture has
            pass
        torch.cuda.synchronize()
        s = want or dict(seq_lens=p["kv"], pages_held=p["held"], free_used=[p["used"]], table=p["table"])
        want = ref.plan(s["seq_lens"], p["new"], s["pages_held"], p["free"], s["free_used"][0], s["table"], T, p["num_pages"])
        for name in attn.PagedPlan._fields:
            assert getattr(out, name).tolist() == want[name], (k, name)
        assert table.tolist() == want["table"]
        p["new"] = [max(0, x - 3) for x in p["new"]]  # the next step adds fewer tokens
        new.copy_(i32(p["new"]))
    assert attn.attn_get_device_status() == 0


def test_plan_on_another_stream():
    p = problem(64, 0, 300, 1, 40, 41)
    s = torch.cuda.Stream()
    args = [i32(p[k]) for k in ("kv", "new", "free", "table", "held")]
    used = i32([p["used"]])
    s.wait_stream(torch.cuda.current_stream())
    kv, new, free, table, held = args
    got = attn.attn_paged_plan(kv, new, free, table, held, used, p["T"], num_pages=p["num_pages"], stream=s)
    s.synchronize()
    want = ref.plan(p["kv"], p["new"], p["held"], p["free"], p["used"], p["table"], p["T"], p["num_pages"])
    assert got.slots.tolist() == want["slots"] and got.pages_held.tolist() == want["pages_held"]
