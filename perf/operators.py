"""The serving and training operators around the attention kernels, as a user's program calls them.

Four groups of operators, each in its plain form (elementary torch operations, 32-bit or wider) and through
the package's public entry points:

* plan        -- block-table rows, slot map, positions and prefix sums of a step, from request lengths
* norm_rope   -- RMS norm of every query and key head with the rotary position encoding, forward
* norm_bwd    -- its gradients (inputs and norm weights)
* to_cache    -- the same forward for serving: K and V go straight into the paged cache by slot
* tree        -- attention of drafted token trees over a paged cache

``own`` selects which of the two ``run`` takes.
"""
import math
import random

import torch

own = False

PAGE = 16
EPS = 1e-6


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # the step plan of a decode batch: one new token for each of 64 requests (latency only)
        dict(name="plan decode 64", op="plan", R=64, lo=256, hi=1024, new_lo=1, new_hi=1),
        # the step plan of a large mixed batch: prompts and continuations, some 500 thousand new tokens
        dict(name="plan prefill 1000", op="plan", R=1000, lo=0, hi=6000, new_lo=1, new_hi=1000),
        # training forward of the sliding-window layers: B 2, S 8192, Hq 32, Hkv 16, head_dim 256
        dict(name="norm_rope train d256", op="norm_rope", T=16384, Hq=32, Hkv=16, D=256, rot=256, inter=False, w32=False,
             fused=True),
        # a short ragged sequence through small heads, interleaved pairs on half of the dims, fp32 weights
        dict(name="norm_rope odd d64", op="norm_rope", T=333, Hq=12, Hkv=3, D=64, rot=32, inter=True, w32=True, fused=False),
        # training backward of the packed head_dim 512 layers (8 sequences), a quarter of the dims rotated
        dict(name="norm_bwd packed d512", op="norm_bwd", T=18001, Hq=32, Hkv=4, D=512, rot=128, inter=False, w32=True,
             fused=True),
        # the backward of one short sequence at head_dim 128
        dict(name="norm_bwd short d128", op="norm_bwd", T=511, Hq=32, Hkv=8, D=128, rot=128, inter=False, w32=False,
             fused=False),
        # one decode step of 64 requests writes its keys and values (latency)
        dict(name="to_cache decode d128", op="to_cache", T=64, Hq=32, Hkv=8, D=128, rot=128, inter=False, w32=False,
             fused=True),
        # a chunked prefill step: 8 requests of 512 new tokens, head_dim 512
        dict(name="to_cache chunk d512", op="to_cache", T=4096, Hq=32, Hkv=4, D=512, rot=128, inter=False, w32=False,
             fused=True),
        # one user's drafted tree (latency)
        dict(name="tree one request d128", op="tree", R=1, lo=900, hi=1000, n_lo=8, n_hi=8, Hq=32, Hkv=8, D=128, window=0),
        # the decode batch with small trees: every cached key is read once for all its rows
        dict(name="tree batch d128", op="tree", R=64, lo=256, hi=1024, n_lo=5, n_hi=16, Hq=32, Hkv=8, D=128, window=0),
        # long contexts, wide trees: several row tiles per KV head
        dict(name="tree long d128", op="tree", R=12, lo=5000, hi=24000, n_lo=33, n_hi=64, Hq=32, Hkv=8, D=128, window=0),
        # sliding-window layers at head_dim 256, contexts past the window
        dict(name="tree window d256", op="tree", R=64, lo=1024, hi=4096, n_lo=4, n_hi=24, Hq=32, Hkv=16, D=256, window=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "norm_rope", "norm_bwd", "to_cache", "tree", "tree"])
    if op == "plan":
        new_hi = _log_int(rng, 1, 1000)
        return dict(op=op, R=_log_int(rng, 1, 1000), lo=rng.randint(0, 500), hi=_log_int(rng, 512, 6000), new_lo=1,
                    new_hi=new_hi)
    D = rng.choice([64, 128, 256, 512])
    Hkv = rng.randint(1, 16)
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op != "tree":
        top = {"norm_rope": 16384 * 48 * 256, "norm_bwd": 18001 * 36 * 512, "to_cache": 4096 * 40 * 512}[op]
        T = _log_int(rng, 1, max(1, min(40000, top // ((G + 2) * Hkv * D))))
        return dict(op=op, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, rot=rng.choice([r for r in (16, 32, 64, 96, 128, 256, 512) if r <= D]),
                    inter=rng.random() < 0.3, w32=rng.random() < 0.5, fused=rng.random() < 0.5)
    n_hi = _log_int(rng, 1, 64)
    R = _log_int(rng, 1, 64)
    # no drawn call reads more of a cache, or multiplies more, than the largest listed one
    most = min(24000, 12 * 14500 * 8 * 128 // (R * Hkv * D), 12 * 14500 * 32 * 128 * 48 // (R * G * Hkv * D * n_hi))
    hi = _log_int(rng, 16, max(17, most))
    return dict(op=op, R=R, lo=rng.randint(0, hi), hi=hi, n_lo=rng.randint(1, n_hi), n_hi=n_hi, Hq=G * Hkv, Hkv=Hkv, D=D,
                window=rng.choice([0, 0, 0, 100, 1024]))


def _lens(case, lo, hi, salt):
    """The requests' lengths: part of the case, not of the seed."""
    r = random.Random("%d %d %d %d" % (case["R"], case[lo], case[hi], salt))
    return [r.randint(case[lo], case[hi]) for _ in range(case["R"])]


# ---------------------------------------------------------------------------------------------
# inputs

def _dev():
    return torch.device("cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def prepare(case, seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed))
    s = {"case": case, "g": g}
    {"plan": _prep_plan, "norm_rope": _prep_norm, "norm_bwd": _prep_norm, "to_cache": _prep_norm, "tree": _prep_tree}[case["op"]](case, g, s)
    del s["g"]
    return s


def _prep_plan(case, g, s):
    R = case["R"]
    kv, new = _lens(case, "lo", "hi", 1), _lens(case, "new_lo", "new_hi", 2)
    s["T"] = sum(new)
    # a request holds the pages of its cached tokens, some of them one page more (left by rejected drafts)
    extra = torch.randint(0, 2, (R,), generator=g, device=_dev(), dtype=torch.int32)
    kv_t, new_t = _i32(kv), _i32(new)
    held = (kv_t + PAGE - 1) // PAGE + extra
    s["max_pages"] = max((a + b + PAGE - 1) // PAGE for a, b in zip(kv, new)) + 2
    pages = sum((a + PAGE - 1) // PAGE + 1 for a in kv) + sum((b + PAGE - 1) // PAGE + 1 for b in new) + 64
    perm = torch.randperm(pages, generator=g, device=_dev()).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(s["max_pages"], device=_dev())
    at = (first[:, None] + col[None, :]).clamp(max=pages - 1)
    s["table"] = torch.where(col[None, :] < held[:, None], perm[at.long()], torch.full_like(at, -1, dtype=torch.int32)).to(torch.int32).contiguous()
    s["free"] = perm.roll(-int(held.sum())).contiguous()[: pages - int(held.sum())].contiguous()
    s["used"] = torch.zeros(1, dtype=torch.int32, device=_dev())
    s.update(kv=kv_t, new=new_t, held=held.to(torch.int32), num_pages=pages)


def _table(rows, rot, theta=10000.0):
    """cos | sin of position * theta^(-2 i / rot), angles in 64 bits, held in 32."""
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=_dev()) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=_dev())[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _prep_norm(case, g, s):
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    n = lambda *shape: torch.randn(shape, generator=g, device=_dev(), dtype=torch.float32)  # noqa: E731
    if case["fused"]:  # q, k, v as the projection leaves them: slices of one row
        qkv = (n(T, (Hq + 2 * Hkv) * D) * 1.7).to(torch.bfloat16)
        q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
        q, k, v = q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D)
    else:
        q, k, v = (n(T, h, D).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    wt = torch.float32 if case["w32"] else torch.bfloat16
    s.update(q=q, k=k, qw=(1 + 0.2 * n(D)).to(wt), kw=(1 + 0.2 * n(D)).to(wt))
    rows = 8192
    s["cs"] = _table(rows, case["rot"])
    s["pos"] = torch.randint(0, rows, (T,), generator=g, device=_dev(), dtype=torch.int32)
    if case["op"] == "norm_bwd":
        s["gq"], s["gk"] = n(T, Hq, D).to(torch.bfloat16), n(T, Hkv, D).to(torch.bfloat16)
    if case["op"] == "to_cache":
        pages = (T + PAGE - 1) // PAGE * 2 + 8
        s["v"] = v
        s["slots"] = torch.randperm(pages * PAGE, generator=g, device=_dev())[:T].to(torch.int32).contiguous()
        s["kc"] = torch.zeros(pages, PAGE, Hkv, D, dtype=torch.bfloat16, device=_dev())
        s["vc"] = torch.zeros_like(s["kc"])


def _prep_tree(case, g, s):
    R, Hq, Hkv, D = case["R"], case["Hq"], case["Hkv"], case["D"]
    ctx, n = _lens(case, "lo", "hi", 1), _lens(case, "n_lo", "n_hi", 2)
    top, T = max(n), sum(n)
    L = [a + b for a, b in zip(ctx, n)]
    npg = [(a + PAGE - 1) // PAGE for a in L]
    pages = sum(npg) + 16
    bf = lambda *shape: torch.randn(shape, generator=g, device=_dev(), dtype=torch.bfloat16)  # noqa: E731
    s.update(q=bf(T, Hq, D), kc=bf(pages, PAGE, Hkv, D), vc=bf(pages, PAGE, Hkv, D))
    perm = torch.randperm(pages, generator=g, device=_dev()).to(torch.int32)
    held = _i32(npg)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(max(npg), device=_dev())
    at = (first[:, None] + col[None, :]).clamp(max=pages - 1)
    s["table"] = torch.where(col[None, :] < held[:, None], perm[at.long()], torch.full_like(at, -1, dtype=torch.int32)).to(torch.int32).contiguous()
    s["lens"] = _i32(L)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s["cu"] = _i32(cu)
    # each drafted token's parent is an earlier one or the last cached token; it sees its ancestors and itself
    words = (top + 31) // 32
    par = (torch.rand(R, top, generator=g, device=_dev()) * (torch.arange(top, device=_dev()) + 1)).long() - 1
    anc = torch.zeros(R, top, words * 32, dtype=torch.bool, device=_dev())
    at = torch.arange(R, device=_dev())
    for i in range(top):
        p = par[:, i]
        if i:
            anc[:, i] = anc[at, p.clamp(min=0)] & (p >= 0)[:, None]
        anc[:, i, i] = True
    live = torch.arange(top, device=_dev())[None, :] < _i32(n)[:, None]
    bits = anc[live].view(T, words, 32).to(torch.int64) << torch.arange(32, device=_dev())
    word = bits.sum(2)
    s["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32).contiguous()
    depth = anc.sum(2) - 1
    s["pos"] = (_i32(ctx).long()[:, None] + depth)[live].to(torch.int32).contiguous()
    s["top"] = top
    s["scale"] = 1.0 / math.sqrt(D)


# ---------------------------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"plan": _plain_plan, "norm_rope": _plain_norm, "norm_bwd": _plain_bwd, "to_cache": _plain_to_cache, "tree": _plain_tree}[op](s)


def _own(op, s):
    import attention_flash_gqa_gb300 as attn

    c = s["case"]
    if op == "plan":
        p = attn.attn_paged_plan(s["kv"], s["new"], s["free"], s["table"], s["held"], s["used"], s["T"], num_pages=s["num_pages"])
        return [p.seq_lens, p.cu_q, p.positions, p.slots, p.pages_held, p.free_used, p.admitted, s["table"]]
    if op == "norm_rope":
        return attn.attn_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["cs"], eps=EPS, interleaved=c["inter"])
    if op == "norm_bwd":
        return attn.attn_qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["cs"], eps=EPS,
                                          interleaved=c["inter"])
    if op == "to_cache":
        q = attn.attn_qk_norm_rope_paged(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["pos"], s["slots"], s["cs"], s["kc"], s["vc"],
                                         eps=EPS, interleaved=c["inter"])
        return [q, s["kc"], s["vc"]]
    return attn.attn_tree_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["cu"], s["mask"], s["top"], positions=s["pos"],
                                window=c["window"], scale=s["scale"])


def _plain_plan(s):
    kv, new, held, used, free, table, T = s["kv"].long(), s["new"].long(), s["held"].long(), s["used"].long(), s["free"], s["table"], s["T"]
    need = ((kv + new + PAGE - 1) // PAGE - held).clamp(min=0)
    fits = (torch.cumsum(new, 0) <= T) & (used + torch.cumsum(need, 0) <= free.numel())
    adm = torch.cumprod(fits.long(), 0)  # in order, up to the first that does not fit
    new, need = new * adm, need * adm
    end, off = torch.cumsum(new, 0), torch.cumsum(need, 0) - need
    cu = torch.cat([torch.zeros_like(end[:1]), end])
    col = torch.arange(table.shape[1], device=table.device)[None, :] - held[:, None]
    take = (col >= 0) & (col < need[:, None])
    at = (used + off[:, None] + col).clamp(0, free.numel() - 1)
    table = torch.where(take, free[at], table)
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(end, t, right=True)
    live = b < kv.numel()
    b = b.clamp(max=kv.numel() - 1)
    pos = kv[b] + t - cu[b]
    slot = table[b, (pos // PAGE).clamp(max=table.shape[1] - 1)].long() * PAGE + pos % PAGE
    pos, slot = torch.where(live, pos, 0), torch.where(live, slot, -1)
    i = lambda x: x.to(torch.int32)  # noqa: E731
    return [i(kv + new), i(cu), i(pos), i(slot), i(held + need), i(used + need.sum()), i(adm.sum()).view(1), table]


def _turn(x, s, back=False):
    """The rotation of the first `rot` dims of x [T, H, D] (its transpose where `back`)."""
    c = s["case"]
    r = c["rot"]
    cs = s["cs"][s["pos"].long()][:, None, :]
    cos, sin = cs[..., : r // 2], cs[..., r // 2:]
    if back:
        sin = -sin
    if c["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _normed(x, w, s):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(x, s).to(torch.bfloat16)


def _plain_norm(s):
    return _normed(s["q"], s["qw"], s), _normed(s["k"], s["kw"], s)


def _plain_to_cache(s):
    at = s["slots"].long()
    q = _normed(s["q"], s["qw"], s)
    s["kc"].view(-1, *s["kc"].shape[2:])[at] = _normed(s["k"], s["kw"], s)
    s["vc"].view(-1, *s["vc"].shape[2:])[at] = s["v"]
    return [q, s["kc"], s["vc"]]


def _grads(x, w, dy, s):
    x, dn = x.float(), _turn(dy.float(), s, back=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dw = (dn * xh).sum((0, 1))
    gw = dn * w.float()
    return (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _plain_bwd(s):
    (dq, dqw), (dk, dkw) = _grads(s["q"], s["qw"], s["gq"], s), _grads(s["k"], s["kw"], s["gk"], s)
    return dq, dk, dqw, dkw


def _plain_tree(s):
    c = s["case"]
    q, table, L, cu, top = s["q"], s["table"], s["lens"].long(), s["cu"].long(), s["top"]
    T, Hq, D = q.shape
    R, Hkv = c["R"], c["Hkv"]
    n = cu[1:] - cu[:-1]
    ctx = L - n
    i = torch.arange(top, device=q.device)
    live = i[None, :] < n[:, None]
    row = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)
    qp = q[row].float().view(R, top, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, -1, D)
    at = table.clamp(min=0).long()
    j = torch.arange(table.shape[1] * PAGE, device=q.device)
    there = (j[None, :] < L[:, None])[:, :, None, None]
    kk = torch.where(there, s["kc"][at].view(R, -1, Hkv, D), 0).float().permute(0, 2, 3, 1)
    vv = torch.where(there, s["vc"][at].view(R, -1, Hkv, D), 0).float().permute(0, 2, 1, 3)
    sc = torch.matmul(qp * s["scale"], kk).view(R, Hkv, Hq // Hkv, top, -1)
    d = j[None, :] - ctx[:, None]  # index among the drafted tokens
    w = s["mask"][row].long()  # [R, top, words]
    dd = d.clamp(0, w.shape[2] * 32 - 1)
    bit = (w.gather(2, (dd // 32)[:, None, :].expand(R, top, -1)) >> (dd % 32)[:, None, :]) & 1
    pos = torch.maximum(s["pos"][row].long(), ctx[:, None])
    near = (pos[:, :, None] - j < c["window"]) if c["window"] else torch.ones_like(bit, dtype=torch.bool)
    see = torch.where(d[:, None, :] < 0, near, (bit > 0) & (d < n[:, None])[:, None, :]) & live[:, :, None]
    sc = sc.masked_fill_(~see[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = (sc - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, Hkv, -1, p.shape[-1]), vv).view(R, Hkv, Hq // Hkv, top, D) / torch.where(l == 0, 1, l)
    lse = (l.log() + m).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(R, top, Hq, D)[live].to(torch.bfloat16)
    return o, lse.permute(0, 3, 1, 2).reshape(R, top, Hq)[live].t().contiguous()


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "tree":
        return _exact_tree(case, s)
    T, D, r = case["T"], case["D"], case["rot"]
    dev = s["q"].device
    # the rotation as complex numbers: pair i is a + i b, turned by cos + i sin
    cs = s["cs"].double()[s["pos"].long()]
    z = torch.complex(cs[:, : r // 2], cs[:, r // 2:])[:, None, :]
    first = torch.arange(0, r, 2, device=dev) if case["inter"] else torch.arange(0, r // 2, device=dev)
    second = first + (1 if case["inter"] else r // 2)

    def turned(x, z):
        y = x.clone()
        p = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = p.real, p.imag
        return y

    def fwd(x, w):
        x = x.double()
        return turned(x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.double(), z)

    if case["op"] == "norm_bwd":
        def bwd(x, w, dy):
            x, g = x.double(), turned(dy.double(), z.conj())
            ms = x.square().sum(-1, keepdim=True) / D + EPS
            dw = (g * x / ms.sqrt()).sum(0).sum(0)
            g = g * w.double()
            return g / ms.sqrt() - x * (g * x).sum(-1, keepdim=True) / (D * ms * ms.sqrt()), dw

        (dq, dqw), (dk, dkw) = bwd(s["q"], s["qw"], s["gq"]), bwd(s["k"], s["kw"], s["gk"])
        return dq, dk, dqw, dkw
    if case["op"] == "norm_rope":
        return fwd(s["q"], s["qw"]), fwd(s["k"], s["kw"])
    kc, vc = torch.zeros_like(s["kc"], dtype=torch.float64), torch.zeros_like(s["vc"], dtype=torch.float64)
    page, at = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    kc[page, at] = fwd(s["k"], s["kw"])
    vc[page, at] = s["v"].double()
    return [fwd(s["q"], s["qw"]), kc, vc]


def _exact_tree(case, s):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out, lses = [], []
    cu, L = s["cu"].tolist(), s["lens"].tolist()
    for b in range(case["R"]):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        used = s["table"][b, : (L[b] + PAGE - 1) // PAGE].long()
        k = s["kc"][used].flatten(0, 1)[: L[b]].double()
        v = s["vc"][used].flatten(0, 1)[: L[b]].double()
        ctx = L[b] - n
        see = torch.ones(n, L[b], dtype=torch.bool, device=k.device)
        if case["window"]:
            at = s["pos"][rows].long().clamp(min=ctx)
            see[:, :ctx] = torch.arange(ctx, device=k.device)[None, :] > at[:, None] - case["window"]
        i = torch.arange(n, device=k.device)
        see[:, ctx:] = (s["mask"][rows].long()[:, i // 32] >> (i % 32)) & 1 == 1
        o, lse = [], []
        for h in range(Hkv):
            q = s["q"][rows, h * (Hq // Hkv): (h + 1) * (Hq // Hkv)].double()
            x = torch.einsum("ngd,kd->gnk", q, k[:, h]) * s["scale"]
            x = x.masked_fill(~see, -math.inf)
            e = torch.logsumexp(x, -1)
            p = torch.where(see, (x - e[..., None]).exp(), 0.0)
            o.append(torch.einsum("gnk,kd->ngd", p, v[:, h]))
            lse.append(e)
        out.append(torch.cat(o, 1))
        lses.append(torch.cat(lse, 0))
    return torch.cat(out, 0), torch.cat(lses, 1)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "plan":
        kv, new = _lens(case, "lo", "hi", 1), _lens(case, "new_lo", "new_hi", 2)
        T = sum(new)
        pages = sum((b + PAGE - 1) // PAGE for b in new)
        # lengths and held pages in, lengths, held pages and prefix sums out, taken pages, slots and positions
        return {"bytes": 4 * case["R"] * 6 + 8 * pages + 8 * T, "flops": 0}
    if op == "tree":
        ctx, n = _lens(case, "lo", "hi", 1), _lens(case, "n_lo", "n_hi", 2)
        Hq, Hkv, D, W = case["Hq"], case["Hkv"], case["D"], case["window"]
        near = [min(c, W - 1) if W else c for c in ctx]
        keys, T = sum(a + b for a, b in zip(near, n)), sum(n)
        return {"bytes": keys * Hkv * D * 4 + T * Hq * (4 * D + 4) + keys // 4, "flops": 4 * D * Hq * sum(b * (a + 1) for a, b in zip(near, n))}
    T, D, H, Hkv = case["T"], case["D"], case["Hq"] + case["Hkv"], case["Hkv"]
    table = min(T, 8192) * case["rot"] * 4
    if op == "norm_rope":
        return {"bytes": T * H * D * 4 + table + 4 * T, "flops": 8 * T * H * D}
    if op == "norm_bwd":
        return {"bytes": T * H * D * 6 + table + 4 * T + 8 * D, "flops": 16 * T * H * D}
    return {"bytes": T * (H + Hkv) * D * 4 + table + 8 * T, "flops": 8 * T * H * D}
