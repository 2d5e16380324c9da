"""Sliding windows with sinks, and a paged cache in 4 bits, as a user's program calls them.

Five operators, each in its plain form (elementary torch operations, 32-bit or wider) and through the package's
public entry points:

* fwd         -- attention forward where a query sees its last `window` keys and the sequence's first `sink` ones
* train       -- the same forward and its gradient: one attention layer's share of a training step
* decode      -- one new token a request over the bf16 paged cache, window and sinks
* kv4_write   -- new keys and values into the 4-bit paged cache, and the pages back as bf16 (what a chunk's
                 attention over the cache reads next)
* kv4_decode  -- one new token a request over the 4-bit paged cache, window and sinks

The 4-bit cache, uint8 [pages, Hkv, 18, D]: one record of 18 D bytes for the 16 tokens of a page and KV head. A
group of 32 consecutive dims of one token is n * s with n in -8 .. 7, held as n + 8 in 4 bits, and s a bf16 number
of 5 significant bits, so that n * s is a bf16 number as well. The record's order is in `_places`.

``own`` selects which of the two ``run`` takes.
"""
import math
import random

import torch

own = False

PAGE = 16
GROUP = 32


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # prompt through the sliding-window layers: B 2, S 8192, 32 and 16 heads of 256, window 1024
        dict(name="fwd window d256", op="fwd", R=2, lo=8192, hi=8192, Hq=32, Hkv=16, D=256, window=1024, sink=4),
        # prompts of different lengths, packed; a window that is no multiple of any tile
        dict(name="fwd packed d128", op="fwd", R=8, lo=1, hi=4096, Hq=32, Hkv=8, D=128, window=500,
             sink=64),
        # a short prompt through small heads (latency)
        dict(name="fwd short d64", op="fwd", R=1, lo=333, hi=333, Hq=12, Hkv=3, D=64, window=100, sink=1),
        # training step of the sliding-window layers
        dict(name="train window d256", op="train", R=2, lo=8192, hi=8192, Hq=32, Hkv=16, D=256, window=1024, sink=4),
        # training step on one long sequence with few KV heads: the sinks' gradient is a sum over all of it
        dict(name="train long d128", op="train", R=1, lo=16000, hi=16000, Hq=8, Hkv=2, D=128, window=700, sink=16),
        # the decode batch through the sliding-window layers, contexts past the window
        dict(name="decode window d256", op="decode", R=64, lo=1024, hi=4096, Hq=32, Hkv=16, D=256, window=1024, sink=4),
        # few long conversations at head_dim 128
        dict(name="decode long d128", op="decode", R=7, lo=3000, hi=30000, Hq=32, Hkv=8, D=128, window=4000, sink=20),
        # one decode step of 64 requests writes its keys and values (latency)
        dict(name="kv4_write step d128", op="kv4_write", T=64, pages=64, Hkv=8, D=128),
        # a chunk of prompts: 8 requests of 1024 new tokens
        dict(name="kv4_write chunk d256", op="kv4_write", T=8192, pages=520, Hkv=16, D=256),
        # the decode batch: 64 requests of 256 to 1024 tokens, all of them visible
        dict(name="kv4_decode batch d128", op="kv4_decode", R=64, lo=256, hi=1024, Hq=32, Hkv=8, D=128, window=0, sink=0),
        # long contexts, what a 4-bit cache is for
        dict(name="kv4_decode long d128", op="kv4_decode", R=12, lo=5000, hi=60000, Hq=32, Hkv=8, D=128, window=0, sink=0),
        # the sliding-window layers over a 4-bit cache
        dict(name="kv4_decode window d256", op="kv4_decode", R=33, lo=100, hi=4096, Hq=32, Hkv=16, D=256, window=1024, sink=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["fwd", "train", "decode", "kv4_write", "kv4_decode", "kv4_decode"])
    Hkv, G = rng.randint(1, 16), rng.randint(1, 8)
    sink = rng.choice([1, 4, 4, 16, _log_int(rng, 1, 128)])
    if op in ("fwd", "train"):
        D = rng.choice([64, 128, 256, 256, 512])
        window = _log_int(rng, 1, 2048)
        # tokens of the largest listed one, at this window
        most = 16384 * 32 * 256 * 1024 // (G * Hkv * D * max(1024, window + sink))
        n = _log_int(rng, 1, 8)
        top = _log_int(rng, 16, max(17, min(16000, most // n)))
        # the plain form holds the whole square of scores: no more of it than the largest listed case
        while n * top * top * G * Hkv > 2 * 8192 * 8192 * 32:
            top = top * 3 // 4
        return dict(op=op, R=n, lo=top if rng.random() < 0.4 else rng.randint(2, top), hi=top, Hq=G * Hkv, Hkv=Hkv, D=D, window=window, sink=sink)
    if op == "kv4_write":
        D = rng.choice([64, 128, 256])
        T = _log_int(rng, 1, min(32768, 8192 * 16 * 256 // (Hkv * D)))
        return dict(op=op, T=T, pages=(T + PAGE - 1) // PAGE + rng.randint(0, 8), Hkv=Hkv, D=D)
    R = _log_int(rng, 1, 64)
    window = rng.choice([100, 500, 1024, 4000])
    if op == "decode":
        D, G = rng.choice([(128, rng.choice([1, 2, 4, 8])), (256, rng.choice([1, 2, 4]))])
        # a context past the window costs no more than the window
        hi = _log_int(rng, 16, min(30000, 64 * 4096 * 16 * 256 // (R * Hkv * D)))
    else:
        D = rng.choice([64, 128, 128, 256])
        if rng.random() < 0.6:
            window, sink = 0, 0
        hi = _log_int(rng, 16, min(60000, 12 * 30000 * 8 * 128 // (R * Hkv * D)))
    return dict(op=op, R=R, lo=rng.randint(1, hi), hi=hi, Hq=G * Hkv, Hkv=Hkv, D=D, window=window, sink=sink)


def _lens(case):
    """Lengths of the sequences or requests: part of the case, not of the seed."""
    r = random.Random("%d %d %d" % (case["R"], case["lo"], case["hi"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["R"])]


# ---------------------------------------------------------------------------------------------
# the 4-bit cache

def _places(D):
    """Where a record holds what: nibble addresses [16, D] of the keys' and the values' codes, and the addresses
    [16, D / 32], in units of 2 bytes, of their scales.

    Codes stand in blocks of 128 dims (64 at D = 64). A key's row of a block is 4 strips (c) of one 4-byte word for
    each of its groups; strip c holds dims 8 c .. 8 c + 7 of every group, the even ones in the word's nibbles 0 to 3, the odd
    ones in nibbles 4 to 7. Values stand token pair by token pair: for every 16 dims (8 at D = 64) the two
    tokens' codes side by side, these chunks exchanged among each other by the pair's number. Key scales are [16][D / 32],
    value scales [D / 32][16].
    """
    W = min(D, 128)  # dims of a block
    t = torch.arange(PAGE)[:, None]
    d = torch.arange(D)[None, :]
    block, e = d // W, d % W
    group, c, i = e // 32, e % 32 // 8, e % 8
    word = c * (W // 32) + group
    key = block * (PAGE * W) + t * W + word * 8 + i // 2 + 4 * (i % 2)
    per = W // 8  # dims of a chunk, for each of 8
    pair, odd, chunk = t // 2, t % 2, e // per
    at = chunk ^ (2 * (pair % 4)) if W == 128 else (pair % 2 * 8 + chunk) ^ (4 * (pair // 2 % 2))
    line = pair * (2 * W) if W == 128 else pair // 2 * (4 * W)
    value = 16 * D + block * (PAGE * W) + line + at * (2 * per) + odd * per + e % per
    g = torch.arange(D // 32)[None, :]
    return key, value, 8 * D + t * (D // 32) + g, 8 * D + D // 2 + g * PAGE + t


def _quantise(x):
    """n in -8 .. 7 and s of every group: s = -(value of largest magnitude) / 8 in 5 significant bits, ties to even (of two
    values that are equal but for their sign the negative one), n = x / s to the nearest whole number, ties to even, at
    most 7. A group whose s would be below 2^-126 is zero; above 31 * 2^118 it stays there; a group with an infinity or a NaN
    is NaN."""
    x = x.float().unflatten(-1, (-1, GROUP))
    hi, lo = x.amax(-1), x.amin(-1)
    a = torch.where(hi > -lo, -hi, -lo) / 8
    m, e = torch.frexp(a)
    s = torch.ldexp(torch.round(m * 32) / 32, e).clamp(-31 * 2.0 ** 118, 31 * 2.0 ** 118)
    s = torch.where(s.abs() < 2.0 ** -126, 0.0, s)
    s = torch.where(x.isfinite().all(-1), s, math.nan)
    n = torch.round(x / s[..., None]).clamp(-8, 7)
    n = torch.where((s == 0)[..., None] | s.isnan()[..., None], 0.0, n)
    return n, s


def _read(records, D):
    """Codes [.., 16, D] (as n) and scales [.., 16, D / 32] of the keys and values of records [.., 18, D]."""
    key, value, ks, vs = (p.to(records.device) for p in _places(D))
    flat = records.flatten(-2)
    nib = torch.stack([flat & 15, flat >> 4], -1).flatten(-2)
    half = flat.view(torch.bfloat16)
    return nib[..., key].float() - 8, half[..., ks].float(), nib[..., value].float() - 8, half[..., vs].float()


def _values(n, s):
    return (n.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _write(records, page, t, k, v):
    """Quantises rows k, v [T, H, D] into the records [P, H, 18, D], row i as token t[i] of page[i]."""
    D, H = k.shape[-1], k.shape[1]
    flat = records.flatten(-2)
    nib = torch.stack([flat & 15, flat >> 4], -1).flatten(-2)
    half = flat.view(torch.int16).clone()
    key, value, ks, vs = (p.to(k.device) for p in _places(D))
    h = torch.arange(H, device=k.device)[None, :, None]
    for x, at, sat in ((k, key, ks), (v, value, vs)):
        n, s = _quantise(x)
        nib[page[:, None, None], h, at[t][:, None, :]] = (n.flatten(-2) + 8).to(torch.uint8)
        half[page[:, None, None], h, sat[t][:, None, :]] = s.to(torch.bfloat16).view(torch.int16)
    codes = nib[..., 0::2] | nib[..., 1::2] << 4
    codes[..., 16 * D:] = half.view(torch.uint8)[..., 16 * D:]
    return codes.view(records.shape)


# ---------------------------------------------------------------------------------------------
# inputs

def _dev():
    return torch.device("cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def prepare(case, seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed))
    bf = lambda *shape: torch.randn(shape, generator=g, device=_dev(), dtype=torch.bfloat16)  # noqa: E731
    s = {"case": case, "scale": 1.0 / math.sqrt(case["D"])}
    {"fwd": _prep_prompt, "train": _prep_prompt, "kv4_write": _prep_write, "decode": _prep_decode,
     "kv4_decode": _prep_decode}[case["op"]](case, s, g, bf)
    return s


def _prep_prompt(case, s, g, bf):
    lens, Hq, Hkv, D = _lens(case), case["Hq"], case["Hkv"], case["D"]
    s["dense"] = case["lo"] == case["hi"]
    lead = (len(lens), lens[0]) if s["dense"] else (sum(lens),)
    s.update(q=bf(*lead, Hq, D), k=bf(*lead, Hkv, D), v=bf(*lead, Hkv, D), top=max(lens))
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu"] = _i32(cu)
    if case["op"] == "train":
        s["do"] = bf(*lead, Hq, D)


def _outliers(x, g):
    """A few dims of a head are larger than the others, as in real keys."""
    return (x * (1 + 4 * (torch.rand(x.shape[-2:], generator=g, device=x.device) < 0.05))).to(torch.bfloat16)


def _prep_write(case, s, g, bf):
    T, P, Hkv, D = case["T"], case["pages"], case["Hkv"], case["D"]
    qkv = bf(T, 4 * Hkv * D)  # as the projection leaves them: slices of one row
    k, v = qkv[:, 2 * Hkv * D: 3 * Hkv * D].view(T, Hkv, D), qkv[:, 3 * Hkv * D:].view(T, Hkv, D)
    k.copy_(_outliers(k, g))
    s.update(k=k, v=v)
    # a pool of pages, of which this step's requests hold some; the tokens' slots anywhere in those
    s["cache"] = torch.randint(0, 128, (P + 32, Hkv, 18, D), generator=g, device=_dev(), dtype=torch.uint8)
    s["cache"][:, :, 16:] = 0  # scale zero: nothing written yet
    s["pages"] = torch.randperm(P + 32, generator=g, device=_dev())[:P].to(torch.int32).contiguous()
    at = torch.randperm(P * PAGE, generator=g, device=_dev())[:T]
    s["slots"] = (s["pages"][at // PAGE] * PAGE + at % PAGE).to(torch.int32).contiguous()


def _prep_decode(case, s, g, bf):
    R, Hq, Hkv, D = case["R"], case["Hq"], case["Hkv"], case["D"]
    L = _lens(case)
    npg = [(a + PAGE - 1) // PAGE for a in L]
    pages = sum(npg) + 16
    s["q"] = bf(R, Hq, D)
    if case["op"] == "decode":
        s.update(kc=bf(pages, PAGE, Hkv, D), vc=bf(pages, PAGE, Hkv, D))
    else:
        page = torch.arange(PAGE, device=_dev()).repeat(256)
        at = torch.arange(256, device=_dev()).repeat_interleave(PAGE)
        parts = []
        for first in range(0, pages, 256):  # some pages at a time: the cache is much smaller than what it is made of
            k, v = _outliers(bf(256 * PAGE, Hkv, D), g), bf(256 * PAGE, Hkv, D)
            empty = torch.zeros(256, Hkv, 18, D, dtype=torch.uint8, device=_dev())
            parts.append(_write(empty, at, page, k, v)[: pages - first])
        s["cache"] = torch.cat(parts)
    perm = torch.randperm(pages, generator=g, device=_dev()).to(torch.int32)
    held = _i32(npg)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(max(npg), device=_dev())
    at = (first[:, None] + col[None, :]).clamp(max=pages - 1)
    s["table"] = torch.where(col[None, :] < held[:, None], perm[at.long()], torch.full_like(at, -1, dtype=torch.int32)).to(torch.int32).contiguous()
    s["lens"] = _i32(L)
    s["most"] = max(L)


# ---------------------------------------------------------------------------------------------
# one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"fwd": _plain_fwd, "train": _plain_train, "kv4_write": _plain_write, "decode": _plain_decode, "kv4_decode": _plain_decode}[op](s)


def _own(op, s):
    import attention_flash_gqa_gb300 as attn

    c = s["case"]
    if op in ("fwd", "train"):
        how = dict(window=c["window"], sink=c["sink"], scale=s["scale"])
        if s["dense"]:
            o, lse = attn.attn_fwd(s["q"], s["k"], s["v"], **how)
        else:
            o, lse = attn.attn_fwd_varlen(s["q"], s["k"], s["v"], s["cu"], s["top"], **how)
        if op == "fwd":
            return o, lse
        packed = {} if s["dense"] else dict(cu_seqlens=s["cu"], max_seqlen=s["top"])
        return [o, lse, *attn.attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], **how, **packed)]
    if op == "decode":
        return attn.attn_decode_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=s["scale"], window=c["window"], sink=c["sink"])
    if op == "kv4_write":
        attn.attn_kv4_append(s["k"], s["v"], s["slots"], s["cache"])
        return attn.attn_kv4_unpack(s["cache"], s["pages"])
    return attn.attn_decode_kv4(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"], window=c["window"], sink=c["sink"])


def _padded(x, s):
    """Rows of every sequence, [n, top, ..] with zeros behind the shorter ones, and where a row is one."""
    i = torch.arange(s["top"], device=x.device)
    cu = s["cu"].long()
    there = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    row = (cu[:-1, None] + i[None, :]).clamp(max=x.numel() // (x.shape[-2] * x.shape[-1]) - 1)
    x = x.view(-1, *x.shape[-2:])[row].float()
    return torch.where(there[:, :, None, None], x, 0), there


def _scores(s):
    """Probabilities [n, Hkv, G, top, top], their log-sum-exp, and q, k, v by KV head."""
    c = s["case"]
    (q, there), (k, _), (v, _) = (_padded(s[x], s) for x in ("q", "k", "v"))
    n, top, Hkv, D = k.shape
    q = q.view(n, top, Hkv, -1, D).permute(0, 2, 3, 1, 4)
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    i = torch.arange(top, device=q.device)
    gap = i[:, None] - i[None, :]
    hidden = (gap < 0) | ((gap >= c["window"]) & (i[None, :] >= c["sink"]))
    x = torch.matmul((q * s["scale"]).reshape(n, Hkv, -1, D), k.transpose(-1, -2)).view(n, Hkv, -1, top, top)
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return p.div_(l), (m + l.log()).squeeze(-1), q, k, v, there


def _rows(x, there, s):
    """[n, top, H, D] back to the caller's layout, rounded."""
    x = x.to(torch.bfloat16)
    return x if s["dense"] else x[there]


def _result(p, lse, v, there, s):
    n, Hkv, G, top, _ = p.shape
    o = torch.matmul(p.view(n, Hkv, G * top, top), v).view(n, Hkv, G, top, -1)
    lse = lse.reshape(n, Hkv * G, top)
    out = _rows(o.permute(0, 3, 1, 2, 4).reshape(n, top, Hkv * G, -1), there, s)
    return o, out, lse if s["dense"] else lse.permute(0, 2, 1)[there].t().contiguous()


def _plain_fwd(s):
    p, lse, _, _, v, there = _scores(s)
    return _result(p, lse, v, there, s)[1:]


def _plain_train(s):
    p, lse, q, k, v, there = _scores(s)
    o, out, lse = _result(p, lse, v, there, s)
    n, Hkv, G, top, D = q.shape
    do, _ = _padded(s["do"], s)
    do = do.view(n, top, Hkv, G, D).permute(0, 2, 3, 1, 4)
    flat = lambda x: x.reshape(n, Hkv, G * top, -1)  # noqa: E731
    dv = torch.matmul(flat(p).transpose(-1, -2), flat(do))
    ds = torch.matmul(flat(do), v.transpose(-1, -2)).view_as(p)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(flat(ds), k).view_as(q) * s["scale"]
    dk = torch.matmul(flat(ds).transpose(-1, -2), flat(q)) * s["scale"]
    back = lambda x: _rows(x.permute(0, 2, 1, 3), there, s)  # noqa: E731
    return [out, lse, _rows(dq.permute(0, 3, 1, 2, 4).reshape(n, top, Hkv * G, D), there, s), back(dk), back(dv)]


def _plain_write(s):
    D = s["case"]["D"]
    slot = s["slots"].long()
    s["cache"].copy_(_write(s["cache"], slot // PAGE, slot % PAGE, s["k"], s["v"]))
    kn, ks, vn, vs = _read(s["cache"][s["pages"].long()], D)
    back = lambda x: x.to(torch.bfloat16).transpose(1, 2).contiguous()  # noqa: E731  ([pages, 16, Hkv, D])
    return back(_values(kn, ks)), back(_values(vn, vs))


def _plain_decode(s):
    c = s["case"]
    q, table, L = s["q"], s["table"], s["lens"].long()
    R, Hq, D = q.shape
    Hkv, W = c["Hkv"], c["window"]
    # visible keys of a request, in order: its sinks that the window does not reach, then the window
    first = (L - W).clamp(min=0) if W else torch.zeros_like(L)
    early = first.clamp(max=c["sink"])
    i = torch.arange(min(s["most"], W + c["sink"]) if W else s["most"], device=q.device)
    key = torch.where(i[None, :] < early[:, None], i[None, :], i[None, :] + (first - early)[:, None])
    there = key < L[:, None]
    key = torch.where(there, key, 0)
    slot = table.gather(1, key // PAGE).long() * PAGE + key % PAGE
    if c["op"] == "decode":
        k, v = (x.view(-1, Hkv, D)[slot].float() for x in (s["kc"], s["vc"]))
    else:
        pages, at = torch.unique(slot // PAGE, return_inverse=True)
        kn, ks, vn, vs = _read(s["cache"][pages], D)  # [pages, Hkv, 16, D]
        k, v = (x.transpose(1, 2)[at, slot % PAGE] for x in (_values(kn, ks), _values(vn, vs)))
    v = torch.where(there[:, :, None, None], v, 0)
    x = torch.matmul((q.float() * s["scale"]).view(R, Hkv, -1, D), k.permute(0, 2, 3, 1))
    x = x.masked_fill_(~there[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / l
    return o.view(R, Hq, D).to(torch.bfloat16), (l.log() + m).view(R, Hq)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "kv4_write":
        return _exact_write(case, s)
    if case["op"] in ("decode", "kv4_decode"):
        return _exact_decode(case, s)
    return _exact_prompt(case, s)


def _exact_prompt(case, s):
    """Block of queries by block of queries, over the keys that they can see: the sinks and one stretch."""
    Hq, Hkv, D, W, sink = case["Hq"], case["Hkv"], case["D"], case["window"], case["sink"]
    G, scale, train = Hq // Hkv, s["scale"], case["op"] == "train"
    flat = {x: s[x].view(-1, *s[x].shape[-2:]) for x in ("q", "k", "v", "do") if x in s}
    T = flat["q"].shape[0]
    z = lambda like: torch.zeros(like.shape, dtype=torch.float64, device=like.device)  # noqa: E731
    o, lse = z(flat["q"]), torch.zeros(Hq, T, dtype=torch.float64, device=_dev())
    dq, dk, dv = z(flat["q"]), z(flat["k"]), z(flat["v"])
    cu = s["cu"].tolist()
    for a, b in zip(cu, cu[1:]):
        for q0 in range(a, b, 1024):
            q1 = min(b, q0 + 1024)
            lo = max(a, q0 - W + 1)
            keys = torch.cat([torch.arange(a, min(a + sink, lo), device=_dev()), torch.arange(lo, q1, device=_dev())])
            rows = torch.arange(q0, q1, device=_dev())
            far = rows[:, None] - keys[None, :]
            see = (far >= 0) & ((far < W) | (keys[None, :] < a + sink))
            q = flat["q"][q0:q1].double().view(-1, Hkv, G, D)
            k, v = flat["k"][keys].double(), flat["v"][keys].double()
            x = torch.einsum("qhgd,khd->hgqk", q, k).mul_(scale).masked_fill_(~see, -math.inf)
            e = torch.logsumexp(x, -1)
            p = x.sub_(e[..., None]).exp_()
            out = torch.einsum("hgqk,khd->qhgd", p, v)
            o[q0:q1] = out.reshape(-1, Hq, D)
            lse[:, q0:q1] = e.reshape(Hq, -1)
            if train:
                do = flat["do"][q0:q1].double().view(-1, Hkv, G, D)
                dv.index_add_(0, keys, torch.einsum("hgqk,qhgd->khd", p, do))
                ds = torch.einsum("qhgd,khd->hgqk", do, v)
                ds = (ds - (do * out).sum(-1).permute(1, 2, 0)[..., None]) * p * scale
                dq[q0:q1] = torch.einsum("hgqk,khd->qhgd", ds, k).reshape(-1, Hq, D)
                dk.index_add_(0, keys, torch.einsum("hgqk,qhgd->khd", ds, q))
    if s["dense"]:
        lse = lse.view(Hq, case["R"], -1).transpose(0, 1).contiguous()
    shaped = lambda x, like: x.view(like.shape)  # noqa: E731
    if not train:
        return shaped(o, s["q"]), lse
    return [shaped(o, s["q"]), lse, shaped(dq, s["q"]), shaped(dk, s["k"]), shaped(dv, s["v"])]


def _exact_write(case, s):
    """Every page's values from its tokens: zero where none was written (the scales there are zero)."""
    D, Hkv = case["D"], case["Hkv"]
    at = torch.full((s["cache"].shape[0],), -1, dtype=torch.long, device=_dev())
    at[s["pages"].long()] = torch.arange(case["pages"], device=_dev())
    slot = s["slots"].long()
    outs = []
    for x in (s["k"], s["v"]):
        x = x.double().reshape(-1, Hkv, D // 32, 32)
        big = torch.where(x.amax(-1) > -x.amin(-1), x.amax(-1), x.amin(-1))  # of largest magnitude, negative if in doubt
        step = -big / 8
        unit = torch.exp2(torch.floor(torch.log2(step.abs().clamp(min=1e-300))) - 4)  # the last of 5 bits
        step = torch.round(step / unit) * unit
        n = torch.where(step[..., None] != 0, torch.round(x / step[..., None]), 0).clamp(-8, 7)
        y = torch.zeros(case["pages"], PAGE, Hkv, D, dtype=torch.float64, device=_dev())
        y[at[slot // PAGE], slot % PAGE] = (n * step[..., None]).view(-1, Hkv, D)
        outs.append(y)
    return tuple(outs)


def _exact_decode(case, s):
    R, Hq, Hkv, D, W = case["R"], case["Hq"], case["Hkv"], case["D"], case["window"]
    out, lses = [], []
    if case["op"] == "kv4_decode":
        key, value, ks, vs = (p.to(_dev()) for p in _places(D))
    for b, L in enumerate(_lens(case)):
        used = s["table"][b, : (L + PAGE - 1) // PAGE].long()
        j = torch.arange(L, device=_dev())
        if W:
            j = j[(j >= L - W) | (j < case["sink"])]
        if case["op"] == "decode":
            k, v = (x[used[j // PAGE], j % PAGE].double() for x in (s["kc"], s["vc"]))
        else:
            rec = s["cache"][used].flatten(-2)  # [pages, Hkv, 18 D]

            def get(codes, scales):
                byte = rec[..., codes // 2]  # [pages, Hkv, 16, D]
                n = torch.where((codes % 2 == 1), byte >> 4, byte & 15).double() - 8
                half = rec.view(torch.bfloat16)[..., scales].double()
                return (n * half.repeat_interleave(32, -1)).permute(0, 2, 1, 3)[j // PAGE, j % PAGE]

            k, v = get(key, ks), get(value, vs)
        q = s["q"][b].double().view(Hkv, -1, D)
        x = torch.einsum("hgd,khd->hgk", q, k) * s["scale"]
        e = torch.logsumexp(x, -1)
        out.append(torch.einsum("hgk,khd->hgd", (x - e[..., None]).exp(), v).reshape(Hq, D))
        lses.append(e.reshape(Hq))
    return torch.stack(out), torch.stack(lses)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def _pairs(n, W, sink):
    """Visible (query, key) pairs of a sequence of n."""
    near = n * (n + 1) // 2 if n <= W else W * (W + 1) // 2 + (n - W) * W
    far = max(0, n - W)  # query W + m (m < far) is past keys 0 .. m
    return near + (far * (far + 1) // 2 if far <= sink else sink * (sink + 1) // 2 + (far - sink) * sink)


def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    if op == "kv4_write":
        T, P = case["T"], case["pages"]
        # rows in, their records out; the pages' records in, their values out
        return {"bytes": T * Hkv * D * 4 + T * Hkv * D * 18 // 16 + 4 * T + P * Hkv * 18 * D + P * PAGE * Hkv * D * 4 + 4 * P, "flops": 0}
    Hq = case["Hq"]
    if op in ("fwd", "train"):
        T, pairs = sum(_lens(case)), sum(_pairs(n, case["window"], case["sink"]) for n in _lens(case))
        fwd = T * (2 * Hq + 2 * Hkv) * D * 2 + T * Hq * 4
        if op == "fwd":
            return {"bytes": fwd, "flops": 4 * D * Hq * pairs}
        return {"bytes": fwd + T * (2 * Hq + 2 * Hkv) * D * 2, "flops": 14 * D * Hq * pairs}
    L, W = _lens(case), case["window"]
    keys = sum(min(x, W + case["sink"]) if W else x for x in L)
    per = 4 * D if op == "decode" else 18 * D // 16  # bytes of a token's key and value in one head
    return {"bytes": keys * Hkv * per + case["R"] * Hq * (4 * D + 4) + 4 * (keys // PAGE + case["R"]), "flops": 4 * D * Hq * keys}
