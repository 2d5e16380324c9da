"""Plain 64-bit implementations of the step plan, the head norm with rotation (and its gradient) and the
tree attention, written from their formulas, with the error bounds that the GPU tests use.

u = 2^-24 is the largest relative error of one fp32 rounding, 2^-8 that of one rounding to bf16.
"""
import math

import torch

U = 2.0 ** -24
BF = 2.0 ** -8
PAGE = 16


# ---- step plan (python integers) -------------------------------------------------------------

def plan(kv, new, held, free, used, table, T, num_pages):
    """Lists in, dict of lists out; `table` (list of rows) is copied. Also whether anything is reported."""
    R, cap = len(kv), (len(table[0]) if table else 0)
    table = [list(r) for r in table]
    bad = not 0 <= used <= len(free)
    room = len(free) - used if not bad else 0
    n, need = [], []
    for b in range(R):
        ok = kv[b] >= 0 and new[b] >= 0 and 0 <= held[b] <= cap and kv[b] <= held[b] * PAGE and kv[b] + new[b] <= cap * PAGE
        bad |= not ok
        n.append(new[b] if ok else 0)
        need.append(max(0, -(-(kv[b] + new[b]) // PAGE) - held[b]) if ok else 0)
    adm = tok = pg = 0
    for b in range(R):
        if tok + n[b] > T or pg + need[b] > room:
            bad = True
            break
        tok, pg, adm = tok + n[b], pg + need[b], adm + 1
    for b in range(adm, R):
        n[b] = need[b] = 0
    cu, off, positions, slots = [0], 0, [0] * T, [-1] * T
    for b in range(R):
        for i in range(need[b]):
            page = free[used + off + i]
            ok = 0 <= page < num_pages
            bad |= not ok
            table[b][held[b] + i] = page if ok else -1
        off += need[b]
        for i in range(n[b]):
            p = kv[b] + i
            page = table[b][p // PAGE]
            ok = 0 <= page < num_pages
            bad |= not ok
            positions[cu[b] + i], slots[cu[b] + i] = p, (page * PAGE + p % PAGE if ok else -1)
        cu.append(cu[b] + n[b])
    return dict(seq_lens=[a + b for a, b in zip(kv, n)], cu_q=cu, positions=positions, slots=slots,
                pages_held=[a + b for a, b in zip(held, need)], free_used=[used + off], admitted=[adm], table=table, bad=bad)


# ---- head norm with rotation ------------------------------------------------------------------

def table(rows, rot, theta=10000.0):
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pairs(rot, inter):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def turn(x, cs, inter, sign=1.0):
    """Rotation of [T, H, D] by [T, rot] cos | sin, and the magnitude |a cos| + |b sin| of each result."""
    rot = cs.shape[1]
    y, mag = x.clone(), x.abs()
    if rot:
        a, b = _pairs(rot, inter)
        c, s = cs[:, None, : rot // 2], sign * cs[:, None, rot // 2:]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def weight(w, offset, D):
    return torch.ones(D, dtype=torch.float64) if w is None else offset + w.double()


def norm_rope(x, w, cs, eps, offset, inter):
    """(y, tolerance) for x [T, H, D], cs [T, rot].

    The sum of squares is a chain of 16 fused steps and 5 exchanges (21 u, halved by the root), rsqrt 2 ulp,
    the weight's sum, mean, eps and the two products 6 u; the rotation 3 more on |a cos| + |b sin|:
    below 32 u = 2^-19. Then one rounding to bf16.
    """
    x = x.double()
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight(w, offset, x.shape[-1])
    y, mag = turn(n, cs.double(), inter)
    return y, BF * y.abs() + 2.0 ** -19 * (1 + BF) * mag


def norm_rope_bwd(dy, x, w, cs, eps, offset, inter):
    """(dx, tolerance, dw, tolerance).

    dn carries 3 u of |a| + |b|, the product with v 1, the sums 21, r 13, the rest a handful: below 64 u of
    the magnitudes. dw sums T * H terms of 20 u each: at most T * 2 + 128 of them one after the other.
    """
    x, dy = x.double(), dy.double()
    T, H, D = x.shape
    v = weight(w, offset, D)
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xh = x * r
    dn, mag = turn(dy, cs.double(), inter, -1.0)
    g, gmag = dn * v, mag * v.abs()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    tol = BF * dx.abs() + 2.0 ** -18 * r * (gmag + xh.abs() * (gmag * xh.abs()).mean(-1, keepdim=True))
    terms = (mag * xh.abs()).sum((0, 1))
    return dx, tol, (dn * xh).sum((0, 1)), (2 * T + 148) * U * terms + 1e-30


# ---- tree attention ----------------------------------------------------------------------------

def tree(q, kc, vc, table, lens, cu, mask, scale, window=0, positions=None):
    """(o, tolerance, lse, tolerance): q [T, Hq, D], caches [pages, 16, Hkv, D], CPU tensors.

    A score's fp32 sum is off by at most (2 D + 8) u scale sum|q k| (each of the D additions may truncate);
    with the exponential's 2^-21 that bounds the relative error e of every p, P rounds to bf16 (2^-8) for the
    product with V, and the result rounds to bf16. lse: e, the sum of up to L terms (L u), the logarithm.
    """
    T, Hq, D = q.shape
    Hkv = kc.shape[2]
    G = Hq // Hkv
    o, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((Hq, T), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(len(lens)):
        n, L = cu[b + 1] - cu[b], lens[b]
        if n == 0:
            continue
        ids = table[b, : -(-L // PAGE)].long()
        k, v = (c[ids].flatten(0, 1)[:L].double() for c in (kc, vc))
        ctx = L - n
        see = torch.zeros(n, L, dtype=torch.bool)
        for i in range(n):
            r = cu[b] + i
            lo = max(0, max(int(positions[r]), ctx) - window + 1) if window else 0
            see[i, min(lo, ctx): ctx] = True
            for d in range(n):
                see[i, ctx + d] = bool(int(mask[r, d // 32]) >> (d % 32) & 1)
        for h in range(Hq):
            qq = q[cu[b]: cu[b + 1], h].double()
            kk, vv = k[:, h // G], v[:, h // G]
            s = qq @ kk.T * scale
            a = qq.abs() @ kk.abs().T * scale
            e = ((2 * D + 8) * U * a + 4 * U * s.abs() + 2.0 ** -21).masked_fill(~see, 0).amax(1) if L else torch.zeros(n)
            s = s.masked_fill(~see, -math.inf)
            x = torch.logsumexp(s, 1)
            p = torch.where(see, (s - x[:, None]).exp(), 0.0)
            rows = slice(cu[b], cu[b + 1])
            o[rows, h], lse[h, rows] = p @ vv, x
            to[rows, h] = (BF + 2 * e + L * U)[:, None] * (p @ vv.abs()) + BF * o[rows, h].abs()
            tl[h, rows] = e + L * U + 2.0 ** -21 * (1 + torch.where(x.isinf(), 0.0, x.abs()))
    return o, to, lse, tl


def random_tree(n, words, gen):
    """Mask words [n][words] and depths of a random tree: a node's parent is an earlier node or the root."""
    anc, depth = [], []
    for i in range(n):
        p = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
        anc.append((anc[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    sign = lambda x: x - (1 << 32) if x >> 31 else x  # noqa: E731
    return [[sign(m >> 32 * w & 0xFFFFFFFF) for w in range(words)] for m in anc], depth


def close(name, got, ref, tol):
    """Every value within its tolerance; infinities equal."""
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, f"{name}: {tuple(got.shape)} against {tuple(ref.shape)}"
    inf = ref.isinf()
    assert torch.equal(got[inf], ref[inf]), f"{name}: infinities differ"
    assert torch.isfinite(got[~inf]).all(), f"{name}: not finite"
    over = ((got - ref).abs() - tol)[~inf]
    assert over.numel() == 0 or over.max() <= 0, f"{name}: {int((over > 0).sum())} of {over.numel()} values are off, by up to {float(over.max()):.3e} more than allowed"
