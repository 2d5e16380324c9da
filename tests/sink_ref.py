"""Plain 64-bit attention with a sliding window and sinks, its gradient, and the error bounds of both, from the
formulas. U = 2^-24 is the largest relative error of one fp32 rounding, BF = 2^-8 that of one rounding to bf16."""
import math

import torch

from operator_ref import BF, U


def visible(n, m, window, sink):
    """[n, m]: which of m keys the last n tokens see."""
    i, j = torch.arange(m - n, m)[:, None], torch.arange(m)[None, :]
    return (j <= i) & ((i - j < window) | (j < sink) if window else torch.ones(1, 1, dtype=torch.bool))


def forward(q, k, v, scale, window, sink):
    """(o, tolerance, lse, tolerance) of q [n, Hq, D], the last n tokens of k, v [m, Hkv, D].

    A score's fp32 sum is off by at most (2 D + 8) U scale sum|q k| (each of the D additions may truncate); with the
    exponential's 2^-21 that bounds the relative error e of every p, P rounds to bf16 for the product with V, and the result
    rounds to bf16. lse: e, the sum of up to m terms (m U), the logarithm.
    """
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    see = visible(n, m, window, sink)
    k, v = (x.double().repeat_interleave(G, 1).transpose(0, 1) for x in (k, v))
    q = q.double().transpose(0, 1)
    s, a = q @ k.transpose(1, 2) * scale, q.abs() @ k.abs().transpose(1, 2) * scale
    e = ((2 * D + 8) * U * a + 4 * U * s.abs() + 2.0 ** -21).masked_fill(~see, 0).amax(2)
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, 2)
    p = torch.where(see, (s - lse[..., None]).exp(), 0.0)
    o = p @ v
    to = (BF + 2 * e + m * U)[..., None] * (p @ v.abs()) + BF * o.abs()
    tl = e + m * U + 2.0 ** -21 * (1 + lse.abs())
    return o.transpose(0, 1), to.transpose(0, 1), lse, tl


def backward(q, k, v, do, scale, window, sink):
    """(dq, tolerance, dk, tolerance, dv, tolerance) for one sequence, o and lse being the forward's own.

    P = exp(s - lse) is off by e (as in the forward) and by lse's error, and rounds to bf16. dP is an fp32 sum over D,
    Delta = sum dO o takes over o's error. dS = P (dP - Delta) rounds to bf16; the three products are fp32 sums
    of n G (dK, dV) or n (dQ) terms, and round to bf16 once more.
    """
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    o, to, lse, tl = forward(q, k, v, scale, window, sink)
    see = visible(n, n, window, sink)
    kk, vv = (x.double().repeat_interleave(G, 1).transpose(0, 1) for x in (k, v))
    qq, dd = q.double().transpose(0, 1), do.double().transpose(0, 1)
    s, a = qq @ kk.transpose(1, 2) * scale, qq.abs() @ kk.abs().transpose(1, 2) * scale
    p = torch.where(see, (s - lse[..., None]).exp(), 0.0)
    ep = (2 * D + 8) * U * a + 4 * U * s.abs() + 2.0 ** -20 + tl[..., None]
    dp = dd @ vv.transpose(1, 2)
    edp = (2 * D + 8) * U * (dd.abs() @ vv.abs().transpose(1, 2))
    oo = o.transpose(0, 1)
    delta = (dd * oo).sum(2, keepdim=True)
    edelta = (dd.abs() * (to.transpose(0, 1) + (2 * D + 8) * U * oo.abs())).sum(2, keepdim=True)
    ds = p * (dp - delta)
    eds = p * ((BF + ep) * (dp - delta).abs() + edp + edelta) + BF * ds.abs()
    eds = eds * (1 + BF)
    acc = 4 * n * U

    def heads(x):  # [Hq, n, D] summed over the groups -> [n, Hkv, D]
        return x.view(Hkv, G, n, D).sum(1).transpose(0, 1)

    dq, tq = ds @ kk * scale, (eds + acc * ds.abs()) @ kk.abs() * scale
    dk, tk = ds.transpose(1, 2) @ qq * scale, (eds + G * acc * ds.abs()).transpose(1, 2) @ qq.abs() * scale
    dv, tv = p.transpose(1, 2) @ dd, ((BF + ep + G * acc) * p).transpose(1, 2) @ dd.abs()
    dq, tq, dk, tk, dv, tv = dq.transpose(0, 1), tq.transpose(0, 1), heads(dk), heads(tk), heads(dv), heads(tv)
    return dq, tq + BF * dq.abs(), dk, tk + BF * dk.abs(), dv, tv + BF * dv.abs()


def packed(fn, lens, *tensors):
    """fn on every sequence's rows of the tensors, the results joined: those of 2 dims (lse) along their last one."""
    outs, at = [], 0
    for n in lens:
        if n:
            outs.append(fn(*(t[at: at + n] for t in tensors)))
        at += n
    return [torch.cat(x, -1 if x[0].dim() == 2 else 0) for x in zip(*outs)]
