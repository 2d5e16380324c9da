"""The 4-bit cache in plain code: the rounding of a group from its definition, the record's layout element by element, and decode
over it in 64 bits with the error bound that the GPU tests use (U = 2^-24: one fp32 rounding, BF = 2^-8: one to bf16)."""
import math

import torch

from operator_ref import BF, U


def quantise(x):
    """n (whole numbers) and s of x [.., D] in 64 bits; NaN as s where the group holds an infinity or a NaN."""
    x = x.double().unflatten(-1, (-1, 32))
    at = x.abs().nan_to_num(0, 0).amax(-1, keepdim=True)
    neg = (x == -at).any(-1)  # of two values that are equal but for their sign the negative one counts
    a = torch.where(neg, -at[..., 0], at[..., 0])
    s = -a / 8
    mant, exp = torch.frexp(s)
    s = torch.ldexp(torch.round(mant * 32) / 32, exp)
    s = torch.where(s.abs() < 2.0 ** -126, 0.0, s.clamp(-31 * 2.0 ** 118, 31 * 2.0 ** 118))
    n = torch.where(s[..., None] == 0, 0.0, torch.round(x / s[..., None]).clamp(-8, 7))
    bad = ~x.isfinite().all(-1)
    return torch.where(bad[..., None], 0.0, n).flatten(-2), torch.where(bad, math.nan, s)


def values(x):
    n, s = quantise(x)
    return n * s.repeat_interleave(32, -1)


def places(D):
    """key[t][d], value[t][d]: nibble of the record that holds the code; sk[t][g], sv[t][g]: byte of the scale."""
    W = min(D, 128)
    key, value = ([[0] * D for _ in range(16)] for _ in range(2))
    for t in range(16):
        for d in range(D):
            block, e = divmod(d, W)
            group, r = divmod(e, 32)
            strip, i = divmod(r, 8)
            word = block * 8 * W + t * W // 2 + (strip * (W // 32) + group) * 4  # byte
            key[t][d] = 2 * word + (i // 2 if i % 2 == 0 else 4 + i // 2)
            chunk, i = divmod(e, W // 8)
            pair = t // 2
            if W == 128:
                byte = 8 * D + block * 8 * W + pair * 128 + (chunk ^ (2 * (pair % 4))) * 16 + (t % 2) * 8
            else:
                byte = 8 * D + (pair // 2) * 128 + (((pair % 2) * 8 + chunk) ^ (4 * (pair // 2 % 2))) * 8 + (t % 2) * 4
            value[t][d] = 2 * byte + i
    sk = [[16 * D + 2 * (t * (D // 32) + g) for g in range(D // 32)] for t in range(16)]
    sv = [[17 * D + 2 * (g * 16 + t) for g in range(D // 32)] for t in range(16)]
    return tuple(torch.tensor(x) for x in (key, value, sk, sv))


def put(cache, slots, k, v):
    """Rows into a cache [pages, Hkv, 18, D] (CPU), slot by slot; -1 and slots outside it are left out."""
    P, H, _, D = cache.shape
    key, value, sk, sv = places(D)
    flat = cache.view(P, H, 18 * D)
    nib = torch.stack([flat & 15, flat >> 4], -1).view(P, H, 36 * D)
    slots = torch.as_tensor(slots)
    live = (slots >= 0) & (slots < 16 * P)
    page, t = slots[live] // 16, slots[live] % 16
    h = torch.arange(H)[None, :, None]
    for x, at in ((k, key), (v, value)):
        n, _ = quantise(x[live])
        nib[page[:, None, None], h, at[t][:, None, :]] = (n + 8).to(torch.uint8)
    flat[:] = nib[..., 0::2] | nib[..., 1::2] << 4
    half = flat.view(torch.int16)
    for x, at in ((k, sk), (v, sv)):
        _, s = quantise(x[live])
        half[page[:, None, None], h, at[t][:, None, :] // 2] = s.to(torch.bfloat16).view(torch.int16)
    return cache


def get(cache):
    """(K, V) [pages, 16, Hkv, D] in 64 bits."""
    P, H, _, D = cache.shape
    flat = cache.view(P, H, 18 * D)
    nib = torch.stack([flat & 15, flat >> 4], -1).view(P, H, 36 * D)
    half = flat.view(torch.bfloat16)
    key, value, sk, sv = places(D)
    out = []
    for at, s in ((key, sk), (value, sv)):
        x = (nib[..., at].double() - 8) * half[..., s // 2].double().repeat_interleave(32, -1)
        out.append(x.transpose(1, 2))
    return out


def decode(q, cache, table, lens, scale, window=0, sink=0):
    """(o, tolerance, lse, tolerance), o [B, Hq, D].

    Scores: in a group of 32 dims products q (16 + code) start from -24 sum q, so that no partial sum is above 55 sum|q|; 34 additions,
    each of which may truncate, are off by 68 U of that, times |s|; the groups' sum by (D / 32 + 2) 2 U sum|q k|. With
    the exponential's 2^-21 that bounds the relative error e of p. P rounds to bf16, V is exact, the sum of up to L terms takes 2 L U,
    the result rounds to bf16. lse: e, L U, the logarithm.
    The exponential is zero below 2^-126 (a subnormal result is flushed). It is taken relative to a running maximum that the row's
    largest score is never more than 2^8 below (the maximum only moves to scores that are there, and each piece is scaled to the
    largest of them), so the sum of the p is at least 2^-8 and a weight is off by 2^-118 at most, o by 2^-118 sum|v|. A result
    below 2^-126 rounds to a multiple of 2^-133. V enters the product times 2^-down, where a bf16 number below 2^-126 is a multiple of
    2^-133: a value of V is off by 2^(down - 134) at most, and only if it is below 2^(down - 126). down is 6 or, with e the exponent of
    the largest scale (2^e or more), at most e + 127 - 121 + 8 = e + 14 (bf16 holds e + 127): 2^-128, or 2^-120 of that scale.
    """
    B, Hq, D = q.shape
    Hkv = cache.shape[1]
    G = Hq // Hkv
    K, V = get(cache)
    step = cache.view(*cache.shape[:2], 18 * D).view(torch.bfloat16)[..., places(D)[2] // 2].double().abs().transpose(1, 2)
    o, lse = torch.zeros(B, Hq, D, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        L = int(lens[b])
        j = torch.arange(L)
        if window:
            j = j[(j >= L - window) | (j < sink)]
        if L == 0:
            continue
        page = table[b].long()[j // 16]
        k, v, st = (x[page, j % 16].transpose(0, 1).repeat_interleave(G, 0) for x in (K, V, step))  # [Hq, n, ..]
        x = q[b].double()
        s = torch.einsum("hd,hnd->hn", x, k) * scale
        a = torch.einsum("hg,hng->hn", x.abs().unflatten(1, (-1, 32)).sum(2), st)
        e = (scale * (68 * 55 * U * a + (D // 32 + 2) * 2 * U * torch.einsum("hd,hnd->hn", x.abs(), k.abs())) + 4 * U * s.abs() + 2.0 ** -21).amax(1)
        y = torch.logsumexp(s, 1)
        p = (s - y[:, None]).exp()
        o[b], lse[b] = torch.einsum("hn,hnd->hd", p, v), y
        to[b] = (BF + 2 * e + 2 * L * U)[:, None] * torch.einsum("hn,hnd->hd", p, v.abs()) + BF * o[b].abs() + 2.0 ** -118 * v.abs().sum(1) + 2.0 ** -134 + 2.0 ** -128 + 2.0 ** -120 * v.abs().amax()
        tl[b] = e + L * U + 2.0 ** -21 * (1 + y.abs())
    return o, to, lse, tl
