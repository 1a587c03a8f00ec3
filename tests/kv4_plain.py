"""Plain binary64 forms of the 4-bit cache and of attention over it, and the
error bounds its tests hold the kernels to (torch, any device, no library code)."""
import math

import torch

from w4_plain import F64, U32, half_step, tiny

PARAM = torch.float16


def quantize(x, group):
    """(codes int32 [.., D], params fp16 [.., D / group, 2]) in binary32, as the definition says."""
    f = x.float()
    bad = ~torch.isfinite(f).unflatten(-1, (-1, group)).all(-1)
    f = torch.nan_to_num(f, nan=0.0, posinf=0.0, neginf=0.0).clamp(-65504, 65504).unflatten(-1, (-1, group))
    lo, hi = f.amin(-1), f.amax(-1)
    step, off = ((hi - lo) / 15).to(PARAM), lo.to(PARAM)
    s = step.float()[..., None]
    c = torch.where(s > 0, ((f - off.float()[..., None]) / s).round().clamp(0, 15), torch.zeros_like(f))
    off = torch.where(bad, torch.full_like(off, math.nan), off)
    step = torch.where(bad, torch.zeros_like(step), step)
    c = torch.where(bad[..., None], torch.zeros_like(c), c)
    return c.flatten(-2).to(torch.int32), torch.stack([step, off], -1)


def words(c):
    sh = torch.arange(0, 32, 4, dtype=torch.int64, device=c.device)
    w = (c.unflatten(-1, (-1, 8)).to(torch.int64) << sh).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def nibbles(w):
    sh = torch.arange(0, 32, 4, dtype=torch.int32, device=w.device)
    return ((w[..., None] >> sh) & 15).flatten(-2)


def k_at(d):
    """Word of a key that holds columns 8 b .., for every b."""
    j = d // 32
    return [(b % 4) * j + b // 4 for b in range(d // 8)]


def store(c_k, p_k, c_v, p_v):
    """The cache's arrays from codes [pages, heads, page, D] and parameters."""
    d = c_k.shape[-1]
    wk, wv = words(c_k), words(c_v)
    kc = torch.empty_like(wk)
    kc[..., k_at(d)] = wk
    pages, h, s, w = wv.shape
    vc = wv.view(pages, h, s // 16, 16, w).transpose(-1, -2).contiguous()
    return kc.contiguous(), vc, p_k.contiguous(), p_v.contiguous()


def read(cache):
    """Values [pages, heads, page, D] of keys and values in binary64."""
    kc, vc, kp, vp = cache
    d = 8 * kc.shape[-1]
    ck = nibbles(kc[..., k_at(d)])
    cv = nibbles(vc.transpose(-1, -2).flatten(2, 3))
    return value(ck, kp), value(cv, vp)


def value(c, p):
    g = c.shape[-1] // p.shape[-2]
    p = p.to(F64)
    return c.to(F64) * p[..., 0].repeat_interleave(g, -1) + p[..., 1].repeat_interleave(g, -1)


def size_of(c, p):
    """What a value's sum runs over in magnitude: codes up to 31 steps above an
    offset that lies 16 steps lower."""
    g = c // p.shape[-2]
    p = p.to(F64).abs()
    return (47 * p[..., 0] + p[..., 1]).repeat_interleave(g, -1)


def attention(q, k, v, size_k, size_v, keys, scale, t):
    """Output and its bound of one query head q [D] over k, v [L, D] of which it
    sees the first `keys`.  All binary64."""
    if keys <= 0:
        z = torch.zeros_like(q)
        return z, z
    k, v, size_k, size_v = k[:keys], v[:keys], size_k[:keys], size_v[:keys]
    d = q.shape[0]
    s = scale * (k @ q)
    # products and sums of up to D + 64 terms, each off by at most a step of
    # binary32; four more roundings of the result and of its product with log2 e
    es = abs(scale) * 2 * (d + 64) * U32 * (size_k @ q.abs()) + 4 * U32 * s.abs()
    top = s.max()
    e = torch.exp(s - top)
    p = e / e.sum()
    # a key's weight: the score's error, the maximum's (common to all, it drops
    # out), the difference's rounding, exp2 within two steps, rescalings within
    # a step for each 32 keys at most
    rel = torch.expm1(es + U32 * ((s - top).abs() + 8)) + (keys / 32 + 8) * 2 * U32
    # numerator and denominator; P step in two bf16 parts (2^-17, and the part's
    # own rounding 2^-18); the sums over keys: 32 in an MFMA, then one by one
    out = p @ v
    n = (keys / 32 + 64) * 2 * U32
    bound = (p * (rel + 2.0 ** -16 + n)) @ size_v + ((p * rel).sum() + n) * (p @ size_v)
    return out, bound + half_step(t) * (out.abs() + bound) + tiny(t)


def attention_all(q, cache, table, lens, starts, scale, t):
    """[tokens, heads, D] outputs and bounds; rows of no sequence are NaN."""
    k, v = read(cache)
    d = q.shape[-1]
    sk, sv = size_of(d, cache[2]), size_of(d, cache[3])
    page, pages, h = k.shape[2], k.shape[0], k.shape[1]
    per = q.shape[1] // h
    out = torch.full(q.shape, math.nan, dtype=F64, device=q.device)
    bound = torch.zeros_like(out)
    for s in range(table.shape[0]):
        n = min(max(int(lens[s]), 0), table.shape[1] * page)
        a, b = (s, s + 1) if starts is None else (int(starts[s]), int(starts[s + 1]))
        at = [(int(table[s, j // page]), j % page) for j in range(n)]
        seen = [0 <= p < pages for p, _ in at]
        pi = torch.tensor([p if ok else 0 for (p, _), ok in zip(at, seen)], dtype=torch.long, device=q.device)
        ui = torch.tensor([u for _, u in at], dtype=torch.long, device=q.device)
        ok = torch.tensor(seen, dtype=torch.bool, device=q.device)
        for t_ in range(a, b):
            see = min(max(n - (b - a) + (t_ - a) + 1, 0), n)
            keep = ok[:see].nonzero()[:, 0]
            for x in range(q.shape[1]):
                g = x // per
                i, j = pi[keep], ui[keep]
                out[t_, x], bound[t_, x] = attention(q[t_, x].to(F64), k[i, g, j], v[i, g, j], sk[i, g, j], sv[i, g, j],
                                                     len(keep), scale, t)
    return out, bound


def make_cache(pages, h, page, d, group, seed, far=0.03):
    """Codes and parameters of random keys, some channels of which stand far from zero, and values (CPU)."""
    g = torch.Generator().manual_seed(seed)
    off = torch.where(torch.rand(h, 1, d, generator=g) < far, 4.0, 0.0)
    ck, pk = quantize((torch.randn(pages, h, page, d, generator=g) + off).half(), group)
    cv, pv = quantize((0.5 * torch.randn(pages, h, page, d, generator=g)).half(), group)
    return store(ck, pk, cv, pv)
