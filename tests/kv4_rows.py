"""The plain binary64 attention of kv4_plain.py for many rows at a time, with the same bound (torch, any device)."""
import math

import torch

import kv4_plain as K
from w4_plain import F64, U32, half_step, tiny


def attention_rows(q, k, v, size_k, size_v, seen, scale, t):
    """Outputs and bounds of queries q [R, D] over k, v [L, D]; row r sees the keys j with seen[r, j]."""
    d = q.shape[1]
    if not k.shape[0]:
        return torch.zeros_like(q), torch.zeros_like(q)
    keys = seen.sum(1, keepdim=True).to(F64)
    s = torch.where(seen, scale * (q @ k.T), -math.inf)
    es = abs(scale) * 2 * (d + 64) * U32 * (q.abs() @ size_k.T) + 4 * U32 * s.abs()
    top = s.amax(1, keepdim=True)
    e = torch.where(seen, torch.exp(s - top), 0.0)
    p = e / e.sum(1, keepdim=True).clamp(min=1)
    rel = torch.expm1(es + U32 * ((s - top).abs() + 8)) + (keys / 32 + 8) * 2 * U32
    prel = torch.where(seen, p * rel, 0.0)
    out = p @ v
    n = (keys / 32 + 64) * 2 * U32
    bound = prel @ size_v + (2.0 ** -16 + n) * (p @ size_v) + (prel.sum(1, keepdim=True) + n) * (p @ size_v)
    bound = bound + half_step(t) * (out.abs() + bound) + tiny(t)
    return out, torch.where(keys > 0, bound, 0.0)


def attention_all(q, cache, table, lens, starts, scale, t):
    """kv4_plain.attention_all, a sequence's rows of a kv head at a time."""
    k, v = K.read(cache)
    sk, sv = K.size_of(q.shape[-1], cache[2]), K.size_of(q.shape[-1], cache[3])
    pages, h, page = k.shape[:3]
    per = q.shape[1] // h
    out = torch.full(q.shape, math.nan, dtype=F64, device=q.device)
    bound = torch.zeros_like(out)
    for s in range(table.shape[0]):
        n = min(max(int(lens[s]), 0), table.shape[1] * page)
        a, b = (s, s + 1) if starts is None else (int(starts[s]), int(starts[s + 1]))
        j = torch.arange(n, device=q.device)
        p = table[s].to(q.device).long()[j // page]
        there = (p >= 0) & (p < pages)
        p, u = torch.where(there, p, 0), j % page
        last = n - (b - a) + torch.arange(b - a, device=q.device)
        seen = ((j[None] <= last[:, None]) & there[None]).repeat_interleave(per, 0)
        for g in range(h):
            x = q[a:b, g * per:(g + 1) * per].to(F64).flatten(0, 1)
            o, e = attention_rows(x, k[p, g, u], v[p, g, u], sk[p, g, u], sv[p, g, u], seen, scale, t)
            out[a:b, g * per:(g + 1) * per] = o.view(b - a, per, o.shape[1])
            bound[a:b, g * per:(g + 1) * per] = e.view(b - a, per, o.shape[1])
    return out, bound
