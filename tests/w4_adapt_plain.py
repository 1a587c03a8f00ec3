"""Plain binary64 forms of the adapters beside a packed product, and their error
bounds (torch, any device, no library code)."""
import torch

from w4_plain import F64, U32, codes, half_step, input_grad, linear, spread, tiny

F16 = torch.float16


def weights(qweight, step, zero):
    """(q - zero) step, exactly: the definition."""
    q = codes(qweight)
    return (q - spread(zero, q.shape[1])) * spread(step, q.shape[1])


def own(ids, count):
    """The tokens of each adapter."""
    return [(ids == a).nonzero()[:, 0] for a in range(count)]


def forward(x, w, a, b, scale, ids):
    x, a, b, scale = x.to(F64), a.to(F64), b.to(F64), scale.to(F64)
    y = x @ w.T
    low = torch.zeros(x.shape[0], a.shape[1], dtype=F64, device=x.device)
    for i, t in enumerate(own(ids, len(scale))):
        low[t] = x[t] @ a[i].T
        y[t] += scale[i] * (low[t] @ b[i].T)
    return y, low


def backward(dy, x, low, w, a, b, scale, ids):
    dy, x, low, a, b, scale = (v.to(F64) for v in (dy, x, low, a, b, scale))
    dx = dy @ w
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i, t in enumerate(own(ids, len(scale))):
        v = scale[i] * (dy[t] @ b[i])
        dx[t] += v @ a[i]
        da[i] = v.T @ x[t]
        db[i] = scale[i] * (dy[t].T @ low[t])
    return dx, da, db


def parts_step(t, nparts):
    """What `nparts` 16-bit parts leave of a value, relative to it: half a step of
    each in turn."""
    return half_step(t) ** nparts


def sum_bound(n):
    """A binary32 sum of n exact products: n + 64 additions, each off by at most a step."""
    return 2 * (n + 64) * U32


def forward_bounds(x, layer, a, b, scale, ids, y_type):
    """(y, bound before the last rounding, low, its bound)."""
    t = x.dtype
    w = weights(*layer)
    _, e = linear(x, w)
    # zeros in two parts: both parts' products run through the same sum
    zs = spread(layer[2], w.shape[1]).abs() * spread(layer[1], w.shape[1]).abs()
    e = e + sum_bound(w.shape[1]) * (x.to(F64).abs() @ (2 * zs).T)
    y, low = forward(x, w, a, b, scale, ids)
    # bf16 rows in fp16: values below 2^-31 of their row's largest off by 2^-39 of it
    if t is torch.bfloat16:
        e = e + 2.0 ** -39 * x.to(F64).abs().amax(1, keepdim=True) * w.abs().sum(1)
    xa, aa, ba = x.to(F64).abs(), a.to(F64).abs(), b.to(F64).abs()
    el = torch.zeros_like(low)
    nparts = 3 if t is torch.bfloat16 and y_type is torch.float32 else 2
    for i, at in enumerate(own(ids, len(scale))):
        s = abs(float(scale[i]))
        el[at] = sum_bound(x.shape[1]) * (xa[at] @ aa[i].T)
        # low's error, the scale's rounding, the parts, fp16's smallest ones, the sum
        part = low[at].abs() * (2 * U32 + parts_step(t, nparts)) + el[at]
        if t is F16:
            part = part + 2.0 ** -39 * low[at].abs().amax(1, keepdim=True)
        e[at] += s * (part @ ba[i].T) + sum_bound(3 * a.shape[1]) * s * (low[at].abs() @ ba[i].T)
    e = e + 2 * U32 * y.abs()
    return y, e, low, el


def backward_bounds(dy, x, low, layer, a, b, scale, ids):
    """((dx, bound before the last rounding), (da, bound), (db, bound)); low as it is given."""
    t = dy.dtype
    w = weights(*layer)
    _, e = input_grad(dy, w, t)
    # q - zero is rounded to 11 bits or a multiple of 2^-15 before the step, the
    # zero first where it is below 2^-5 (2^-16 more)
    q = codes(layer[0]) - spread(layer[2], w.shape[1])
    st = spread(layer[1], w.shape[1]).abs()
    e = e + dy.to(F64).abs() @ ((2.0 ** -11 * q.abs() + 2.0 ** -14) * st)
    if t is torch.bfloat16:
        e = e + 2.0 ** -39 * dy.to(F64).abs().amax(1, keepdim=True) * w.abs().sum(0)
    dx, da, db = backward(dy, x, low, w, a, b, scale, ids)
    ea, eb = torch.zeros_like(da), torch.zeros_like(db)
    dya, xa, aa, ba, la = dy.to(F64).abs(), x.to(F64).abs(), a.to(F64).abs(), b.to(F64).abs(), low.to(F64).abs()
    two = parts_step(t, 2)
    all_ = parts_step(t, 2 if t is F16 else 3)
    far = 2.0 ** -39 if t is F16 else 0.0
    for i, at in enumerate(own(ids, len(scale))):
        if not len(at):
            continue
        s = abs(float(scale[i]))
        v = (s * (dy[at].to(F64) @ b[i].to(F64))).abs()
        ev = s * sum_bound(dy.shape[1]) * (dya[at] @ ba[i]) + 2 * U32 * v
        e[at] += (ev + two * v + far * v.amax(1, keepdim=True)) @ aa[i] + sum_bound(3 * a.shape[1]) * (v @ aa[i])
        n = sum_bound(3 * len(at))
        ea[i] = (ev + all_ * v + far * v.max()).T @ xa[at] + n * (v.T @ xa[at])
        eb[i] = s * (dya[at].T @ (all_ * la[at] + far * la[at].max()) + (n + 2 * U32) * (dya[at].T @ la[at]))
    return (dx, e + 2 * U32 * dx.abs()), (da, ea), (db, eb)


def rounded(y, bound, t):
    return bound + half_step(t) * (y.abs() + bound) + (tiny(t) if t is not torch.float32 else 2.0 ** -149)
