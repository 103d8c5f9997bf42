"""Plain forms in 64 bits of attention within segments, dropout and the loss of a
linear classifier, with bounds on what rounding may do to the kernels' results.

u = 2^-24 is half a step of fp32.  A sum of n products on the matrix cores is
taken to be off by at most 2 n u of the magnitudes that it adds (they may truncate
where they add), an exponential or a quotient by 4 u.  `half` is half a step of
the rows' type where it has 16 bits (a probability, or the gradient of a score or
logit, is rounded to it once), else 0; `tiny` is half its smallest subnormal, what
that rounding may be off by at least.  Every bound is of first order; the callers
multiply by a slack of 1.02.
"""
import numpy as np
import torch

U = 2.0 ** -24


def steps(dtype):
    f = torch.finfo(dtype)
    if dtype == torch.float32:
        return 0.0, 0.0
    return f.eps / 2, f.smallest_normal * f.eps / 2


def attention(q, k, v, rows, keys, causal, scale, dout=None):
    """(value, bound) of out and, with dout, of dq, dk and dv; rows and keys: the
    bounds of the segments, as lists.  All on the CPU."""
    half, tiny = steps(q.dtype)
    R, H, D = q.shape
    G = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, oute = torch.zeros_like(q), torch.zeros_like(q)
    grads = [torch.zeros_like(t) for t in (q, q, k, k, v, v)]
    dq, dqe, dk, dke, dv, dve = grads
    for a, b, c, d in zip(rows, rows[1:], keys, keys[1:]):
        n, m = b - a, d - c
        if n <= 0 or m <= 0:
            continue
        seen = torch.ones(n, m, dtype=torch.bool)
        if causal:
            seen = torch.arange(m)[None, :] <= torch.arange(n)[:, None] + (m - n)
        for h in range(H):
            x, y, z = q[a:b, h], k[c:d, h // G], v[c:d, h // G]
            s = scale * (x @ y.T)
            # the score's error, and its exponent's: the products, the scale's
            # rounding and the sum with the running maximum
            mag = scale * (x.abs() @ y.abs().T)
            top = torch.where(seen, s, torch.full_like(s, -np.inf)).amax(1, keepdim=True)
            top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
            e = torch.where(seen, torch.exp(s - top), torch.zeros_like(s))
            total = e.sum(1, keepdim=True)
            p = e / torch.where(total == 0, torch.ones_like(total), total)
            eps = 2 * D * U * mag + 8 * U * (mag + top.abs()) + 8 * U
            # a normalised weight: its own exponent's error, the mean one of the
            # sum, and the sum's n additions
            rel = eps + (p * eps).sum(1, keepdim=True) + 2 * m * U + 8 * U
            az = z.abs()
            out[a:b, h] = p @ z
            ferr = (p * (rel + half + 2 * m * U)) @ az + tiny * (seen.double() @ az)
            oute[a:b, h] = ferr
            if dout is None:
                continue
            g = dout[a:b, h].double()
            ag = g.abs()
            dv[c:d, h // G] += p.T @ g
            dve[c:d, h // G] += (p * (rel + half + 2 * (n * G) * U)).T @ ag + tiny * (seen.double().T @ ag)
            dp = g @ z.T
            dpe = 2 * D * U * (ag @ az.T)
            delta = (g * out[a:b, h]).sum(1, keepdim=True)
            # out's error before its rounding, what the kept rest of that rounding
            # leaves, and the sum's
            o = out[a:b, h].abs()
            deltae = (ag * (ferr + (half * half + 2 * D * U) * (o + ferr) + tiny)).sum(1, keepdim=True)
            ds = p * (dp - delta)
            dse = p * (rel * (dp - delta).abs() + dpe + deltae + 2 * U * (dp.abs() + delta.abs())) + half * ds.abs() + \
                tiny * seen.double()
            dq[a:b, h] = scale * (ds @ y)
            dqe[a:b, h] = scale * ((dse + 2 * m * U * ds.abs()) @ y.abs())
            dk[c:d, h // G] += scale * (ds.T @ x)
            dke[c:d, h // G] += scale * ((dse + 2 * (n * G) * U * ds.abs()).T @ x.abs())
    if dout is None:
        return [(out, oute)]
    return [(out, oute), (dq, dqe), (dk, dke), (dv, dve)]


MASK = (1 << 32) - 1


def words(n, seed, offset):
    """Philox 4x32 with 10 rounds (Salmon et al. 2011): 32 random bits for each of n elements."""
    c = np.zeros(((n + 3) // 4, 4), dtype=np.uint64)
    group = np.arange(c.shape[0], dtype=np.uint64)
    c[:, 0], c[:, 1] = group & np.uint64(MASK), group >> np.uint64(32)
    c[:, 2], c[:, 3] = offset & MASK, offset >> 32 & MASK
    return philox(c, seed & MASK, seed >> 32 & MASK).reshape(-1)[:n]


def philox(c, k0, k1):
    """Ten rounds over counters c [n, 4] of 32-bit words."""
    for _ in range(10):
        p0, p1 = c[:, 0] * np.uint64(0xD2511F53), c[:, 2] * np.uint64(0xCD9E8D57)
        c = np.stack([(p1 >> np.uint64(32)) ^ c[:, 1] ^ np.uint64(k0), p1 & np.uint64(MASK),
                      (p0 >> np.uint64(32)) ^ c[:, 3] ^ np.uint64(k1), p0 & np.uint64(MASK)], 1)
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    return c


def kept(n, p, seed, offset):
    return torch.from_numpy(words(n, seed, offset) >= np.uint64(round(p * 2 ** 32)))


def loss(x, w, target, reduction, dloss=None):
    """(value, bound) of the loss and, with dloss, of dx and dw.  All on the CPU."""
    half, tiny = steps(x.dtype)
    if x.dtype == torch.float16:
        tiny /= 4096                                   # the logits' gradient is held times 2^12
    x, w = x.double(), w.double()
    (R, I), V = x.shape, w.shape[0]
    live = (target >= 0) & (target < V)
    at = torch.nonzero(live)[:, 0]
    xs, t = x[at], target[at]
    count = max(1, at.numel())
    logits = xs @ w.T
    mag = xs.abs() @ w.abs().T
    le = 2 * I * U * mag
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    one = torch.zeros_like(p)
    one[torch.arange(at.numel()), t] = 1.0
    own = (logits * one).sum(1)
    top = logits.amax(1) if at.numel() else lse
    # the exponents' errors, and a sum of up to 32 + 4 + V / 64 terms in a row
    rel = le + 8 * U * (logits - top[:, None]).abs() + 8 * U
    mean = (p * rel).sum(1) + 2 * (40 + V / 64) * U
    rows = lse - own
    rowse = mean + (le * one).sum(1) + 4 * U * ((top - own).abs() + (lse - top).abs() + rows.abs()) + \
        (le.gather(1, logits.argmax(1, keepdim=True))[:, 0] if at.numel() else 0)
    value, bound = torch.zeros(R, dtype=torch.float64), torch.zeros(R, dtype=torch.float64)
    value[at], bound[at] = rows, rowse
    if reduction != "none":
        by = count if reduction == "mean" else 1
        value, bound = value.sum() / by, (bound.sum() + 2 * (64 + R / 1024) * U * value.abs().sum()) / by
    if dloss is None:
        return [(value, bound)]
    g = dloss.double()[at] if reduction == "none" else dloss.double() / (count if reduction == "mean" else 1)
    unit = 2.0 ** float(torch.ceil(torch.log2(g.abs().max()))) * 2 if reduction == "none" and at.numel() else 1.0
    g = g[:, None] if reduction == "none" else g
    scale = unit if reduction == "none" else g.abs()
    d = (p - one) * g
    de = p * (rel + mean[:, None]) * g.abs() + half * d.abs() + 4 * U * (p + one) * g.abs() + tiny * scale
    dx, dxe = torch.zeros_like(x), torch.zeros_like(x)
    dx[at] = d @ w
    dxe[at] = (de + 2 * (V + 8) * U * d.abs()) @ w.abs()
    dw, dwe = d.T @ xs, (de + 2 * (R + 8) * U * d.abs()).T @ xs.abs()
    return [(value, bound), (dx, dxe), (dw, dwe)]
