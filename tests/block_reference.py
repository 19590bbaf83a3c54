"""float64 references of the operators around the recurrence, written from their formulas.

``decay_attention`` also returns the same sums over absolute values, from which the tests take
element-wise error bounds: a product's operand rounded to a type of half step u changes a result
by at most u times the sum of the absolute values of its terms.
"""
import math

import torch

F32 = 2.0 ** -24  # half a float32 step, relative
HALF = {torch.float32: F32, torch.bfloat16: 2.0 ** -8}


def decay_attention(q, k, v, decay, S0=None, edges=None):
    """(o, final state, |o|, |final state|), token by token; edges: packed offsets as a list."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    q, k = (x.double().repeat_interleave(H // Hk, 2).reshape(B * T, H, K) for x in (q, k))
    v = v.double().reshape(B * T, H, V)
    a = decay.double().expand(B, T, H).reshape(B * T, H)
    spans = [(b * T, (b + 1) * T) for b in range(B)] if edges is None else list(zip(edges, edges[1:]))
    o, oa = torch.zeros(B * T, H, V, dtype=torch.float64), torch.zeros(B * T, H, V, dtype=torch.float64)
    last, lasta = [], []
    for n, (lo, hi) in enumerate(spans):
        S = torch.zeros(H, K, V, dtype=torch.float64) if S0 is None else S0[n].double().clone()
        A = S.abs()
        for t in range(lo, hi):
            g = a[t].exp()[:, None, None]
            kv = k[t][:, :, None] * v[t][:, None, :]
            S = torch.where(g == 0, kv, g * S + kv)
            A = torch.where(g == 0, kv.abs(), g * A + kv.abs())
            o[t] = (q[t][:, :, None] * S).sum(1) / math.sqrt(K)
            oa[t] = (q[t].abs()[:, :, None] * A).sum(1) / math.sqrt(K)
        last.append(S)
        lasta.append(A)
    shape = (B, T, H, V)
    empty = torch.zeros(0, H, K, V, dtype=torch.float64)
    return (o.reshape(shape), torch.stack(last) if last else empty, oa.reshape(shape),
            torch.stack(lasta) if lasta else empty)


def act(z, kind):
    if kind == 0:
        return z
    s = torch.sigmoid(z)
    return s if kind == 1 else z * s


def norm(x, w, eps):
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def gated_norm(x, z, w, eps, kind):
    return norm(x.double(), w, eps) * act(z.double(), kind)


def block_norm(x, r, wp, z, kind, scale, c, wn, eps):
    n = x.double()
    if wp is not None:
        n = norm(n, wp, eps)
    if z is not None:
        n = n * act(z.double(), kind)
    if c is not None:
        n = n * c.double()
    scale = torch.tensor(scale, dtype=torch.float32).double()  # the C ABI carries a float
    h = n * scale + (0 if r is None else r.double())
    return h, h if wn is None else norm(h, wn, eps)


def short_conv(x, w, b, kind, S0, edges=None):
    """(y before the activation, y, final state)."""
    B, T, D = x.shape
    W = w.shape[1]
    spans = [(i * T, (i + 1) * T) for i in range(B)] if edges is None else list(zip(edges, edges[1:]))
    flat = x.double().reshape(B * T, D)
    y, last = torch.zeros_like(flat), []
    for n, (lo, hi) in enumerate(spans):
        hist = torch.zeros(W - 1, D, dtype=torch.float64) if S0 is None else S0[n].double()
        rows = torch.cat([hist, flat[lo:hi]])
        for t in range(hi - lo):
            y[lo + t] = (rows[t:t + W] * w.double().T).sum(0) + (0 if b is None else b.double())
        last.append(rows[rows.shape[0] - (W - 1):])
    y = y.reshape(B, T, D)
    return y, (y if kind == 0 else act(y, kind)), torch.stack(last)
