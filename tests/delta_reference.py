"""float64 references of the gated delta rule with a decay for each head and of the norm and rotation of
queries and keys, written from their formulas."""
import math

import torch

F32 = 2.0 ** -24  # half a float32 step, relative
HALF = {torch.float32: F32, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


def gate(g, A_log=None, dt_bias=None):
    """The natural-log decay, float64."""
    if A_log is None:
        return g.double()
    z = g.double() + (0 if dt_bias is None else dt_bias.double())
    return -torch.exp(A_log.double()) * (z.clamp_min(0) + torch.log1p(torch.exp(-z.abs())))


def unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


def delta(q, k, v, a, beta, S0=None, edges=None, q_unit=False, k_unit=False, chunk=64):
    """(o, final state, inter, intra): token by token; edges: packed offsets as a list; a, beta: decay and rate as used.

    inter and intra bound what an output is made of where it is formed in chunks: s |q_t| e^G |S[:, v]| with the
    chunk's incoming state, and s sum_j e^(G_t - G_j) |q_t . k_j| |u_j| with the corrections u of the chunk's tokens."""
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    q, k = (x.double().repeat_interleave(H // Hk, 2).reshape(B * T, H, K) for x in (q, k))
    q, k = unit(q) if q_unit else q, unit(k) if k_unit else k
    v = v.double().reshape(B * T, H, V)
    a, b = a.double().reshape(B * T, H), beta.double().reshape(B * T, H)
    spans = [(i * T, (i + 1) * T) for i in range(B)] if edges is None else list(zip(edges, edges[1:]))
    o, inter, intra = (torch.zeros(B * T, H, V, dtype=torch.float64) for _ in range(3))
    s, last = 1 / math.sqrt(K), []
    for n, (lo, hi) in enumerate(spans):
        S = torch.zeros(H, K, V, dtype=torch.float64) if S0 is None else S0[n].double().clone()
        for t in range(lo, hi):
            if (t - lo) % chunk == 0:
                start, us = S.norm(dim=1), []
            e = a[t].exp()
            S = torch.where(e[:, None, None] == 0, 0.0, e[:, None, None] * S)
            u = b[t][:, None] * (v[t] - (k[t][:, :, None] * S).sum(1))
            S = S + k[t][:, :, None] * u[:, None, :]
            o[t] = s * (q[t][:, :, None] * S).sum(1)
            start = start * e[:, None]
            us = [(w * e, kj, uj) for w, kj, uj in us] + [(torch.ones_like(e), k[t], u.abs())]
            inter[t] = s * q[t].norm(dim=-1)[:, None] * start
            for w, kj, uj in us:
                intra[t] += s * (w * (q[t] * kj).sum(-1).abs())[:, None] * uj
        last.append(S)
    shape = (B, T, H, V)
    empty = torch.zeros(0, H, K, V, dtype=torch.float64)
    return o.reshape(shape), torch.stack(last) if last else empty, inter.reshape(shape), intra.reshape(shape)


def qk(x, weight, norm, positions=None, inv_freq=None, pair_axes=None, interleaved=False, m=1.0, eps=EPS):
    """One side: x [B, T, heads, D]; norm 0 none, 1 rms, 2 l2."""
    y = x.double()
    if norm:
        n = (y * y).sum(-1, keepdim=True)
        y = y / torch.sqrt((n / x.shape[-1] if norm == 1 else n) + eps)
    if weight is not None:
        y = y * weight.double()
    if positions is None:
        return y
    y = y.clone()
    half = inv_freq.numel()
    pos = positions if positions.dim() == 3 else positions[None]
    m = torch.tensor(m, dtype=torch.float32).double()  # the C ABI carries a float
    for i in range(half):
        angle = (pos[pair_axes[i] if pair_axes is not None else 0].double() * inv_freq[i].double())[:, :, None]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y[..., a] = m * (ya * torch.cos(angle) - yb * torch.sin(angle))
        y[..., b] = m * (yb * torch.cos(angle) + ya * torch.sin(angle))
    return y
