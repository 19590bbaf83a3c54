"""Operators in front of and in place of the recurrence, their cases, inputs and plain forms.

Three operators: the gated delta rule with one decay for each head (in chunks for prompts, token by
token for decoding), and the norm of each query and key head with the rotation of its positions in
the same pass.  `run` makes one pass through one of them: with `own` through the library's entry
points, else in elementary torch operations.
"""
import math
import random  # noqa: F401  (the type of draw's argument)

import torch

own = False

EPS = 1e-6
PLAIN_CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a short float32 prompt: the smallest chunked call, latency
        chunk("delta_f32_b1_t128_h2_d64", "f32", B=1, T=128, H=2, K=64, V=64, state=False),
        # a batch of packed prompts of uneven lengths, two query heads to a key head, continued from
        # states, everything as the projections leave it: raw gates, logits, rows that have no norm yet
        chunk("delta_packed_raw_n16_t20480_h32_d128", "bf16", B=1, T=20480, H=32, Hk=16, K=128, V=128,
              n_seqs=16, raw=True),
        # long prompts of a wide model: the largest work
        chunk("delta_b4_t4096_h64_d128", "bf16", B=4, T=4096, H=64, K=128, V=128, state=False),
        # one long prompt
        chunk("delta_b1_t8192_h96_d128", "bf16", B=1, T=8192, H=96, K=128, V=128),
        # one token for each of a full server's sequences
        token("delta_token_n512_h32_d128", "bf16", N=512, H=32, K=128, V=128),
        # one token for a few sequences, straight from the projections: latency
        token("delta_token_raw_n3_h32_d128", "bf16", N=3, H=32, Hk=16, K=128, V=128, raw=True),
        # queries and keys of a prompt, slices of the projection's rows: norm with weights, rotation
        # of all channels at positions that go on behind a long context
        rope("qk_rope_t16384_h64_d128", "bf16", B=1, T=16384, Hq=64, Hk=8, D=128, R=128, norm="rms", past=100000),
        # images and video between text: three axes, half of the channels rotated
        rope("qk_rope_axes3_b2_t2048_h32_d128", "bf16", B=2, T=2048, Hq=32, Hk=8, D=128, R=64, norm="rms", axes=3),
        # one token for some sequences: latency
        rope("qk_rope_t77_h32_d128", "bf16", B=77, T=1, Hq=32, Hk=8, D=128, R=128, norm="rms", past=30000),
        # queries and keys in front of the delta rule: rows of norm 1, no positions
        rope("qk_l2_t20480_h16_d128", "bf16", B=1, T=20480, Hq=16, Hk=16, D=128, R=0, norm="l2"),
    ]


def chunk(name, dtype, B, T, H, K, V, Hk=0, n_seqs=0, raw=False, state=True):
    return {"name": name, "op": "chunk", "dtype": dtype, "B": B, "T": T, "H": H, "Hk": Hk or H, "K": K,
            "V": V, "n_seqs": n_seqs, "raw": raw, "state": state}


def token(name, dtype, N, H, K, V, Hk=0, raw=False):
    return {"name": name, "op": "token", "dtype": dtype, "N": N, "H": H, "Hk": Hk or H, "K": K, "V": V, "raw": raw}


def rope(name, dtype, B, T, Hq, Hk, D, R, norm, axes=1, past=0, interleaved=False, sliced=True):
    return {"name": name, "op": "rope", "dtype": dtype, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R,
            "norm": norm, "axes": axes, "past": past, "interleaved": interleaved, "sliced": sliced}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "chunk", "token", "rope", "rope"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    H = _log_int(rng, 1, 96)
    Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0 and H // h <= 8])
    raw = rng.random() < 0.5
    if op == "chunk":
        K, V = rng.choice(((128, 128), (128, 128), (64, 64), (64, 128), (128, 256), (96, 96)))
        most = 2 ** 20 if dtype == "bf16" else 2 ** 17  # tokens times heads
        most = max(1, int(most * min(1.0, 128 * 128 / (K * V))) // H)
        T = _log_int(rng, 1, min(most, 32768))
        if rng.random() < 0.4:
            n = _log_int(rng, 1, min(64, 2 * T))
            return chunk("", dtype, 1, T, H, K, V, Hk, n, raw) | _unnamed()
        B = _log_int(rng, 1, max(1, min(32, most // T)))
        return chunk("", dtype, B, T, H, K, V, Hk, 0, raw, rng.random() < 0.5) | _unnamed()
    if op == "token":
        K, V = rng.choice((128, 128, 64, 256, rng.randint(16, 256))), rng.choice((128, 128, 64, 256, rng.randint(16, 256)))
        N = _log_int(rng, 1, max(1, min(1024, (512 * 32 * 128 * 128) // (H * K * V))))
        return token("", dtype, N, H, K, V, Hk, raw) | _unnamed()
    D = rng.choice((128, 128, 64, 256, 2 * rng.randint(8, 128)))
    R = rng.choice((D, D, 2 * rng.randint(0, D // 2)))
    rows = _log_int(rng, 1, max(1, min(65536, 2 ** 27 // ((H + Hk) * D))))
    B = rng.choice([b for b in range(1, 33) if rows % b == 0])
    return rope("", dtype, B, rows // B, H, Hk, D, R, rng.choice(("rms", "rms", "l2", "none")), rng.randint(1, 3),
                rng.choice((0, 1000, 1000000)), rng.random() < 0.3, rng.random() < 0.7) | _unnamed()


def _unnamed():
    return {"name": "drawn"}


def _lengths(n, total, seed):
    """n lengths with the given sum: uneven, some of them zero."""
    gen = torch.Generator().manual_seed(seed)
    part = torch.rand(n, generator=gen, dtype=torch.float64) ** 1.5
    part[torch.rand(n, generator=gen) < 0.1] = 0
    part[int(torch.randint(n, (1,), generator=gen))] = 1.0
    edges = torch.round(torch.cumsum(part, 0) / part.sum() * total).to(torch.int64)
    return [0] + edges.tolist()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(1000003 * (seed % 1000003) + 29)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    s = {"case": dict(case)}
    if case["op"] == "rope":
        B, T, Hq, Hk, D, R = (case[n] for n in ("B", "T", "Hq", "Hk", "D", "R"))
        if case["sliced"]:  # queries, keys and values of a token side by side, as the projection leaves them
            rows = randn(B, T, Hq + 2 * Hk, D)
            s["q"], s["k"] = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = randn(B, T, Hq, D), randn(B, T, Hk, D)
        weights = case["norm"] == "rms"
        s["q_weight"] = 1.0 + randn(D, std=0.1, dtype=torch.float32) if weights else None
        s["k_weight"] = 1.0 + randn(D, std=0.1, dtype=torch.float32) if weights else None
        s["positions"] = s["inv_freq"] = s["pair_axes"] = None
        if R:
            first = torch.randint(case["past"] + 1, (B, 1), generator=gen, device=dev, dtype=torch.int32)
            pos = first + torch.arange(T, device=dev, dtype=torch.int32)
            if case["axes"] > 1:  # a height and a width beside the time
                more = torch.randint(64, (case["axes"] - 1, B, T), generator=gen, device=dev, dtype=torch.int32)
                pos = torch.cat([pos[None], first + more])
            s["positions"] = pos.contiguous()
            s["inv_freq"] = torch.exp(torch.arange(R // 2, device=dev) * (-2.0 * math.log(1e6) / R)).float()
            s["pair_axes"] = [i % case["axes"] for i in range(R // 2)] if case["axes"] > 1 else None
        return s
    H, Hk, K, V = (case[n] for n in ("H", "Hk", "K", "V"))
    B, T = (1, case["N"]) if case["op"] == "token" else (case["B"], case["T"])

    def rows(*shape):  # as a convolution's activation leaves them, and of norm 1 unless the call does that
        x = torch.nn.functional.silu(torch.randn(shape, generator=gen, device=dev))
        return (x if case["raw"] else x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dt)

    s["q"], s["k"], s["v"] = rows(B, T, Hk, K), rows(B, T, Hk, K), randn(B, T, H, V)
    A_log = torch.log(1.0 + 15.0 * rand(H))
    step = torch.exp(math.log(1e-3) + rand(H) * (math.log(0.1) - math.log(1e-3)))
    dt_bias = step + torch.log(-torch.expm1(-step))  # softplus of it is the head's step
    if case["raw"]:
        s["g"], s["beta"], s["A_log"], s["dt_bias"] = randn(B, T, H), randn(B, T, H), A_log, dt_bias
    else:
        x = randn(B, T, H, dtype=torch.float32)
        s["g"] = -torch.exp(A_log) * torch.nn.functional.softplus(x + dt_bias)
        s["beta"], s["A_log"], s["dt_bias"] = torch.sigmoid(randn(B, T, H, dtype=torch.float32)).to(dt), None, None
    edges = None
    if case["op"] == "token":
        edges = list(range(T + 1))
    elif case["n_seqs"]:
        edges = _lengths(case["n_seqs"], T, seed)
    if edges is not None:
        s["edges"] = edges
        s["cu"] = torch.tensor(edges, dtype=torch.int32, device=dev)
    N = len(edges) - 1 if edges is not None else B
    s["state"] = randn(N, H, K, V, std=0.05, dtype=torch.float32) if case.get("state", True) else None
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


# ------------------------------------------------------------------ the library's calls

def _gate(s):
    import chunked_kda_gb300 as kda

    if not s["case"]["raw"]:
        return {}
    return {"A_log": s["A_log"], "dt_bias": s["dt_bias"], "mode": kda.GATE_NONSAFE,
            "flags": kda.FLAG_Q_L2NORM | kda.FLAG_K_L2NORM | kda.FLAG_BETA_LOGITS}


def _own_chunk(s):
    import chunked_kda_gb300 as kda

    return kda.kda_delta_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], initial_state=s["state"],
                                   output_final_state=True, cu_seqlens=s.get("cu"), **_gate(s))


def _own_token(s):
    import chunked_kda_gb300 as kda

    return kda.kda_delta_recurrent_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], initial_state=s["state"],
                                       final_state=s["state"], cu_seqlens=s["cu"], **_gate(s))


def _own_rope(s):
    import chunked_kda_gb300 as kda

    norm = {"rms": kda.NORM_RMS, "l2": kda.NORM_L2, "none": kda.NORM_NONE}[s["case"]["norm"]]
    return kda.kda_qk_norm_rope_fwd(s["q"], s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"], norm=norm,
                                    eps=EPS, positions=s["positions"], inv_freq=s["inv_freq"],
                                    pair_axes=s["pair_axes"], interleaved=s["case"]["interleaved"])


# ------------------------------------------------------------------ the plain forms

def _inputs(s):
    """q, k, v, the natural-log decay in 64 bits and beta: float32, heads repeated, activated and normed."""
    H = s["v"].shape[2]
    q, k, v, b, g = s["q"].float(), s["k"].float(), s["v"].float(), s["beta"].float(), s["g"]
    if s["case"]["raw"]:
        g = -torch.exp(s["A_log"].double()) * torch.nn.functional.softplus(g.double() + s["dt_bias"].double())
        b = torch.sigmoid(b)
        q, k = (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS) for x in (q, k))
    q, k = (x.repeat_interleave(H // x.shape[2], dim=2) for x in (q, k))
    return q, k, v, g.double(), b


def _rows(edges, cu):
    """Indices [N, L] of each sequence's rows (clamped to a row of its own padding) and which of them are real."""
    longest = max(1, max(b - a for a, b in zip(edges, edges[1:])))
    at = torch.arange(longest, device=cu.device)
    lens = (cu[1:] - cu[:-1]).long()
    real = at < lens[:, None]
    return torch.where(real, cu[:-1, None].long() + at, 0), real


def _inverse(A):
    """(1 + A)^-1 of strictly lower triangular 64 x 64 matrices: blocks of 16 row by row, then merged."""
    n = A.shape[:-2]
    D = torch.stack([A[..., i:i + 16, i:i + 16] for i in range(0, 64, 16)], -3)
    X = torch.eye(16, device=A.device).expand(D.shape).clone()
    for i in range(1, 16):
        X[..., i:i + 1, :i] -= D[..., i:i + 1, :i] @ X[..., :i, :i]
    X = list(X.unbind(-3))
    for w in (16, 32):
        for b in range(64 // (2 * w)):
            a, c = X[2 * b], X[2 * b + 1]
            low = A[..., (2 * b + 1) * w:(2 * b + 2) * w, 2 * b * w:(2 * b + 1) * w]
            top = torch.cat([a, torch.zeros(n + (w, w), device=A.device)], -1)
            X[2 * b] = torch.cat([top, torch.cat([-(c @ (low @ a)), c], -1)], -2)
        X = X[::2]
    return X[0]


def _plain_chunk(s):
    q, k, v, g, b = _inputs(s)
    S, C = s["state"], PLAIN_CHUNK
    packed = "cu" in s
    if packed:  # one row for each sequence
        index, real = _rows(s["edges"], s["cu"])
        q, k, v = (torch.where(real[..., None, None], x[0][index], 0) for x in (q, k, v))
        g, b = (torch.where(real[..., None], x[0][index], 0) for x in (g, b))
    N, L, H, V = v.shape
    K, n = q.shape[3], -(-L // C)

    def chunks(x):  # [N, L, H, d] -> [n, N, H, C, d]
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * C - L))
        return x.reshape(N, n, C, H, -1).permute(1, 0, 3, 2, 4).contiguous()

    q, k, v, b = chunks(q), chunks(k), chunks(v), chunks(b[..., None])
    G = chunks(g[..., None])[..., 0].cumsum(-1)
    causal = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    M = torch.where(causal, G[..., :, None] - G[..., None, :], -math.inf).float().exp()
    T = _inverse((b * (k @ k.transpose(-1, -2)) * M).tril(-1)) * b.transpose(-1, -2)
    P = (q @ k.transpose(-1, -2)) * M
    row, last = G.float().exp()[..., None], (G[..., -1:] - G).float().exp()[..., None]
    S = torch.zeros(N, H, K, V, device=q.device) if S is None else S
    o = []
    for c in range(n):  # the state goes from chunk to chunk
        U = T[c] @ (v[c] - row[c] * (k[c] @ S))
        o.append(row[c] * (q[c] @ S) + P[c] @ U)
        S = row[c][..., -1:, :] * S + (k[c] * last[c]).transpose(-1, -2) @ U
    o = torch.stack(o).permute(1, 0, 3, 2, 4).reshape(N, n * C, H, V)[:, :L] * K ** -0.5
    if packed:
        o = o[real][None]
    return o.to(s["q"].dtype), S


def _plain_token(s):
    state = s["state"]
    q, k, v, g, b = (x[0] for x in _inputs(s))
    state.mul_(g.float().exp()[..., None, None])
    u = b[..., None] * (v - (state * k[..., :, None]).sum(-2))
    state.add_(k[..., :, None] * u[..., None, :])
    o = (state * q[..., :, None]).sum(-2) * q.shape[-1] ** -0.5
    return o[None].to(s["q"].dtype), state


def _plain_rope(s):
    case, out = s["case"], []
    R = case["R"]
    if R:
        pos = s["positions"]
        if s["pair_axes"] is None:
            pos = pos[..., None]
        else:
            pos = pos[torch.tensor(s["pair_axes"], device=pos.device)].permute(1, 2, 0)
        angle = pos.double() * s["inv_freq"].double()  # in 64 bits: far positions
        cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if case["norm"] == "rms":
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
        elif case["norm"] == "l2":
            y = y * torch.rsqrt(y.square().sum(-1, keepdim=True) + EPS)
        if R:
            turn, rest = y[..., :R], y[..., R:]
            if case["interleaved"]:
                a, b = turn[..., 0::2], turn[..., 1::2]
                turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            else:
                a, b = turn[..., :R // 2], turn[..., R // 2:]
                turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            y = torch.cat([turn, rest], -1)
        out.append(y.to(x.dtype))
    return tuple(out)


_PLAIN = {"chunk": _plain_chunk, "token": _plain_token, "rope": _plain_rope}
_OWN = {"chunk": _own_chunk, "token": _own_token, "rope": _own_rope}


# ------------------------------------------------------------------ work and the 64-bit results

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        positions = 4 * case["axes"] * case["B"] * case["T"] if case["R"] else 0
        return {"bytes": 2 * n * e + positions, "flops": 7 * n}
    H, Hk, K, V = (case[n] for n in ("H", "Hk", "K", "V"))
    single = case["op"] == "token"
    tokens = case["N"] if single else case["B"] * case["T"]
    N = case["N"] if single else (case["n_seqs"] or case["B"])
    states = 2 if case.get("state", True) else 1
    gates = tokens * H * (2 * e if case["raw"] else 4 + e)
    # the recurrence itself: decay, product with the key, update, and product with the query
    return {"bytes": tokens * (2 * Hk * K + 2 * H * V) * e + gates + states * 4 * N * H * K * V,
            "flops": tokens * H * 7 * K * V}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_delta(s)


def _exact_delta(s):
    """The recurrence token by token, all sequences side by side."""
    case = s["case"]
    q, k, v, b, a = (s[n].double() for n in ("q", "k", "v", "beta", "g"))
    H, K, V = v.shape[2], q.shape[3], v.shape[3]
    B, T = v.shape[:2]
    if case["raw"]:
        z = a + s["dt_bias"].double()
        a = -torch.exp(s["A_log"].double()) * (z.clamp_min(0) + torch.log1p(torch.exp(-z.abs())))
        b = 1.0 / (1.0 + torch.exp(-b))
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
    share = torch.arange(H, device=q.device) // (H // q.shape[2])
    edges = s.get("edges")
    if edges is None:
        starts, lens = [i * T for i in range(B)], [T] * B
    else:
        starts, lens = edges[:-1], [y - x for x, y in zip(edges, edges[1:])]
    N = len(lens)
    if max(lens) * max(1.0, N * H * K * V / 2 ** 22) > 40000:
        return None
    q, k, v = q.reshape(B * T, -1, K), k.reshape(B * T, -1, K), v.reshape(B * T, H, V)
    a, b = torch.exp(a).reshape(B * T, H), b.reshape(B * T, H)
    S = s["state"].double().clone() if s["state"] is not None else torch.zeros(N, H, K, V, dtype=torch.float64, device=q.device)
    order = sorted(range(N), key=lambda i: -lens[i])  # the longest first: those still running are a prefix
    S = S[order]
    first = torch.tensor([starts[i] for i in order], device=q.device)
    o = torch.zeros(B * T, H, V, dtype=torch.float64, device=q.device)
    live = N
    for t in range(max(lens)):
        while live and lens[order[live - 1]] <= t:
            live -= 1
        row = first[:live] + t
        cur, key = S[:live], k[row][:, share]
        cur.mul_(a[row][..., None, None])
        u = b[row][..., None] * (v[row] - torch.einsum("nhkv,nhk->nhv", cur, key))
        cur.addcmul_(key[..., :, None], u[..., None, :])
        o[row] = torch.einsum("nhkv,nhk->nhv", cur, q[row][:, share]) / math.sqrt(K)
    back = torch.empty_like(S)
    back[order] = S
    return o.reshape(B, T, H, V), back


def _exact_rope(s):
    case, out = s["case"], []
    half, D = case["R"] // 2, case["D"]
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        if case["norm"] != "none":
            norm = (y * y).sum(-1, keepdim=True)
            y = y / torch.sqrt((norm / D if case["norm"] == "rms" else norm) + EPS)
        if w is not None:
            y = y * w.double()
        y = y.clone()
        for i in range(half):  # one pair of channels after another
            p = s["positions"] if s["pair_axes"] is None else s["positions"][s["pair_axes"][i]]
            at = (p.double() * s["inv_freq"][i].double())[:, :, None]
            m, n = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
            a, b = y[..., m].clone(), y[..., n].clone()
            y[..., m] = a * torch.cos(at) - b * torch.sin(at)
            y[..., n] = a * torch.sin(at) + b * torch.cos(at)
        out.append(y)
    return tuple(out)
