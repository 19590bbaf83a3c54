"""The operators of a linear-attention block, their cases, inputs and plain forms.

Four operators: linear attention with a decay for each head (chunked for prompts, recurrent for
single tokens), the gated norm of its heads, the norm around a block with its gate, residual and
scale, and the short causal convolution in front of the recurrence.  `run` makes one pass through
one of them: with `own` through the library's entry points, else in elementary torch operations.
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
        chunk("chunk_f32_b1_t128_h2_d64", "f32", B=1, T=128, H=2, K=64, V=64, state=False),
        # a batch of packed prompts of uneven lengths, two of them empty, continued from states
        chunk("chunk_packed_n16_t20480_h32_d128", "bf16", B=1, T=20480, H=32, K=128, V=128, n_seqs=16),
        # long prompts of a wide model, a decay for each token: the largest work
        chunk("chunk_b4_t4096_h64_d128", "bf16", B=4, T=4096, H=64, K=128, V=128, state=False),
        # one very long prompt with few heads and a fixed decay for each head
        chunk("chunk_b1_t32767_h16_d128_fixed", "bf16", B=1, T=32767, H=16, K=128, V=128, fixed=True),
        # one token for each of a full server's sequences
        recurrent("recurrent_n512_h32_d128", "bf16", N=512, H=32, K=128, V=128),
        # one token for a few sequences: latency
        recurrent("recurrent_n3_h32_d128", "bf16", N=3, H=32, K=128, V=128),
        # the heads' outputs of a prompt, and of one decode step
        head_norm("gated_norm_t16384_h64_d128", "bf16", rows=16384, H=64, V=128, act="sigmoid"),
        head_norm("gated_norm_t128_h32_d128", "bf16", rows=128, H=32, V=128, act="silu"),
        # the residual stream (float32) of a prompt through a norm after and one before a block
        block_norm("block_norm_t16384_d8192", "bf16", rows=16384, D=8192, res="f32", post=True, gate=False),
        # one token for some sequences, bf16 stream, gated block
        block_norm("block_norm_t77_d4096_gate", "bf16", rows=77, D=4096, res="bf16", post=True, gate=True),
        # packed prompts through the convolution, and one token for each of a server's sequences
        conv("conv_packed_n16_t20480_d12288", "bf16", N=16, T=20480, D=12288, W=4),
        conv("conv_n512_t1_d12288", "bf16", N=512, T=512, D=12288, W=4, single=True),
    ]


def chunk(name, dtype, B, T, H, K, V, Hk=0, n_seqs=0, fixed=False, state=True):
    return {"name": name, "op": "chunk", "dtype": dtype, "B": B, "T": T, "H": H, "Hk": Hk or H, "K": K,
            "V": V, "n_seqs": n_seqs, "fixed": fixed, "state": state}


def recurrent(name, dtype, N, H, K, V, Hk=0, fixed=False):
    return {"name": name, "op": "recurrent", "dtype": dtype, "N": N, "H": H, "Hk": Hk or H, "K": K, "V": V,
            "fixed": fixed}


def head_norm(name, dtype, rows, H, V, act):
    return {"name": name, "op": "head_norm", "dtype": dtype, "rows": rows, "H": H, "V": V, "act": act}


def block_norm(name, dtype, rows, D, res, post, gate, channel_scale=False):
    return {"name": name, "op": "block_norm", "dtype": dtype, "rows": rows, "D": D, "res": res,
            "post": post, "gate": gate, "channel_scale": channel_scale}


def conv(name, dtype, N, T, D, W, single=False, bias=False):
    return {"name": name, "op": "conv", "dtype": dtype, "N": N, "T": T, "D": D, "W": W, "single": single,
            "bias": bias}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "chunk", "recurrent", "head_norm", "block_norm", "conv"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    H = _log_int(rng, 1, 96)
    Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0 and H // h <= 8])
    if op == "chunk":
        K, V = rng.choice(((128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (256, 256)))
        most = 2 ** 20 if dtype == "bf16" else 2 ** 17  # tokens times heads
        most = max(1, int(most * min(1.0, 128 * 128 / (K * V))) // H)
        T = _log_int(rng, 1, min(most, 32768))
        if rng.random() < 0.4:
            n = _log_int(rng, 1, min(64, 2 * T))
            return chunk("", dtype, 1, T, H, K, V, Hk, n, rng.random() < 0.3) | _unnamed()
        B = _log_int(rng, 1, max(1, min(32, most // T)))
        return chunk("", dtype, B, T, H, K, V, Hk, 0, rng.random() < 0.3, rng.random() < 0.5) | _unnamed()
    if op == "recurrent":
        K, V = rng.choice((128, 128, 64, 256, rng.randint(16, 256))), rng.choice((128, 128, 64, 256, rng.randint(16, 256)))
        N = _log_int(rng, 1, max(1, min(1024, (512 * 32 * 128 * 128) // (H * K * V))))
        return recurrent("", dtype, N, H, K, V, Hk, rng.random() < 0.3) | _unnamed()
    if op == "head_norm":
        V = rng.choice((128, 128, 64, 256, rng.randint(16, 512)))
        rows = _log_int(rng, 1, max(1, min(65536, 2 ** 27 // (H * V))))
        return head_norm("", dtype, rows, H, V, rng.choice(("sigmoid", "silu"))) | _unnamed()
    D = rng.choice((128 * H, 128 * H, _log_int(rng, 8, 12288)))
    if op == "block_norm":
        rows = _log_int(rng, 1, max(1, min(65536, 2 ** 26 // D)))
        return block_norm("", dtype, rows, D, rng.choice(("f32", "bf16")), rng.random() < 0.6,
                          rng.random() < 0.5, rng.random() < 0.3) | _unnamed()
    T = _log_int(rng, 1, max(1, min(65536, 2 ** 26 // D)))
    single = rng.random() < 0.3
    if single:
        T = min(T, 1024)
    return conv("", dtype, T if single else _log_int(rng, 1, min(32, 2 * T)), T, D, rng.randint(2, 6), single,
                rng.random() < 0.3) | _unnamed()


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
    gen = torch.Generator(device=dev).manual_seed(1000003 * (seed % 1000003) + 17)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def unit(*shape):  # rows of norm 1, as the recurrence gets its queries and keys
        x = torch.randn(shape, generator=gen, device=dev)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dt)

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("chunk", "recurrent"):
        H, Hk, K, V = (case[n] for n in ("H", "Hk", "K", "V"))
        B, T = (1, case["N"]) if op == "recurrent" else (case["B"], case["T"])
        s["q"], s["k"], s["v"] = unit(B, T, Hk, K), unit(B, T, Hk, K), randn(B, T, H, V)
        slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev) / H)  # from a few tokens to hundreds
        if case["fixed"]:
            s["decay"] = (-slope * (0.5 + rand(H))).contiguous()
        else:  # a step size for each token, as a softplus gives it, times the head's slope
            s["decay"] = -slope * torch.nn.functional.softplus(randn(B, T, H, dtype=torch.float32) * 1.5)
        edges = None
        if op == "recurrent":
            edges = list(range(T + 1))
        elif case["n_seqs"]:
            edges = _lengths(case["n_seqs"], T, seed)
        if edges is not None:
            s["edges"] = edges
            s["cu"] = torch.tensor(edges, dtype=torch.int32, device=dev)
        N = len(edges) - 1 if edges is not None else B
        s["state"] = randn(N, H, K, V, std=0.05, dtype=torch.float32) if case.get("state", True) else None
    elif op == "head_norm":
        shape = (1, case["rows"], case["H"], case["V"])
        s["x"], s["gate"] = randn(*shape, std=0.3), randn(*shape)
        s["weight"] = 1.0 + randn(case["V"], std=0.1, dtype=torch.float32)
    elif op == "block_norm":
        rows, D = case["rows"], case["D"]
        s["x"] = randn(rows, D, std=0.5)
        s["residual"] = randn(rows, D, std=2.0, dtype=DTYPES[case["res"]])
        s["gate"] = randn(rows, D) if case["gate"] else None
        s["post_weight"] = 1.0 + randn(D, std=0.1, dtype=torch.float32) if case["post"] else None
        s["pre_weight"] = 1.0 + randn(D, std=0.1, dtype=torch.float32)
        s["channel_scale"] = 0.5 + rand(D) if case["channel_scale"] else None
        s["scale"] = 0.7
    else:
        N, T, D, W = (case[n] for n in ("N", "T", "D", "W"))
        s["x"] = randn(1, T, D)
        s["weight"] = randn(D, W, std=0.5, dtype=torch.float32)
        s["bias"] = randn(D, std=0.1, dtype=torch.float32) if case["bias"] else None
        s["edges"] = list(range(T + 1)) if case["single"] else _lengths(N, T, seed)
        s["cu"] = torch.tensor(s["edges"], dtype=torch.int32, device=dev)
        s["state"] = randn(len(s["edges"]) - 1, W - 1, D)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


# ------------------------------------------------------------------ the library's calls

def _own_chunk(s):
    import chunked_kda_gb300 as kda

    return kda.kda_decay_chunk_fwd(s["q"], s["k"], s["v"], s["decay"], initial_state=s["state"],
                                   output_final_state=True, cu_seqlens=s.get("cu"))


def _own_recurrent(s):
    import chunked_kda_gb300 as kda

    return kda.kda_decay_recurrent_fwd(s["q"], s["k"], s["v"], s["decay"], initial_state=s["state"],
                                       final_state=s["state"], cu_seqlens=s["cu"])


def _own_head_norm(s):
    import chunked_kda_gb300 as kda

    act = kda.ACT_SIGMOID if s["case"]["act"] == "sigmoid" else kda.ACT_SILU
    return kda.kda_gated_norm_fwd(s["x"], s["gate"], s["weight"], eps=EPS, act=act)


def _own_block_norm(s):
    import chunked_kda_gb300 as kda

    return kda.kda_block_norm_fwd(s["x"], residual=s["residual"], post_weight=s["post_weight"], gate=s["gate"],
                                  pre_weight=s["pre_weight"], scale=s["scale"],
                                  channel_scale=s["channel_scale"], eps=EPS, act=kda.ACT_SIGMOID)


def _own_conv(s):
    import chunked_kda_gb300 as kda

    final = s["state"] if s["case"]["single"] else None  # a decode step works in place
    return kda.kda_short_conv_fwd(s["x"], s["weight"], s["bias"], act=kda.ACT_SILU, initial_state=s["state"],
                                  output_final_state=True, final_state=final, cu_seqlens=s["cu"])


# ------------------------------------------------------------------ the plain forms

def _rows(edges, cu):
    """Indices [N, L] of each sequence's rows (clamped to a row of its own padding) and which of them are real."""
    longest = max(1, max(b - a for a, b in zip(edges, edges[1:])))
    at = torch.arange(longest, device=cu.device)
    lens = (cu[1:] - cu[:-1]).long()
    real = at < lens[:, None]
    return torch.where(real, cu[:-1, None].long() + at, 0), real


def _heads(x, H):
    """[N, L, Hk, K] in float32, each head repeated for the value heads that share it."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2)


def _plain_chunk(s):
    q, k, v, decay, S0 = s["q"], s["k"], s["v"], s["decay"], s["state"]
    H, K, V, C = v.shape[2], q.shape[3], v.shape[3], PLAIN_CHUNK
    a = decay.expand(v.shape[:3]) if decay.dim() == 1 else decay
    packed = "cu" in s
    if packed:  # one row for each sequence
        index, real = _rows(s["edges"], s["cu"])
        q, k, v = (torch.where(real[..., None, None], x[0][index], 0) for x in (q, k, v))
        a = torch.where(real[..., None], a[0][index], 0.0)
    N, L = v.shape[:2]
    n = -(-L // C)

    def chunks(x):  # [N, L, H, d] -> [N, H, n, C, d]
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * C - L))
        return x.reshape(N, n, C, H, -1).permute(0, 3, 1, 2, 4)

    qc, kc, vc = chunks(_heads(q, H)), chunks(_heads(k, H)), chunks(v.float())
    G = chunks(a.double()[..., None])[..., 0].cumsum(-1)  # in 64 bits: far positions' differences
    causal = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    M = torch.where(causal, G[..., :, None] - G[..., None, :], -math.inf).float().exp()
    inside = (qc @ kc.transpose(-1, -2) * M) @ vc
    kd = kc * (G[..., -1:] - G).float().exp()[..., None]
    dS = (kd.transpose(-1, -2) @ vc).reshape(N, H, n, K * V)
    E = torch.nn.functional.pad(G[..., -1].cumsum(-1), (1, 0))  # log decay up to each chunk's start
    before = torch.ones(n + 1, n, dtype=torch.bool, device=q.device).tril(-1)
    W = torch.where(before, E[..., :, None] - E[..., None, 1:], -math.inf).float().exp()
    S = (W @ dS).reshape(N, H, n + 1, K, V)  # each chunk's incoming state, and the last one's outgoing
    if S0 is not None:
        S = S + E.float().exp()[..., None, None] * S0[:, :, None]
    o = (inside + G.float().exp()[..., None] * (qc @ S[:, :, :n])) * K ** -0.5
    o = o.permute(0, 2, 3, 1, 4).reshape(N, n * C, H, V)[:, :L]
    if packed:
        o = o[real][None]
    return o.to(s["q"].dtype), S[:, :, n].contiguous()


def _plain_recurrent(s):
    q, k, v, state = s["q"], s["k"], s["v"], s["state"]
    H, K = v.shape[2], q.shape[3]
    q, k, v = _heads(q, H)[0], _heads(k, H)[0], v[0].float()
    decay = s["decay"].expand(v.shape[:2]) if s["decay"].dim() == 1 else s["decay"][0]
    state.mul_(decay.exp()[..., None, None]).add_(k[..., :, None] * v[..., None, :])
    o = (state * q[..., :, None]).sum(-2) * K ** -0.5
    return o[None].to(s["q"].dtype), state


def _act(z, name):
    return torch.sigmoid(z) if name == "sigmoid" else z * torch.sigmoid(z)


def _norm(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _plain_head_norm(s):
    y = _norm(s["x"].float(), s["weight"]) * _act(s["gate"].float(), s["case"]["act"])
    return y.to(s["x"].dtype)


def _plain_block_norm(s):
    n = s["x"].float()
    if s["post_weight"] is not None:
        n = _norm(n, s["post_weight"])
    if s["gate"] is not None:
        n = n * torch.sigmoid(s["gate"].float())
    if s["channel_scale"] is not None:
        n = n * s["channel_scale"]
    h = s["residual"].float() + s["scale"] * n
    return h.to(s["residual"].dtype), _norm(h, s["pre_weight"]).to(s["x"].dtype)


def _plain_conv(s):
    x, weight, state = s["x"], s["weight"], s["state"]
    W = weight.shape[1]
    index, real = _rows(s["edges"], s["cu"])
    rows = torch.cat([state, torch.where(real[..., None], x[0][index], 0)], 1)  # [N, W - 1 + L, D]
    y = (rows.float().unfold(1, W, 1) * weight).sum(-1)
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, "silu")[real][None].to(x.dtype)
    last = (s["cu"][1:] - s["cu"][:-1]).long()[:, None] + torch.arange(W - 1, device=x.device)
    final = torch.gather(rows, 1, last[..., None].expand(-1, -1, x.shape[2]))
    return y, state.copy_(final) if s["case"]["single"] else final


_PLAIN = {"chunk": _plain_chunk, "recurrent": _plain_recurrent, "head_norm": _plain_head_norm,
          "block_norm": _plain_block_norm, "conv": _plain_conv}
_OWN = {"chunk": _own_chunk, "recurrent": _own_recurrent, "head_norm": _own_head_norm,
        "block_norm": _own_block_norm, "conv": _own_conv}


# ------------------------------------------------------------------ work and the 64-bit results

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("chunk", "recurrent"):
        H, Hk, K, V = (case[n] for n in ("H", "Hk", "K", "V"))
        tokens = case["N"] if op == "recurrent" else case["B"] * case["T"]
        N = case["N"] if op == "recurrent" else (case["n_seqs"] or case["B"])
        states = 2 if case.get("state", True) else 1
        data = tokens * (2 * Hk * K + 2 * H * V) * e + (4 * H if case["fixed"] else 4 * H * tokens)
        # the recurrence itself: decay and update of the state, and its product with the query
        return {"bytes": data + states * 4 * N * H * K * V, "flops": tokens * H * 5 * K * V}
    if op == "head_norm":
        n = case["rows"] * case["H"] * case["V"]
        return {"bytes": 3 * n * e, "flops": 10 * n}
    if op == "block_norm":
        n, r = case["rows"] * case["D"], 2 if case["res"] == "bf16" else 4
        return {"bytes": n * ((3 if case["gate"] else 2) * e + 2 * r), "flops": 12 * n}
    n, N = case["T"] * case["D"], case["N"]
    return {"bytes": 2 * n * e + 2 * N * (case["W"] - 1) * case["D"] * e, "flops": n * (2 * case["W"] + 5)}


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _exact_attention(s):
    """The recurrence token by token, all sequences side by side."""
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    H, K, V = v.shape[2], q.shape[3], v.shape[3]
    B, T = v.shape[:2]
    g = torch.exp(s["decay"].double())
    g = g.expand(B, T, H) if g.dim() == 1 else g
    share = torch.arange(H, device=q.device) // (H // q.shape[2])
    edges = s.get("edges")
    if edges is None:
        starts, lens = [b * T for b in range(B)], [T] * B
    else:
        starts, lens = edges[:-1], [b - a for a, b in zip(edges, edges[1:])]
    N = len(lens)
    if max(lens) * max(1.0, N * H * K * V / 2 ** 22) > 60000:
        return None
    q, k, v, g = q.reshape(B * T, -1, K), k.reshape(B * T, -1, K), v.reshape(B * T, H, V), g.reshape(B * T, H)
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
        cur = S[:live]
        cur.mul_(g[row][..., None, None])
        cur.add_(k[row][:, share][..., :, None] * v[row][..., None, :])
        o[row] = torch.einsum("nhkv,nhk->nhv", cur, q[row][:, share]) / math.sqrt(K)
    back = torch.empty_like(S)
    back[order] = S
    return o.reshape(B, T, H, V), back


def _sig64(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _exact_head_norm(s):
    x, z = s["x"].double(), s["gate"].double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].double() * _sig64(z)
    return y * z if s["case"]["act"] == "silu" else y


def _exact_block_norm(s):
    n = s["x"].double()
    if s["post_weight"] is not None:
        n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS) * s["post_weight"].double()
    if s["gate"] is not None:
        n = n * _sig64(s["gate"].double())
    if s["channel_scale"] is not None:
        n = n * s["channel_scale"].double()
    h = s["residual"].double() + s["scale"] * n
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["pre_weight"].double()


def _exact_conv(s):
    W, T = s["weight"].shape[1], s["x"].shape[1]
    lens = [b - a for a, b in zip(s["edges"], s["edges"][1:])]
    owner = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(s["x"].device)
    x, w, hist = s["x"][0].double(), s["weight"].double(), s["state"].double()
    place = torch.arange(T, device=x.device) - s["cu"].long()[owner]
    y = torch.zeros_like(x) if s["bias"] is None else s["bias"].double().expand_as(x).clone()
    for tap in range(W):
        back = W - 1 - tap
        past = place < back
        src = x[(torch.arange(T, device=x.device) - back).clamp_min(0)]
        old = hist[owner, (place - back + W - 1).clamp(0, W - 2)]
        y += w[:, tap] * torch.where(past[:, None], old, src)
    final = hist.clone()
    for n, (a, b) in enumerate(zip(s["edges"], s["edges"][1:])):
        m = min(b - a, W - 1)
        if m:
            final[n] = torch.cat([hist[n, m:], x[b - m:b]])
    return (y * _sig64(y))[None], final


_EXACT = {"chunk": _exact_attention, "recurrent": _exact_attention, "head_norm": _exact_head_norm,
          "block_norm": _exact_block_norm, "conv": _exact_conv}
