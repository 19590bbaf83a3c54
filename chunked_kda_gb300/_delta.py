"""The gated delta rule with one decay for each head, and the norm and rotation of its queries and keys.
The functions carry the C ABI's names and only check and marshal their arguments, in the manner of
the other operators around the recurrence.
"""
from __future__ import annotations

from operator import index

import torch

import chunked_kda_gb300 as _kda

from ._block import _CODES, _F32, _I32, _arg, _code, _device, _elsewhere, _library, _opt, _packed, _raw_stream


def kda_delta_chunk_workspace_bytes(dtype, B, T, H, K, V, n_seqs=0, o_dtype=None) -> int:
    """Scratch bytes of kda_delta_chunk_fwd for these sizes (n_seqs 0: dense)."""
    return int(_library().kda_delta_chunk_workspace_bytes(_CODES[dtype], _CODES[o_dtype or dtype], B, T, H, K, V, n_seqs))


def _delta(chunked, q, k, v, g, beta, A_log, dt_bias, mode, initial_state, output_final_state, cu_seqlens, o, final_state,
           stream, o_dtype, flags, workspace=None, status=None):
    dev, here = _device(q)
    if stream is not None or not here:
        return _elsewhere(_delta, q, stream, (chunked, q, k, v, g, beta, A_log, dt_bias, mode, initial_state,
                                              output_final_state, cu_seqlens, o, final_state, None, o_dtype, flags,
                                              workspace, status))
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must have four dimensions [B, T, heads, channels]")
    B, T, Hk, K = shape = q.shape
    H, V = v.shape[2:]
    if Hk < 1 or H % Hk != 0:
        raise ValueError("the q/k heads must divide v's heads")
    dtype, dt = q.dtype, _code(q, "q")
    out_shape, gate_shape, head_shape = (B, T, H, V), (B, T, H), (H,)
    pq, pk = _arg(q, "q", dev, dtype, shape), _arg(k, "k", dev, dtype, shape)
    pv = _arg(v, "v", dev, dtype, out_shape)
    gt, bt = _code(g, "g"), _code(beta, "beta")
    pg, pb = _arg(g, "g", dev, g.dtype, gate_shape), _arg(beta, "beta", dev, beta.dtype, gate_shape)
    pa, pd = _opt(A_log, "A_log", dev, _F32, head_shape), _opt(dt_bias, "dt_bias", dev, _F32, head_shape)
    pcu, n_seqs, N = _packed(cu_seqlens, B, dev)
    state_shape = (N, H, K, V)
    p0 = _opt(initial_state, "initial_state", dev, _F32, state_shape)
    if o is None:
        if o_dtype is None:
            o, ot = torch.empty_like(v), dt
        else:
            o = torch.empty(out_shape, device=v.device, dtype=o_dtype)
            ot = _code(o, "o")
        po = o.data_ptr()
    else:
        po, ot = _arg(o, "o", dev, o.dtype, out_shape), _code(o, "o")
    if final_state is None:
        p1 = None
        if output_final_state:
            final_state = torch.empty(state_shape, device=q.device, dtype=_F32)
            p1 = final_state.data_ptr()
    else:
        p1 = p0 if final_state is initial_state else _arg(final_state, "final_state", dev, _F32, state_shape)
    lib = _library()
    if not chunked:
        code = lib.kda_delta_recurrent_fwd(pq, pk, pv, dt, pg, gt, pa, pd, mode, pb, bt, p0, p1, pcu, n_seqs, B, T, H, Hk,
                                           K, V, po, ot, flags, _raw_stream(dev))
        if code:
            _kda._check("kda_delta_recurrent_fwd", code)
        return o, final_state
    if workspace is None:
        need = lib.kda_delta_chunk_workspace_bytes(dt, ot, B, T, H, K, V, n_seqs)
        if need > 0:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    pw, size = None, 0
    if workspace is not None:
        pw, size = _arg(workspace, "workspace", dev, workspace.dtype, workspace.shape), workspace.nbytes
    if status is not None and status.numel() < 1:
        raise ValueError("status needs one int32 element")
    code = lib.kda_delta_chunk_fwd(pq, pk, pv, dt, pg, gt, pa, pd, mode, pb, bt, p0, p1, pcu, n_seqs, B, T, H, Hk, K, V,
                                   po, ot, flags, pw, size,
                                   None if status is None else _arg(status, "status", dev, _I32, status.shape),
                                   _raw_stream(dev))
    if code:
        _kda._check("kda_delta_chunk_fwd", code)
    return o, final_state


def kda_delta_chunk_fwd(q, k, v, g, beta, A_log=None, dt_bias=None, mode=_kda.GATE_PRE, initial_state=None,
                        output_final_state=False, cu_seqlens=None, o=None, final_state=None, workspace=None,
                        stream=None, o_dtype=None, flags=0, status=None):
    """The gated delta rule with a decay for each head, in chunks (prompts); (o, final_state or None).

        S_t = exp(a_t) S_{t-1};   S_t += beta_t k_t (v_t - S_t^T k_t)^T;   o_t = S_t^T q_t / sqrt(K)

    q, k [B, T, Hk, K], v [B, T, H, V] (float32 or bfloat16, Hk a divisor of H); g [B, T, H], float32 or
    bfloat16: the natural-log decay a (GATE_PRE), or with GATE_NONSAFE the raw gate of
    a = -exp(A_log) softplus(g + dt_bias), A_log and dt_bias float32 [H]; beta [B, T, H] in q's dtype or
    float32.  ``flags``: FLAG_Q_L2NORM, FLAG_K_L2NORM, FLAG_BETA_LOGITS.  States float32 [N, H, K, V];
    ``o_dtype`` is q's dtype or torch.float32 (for bf16 inputs the exact one: computed in FP32).  Packed
    sequences, in-place states, ``workspace``, ``status`` and ``stream`` as for kda_chunk_fwd."""
    return _delta(True, q, k, v, g, beta, A_log, dt_bias, mode, initial_state, output_final_state, cu_seqlens, o,
                  final_state, stream, o_dtype, flags, workspace, status)


def kda_delta_recurrent_fwd(q, k, v, g, beta, A_log=None, dt_bias=None, mode=_kda.GATE_PRE, initial_state=None,
                            output_final_state=False, cu_seqlens=None, o=None, final_state=None, stream=None,
                            o_dtype=None, flags=0):
    """kda_delta_chunk_fwd's function token by token in float32 (single tokens; ``final_state`` may be
    ``initial_state``)."""
    return _delta(False, q, k, v, g, beta, A_log, dt_bias, mode, initial_state, output_final_state, cu_seqlens, o,
                  final_state, stream, o_dtype, flags)


def _rows(x, name, dev, dtype, shape):
    """(address, elements from one token to the next) of a checked tensor [B, T, heads, D] whose tokens lie
    evenly apart, each one's heads together."""
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.dim() != 4 or (shape is not None and x.shape != shape):
        raise ValueError(f"{name} must have shape {'[B, T, heads, D]' if shape is None else tuple(shape)}, got {tuple(x.shape)}")
    if x.requires_grad:
        raise ValueError(f"{name} requires grad: this library is forward-only (inference)")
    if x.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor, all arguments on one device")
    B, T, H, D = x.shape
    if x.is_contiguous():
        return x.data_ptr(), H * D
    sb, st, sh, sd = x.stride()
    step = st if T > 1 else sb
    if (D > 1 and sd != 1) or (H > 1 and sh != D) or (B > 1 and T > 1 and sb != T * st):
        raise ValueError(f"{name}: a token's heads must lie together, and its tokens evenly apart")
    return x.data_ptr(), step if B * T > 1 else H * D


def kda_qk_norm_rope_fwd(q, k=None, q_weight=None, k_weight=None, norm=_kda.NORM_RMS, eps=1e-6, positions=None,
                         inv_freq=None, pair_axes=None, interleaved=False, rope_scale=1.0, q_out=None, k_out=None,
                         stream=None):
    """The norm of each query and key head and the rotation of its position in one pass; (q_out, k_out).

        y = x / sqrt(mean(x^2) + eps) * weight   (NORM_RMS; NORM_L2: the sum for the mean; NORM_NONE: x * weight)
        (y_a, y_b) <- rope_scale (y_a cos - y_b sin, y_b cos + y_a sin),   angle = position * inv_freq

    q [B, T, Hq, D] and k [B, T, Hk, D] or None (float32 or bfloat16), each contiguous or a part of wider rows
    (a slice of the projection's output); weights float32 [D] or None.  ``positions`` int32 [B, T] or
    [axes, B, T] (up to four axes) and ``inv_freq`` float32 [R/2] rotate the first R channels, pair i being
    (i, R/2 + i) or, ``interleaved``, (2i, 2i + 1); ``pair_axes``, a sequence of R/2 integers, says which
    axis each pair follows (default: the first).  Without positions nothing is rotated.  ``q_out`` may be q and
    ``k_out`` k; allocated ones are contiguous."""
    dev, here = _device(q)
    if stream is not None or not here:
        return _elsewhere(kda_qk_norm_rope_fwd, q, stream, (q, k, q_weight, k_weight, norm, eps, positions, inv_freq,
                                                            pair_axes, interleaved, rope_scale, q_out, k_out))
    dtype, dt = q.dtype, _code(q, "q")
    pq, sq = _rows(q, "q", dev, dtype, None)
    B, T, Hq, D = q.shape
    pk = pko = None
    Hk = sk = sko = 0
    if k is not None:
        Hk = k.shape[2] if k.dim() == 4 else 0
        pk, sk = _rows(k, "k", dev, dtype, (B, T, Hk, D))
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    pwq, pwk = _opt(q_weight, "q_weight", dev, _F32, (D,)), _opt(k_weight, "k_weight", dev, _F32, (D,))
    pp = pf = axes = None
    R = n_axes = 0
    if positions is not None:
        if inv_freq is None or inv_freq.dim() != 1:
            raise ValueError("positions need inv_freq [R/2]")
        R, n_axes = 2 * inv_freq.shape[0], 1 if positions.dim() == 2 else positions.shape[0]
        pp = _arg(positions, "positions", dev, _I32, (B, T) if positions.dim() == 2 else (n_axes, B, T))
        pf = _arg(inv_freq, "inv_freq", dev, _F32, inv_freq.shape)
        if pair_axes is not None:
            pair_axes = [index(a) for a in pair_axes]  # (bytes() of an array would be its memory)
            if len(pair_axes) != R // 2 or not set(pair_axes) <= set(range(n_axes)):
                raise ValueError("pair_axes needs R/2 integers below the number of axes")
            axes = bytes(pair_axes)
    elif inv_freq is not None or pair_axes is not None:
        raise ValueError("inv_freq and pair_axes need positions")
    if q_out is None:
        q_out, sqo = torch.empty(q.shape, device=q.device, dtype=dtype), Hq * D
        pqo = q_out.data_ptr()
    else:
        pqo, sqo = _rows(q_out, "q_out", dev, dtype, q.shape)
    if k is not None:
        if k_out is None:
            k_out, sko = torch.empty(k.shape, device=q.device, dtype=dtype), Hk * D
            pko = k_out.data_ptr()
        else:
            pko, sko = _rows(k_out, "k_out", dev, dtype, k.shape)
    code = _library().kda_qk_norm_rope_fwd(pq, sq, pk, sk, dt, pwq, pwk, norm, eps, pp, n_axes, pf, axes, R, interleaved,
                                           rope_scale, B * T, Hq, Hk, D, pqo, sqo, pko, sko, _raw_stream(dev))
    if code:
        _kda._check("kda_qk_norm_rope_fwd", code)
    return q_out, k_out
