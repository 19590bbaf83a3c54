"""The operators around the recurrence: decayed linear attention, gated and block norms, short
convolution.  As in the rest of the binding, the functions carry the C ABI's names and only check
and marshal their arguments.

A decode step makes these calls for every layer with kernels of a few microseconds, so the checks
stay short and the library's functions are looked up once.  Outputs and scratch are allocated on the
stream that the kernels run on (torch's current one unless ``stream`` is given).
"""
from __future__ import annotations

import torch

import chunked_kda_gb300 as _kda

_CODES = {torch.float32: 0, torch.bfloat16: 1}
_F32, _I32 = torch.float32, torch.int32
_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = _kda.load_library()
    return _lib


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the handle of torch's current stream without building a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(fn, x, stream, args):
    """fn's call with the given stream, or with the inputs' device, made current around it."""
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(x.get_device()):
        return fn(*args)


def _device(x):
    """The inputs' device, and whether it is the current one."""
    if not x.is_cuda:
        raise ValueError("the inputs must be CUDA tensors")
    index = x.get_device()
    return index, index == _current_device()


def _arg(t, name, index, dtype, shape):
    """The device address of a checked tensor."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.requires_grad or t.get_device() != index:
        _refuse(t, name, dtype, shape)
    return t.data_ptr()


def _opt(t, name, index, dtype, shape):
    return None if t is None else _arg(t, name, index, dtype, shape)


def _refuse(t, name, dtype, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.requires_grad:
        raise ValueError(f"{name} requires grad: this library is forward-only (inference)")
    raise ValueError(f"{name} must be a CUDA tensor, all arguments on one device")


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} is not float32 or bfloat16")
    return code


def _packed(cu_seqlens, B, index):
    """(pointer, n_seqs, logical sequences)."""
    if cu_seqlens is None:
        return None, 0, B
    if B != 1:
        raise ValueError("packed mode (cu_seqlens given) needs B == 1")
    n = cu_seqlens.numel()
    if n < 1:
        raise ValueError("cu_seqlens needs at least one offset")
    return _arg(cu_seqlens, "cu_seqlens", index, _I32, (n,)), n - 1, n - 1


def kda_decay_chunk_workspace_bytes(dtype, B, T, H, K, V, n_seqs=0) -> int:
    """Scratch bytes of kda_decay_chunk_fwd for these sizes (n_seqs 0: dense)."""
    return int(_library().kda_decay_chunk_workspace_bytes(_CODES[dtype], B, T, H, K, V, n_seqs))


def _decay(chunked, q, k, v, decay, initial_state, output_final_state, cu_seqlens, o, final_state, stream, o_dtype,
           workspace=None, status=None):
    dev, here = _device(q)
    if stream is not None or not here:
        return _elsewhere(_decay, q, stream, (chunked, q, k, v, decay, initial_state, output_final_state, cu_seqlens, o,
                                              final_state, None, o_dtype, workspace, status))
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must have four dimensions [B, T, heads, channels]")
    B, T, Hk, K = shape = q.shape
    H, V = v.shape[2:]
    if Hk < 1 or H % Hk != 0:
        raise ValueError("the q/k heads must divide v's heads")
    dtype, dt = q.dtype, _code(q, "q")
    out_shape = (B, T, H, V)
    pq, pk = _arg(q, "q", dev, dtype, shape), _arg(k, "k", dev, dtype, shape)
    pv = _arg(v, "v", dev, dtype, out_shape)
    per_token = decay.dim() == 3
    pd = _arg(decay, "decay", dev, _F32, (B, T, H) if per_token else (H,))
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
        code = lib.kda_decay_recurrent_fwd(pq, pk, pv, dt, pd, per_token, p0, p1, pcu, n_seqs, B, T, H, Hk, K, V, po,
                                           ot, _raw_stream(dev))
        if code:
            _kda._check("kda_decay_recurrent_fwd", code)
        return o, final_state
    if workspace is None:
        need = lib.kda_decay_chunk_workspace_bytes(dt, B, T, H, K, V, n_seqs)
        if need > 0:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    pw, size = None, 0
    if workspace is not None:
        pw, size = _arg(workspace, "workspace", dev, workspace.dtype, workspace.shape), workspace.nbytes
    if status is not None and status.numel() < 1:
        raise ValueError("status needs one int32 element")
    code = lib.kda_decay_chunk_fwd(pq, pk, pv, dt, pd, per_token, p0, p1, pcu, n_seqs, B, T, H, Hk, K, V, po, ot, pw,
                                   size, None if status is None else _arg(status, "status", dev, _I32, status.shape),
                                   _raw_stream(dev))
    if code:
        _kda._check("kda_decay_chunk_fwd", code)
    return o, final_state


def kda_decay_chunk_fwd(q, k, v, decay, initial_state=None, output_final_state=False, cu_seqlens=None, o=None,
                        final_state=None, workspace=None, stream=None, o_dtype=None, status=None):
    """Linear attention with a decay for each head, in chunks (prompts); (o, final_state or None).

        S_t = exp(decay_t) S_{t-1} + k_t v_t^T;   o_t = S_t^T q_t / sqrt(K)

    q, k [B, T, Hk, K], v [B, T, H, V] (float32 or bfloat16, Hk a divisor of H), ``decay`` float32
    natural log, [B, T, H] or [H]; states float32 [N, H, K, V].  ``o_dtype`` is q's dtype or
    torch.float32 (for bf16 inputs the exact one: no operand is rounded to bf16, about twice the time).  Packed sequences, in-place states, ``workspace``, ``status`` and ``stream`` as
    for kda_chunk_fwd."""
    return _decay(True, q, k, v, decay, initial_state, output_final_state, cu_seqlens, o, final_state, stream, o_dtype,
                  workspace, status)


def kda_decay_recurrent_fwd(q, k, v, decay, initial_state=None, output_final_state=False, cu_seqlens=None,
                            o=None, final_state=None, stream=None, o_dtype=None):
    """kda_decay_chunk_fwd's function token by token in float32 (single tokens; ``final_state`` may
    be ``initial_state``)."""
    return _decay(False, q, k, v, decay, initial_state, output_final_state, cu_seqlens, o, final_state, stream, o_dtype)


def kda_gated_norm_fwd(x, gate, weight=None, eps=1e-6, act=_kda.ACT_SIGMOID, out=None, stream=None):
    """y = x / sqrt(mean(x^2) + eps) * weight * act(gate) over the last dimension (one head's channels).

    x and gate of one shape and dtype (float32 or bfloat16), weight float32 [V] or None; ``out`` may
    be x or gate."""
    dev, here = _device(x)
    if stream is not None or not here:
        return _elsewhere(kda_gated_norm_fwd, x, stream, (x, gate, weight, eps, act, out))
    shape, dtype, dt = x.shape, x.dtype, _code(x, "x")
    V = shape[-1]
    px, pg = _arg(x, "x", dev, dtype, shape), _arg(gate, "gate", dev, dtype, shape)
    pw = _opt(weight, "weight", dev, _F32, (V,))
    if out is None:
        out = torch.empty_like(x)
        py = out.data_ptr()
    else:
        py = _arg(out, "out", dev, dtype, shape)
    code = _library().kda_gated_norm_fwd(px, pg, dt, pw, eps, act, x.numel() // V if V else 0, V, py, _raw_stream(dev))
    if code:
        _kda._check("kda_gated_norm_fwd", code)
    return out


def kda_block_norm_fwd(x, residual=None, post_weight=None, gate=None, pre_weight=None, scale=1.0,
                       channel_scale=None, eps=1e-6, act=_kda.ACT_SIGMOID, out=None, residual_out=None,
                       stream=None):
    """The norm around a block over the last dimension; returns (h, y).

        n = x [/ sqrt(mean(x^2) + eps) * post_weight] [* act(gate)]
        h = [residual +] scale [* channel_scale] * n
        y = h [/ sqrt(mean(h^2) + eps) * pre_weight]

    Each bracket is there when its tensor is given.  x, gate and y share a dtype, residual and h
    another (float32 or bfloat16 each; x's when there is no residual); weights and channel_scale
    are float32 [D].  ``residual_out`` (h) may be ``residual``."""
    dev, here = _device(x)
    if stream is not None or not here:
        return _elsewhere(kda_block_norm_fwd, x, stream, (x, residual, post_weight, gate, pre_weight, scale, channel_scale,
                                                          eps, act, out, residual_out))
    shape, dtype, dt = x.shape, x.dtype, _code(x, "x")
    D = shape[-1]
    per = (D,)
    like = residual if residual is not None else residual_out if residual_out is not None else x
    rt = _code(like, "residual")
    px, pr = _arg(x, "x", dev, dtype, shape), _opt(residual, "residual", dev, like.dtype, shape)
    pg = _opt(gate, "gate", dev, dtype, shape)
    pp, pn = _opt(post_weight, "post_weight", dev, _F32, per), _opt(pre_weight, "pre_weight", dev, _F32, per)
    pc = _opt(channel_scale, "channel_scale", dev, _F32, per)
    if residual_out is None:
        residual_out = torch.empty_like(like)
        ph = residual_out.data_ptr()
    else:
        ph = pr if residual_out is residual else _arg(residual_out, "residual_out", dev, like.dtype, shape)
    if out is None:
        out = torch.empty_like(x)
        py = out.data_ptr()
    else:
        py = _arg(out, "out", dev, dtype, shape)
    code = _library().kda_block_norm_fwd(px, dt, pr, rt, pp, pg, act, scale, pc, pn, eps, x.numel() // D if D else 0, D,
                                         ph, py, _raw_stream(dev))
    if code:
        _kda._check("kda_block_norm_fwd", code)
    return residual_out, out


def kda_short_conv_fwd(x, weight, bias=None, act=_kda.ACT_SILU, initial_state=None, output_final_state=False,
                       cu_seqlens=None, out=None, final_state=None, stream=None):
    """Causal convolution of each channel over its last W tokens; returns (y, final_state or None).

        y_t[d] = act(bias[d] + sum_w weight[d, w] x_{t-W+1+w}[d])

    x [B, T, D] (float32 or bfloat16), weight float32 [D, W] with 2 <= W <= 8, bias float32 [D] or
    None; states [N, W - 1, D] in x's dtype hold the last W - 1 inputs, the oldest first, and
    ``final_state`` may be ``initial_state``."""
    dev, here = _device(x)
    if stream is not None or not here:
        return _elsewhere(kda_short_conv_fwd, x, stream, (x, weight, bias, act, initial_state, output_final_state,
                                                          cu_seqlens, out, final_state))
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, D] and weight [D, W]")
    B, T, D = shape = x.shape
    W, dtype, dt = weight.shape[1], x.dtype, _code(x, "x")
    px, pw = _arg(x, "x", dev, dtype, shape), _arg(weight, "weight", dev, _F32, (D, W))
    pb = _opt(bias, "bias", dev, _F32, (D,))
    pcu, n_seqs, N = _packed(cu_seqlens, B, dev)
    state_shape = (N, W - 1, D)
    p0 = _opt(initial_state, "initial_state", dev, dtype, state_shape)
    if out is None:
        out = torch.empty_like(x)
        py = out.data_ptr()
    else:
        py = _arg(out, "out", dev, dtype, shape)
    if final_state is None and output_final_state:
        final_state = torch.empty(state_shape, device=x.device, dtype=dtype)
    p1 = p0 if final_state is initial_state else _opt(final_state, "final_state", dev, dtype, state_shape)
    code = _library().kda_short_conv_fwd(px, dt, pw, pb, act, W, p0, p1, pcu, n_seqs, B, T, D, py, _raw_stream(dev))
    if code:
        _kda._check("kda_short_conv_fwd", code)
    return out, final_state
