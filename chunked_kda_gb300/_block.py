"""The operators around the recurrence: decayed linear attention, gated and block norms, short
convolution.  As in the rest of the binding, the functions carry the C ABI's names and only check
and marshal their arguments.

A decode step calls each of them once per layer, so the checks are kept short.  Outputs and scratch
are allocated on the stream that the kernels run on (torch's current one unless ``stream`` is given).
"""
from __future__ import annotations

import torch

import chunked_kda_gb300 as _kda

_CODES = {torch.float32: 0, torch.bfloat16: 1}


def _dtype(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} is not float32 or bfloat16")
    return code


def _arg(t, name, device, dtype=None, shape=None):
    """The device address of a checked tensor (None stays None)."""
    if t is None:
        return None
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, all arguments on one device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.requires_grad:
        raise ValueError(f"{name} requires grad: this library is forward-only (inference)")
    return t.data_ptr()


class _On:
    """The device and stream of a call: both current inside the block, ``raw`` the stream's handle."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError("the inputs must be CUDA tensors")
        self.enter = None
        if stream is not None:
            self.enter = torch.cuda.stream(stream)
        elif device.index != torch.cuda.current_device():
            self.enter = torch.cuda.device(device)
        self.device, self.stream = device, stream

    def __enter__(self):
        if self.enter is not None:
            self.enter.__enter__()
        s = self.stream if self.stream is not None else torch.cuda.current_stream(self.device)
        return s.cuda_stream

    def __exit__(self, *exc):
        if self.enter is not None:
            self.enter.__exit__(*exc)


def _packed(cu_seqlens, B, device):
    """(pointer, n_seqs, logical sequences)."""
    if cu_seqlens is None:
        return None, 0, B
    p = _arg(cu_seqlens, "cu_seqlens", device, torch.int32)
    if B != 1:
        raise ValueError("packed mode (cu_seqlens given) needs B == 1")
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens needs at least one offset")
    n = cu_seqlens.numel() - 1
    return p, n, n


def kda_decay_chunk_workspace_bytes(dtype, B, T, H, K, V, n_seqs=0) -> int:
    """Scratch bytes of kda_decay_chunk_fwd for these sizes (n_seqs 0: dense)."""
    return int(_kda.load_library().kda_decay_chunk_workspace_bytes(_CODES[dtype], B, T, H, K, V, n_seqs))


def _decay(fn, q, k, v, decay, initial_state, output_final_state, cu_seqlens, o, final_state, stream, o_dtype,
           workspace=None, status=None):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must have four dimensions [B, T, heads, channels]")
    dev, (B, T, Hk, K), (H, V) = q.device, q.shape, v.shape[2:]
    if Hk < 1 or H % Hk != 0:
        raise ValueError("the q/k heads must divide v's heads")
    dt = _dtype(q, "q")
    with _On(dev, stream) as raw:
        pq, pk = _arg(q, "q", dev), _arg(k, "k", dev, q.dtype, q.shape)
        pv = _arg(v, "v", dev, q.dtype, (B, T, H, V))
        per_token = decay.dim() == 3
        pd = _arg(decay, "decay", dev, torch.float32, (B, T, H) if per_token else (H,))
        pcu, n_seqs, N = _packed(cu_seqlens, B, dev)
        p0 = _arg(initial_state, "initial_state", dev, torch.float32, (N, H, K, V))
        if o is None:
            o = torch.empty((B, T, H, V), device=dev, dtype=o_dtype or q.dtype)
        po = _arg(o, "o", dev, None, (B, T, H, V))
        if final_state is None and output_final_state:
            final_state = torch.empty((N, H, K, V), device=dev, dtype=torch.float32)
        p1 = _arg(final_state, "final_state", dev, torch.float32, (N, H, K, V))
        lib = _kda.load_library()
        args = (pq, pk, pv, dt, pd, int(per_token), p0, p1, pcu, n_seqs, B, T, H, Hk, K, V, po, _dtype(o, "o"))
        if fn == "kda_decay_chunk_fwd":
            need = lib.kda_decay_chunk_workspace_bytes(dt, B, T, H, K, V, n_seqs)
            if workspace is None and need > 0:
                workspace = torch.empty(need, device=dev, dtype=torch.uint8)
            size = 0 if workspace is None else workspace.numel() * workspace.element_size()
            args += (_arg(workspace, "workspace", dev), size, _arg(status, "status", dev, torch.int32))
        code = getattr(lib, fn)(*args, raw)
        if code:
            _kda._check(fn, code)
    return o, final_state


def kda_decay_chunk_fwd(q, k, v, decay, initial_state=None, output_final_state=False, cu_seqlens=None, o=None,
                        final_state=None, workspace=None, stream=None, o_dtype=None, status=None):
    """Linear attention with a decay for each head, in chunks (prompts); (o, final_state or None).

        S_t = exp(decay_t) S_{t-1} + k_t v_t^T;   o_t = S_t^T q_t / sqrt(K)

    q, k [B, T, Hk, K], v [B, T, H, V] (float32 or bfloat16, Hk a divisor of H), ``decay`` float32
    natural log, [B, T, H] or [H]; states float32 [N, H, K, V].  ``o_dtype`` is q's dtype or
    torch.float32.  Packed sequences, in-place states, ``workspace`` and ``status`` as for
    kda_chunk_fwd."""
    return _decay("kda_decay_chunk_fwd", q, k, v, decay, initial_state, output_final_state, cu_seqlens, o,
                  final_state, stream, o_dtype, workspace, status)


def kda_decay_recurrent_fwd(q, k, v, decay, initial_state=None, output_final_state=False, cu_seqlens=None,
                            o=None, final_state=None, stream=None, o_dtype=None):
    """kda_decay_chunk_fwd's function token by token in float32 (single tokens; ``final_state`` may
    be ``initial_state``)."""
    return _decay("kda_decay_recurrent_fwd", q, k, v, decay, initial_state, output_final_state, cu_seqlens, o,
                  final_state, stream, o_dtype)


def kda_gated_norm_fwd(x, gate, weight=None, eps=1e-6, act=_kda.ACT_SIGMOID, out=None, stream=None):
    """y = x / sqrt(mean(x^2) + eps) * weight * act(gate) over the last dimension (one head's channels).

    x and gate of one shape and dtype (float32 or bfloat16), weight float32 [V] or None; ``out`` may
    be x or gate."""
    dev = x.device
    dt = _dtype(x, "x")
    V = x.shape[-1]
    with _On(dev, stream) as raw:
        px, pg = _arg(x, "x", dev), _arg(gate, "gate", dev, x.dtype, x.shape)
        pw = _arg(weight, "weight", dev, torch.float32, (V,))
        if out is None:
            out = torch.empty_like(x)
        py = _arg(out, "out", dev, x.dtype, x.shape)
        code = _kda.load_library().kda_gated_norm_fwd(px, pg, dt, pw, eps, act, x.numel() // V if V else 0, V, py, raw)
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
    dev = x.device
    dt = _dtype(x, "x")
    D = x.shape[-1]
    rt = x.dtype if residual is None else residual.dtype
    if residual is None and residual_out is not None:
        rt = residual_out.dtype
    with _On(dev, stream) as raw:
        px, pr = _arg(x, "x", dev), _arg(residual, "residual", dev, None, x.shape)
        pg = _arg(gate, "gate", dev, x.dtype, x.shape)
        pp, pn = (_arg(w, n, dev, torch.float32, (D,)) for w, n in ((post_weight, "post_weight"), (pre_weight, "pre_weight")))
        pc = _arg(channel_scale, "channel_scale", dev, torch.float32, (D,))
        if residual_out is None:
            residual_out = torch.empty(x.shape, device=dev, dtype=rt)
        if out is None:
            out = torch.empty_like(x)
        ph, py = _arg(residual_out, "residual_out", dev, rt, x.shape), _arg(out, "out", dev, x.dtype, x.shape)
        code = _kda.load_library().kda_block_norm_fwd(px, dt, pr, _dtype(residual_out, "residual"), pp, pg, act, scale, pc,
                                                      pn, eps, x.numel() // D if D else 0, D, ph, py, raw)
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
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, D] and weight [D, W]")
    dev, (B, T, D), W = x.device, x.shape, weight.shape[1]
    dt = _dtype(x, "x")
    with _On(dev, stream) as raw:
        px, pw = _arg(x, "x", dev), _arg(weight, "weight", dev, torch.float32, (D, W))
        pb = _arg(bias, "bias", dev, torch.float32, (D,))
        pcu, n_seqs, N = _packed(cu_seqlens, B, dev)
        p0 = _arg(initial_state, "initial_state", dev, x.dtype, (N, W - 1, D))
        if out is None:
            out = torch.empty_like(x)
        py = _arg(out, "out", dev, x.dtype, x.shape)
        if final_state is None and output_final_state:
            final_state = torch.empty((N, W - 1, D), device=dev, dtype=x.dtype)
        p1 = _arg(final_state, "final_state", dev, x.dtype, (N, W - 1, D))
        code = _kda.load_library().kda_short_conv_fwd(px, dt, pw, pb, act, W, p0, p1, pcu, n_seqs, B, T, D, py, raw)
        if code:
            _kda._check("kda_short_conv_fwd", code)
    return out, final_state
