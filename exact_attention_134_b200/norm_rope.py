"""Queries and keys between their projection and attention: the RMS norm of
every head and the rotation by the position, in one pass, and its gradients.

    q, k = qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight)
    q, k = norm_rope(q, k, positions, inv_freq, q_weight, k_weight)   # torch autograd

With xhat = x / sqrt(mean(x^2) + eps) and n = xhat * w, pair i = (a, b) of n
becomes (a cos t - b sin t, a sin t + b cos t), t = position * inv_freq[i]. q and
k are read where the projection left them (any strides that are multiples of 8
elements, channels contiguous) and written as attn_fwd (4-D) or attn_fwd_varlen
and attn_fwd_kv4 (3-D) read them.
"""
from __future__ import annotations

from . import _check, _current_device, _ll, _c_int, _stream_handle, lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(name, t, shape=None):
    """(batch, head, token) strides of a [B, H, N, d] or [total, H, d] tensor."""
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() not in (3, 4):
        raise ValueError(f"{name} must be a bf16 CUDA tensor [B, H, N, d] or [total, H, d]")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have contiguous channels")
    s = (0, s[1], s[0]) if t.dim() == 3 else s[:3]
    # the stride of an axis of one is never used: torch leaves anything there
    n = (1, t.shape[1], t.shape[0]) if t.dim() == 3 else t.shape[:3]
    return [x if m > 1 else 0 for x, m in zip(s, n)]


def _written(name, t):
    if any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
        raise ValueError(f"{name} is written to and must not be expanded")


def _shapes(q, k):
    if q.dim() != k.dim() or q.shape[-1] != k.shape[-1]:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)}")
    if q.dim() == 3:
        (N, Hq, d), B, Hkv = q.shape, 1, k.shape[1]
        same = k.shape[0] == N
    else:
        B, Hq, N, d = q.shape
        Hkv = k.shape[1]
        same = k.shape[0] == B and k.shape[2] == N
    if not same:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)}")
    return B, N, Hq, Hkv, d


def _rotation(positions, inv_freq, sections, B, N, packed, device):
    """(positions, axis stride, batch stride, inv_freq, sections, axes, rotary_dim) as the C call takes them."""
    import torch
    if inv_freq is None:
        if positions is not None or sections is not None:
            raise ValueError("positions and sections need inv_freq")
        return None, 0, 0, None, None, 0, 0
    if inv_freq.dtype != torch.float32 or inv_freq.device != device or not inv_freq.is_contiguous() or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a contiguous fp32 CUDA vector on the device of q")
    half = inv_freq.numel()
    sections = [half] if sections is None else [int(x) for x in sections]
    axes = len(sections)
    if not 1 <= axes <= 4 or min(sections) < 0 or sum(sections) != half:
        raise ValueError("sections must be 1 to 4 counts that add up to the length of inv_freq")
    p = positions
    if p is None or p.dtype != torch.int32 or p.device != device:
        raise ValueError("positions must be an int32 CUDA tensor on the device of q")
    want = ([(N,)] if packed else [(N,), (B, N)]) if axes == 1 else []
    want += [(axes, N)] if packed else [(axes, B, N), (axes, 1, N)]
    if tuple(p.shape) not in want:
        raise ValueError(f"positions must be one of {want}, not {tuple(p.shape)}")
    if N > 1 and p.stride(-1) != 1:
        raise ValueError("positions must be contiguous along the tokens")
    if p.dim() == 3:
        axis, batch = p.stride(0), p.stride(1) if p.shape[1] > 1 else 0
    elif p.dim() == 2:
        axis, batch = (p.stride(0), 0) if packed else (0, p.stride(0))
    else:
        axis, batch = 0, 0
    return p.data_ptr(), axis, batch, inv_freq.data_ptr(), (_c_int * axes)(*sections), axes, 2 * half


def _weights(q_weight, k_weight, d, device):
    import torch
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if q_weight is None:
        return 0
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t.dtype not in (torch.float32, torch.bfloat16) or t.device != device or tuple(t.shape) != (d,) or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 or bf16 CUDA vector [{d}] on the device of q")
    if q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must have the same type")
    return int(q_weight.dtype == torch.bfloat16)


def _same_device(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"all tensors of a call must be on one device: {t.device} and {device}")


def qk_norm_rope(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 sections=None, interleaved: bool = False, q_out=None, k_out=None):
    """RMS norm of every query and key head, then their rotation, in one launch.

    q: bf16 cuda [B, Hq, N, d] or packed [total, Hq, d], k with Hkv heads; any
    strides that are multiples of 8 elements, channels contiguous (views of the
    projection's result as it is). d = 64, 96, 128 or 256.
    positions: int32 cuda; [N] or [B, N] ([total] packed), or one row for each of
    the 1 to 4 axes of `sections` before that ([axes, B, N], [axes, 1, N] or
    [axes, total]).
    inv_freq: fp32 cuda [rotary_dim / 2] (rotary_dim a multiple of 16, at most d;
    the channels behind it are not rotated); None: norm only.
    sections: how many pairs turn with each axis, in order (time, height, width,
    say); None: all with one.
    q_weight, k_weight: fp32 or bf16 cuda [d]; both None: rotation only.
    interleaved: pairs of channels (2i, 2i + 1) instead of (i, i + rotary_dim / 2).
    Returns (q, k) in the shapes of q and k, contiguous unless q_out / k_out say
    otherwise; q_out may be q itself and k_out k (in place).
    """
    import torch
    sq, sk = _rows("q", q), _rows("k", k)
    B, N, Hq, Hkv, d = _shapes(q, k)
    packed = q.dim() == 3
    rot = _rotation(positions, inv_freq, sections, B, N, packed, q.device)
    bf16 = _weights(q_weight, k_weight, d, q.device)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
    k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device) if k_out is None else k_out
    _same_device(q.device, k, q_out, k_out)
    strides = sq + sk + _rows("q_out", q_out, q.shape) + _rows("k_out", k_out, k.shape)
    _written("q_out", q_out)
    _written("k_out", k_out)
    with _current_device(q.device):
        st = lib().attn_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
                                     (_ll * 12)(*strides), _ptr(q_weight), _ptr(k_weight), bf16, rot[0], rot[1], rot[2],
                                     rot[3], rot[4], rot[5], rot[6], int(bool(interleaved)), B, N, Hq, Hkv, d,
                                     float(eps), _stream_handle(q.device))
    _check(st, "attn_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd(q, k, dq_out, dk_out, positions=None, inv_freq=None, q_weight=None, k_weight=None,
                     eps: float = 1e-6, sections=None, interleaved: bool = False, workspace=None, dq=None, dk=None):
    """Gradients of qk_norm_rope: dq_out, dk_out are those of its results (bf16
    cuda, shapes and strides as for q and k), the other arguments its own; q and
    k may be None without a norm. Returns (dq, dk, dq_weight, dk_weight): bf16 in
    the shapes of q and k, and fp32 [d] (None without a norm), summed over
    batch, heads and tokens in a fixed order. dq may be dq_out itself and dk
    dk_out. `workspace` (uint8 cuda, attn_qk_norm_rope_bwd_workspace_size bytes)
    is allocated when not given.
    """
    import torch
    norm = q_weight is not None
    if not norm:
        q, k = dq_out, dk_out  # their shapes: nothing of q and k is read
    if q is None or k is None:
        raise ValueError("q and k are needed with a norm")
    sq, sk = _rows("q", q), _rows("k", k)
    B, N, Hq, Hkv, d = _shapes(q, k)
    packed = q.dim() == 3
    rot = _rotation(positions, inv_freq, sections, B, N, packed, q.device)
    bf16 = _weights(q_weight, k_weight, d, q.device)
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=k.dtype, device=k.device) if dk is None else dk
    _same_device(q.device, k, dq_out, dk_out, dq, dk, workspace)
    strides = sq + sk + _rows("dq_out", dq_out, q.shape) + _rows("dk_out", dk_out, k.shape) + \
        _rows("dq", dq, q.shape) + _rows("dk", dk, k.shape)
    _written("dq", dq)
    _written("dk", dk)
    dwq = dwk = None
    nbytes = 0
    if norm:
        dwq, dwk = torch.empty((2, d), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = torch.empty(int(lib().attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d)),
                                    dtype=torch.uint8, device=q.device)
        nbytes = workspace.numel() * workspace.element_size()
    else:
        workspace = None
    with _current_device(q.device):
        st = lib().attn_qk_norm_rope_bwd(q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(),
                                         dk.data_ptr(), (_ll * 18)(*strides), _ptr(q_weight), _ptr(k_weight), bf16,
                                         _ptr(dwq), _ptr(dwk), rot[0], rot[1], rot[2], rot[3], rot[4], rot[5], rot[6],
                                         int(bool(interleaved)), B, N, Hq, Hkv, d, float(eps), _ptr(workspace), nbytes,
                                         _stream_handle(q.device))
    _check(st, "attn_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


_AUTOGRAD_FN = None


def _readable(t):
    """A gradient as the kernel can read it (autograd hands over any strides)."""
    ok = t.stride(-1) == 1 and all(s % 8 == 0 for s in t.stride()[:-1]) and t.data_ptr() % 16 == 0
    return t if ok else t.contiguous()


def _autograd_fn():
    global _AUTOGRAD_FN
    if _AUTOGRAD_FN is None:
        import torch

        class _NormRope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, positions, inv_freq, q_weight, k_weight, eps, sections, interleaved):
                out = qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, sections, interleaved)
                norm = q_weight is not None
                ctx.save_for_backward(q if norm else None, k if norm else None, positions, inv_freq, q_weight, k_weight)
                ctx.args = (eps, sections, interleaved)
                return out

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dq_out, dk_out):
                q, k, positions, inv_freq, q_weight, k_weight = ctx.saved_tensors
                eps, sections, interleaved = ctx.args
                dq, dk, dwq, dwk = qk_norm_rope_bwd(q, k, _readable(dq_out), _readable(dk_out), positions, inv_freq,
                                                    q_weight, k_weight, eps, sections, interleaved)
                if q_weight is not None:
                    dwq, dwk = dwq.to(q_weight.dtype), dwk.to(k_weight.dtype)
                return dq, dk, None, None, dwq, dwk, None, None, None

        _AUTOGRAD_FN = _NormRope
    return _AUTOGRAD_FN


def norm_rope(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
              sections=None, interleaved: bool = False):
    """Differentiable qk_norm_rope (gradients of q, k, q_weight and k_weight):
    forward attn_qk_norm_rope, backward attn_qk_norm_rope_bwd. Same arguments."""
    return _autograd_fn().apply(q, k, positions, inv_freq, q_weight, k_weight, float(eps),
                                None if sections is None else tuple(sections), bool(interleaved))
