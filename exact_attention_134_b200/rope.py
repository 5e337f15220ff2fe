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

import struct

from . import _call, _changed, _check_scratch, lib

# arrays of long long and int as the C calls read them
_pack12, _pack18 = struct.Struct("12q").pack, struct.Struct("18q").pack
_pack_ints = [None] + [struct.Struct(f"{n}i").pack for n in range(1, 5)]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _shapes(q, k):
    """(B, N, Hq, Hkv, d) of q and k."""
    sq, sk = q.shape, k.shape
    if len(sq) == 4 and len(sk) == 4:
        B, Hq, N, d = sq
        Bk, Hkv, Nk, dk = sk
    elif len(sq) == 3 and len(sk) == 3:
        (N, Hq, d), (Nk, Hkv, dk), B, Bk = sq, sk, 1, 1
    else:
        raise ValueError("q and k must both be [B, H, N, d] or [total, H, d]")
    if B != Bk or N != Nk or d != dk:
        raise ValueError(f"shape mismatch: q {tuple(sq)} k {tuple(sk)}")
    return B, N, Hq, Hkv, d


def _rows(name, t, shape, index, written=False):
    """(batch, head, token) strides of a tensor of that shape on that device."""
    import torch
    if t.dtype is not torch.bfloat16 or t.get_device() != index or index < 0:
        raise ValueError(f"{name} must be a bf16 CUDA tensor [B, H, N, d] or [total, H, d] on the device of q")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have contiguous channels")
    # the stride of an axis of one is never used: torch leaves anything there
    if len(shape) == 4:
        B, H, N, _ = shape
        r = (s[0] if B > 1 else 0, s[1] if H > 1 else 0, s[2] if N > 1 else 0)
    else:
        B, (N, H, _) = 1, shape
        r = (0, s[1] if H > 1 else 0, s[0] if N > 1 else 0)
    if written and ((H > 1 and r[1] == 0) or (N > 1 and r[2] == 0) or (B > 1 and r[0] == 0)):
        raise ValueError(f"{name} is written to and must not be expanded")
    return r


def _rotation(positions, inv_freq, sections, B, N, packed, index):
    """(positions, axis stride, batch stride, inv_freq, sections, axes, rotary_dim) as the C call takes them."""
    import torch
    if inv_freq is None:
        if positions is not None or sections is not None:
            raise ValueError("positions and sections need inv_freq")
        return None, 0, 0, None, None, 0, 0
    if inv_freq.dtype is not torch.float32 or inv_freq.get_device() != index or inv_freq.dim() != 1 or \
            not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous fp32 CUDA vector on the device of q")
    half = inv_freq.shape[0]
    sections = (half,) if sections is None else [int(x) for x in sections]
    axes = len(sections)
    if not 1 <= axes <= 4 or min(sections) < 0 or sum(sections) != half:
        raise ValueError("sections must be 1 to 4 counts that add up to the length of inv_freq")
    p = positions
    if p is None or p.dtype is not torch.int32 or p.get_device() != index:
        raise ValueError("positions must be an int32 CUDA tensor on the device of q")
    shape, stride = tuple(p.shape), p.stride()
    if shape == ((axes, N) if packed else (axes, B, N)):
        axis, batch = stride[0], 0 if packed or B == 1 else stride[1]
    elif shape == (axes, 1, N) and not packed:
        axis, batch = stride[0], 0
    elif axes == 1 and shape == (N,):
        axis, batch = 0, 0
    elif axes == 1 and shape == (B, N) and not packed:
        axis, batch = 0, stride[0]
    else:
        raise ValueError(f"positions {shape} do not fit {axes} axes, batch {B} and {N} tokens")
    if N > 1 and stride[-1] != 1:
        raise ValueError("positions must be contiguous along the tokens")
    return p.data_ptr(), axis, batch, inv_freq.data_ptr(), _pack_ints[axes](*sections), axes, 2 * half


def _weights(q_weight, k_weight, d, index):
    """1 for bf16 weights, 0 for fp32 or none."""
    import torch
    if q_weight is None and k_weight is None:
        return 0
    if q_weight is None or k_weight is None:
        raise ValueError("q_weight and k_weight go together")
    dtype = q_weight.dtype
    if k_weight.dtype is not dtype:
        raise ValueError("q_weight and k_weight must have the same type")
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if (dtype is not torch.float32 and dtype is not torch.bfloat16) or t.get_device() != index or \
                t.shape != (d,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 or bf16 CUDA vector [{d}] on the device of q")
    return int(dtype is torch.bfloat16)


def _written(name, t, like, index):
    """The tensor to write a result in the shape of `like` to, a new contiguous one if None, and its strides."""
    import torch
    if t is not None:
        return t, _rows(name, t, like.shape, index, True)
    t = torch.empty_like(like) if like.is_contiguous() else torch.empty_like(like, memory_format=torch.contiguous_format)
    if t.dim() == 4:
        _, H, N, d = t.shape
        return t, (H * N * d, N * d, d)
    _, H, d = t.shape
    return t, (0, d, H * d)


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
    B, N, Hq, Hkv, d = _shapes(q, k)
    index = q.get_device()
    strides = _rows("q", q, q.shape, index) + _rows("k", k, k.shape, index)
    rot = _rotation(positions, inv_freq, sections, B, N, q.dim() == 3, index)
    bf16 = _weights(q_weight, k_weight, d, index)
    given = q_out, k_out
    q_out, sq = _written("q_out", q_out, q, index)
    k_out, sk = _written("k_out", k_out, k, index)
    _call("attn_qk_norm_rope", index, q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), _pack12(*strides, *sq, *sk),
          _ptr(q_weight), _ptr(k_weight), bf16, *rot, 1 if interleaved else 0, B, N, Hq, Hkv, d, float(eps))
    _changed(*given)
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
    B, N, Hq, Hkv, d = _shapes(q, k)
    index = q.get_device()
    strides = _rows("q", q, q.shape, index) + _rows("k", k, k.shape, index)
    rot = _rotation(positions, inv_freq, sections, B, N, q.dim() == 3, index)
    bf16 = _weights(q_weight, k_weight, d, index)
    strides += _rows("dq_out", dq_out, q.shape, index) + _rows("dk_out", dk_out, k.shape, index)
    given = dq, dk
    dq, sq = _written("dq", dq, q, index)
    dk, sk = _written("dk", dk, k, index)
    dwq = dwk = None
    nbytes = 0
    if norm:
        if bf16:
            dwq, dwk = (torch.empty_like(q_weight, dtype=torch.float32) for _ in range(2))
        else:
            dwq, dwk = torch.empty_like(q_weight), torch.empty_like(q_weight)
        if workspace is None:
            workspace = dwq.new_empty((lib().attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d) // 4,))
        else:
            _check_scratch("workspace", workspace, index)
        nbytes = workspace.nbytes
    else:
        workspace = None
    _call("attn_qk_norm_rope_bwd", index, q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(),
          dq.data_ptr(), dk.data_ptr(), _pack18(*strides, *sq, *sk), _ptr(q_weight), _ptr(k_weight), bf16, _ptr(dwq), _ptr(dwk),
          *rot, 1 if interleaved else 0, B, N, Hq, Hkv, d, float(eps), _ptr(workspace), nbytes)
    _changed(*given)
    return dq, dk, dwq, dwk


_AUTOGRAD_FN = None


def _readable(t):
    """A gradient as the kernel can read it (autograd hands over any strides, and
    views that begin anywhere: contiguous() would return such a one as it is)."""
    import torch
    ok = t.stride(-1) == 1 and all(s % 8 == 0 for s in t.stride()[:-1]) and t.data_ptr() % 16 == 0
    return t if ok else t.clone(memory_format=torch.contiguous_format)


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
    forward attn_qk_norm_rope, backward attn_qk_norm_rope_bwd. Same arguments.
    A step with its backward can be captured as torch asks for it: after warm-up
    on a side stream, with no eager graph of the same leaves alive."""
    return _autograd_fn().apply(q, k, positions, inv_freq, q_weight, k_weight, float(eps),
                                None if sections is None else tuple(sections), bool(interleaved))
