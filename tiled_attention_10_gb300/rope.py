"""RMS norm of query and key heads with the rotation by position, over torch CUDA
tensors (fa_qk_norm_rope and its backward; formulas in include/fa_api.h)."""
from __future__ import annotations

import functools
import struct

import torch

from .binding import FaError, fa_qk_norm_rope_bwd_workspace_size, load
from .paged import _call, _check, _dtype_of, _I32, _is, _no_tangents, _written, forward_ad

_F64 = torch.float64


def _sizes(q, k, layout):
    """(B, S, H, H_kv, D, sequence dimension before the heads') of q and k in a layout; packed
    [T, H, D] tensors are one batch."""
    if q.dim() == 3:
        (S, H, D), B, bsnd = q.shape, 1, True
        h_kv = k.shape[1] if k.dim() == 3 else -1
        want = (S, h_kv, D)
    elif layout == "BNSD":
        (B, H, S, D), bsnd = q.shape, False
        h_kv = k.shape[1]
        want = (B, h_kv, S, D)
    elif layout == "BSND":
        (B, S, H, D), bsnd = q.shape, True
        h_kv = k.shape[2] if k.dim() == 4 else -1
        want = (B, S, h_kv, D)
    else:
        raise ValueError(f"layout {layout!r}: BNSD or BSND")
    if k.shape != want:
        raise ValueError(f"k: shape {tuple(k.shape)} does not go with q's {tuple(q.shape)}")
    if k.dtype is not q.dtype:
        raise TypeError(f"k: {k.dtype}, q: {q.dtype}")
    if not q.is_cuda or k.get_device() != q.get_device():
        raise ValueError(f"q is on {q.device}, k on {k.device}: one CUDA device expected")
    return B, S, H, h_kv, D, bsnd


def _place(t, bsnd):
    """(t, address, batch, head and seq stride) of a tensor of q's or k's dims; t is a dense copy
    where the strides (of a transposed or expanded view, an odd offset) are none that the kernels
    take.  Dimensions of one element get a stride that passes the checks, whatever torch keeps."""
    ptr, st = t.data_ptr(), t.stride()
    if len(st) == 4:
        b, x, y, one = st
        if one == 1 and not ptr & 15 and not (b | x | y) & 7 and b > 0 and x > 0 and y > 0:
            return (t, ptr, b, y, x) if bsnd else (t, ptr, b, x, y)
    fine = st[-1] == 1 and ptr % 16 == 0
    for s, n in zip(st[:-1], t.shape):
        fine = fine and (n <= 1 or (s > 0 and s % 8 == 0))
    if not fine:
        t = t.clone(memory_format=torch.contiguous_format)
    st = [s if n > 1 else 8 for s, n in zip(t.stride(), t.shape)]
    if len(st) == 3:
        return t, t.data_ptr(), 8, st[1], st[0]
    return (t, t.data_ptr(), st[0], st[2], st[1]) if bsnd else (t, t.data_ptr(), st[0], st[1], st[2])


def _new(t, B, S, H, D, bsnd):
    """_place of a new dense tensor of t's shape."""
    o = torch.empty_like(t, memory_format=torch.contiguous_format)
    if bsnd:
        return o, o.data_ptr(), S * H * D or 8, D, H * D
    return o, o.data_ptr(), S * H * D or 8, S * D or 8, D


def _positions(positions, inv_freq, pair_axis, B, S, packed, index):
    """(positions [n_axes, B, S] or None, n_axes, rot_dim, pair_axis as bytes or None)."""
    if inv_freq is None:
        return None, 1, 0, None
    if inv_freq.dtype is not _F64 or inv_freq.dim() != 1 or inv_freq.get_device() != index or not inv_freq.is_contiguous():
        _check("inv_freq", inv_freq, _F64, (None,), index)
    rot = 2 * inv_freq.shape[0]
    if positions is None:
        raise ValueError("a rotation (inv_freq) needs positions")
    if positions.dtype is not _I32:
        raise TypeError(f"positions: {positions.dtype}, expected {_I32}")
    if positions.get_device() != index:
        raise ValueError(f"positions are on {positions.device}, expected cuda:{index}")
    n = positions.shape
    dims = len(n)
    axes = n[0] if dims == 3 or (packed and dims == 2) else 1
    if n != (S,) and (n != (axes, S) if packed else n != (B, S) and n != (axes, B, S)):
        raise ValueError(f"positions: shape {tuple(n)} does not go with {B} x {S} tokens")
    if dims == 1 and B > 1:
        positions = positions.expand(B, S)
    if not positions.is_contiguous():
        positions = positions.contiguous()
    if pair_axis is not None:
        pair_axis = bytes(pair_axis)
        if len(pair_axis) != rot // 2:
            raise ValueError(f"pair_axis: {len(pair_axis)} entries for {rot // 2} pairs")
    return positions, axes, rot, pair_axis


def _weight(name, w, D, dtype, index):
    """A weight's address (None for none)."""
    if w is None:
        return None
    if not _is(w, dtype, (D,), index):
        _check(name, w, dtype, (D,), index)
    return w.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


_four_strides = struct.Struct("12q").pack
_six_strides = struct.Struct("18q").pack


def _forward(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, pair_axis, interleaved, layout, out):
    dt = _dtype_of("q", q)
    B, S, H, H_kv, D, bsnd = _sizes(q, k, layout)
    index = q.get_device()
    pos, axes, rot, axis = _positions(positions, inv_freq, pair_axis, B, S, q.dim() == 3, index)
    wq = _weight("q_weight", q_weight, D, q.dtype, index)
    wk = _weight("k_weight", k_weight, D, q.dtype, index)
    q, qp, *qs = _place(q, bsnd)
    k, kp, *ks = _place(k, bsnd)
    given = out
    if out is None:
        qo, qop, *qos = _new(q, B, S, H, D, bsnd)
        ko, kop, *kos = _new(k, B, S, H_kv, D, bsnd)
        out = qo, ko
    else:
        for name, t, x in (("out[0]", out[0], q), ("out[1]", out[1], k)):
            if t.dtype is not x.dtype or t.shape != x.shape or t.get_device() != index or t.stride(-1) != 1:
                raise ValueError(f"{name}: expected {tuple(x.shape)} of {x.dtype} on {x.device}, the head dimension contiguous")
        qo, qop, *qos = _place(out[0], bsnd)
        ko, kop, *kos = _place(out[1], bsnd)
        if qo is not out[0] or ko is not out[1]:
            raise ValueError("out: strides and addresses have to be positive multiples of 16 bytes")
    _call("fa_qk_norm_rope", load().fa_qk_norm_rope, index, qp, kp, qop, kop, wq, wk, _ptr(pos), _ptr(inv_freq), B, S,
          H, H_kv, D, rot, axes, axis, 1 if interleaved else 0, 1 if norm else 0, eps,
          _four_strides(*qs, *ks, *qos, *kos), dt)
    if given is not None:
        _written(given)
    return out


@functools.lru_cache(None)
def _workspace_bytes(D):
    st, nbytes = fa_qk_norm_rope_bwd_workspace_size(D)
    if st != 0:
        raise FaError(st, "fa_qk_norm_rope_bwd_workspace_size")
    return nbytes


def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, *, q_weight=None, k_weight=None,
                          norm=True, eps=1e-6, pair_axis=None, interleaved=False, layout="BNSD",
                          weight_grads=True):
    """dq, dk, dq_weight, dk_weight of qk_norm_rope from the gradients of its
    outputs and its inputs.  A weight's gradient is None where the forward had no
    such weight, or with weight_grads=False."""
    if forward_ad._current_level >= 0:
        _no_tangents("qk_norm_rope_backward", dq_out, dk_out, q, k, q_weight, k_weight, inv_freq)
    dt = _dtype_of("q", q)
    B, S, H, H_kv, D, bsnd = _sizes(q, k, layout)
    index = q.get_device()
    pos, axes, rot, axis = _positions(positions, inv_freq, pair_axis, B, S, q.dim() == 3, index)
    wq = _weight("q_weight", q_weight, D, q.dtype, index)
    wk = _weight("k_weight", k_weight, D, q.dtype, index)
    for name, t, x in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if t.dtype is not x.dtype or t.shape != x.shape or t.get_device() != index:
            raise ValueError(f"{name}: expected {tuple(x.shape)} of {x.dtype} on {x.device}")
    dq_out, gqp, *gqs = _place(dq_out, bsnd)
    dk_out, gkp, *gks = _place(dk_out, bsnd)
    q, qp, *qs = _place(q, bsnd)
    k, kp, *ks = _place(k, bsnd)
    dq, dqp, *dqs = _new(q, B, S, H, D, bsnd)
    dk, dkp, *dks = _new(k, B, S, H_kv, D, bsnd)
    dqw = torch.empty_like(q_weight) if weight_grads and q_weight is not None else None
    dkw = torch.empty_like(k_weight) if weight_grads and k_weight is not None else None
    ws, nbytes = None, 0
    if dqw is not None or dkw is not None:
        nbytes = _workspace_bytes(D)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _call("fa_qk_norm_rope_bwd", load().fa_qk_norm_rope_bwd, index, gqp, gkp, qp, kp, dqp, dkp, wq, wk, _ptr(dqw),
          _ptr(dkw), _ptr(pos), _ptr(inv_freq), B, S, H, H_kv, D, rot, axes, axis, 1 if interleaved else 0,
          1 if norm else 0, eps, _six_strides(*gqs, *gks, *qs, *ks, *dqs, *dks), dt, _ptr(ws), nbytes)
    return dq, dk, dqw, dkw


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, norm, eps, pair_axis, interleaved, layout):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        ctx.opts = dict(norm=norm, eps=eps, pair_axis=pair_axis, interleaved=interleaved, layout=layout)
        return _forward(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, pair_axis, interleaved, layout, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
        dq, dk, dqw, dkw = qk_norm_rope_backward(
            dq_out, dk_out, q, k, positions, inv_freq, q_weight=q_weight, k_weight=k_weight,
            weight_grads=ctx.needs_input_grad[2] or ctx.needs_input_grad[3], **ctx.opts)
        return dq, dk, dqw, dkw, None, None, None, None, None, None, None


def qk_norm_rope(q, k, positions=None, inv_freq=None, *, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                 pair_axis=None, interleaved=False, layout="BNSD", out=None):
    """q_out, k_out: RMS norm of every head of q and k and the rotation of its
    first 2 * len(inv_freq) elements, in one pass; differentiable in q, k and the
    weights (fp16 / bf16; k may have fewer heads; any strides with the head
    dimension contiguous; packed [T, H, D] tensors too).

    positions: int32 [S], [B, S] or [n_axes, B, S] (packed: [T] or [n_axes, T]);
    inv_freq: float64, radians a position of each pair; pair_axis: the axis of
    each pair, a sequence of ints (default: the first).  Pairs are elements
    (i, i + rot / 2), or neighbours with `interleaved`.  norm=False leaves out
    the norm, inv_freq=None the rotation.  `out`: a pair to write into, which may
    be (q, k) themselves; only where no gradient is asked for.  Gradients of
    inv_freq and forward-mode derivatives (torch.autograd.forward_ad) are refused."""
    if forward_ad._current_level >= 0:
        _no_tangents("qk_norm_rope", q, k, q_weight, k_weight, inv_freq)
    if inv_freq is not None and inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("inv_freq has no gradient: detach it")
    wants = torch.is_grad_enabled() and (q.requires_grad or k.requires_grad
                                         or (q_weight is not None and q_weight.requires_grad)
                                         or (k_weight is not None and k_weight.requires_grad))
    if not wants:
        return _forward(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, pair_axis, interleaved, layout, out)
    if out is not None:
        raise ValueError("out cannot be given where gradients are wanted")
    return _QkNormRope.apply(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, pair_axis, interleaved, layout)
