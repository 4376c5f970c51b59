"""RMS norm of query and key heads with the rotation by position, over torch CUDA
tensors (fa_qk_norm_rope and its backward; formulas in include/fa_api.h)."""
from __future__ import annotations

import torch

from .binding import FaError, Strides, fa_qk_norm_rope_bwd_workspace_size, load
from .paged import _check, _dtype_of, _on


class _Shape:
    """Sizes of q and k in a layout; packed [T, H, D] tensors are one batch, BSND."""

    __slots__ = ("B", "S", "H", "H_kv", "D", "bnsd")

    def __init__(self, q, k, layout):
        if q.dim() == 3:
            self.B, (self.S, self.H, self.D), self.bnsd = 1, q.shape, False
            want, self.H_kv = (self.S, None, self.D), k.shape[1]
        elif layout == "BNSD":
            (self.B, self.H, self.S, self.D), self.bnsd = q.shape, True
            want, self.H_kv = (self.B, None, self.S, self.D), k.shape[1]
        elif layout == "BSND":
            (self.B, self.S, self.H, self.D), self.bnsd = q.shape, False
            want, self.H_kv = (self.B, self.S, None, self.D), k.shape[2]
        else:
            raise ValueError(f"layout {layout!r}: BNSD or BSND")
        if len(k.shape) != len(want) or any(w is not None and w != n for w, n in zip(want, k.shape)):
            raise ValueError(f"k: shape {tuple(k.shape)} does not go with q's {tuple(q.shape)}")
        if k.dtype != q.dtype:
            raise TypeError(f"k: {k.dtype}, q: {q.dtype}")
        if k.device != q.device or not q.is_cuda:
            raise ValueError(f"q is on {q.device}, k on {k.device}: one CUDA device expected")

    def strides(self, t):
        """(batch, head, seq) of a tensor of q's or k's dims; dimensions of one
        element get a stride that passes the checks, whatever torch keeps."""
        st, n = t.stride(), t.shape
        if len(n) == 3:
            st, n = (8,) + st, (1,) + tuple(n)
        st = [s if m > 1 else 8 for s, m in zip(st, n)]
        return Strides(st[0], st[1], st[2]) if self.bnsd else Strides(st[0], st[2], st[1])


def _usable(t):
    """t, or a dense copy where its strides (a transposed or expanded view, an odd
    offset) are none that the kernels take."""
    st, n = t.stride(), t.shape
    fine = st[-1] == 1 and t.data_ptr() % 16 == 0
    for s, m in zip(st[:-1], n[:-1]):
        fine = fine and (m <= 1 or (s > 0 and s % 8 == 0))
    return t if fine else t.clone(memory_format=torch.contiguous_format)


def _positions(positions, inv_freq, pair_axis, sh, packed, dev):
    """(positions [n_axes, B, S] or None, n_axes, rot_dim, pair_axis as bytes or None)."""
    if inv_freq is None:
        return None, 1, 0, None
    _check("inv_freq", inv_freq, torch.float64, (None,), dev)
    rot = 2 * inv_freq.shape[0]
    if positions is None:
        raise ValueError("a rotation (inv_freq) needs positions")
    if positions.dtype != torch.int32:
        raise TypeError(f"positions: {positions.dtype}, expected {torch.int32}")
    if positions.device != dev:
        raise ValueError(f"positions are on {positions.device}, expected {dev}")
    axes, dims, n = 1, positions.dim(), tuple(positions.shape)
    if dims == 3 or (packed and dims == 2):
        axes = n[0]
    want = ((sh.S,), (axes, sh.S)) if packed else ((sh.S,), (sh.B, sh.S), (axes, sh.B, sh.S))
    if n not in want:
        raise ValueError(f"positions: shape {n} does not go with {sh.B} x {sh.S} tokens")
    if dims == 1 and sh.B > 1:
        positions = positions.expand(sh.B, sh.S)
    if not positions.is_contiguous():
        positions = positions.contiguous()
    if pair_axis is not None:
        pair_axis = bytes(pair_axis)
        if len(pair_axis) != rot // 2:
            raise ValueError(f"pair_axis: {len(pair_axis)} entries for {rot // 2} pairs")
    return positions, axes, rot, pair_axis


def _weights(q_weight, k_weight, sh, dtype, dev):
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check(name, w, dtype, (sh.D,), dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _forward(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, pair_axis, interleaved, layout, out):
    dt = _dtype_of("q", q)
    sh = _Shape(q, k, layout)
    dev = q.device
    pos, axes, rot, axis = _positions(positions, inv_freq, pair_axis, sh, q.dim() == 3, dev)
    _weights(q_weight, k_weight, sh, q.dtype, dev)
    q, k = _usable(q), _usable(k)
    if out is None:
        out = (torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=q.dtype, device=dev))
    else:
        for name, t, x in (("out[0]", out[0], q), ("out[1]", out[1], k)):
            if t.dtype != x.dtype or t.shape != x.shape or t.device != dev or t.stride(-1) != 1:
                raise ValueError(f"{name}: expected {tuple(x.shape)} of {x.dtype} on {dev}, the head dimension contiguous")
    strides = (Strides * 4)(sh.strides(q), sh.strides(k), sh.strides(out[0]), sh.strides(out[1]))
    with _on(dev):
        st = load().fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), out[0].data_ptr(), out[1].data_ptr(),
                                    _ptr(q_weight), _ptr(k_weight), _ptr(pos), _ptr(inv_freq), sh.B, sh.S,
                                    sh.H, sh.H_kv, sh.D, rot, axes, axis, int(bool(interleaved)),
                                    int(bool(norm)), eps, strides, dt,
                                    torch.cuda.current_stream(dev).cuda_stream)
    if st != 0:
        raise FaError(st, "fa_qk_norm_rope")
    return out


def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, *, q_weight=None, k_weight=None,
                          norm=True, eps=1e-6, pair_axis=None, interleaved=False, layout="BNSD",
                          weight_grads=True):
    """dq, dk, dq_weight, dk_weight of qk_norm_rope from the gradients of its
    outputs and its inputs.  A weight's gradient is None where the forward had no
    such weight, or with weight_grads=False."""
    dt = _dtype_of("q", q)
    sh = _Shape(q, k, layout)
    dev = q.device
    pos, axes, rot, axis = _positions(positions, inv_freq, pair_axis, sh, q.dim() == 3, dev)
    _weights(q_weight, k_weight, sh, q.dtype, dev)
    for name, t, x in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if t.dtype != x.dtype or t.shape != x.shape or t.device != dev:
            raise ValueError(f"{name}: expected {tuple(x.shape)} of {x.dtype} on {dev}")
    dq_out, dk_out, q, k = _usable(dq_out), _usable(dk_out), _usable(q), _usable(k)
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
    dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
    dqw = torch.empty_like(q_weight) if q_weight is not None and weight_grads else None
    dkw = torch.empty_like(k_weight) if k_weight is not None and weight_grads else None
    ws, nbytes = None, 0
    if dqw is not None or dkw is not None:
        st, nbytes = fa_qk_norm_rope_bwd_workspace_size(sh.D)
        if st != 0:
            raise FaError(st, "fa_qk_norm_rope_bwd_workspace_size")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    strides = (Strides * 6)(*(sh.strides(t) for t in (dq_out, dk_out, q, k, dq, dk)))
    with _on(dev):
        st = load().fa_qk_norm_rope_bwd(dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(),
                                        dq.data_ptr(), dk.data_ptr(), _ptr(q_weight), _ptr(k_weight),
                                        _ptr(dqw), _ptr(dkw), _ptr(pos), _ptr(inv_freq), sh.B, sh.S, sh.H,
                                        sh.H_kv, sh.D, rot, axes, axis, int(bool(interleaved)),
                                        int(bool(norm)), eps, strides, dt, _ptr(ws), nbytes,
                                        torch.cuda.current_stream(dev).cuda_stream)
    if st != 0:
        raise FaError(st, "fa_qk_norm_rope_bwd")
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
    be (q, k) themselves; only where no gradient is asked for."""
    wants = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, q_weight, k_weight))
    if not wants:
        return _forward(q, k, positions, inv_freq, q_weight, k_weight, norm, eps, pair_axis, interleaved, layout, out)
    if out is not None:
        raise ValueError("out cannot be given where gradients are wanted")
    return _QkNormRope.apply(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, pair_axis, interleaved, layout)
