"""Plain 64-bit implementations of the operators around paged attention (numpy, CPU), written
from the formulas in include/fa_api.h, and the error bounds their kernels' arithmetic gives.
(Test infrastructure.)"""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U32 = 2.0 ** -24      # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half a step of the type's smallest numbers."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------- slots
def slots(past_k, new_q, free, table, ps, total_q):
    """(cu_q, used, table, positions, slot_map, taken) of one step, by loops over requests."""
    table = table.copy()
    n, cols = table.shape
    cap = cols * ps
    cu, used, pos, slot, taken, rows = [0], [], [], [], 0, 0
    for s in range(n):
        past, new = min(max(int(past_k[s]), 0), cap), max(int(new_q[s]), 0)
        held = min(past + new, cap)
        for col in range(-(-past // ps), -(-held // ps)):
            table[s, col] = free[taken] if taken < len(free) else -1
            taken += 1
        for i in range(min(new, total_q - rows)):
            p = past + i
            page = int(table[s, p // ps]) if p < cap else -1
            pos.append(p)
            slot.append(page * ps + p % ps if page >= 0 else -1)
        rows = min(rows + new, total_q)
        cu.append(rows)
        used.append(held)
    pad = total_q - rows
    return (np.array(cu, np.int32), np.array(used, np.int32), table, np.array(pos + [0] * pad, np.int32),
            np.array(slot + [-1] * pad, np.int64), taken)


# ---------------------------------------------------------------- 4-bit cache
def e4m3_values():
    c = np.arange(128)
    e, m = c >> 3, (c & 7).astype(np.float64)
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[127] = np.nan
    return v


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0, ties to the even index, saturated."""
    i = np.clip(np.searchsorted(grid, x, side="right") - 1, 0, len(grid) - 2)
    lo, hi = grid[i], grid[i + 1]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 1))
    return np.where(up, i + 1, i)


def to_cache(x, descale):
    """codes [..., D / 2], scales [..., D / 16] (uint8) of x [..., D] in float64; NaN and
    infinities by the documented rule."""
    d = x.shape[-1]
    g = float(np.float32(descale))
    y = x.reshape(*x.shape[:-1], d // 16, 16).astype(np.float64)
    a = np.abs(y)
    amax = np.where(np.isnan(a), 0.0, a).max(-1)
    s = nearest(np.minimum(amax / (6 * g), 1e30), e4m3_values()[:127])
    step = (e4m3_values()[s] * g)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(np.isnan(a), 1e9, np.minimum(a, 1e300) / step)
    code = nearest(np.where(step > 0, z, 0.0), E2M1)
    code = np.where(step > 0, code | (np.signbit(y) * 8), 0).reshape(*x.shape[:-1], d // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).astype(np.uint8), s.astype(np.uint8)


def values(codes, scales, descale):
    """The float64 values of codes [..., D / 2] and scales [..., D / 16]."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2)
    v = E2M1[c & 7] * np.where(c >= 8, -1.0, 1.0)
    full = np.concatenate((e4m3_values(), -e4m3_values()))
    return v * np.repeat(full[scales], 16, -1) * float(np.float32(descale))


def gather(codes, scales, descale, pages, n, num_pages):
    """Keys (or values) [H_kv, n, D] of a sequence with these pages; pages outside read as zeros."""
    ps = codes.shape[2]
    got = []
    for i in range(-(-n // ps)):
        p = int(pages[i])
        if 0 <= p < num_pages:
            got.append(values(codes[p], scales[p], descale))
        else:
            got.append(np.zeros((codes.shape[1], ps, codes.shape[3] * 2)))
    return np.concatenate(got, 1)[:, :n] if got else np.zeros((codes.shape[1], 0, codes.shape[3] * 2))


# ---------------------------------------------------------------- attention
def attend(q, k, v, scale, causal):
    """One sequence: q [n, H, D], k and v [H_kv, m, D] -> O [n, H, D], lse [H, n], and the two
    sums the error bounds need: sum p |v| [n, H, D] and max over keys of scale * sum |q k|."""
    n, H, D = q.shape
    hk, m = k.shape[0], k.shape[1]
    O, L = np.zeros((n, H, D)), np.full((H, n), -np.inf)
    PV, A = np.zeros((n, H, D)), np.zeros((H, n))
    for h in range(H):
        kk, vv = k[h // (H // hk)], v[h // (H // hk)]
        s = scale * (q[:, h] @ kk.T)
        reach = abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T)
        i, j = np.arange(n)[:, None], np.arange(m)[None, :]
        seen = np.ones((n, m), bool) if causal == 0 else j <= i + (0 if causal == 1 else m - n)
        s = np.where(seen, s, -np.inf)
        rows = seen.any(1) if m else np.zeros(n, bool)
        if not rows.any():
            continue
        top = s[rows].max(1, keepdims=True)
        p = np.exp(s[rows] - top)
        l = p.sum(1, keepdims=True)
        O[rows, h] = p / l @ vv
        PV[rows, h] = p / l @ np.abs(vv)
        L[h, rows] = (top + np.log(l))[:, 0]
        A[h, rows] = reach[rows].max(1)
    return O, L, PV, A


def attend_bounds(O, PV, A, n_keys, D, dtype, p_step, v_step):
    """Bounds on |O - exact| and |lse - exact|: P rounded to a type of half step p_step, V to one
    of v_step (0: exact), O once; scores in fp32 (D products and the scaling) and 2^x to 2 ulp."""
    score = (D + 8) * U32 * A + 4 * U32 * (A + 32)     # absolute, natural log units
    rel = 2 * score.T[:, :, None] + p_step + v_step + 64 * U32 + n_keys * 2.0 ** -24 / 32
    bo = PV * rel + n_keys * 2.0 ** -33 * np.abs(PV).max(initial=0.0) + half_step(dtype) * np.abs(O) * (1 + rel) + tiny(dtype)
    return bo * 1.001, score + (n_keys / 32 + 64) * U32


# ---------------------------------------------------------------- norm and rotation
def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, ang, interleaved):
    """x [..., D] with its first pairs turned by ang [..., rot / 2]."""
    y = x.copy()
    rot = 2 * ang.shape[-1]
    if rot:
        a, b = pairs(rot, interleaved)
        c, s = np.cos(ang), np.sin(ang)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def partner_size(x, rot, interleaved):
    """|x| of each element and its partner together."""
    y = np.abs(x)
    if rot:
        a, b = pairs(rot, interleaved)
        both = y[..., a] + y[..., b]
        y[..., a], y[..., b] = both, both
    return y


def angles(positions, inv_freq, pair_axis):
    """[B, S, 1, rot / 2] from positions [n_axes, B, S]: exact products, reduced modulo a turn."""
    pos = np.asarray(positions, dtype=np.int64)
    ax = np.zeros(len(inv_freq), int) if pair_axis is None else np.asarray(pair_axis)
    # far positions: the product in two parts of 26 bits, each exact in float64
    f = np.asarray(inv_freq, np.float64)
    hi = np.float64(np.float32(f))
    lo = f - hi
    p = pos[ax].astype(np.float64).transpose(1, 2, 0)
    return (np.fmod(p * hi, 2 * math.pi) + p * lo)[:, :, None, :]


def norm_rope(x, w, ang, norm, eps, interleaved):
    """x [B, S, H, D] float64 -> output."""
    u = x
    if norm:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    return turn(u, ang, interleaved)


def norm_rope_bound(x, w, ang, norm, eps, interleaved, dtype):
    """Bound on |kernel - norm_rope|: one rounding of the result; fp32 before it (a sum of D
    squares, the root, three products, a turn whose sine and cosine are good to 2^-21)."""
    D = x.shape[-1]
    u = x
    if norm:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    big = partner_size(u, 2 * ang.shape[-1], interleaved)
    y = turn(u, ang, interleaved)
    return half_step(dtype) * np.abs(y) * 1.01 + tiny(dtype) + big * ((D if norm else 0) / 2 + 24) * U32


def norm_rope_grad(dy, x, w, ang, norm, eps, interleaved):
    """(dx, dw or None) in float64."""
    g = turn(dy, -ang, interleaved)
    if not norm:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h, u = x * r, g * (1.0 if w is None else w)
    return r * (u - h * (u * h).mean(-1, keepdims=True)), (g * h).sum((0, 1, 2))


def norm_rope_grad_bounds(dy, x, w, ang, norm, eps, interleaved, dtype):
    """Bounds on dx and dw, as norm_rope_bound; dw adds its terms in fp32 in some order."""
    D, rot = x.shape[-1], 2 * ang.shape[-1]
    dx, dw = norm_rope_grad(dy, x, w, ang, norm, eps, interleaved)
    g = partner_size(dy, rot, interleaved)
    if not norm:
        return half_step(dtype) * np.abs(dx) * 1.01 + tiny(dtype) + g * 24 * U32, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h, u = np.abs(x * r), g * (1.0 if w is None else np.abs(w))
    size = r * (u + h * (u * h).mean(-1, keepdims=True))
    bx = half_step(dtype) * np.abs(dx) * 1.01 + tiny(dtype) + size * (2 * D + 48) * U32
    terms = (g * h).sum((0, 1, 2))
    count = x.shape[0] * x.shape[1] * x.shape[2]
    bw = half_step(dtype) * np.abs(dw) * 1.01 + tiny(dtype) + terms * (D / 2 + 48 + count) * U32
    return bx, bw
