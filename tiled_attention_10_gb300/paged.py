"""A paged serving step around attention, over torch CUDA tensors: slots of a
step's tokens, the 4-bit K/V cache and attention over it.

    slots = paged_slots(past, new, free_pages, block_table, page_size=64, total_q=rows)
    q, k  = qk_norm_rope(q, k, slots.positions, inv_freq, ...)
    kv4_write(k, v, slots.slot_map, cache)
    o, lse = paged_attention_kv4(q, cache, slots.cu_seqlens_q, slots.seqused_k, block_table,
                                 max_seqlen_q=..., total_k=...)

Allocation, checks and argument marshalling only; the formulas and limits stand
in include/fa_api.h.  Every call runs on the current stream of its tensors'
device, does not synchronise, and can be captured into a CUDA graph.
"""
from __future__ import annotations

import math
import struct
from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from .binding import CAUSAL, FA_DTYPE, FaError, fa_fwd_paged_kv4_workspace_size, load

_I32, _I64, _U8 = torch.int32, torch.int64, torch.uint8
_DTYPE = {torch.float16: FA_DTYPE["f16"], torch.bfloat16: FA_DTYPE["bf16"]}
_written = torch._C._increment_version      # (tensors): the kernels write by address, autograd is told
_two_strides = struct.Struct("6q").pack     # two fa_strides_t


def _stream(index):
    """The current stream of a device (torch.cuda.current_stream without the object)."""
    return torch._C._cuda_getCurrentRawStream(index)



# A decoding step makes several of these calls in the time its kernels take, so
# the checks are single expressions over cheap attributes; only a failed one
# goes through _check, which says what is wrong.


def _call(name, fn, index, *args):
    """fn(*args, stream) with device `index` current, on its current stream."""
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _stream(index))
    if st != 0:
        raise FaError(st, name)


def _is(t, dtype, shape, index):
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _check(name, t, dtype, shape, index):
    """Raises unless t is a dense tensor of this type and shape (None: any size) on CUDA
    device `index`."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{max(index, 0)}")
    if len(t.shape) != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _no_tangents(name, *tensors):
    """Raises where a tensor carries a forward-mode derivative: the kernels would drop it."""
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{name} has no forward-mode derivative")


def _no_gradients(name, *tensors):
    """Raises where a gradient of one of the tensors is asked for: there is none."""
    for t in tensors:
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} has no gradient: detach what goes in, or use torch.no_grad()")
    _no_tangents(name, *tensors)


def _dtype_of(name, t):
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


class PagedSlots(NamedTuple):
    """What paged_slots writes: int32 but for slot_map (int64)."""
    cu_seqlens_q: torch.Tensor   # [n_seqs + 1]
    seqused_k: torch.Tensor      # [n_seqs]
    positions: torch.Tensor      # [total_q]
    slot_map: torch.Tensor       # [total_q]
    pages_taken: torch.Tensor    # [1]


def paged_slots(past_k, new_q, free_pages, block_table, *, page_size, total_q, out=None):
    """The arrays of one paged step from its request lengths (fa_paged_slots).

    past_k, new_q: int32 [n_seqs], tokens each request holds and adds;
    free_pages: int32 page ids to hand out, from the front; block_table: int32
    [n_seqs, max_pages], its new entries are written.  total_q: rows of the step
    (at least the sum of new_q; rows behind it get slot -1, position 0).  `out`:
    a PagedSlots to write into.  pages_taken above free_pages' length says that
    the list ran out (the tokens without a page have slot -1)."""
    dev, n = past_k.get_device(), past_k.shape[0]
    if not (dev >= 0 and _is(past_k, _I32, (n,), dev) and _is(new_q, _I32, (n,), dev)):
        _check("past_k", past_k, _I32, (n,), dev)
        _check("new_q", new_q, _I32, (n,), dev)
    if free_pages.dtype is not _I32 or free_pages.get_device() != dev or free_pages.dim() != 1 or not free_pages.is_contiguous():
        _check("free_pages", free_pages, _I32, (None,), dev)
    if block_table.dim() != 2 or not _is(block_table, _I32, (n, block_table.shape[1]), dev):
        _check("block_table", block_table, _I32, (n, None), dev)
    given = out
    if out is None:
        i32 = {"dtype": _I32, "device": past_k.device}
        out = PagedSlots(torch.empty(n + 1, **i32), torch.empty(n, **i32), torch.empty(total_q, **i32),
                         torch.empty(total_q, dtype=_I64, device=past_k.device), torch.empty(1, **i32))
        cu, used, pos, slot, taken = out
    else:
        cu, used, pos, slot, taken = out
        if not (_is(cu, _I32, (n + 1,), dev) and _is(used, _I32, (n,), dev) and _is(pos, _I32, (total_q,), dev)
                and _is(slot, _I64, (total_q,), dev) and _is(taken, _I32, (1,), dev)):
            for name, t, dtype, size in (("cu_seqlens_q", cu, _I32, n + 1), ("seqused_k", used, _I32, n),
                                         ("positions", pos, _I32, total_q), ("slot_map", slot, _I64, total_q),
                                         ("pages_taken", taken, _I32, 1)):
                _check(name, t, dtype, (size,), dev)
    _call("fa_paged_slots", load().fa_paged_slots, dev, past_k.data_ptr(), new_q.data_ptr(), free_pages.data_ptr(),
          free_pages.shape[0], block_table.data_ptr(), n, block_table.shape[1], page_size, total_q, cu.data_ptr(),
          used.data_ptr(), pos.data_ptr(), slot.data_ptr(), taken.data_ptr())
    _written((block_table,) if given is None else (block_table, *given))
    return out


class KV4Cache:
    """A paged K/V cache of 4-bit values: value = e2m1 code * e4m3 scale of its
    16 elements * the tensor's descale.

    k_codes, v_codes: uint8 [num_pages, H_kv, page_size, D / 2]; k_scales,
    v_scales: float8_e4m3fn (or uint8) [num_pages, H_kv, page_size, D / 16].
    k_descale, v_descale: floats, or tensors of one fp32 on the cache's device: those
    are read by the kernels when they run (nothing synchronises, and a captured graph
    follows them).  A descale of largest value / (6 * 448) uses the scales' whole
    range."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "_descales", "_at", "_held", "_geometry")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_descale=1.0, v_descale=1.0):
        if k_codes.dim() != 4:
            raise ValueError(f"k_codes: shape {tuple(k_codes.shape)}, expected [num_pages, H_kv, page_size, D / 2]")
        pages, heads, rows, half = k_codes.shape
        index = k_codes.get_device()
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            _check(name, t, _U8, (pages, heads, rows, half), index)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            kind = _U8 if t.dtype == _U8 else torch.float8_e4m3fn
            _check(name, t, kind, (pages, heads, rows, half // 8), index)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self._geometry = (pages, heads, rows, 2 * half, index)
        self._set_descales(k_descale, v_descale)

    def _set_descales(self, *descales):
        got = []
        for name, x in zip(("k_descale", "v_descale"), descales):
            if isinstance(x, torch.Tensor):
                if x.numel() != 1:
                    raise ValueError(f"{name}: shape {tuple(x.shape)}, expected one number")
                _no_gradients(name, x)
                _check(name, x, torch.float32, x.shape, self._geometry[4])
                got.append(x.detach())
            else:
                got.append(float(x))
        self._descales, self._at = tuple(got), None
        # If either is a tensor, both as tensors (a float goes to the device once) and their places.
        if any(isinstance(x, torch.Tensor) for x in got):
            at = [x if isinstance(x, torch.Tensor) else torch.full((1,), x, dtype=torch.float32, device=self.device) for x in got]
            self._at, self._held = (at[0].data_ptr(), at[1].data_ptr()), at

    @classmethod
    def allocate(cls, num_pages, page_size, H_kv, D, device="cuda", k_descale=1.0, v_descale=1.0):
        """A cache of zeros."""
        shape = (num_pages, H_kv, page_size)
        codes = [torch.zeros(*shape, D // 2, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(*shape, D // 16, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1], k_descale, v_descale)

    @property
    def k_descale(self):
        return self._descales[0]

    @k_descale.setter
    def k_descale(self, x):
        self._set_descales(x, self._descales[1])

    @property
    def v_descale(self):
        return self._descales[1]

    @v_descale.setter
    def v_descale(self, x):
        self._set_descales(self._descales[0], x)

    @property
    def num_pages(self):
        return self._geometry[0]

    @property
    def H_kv(self):
        return self._geometry[1]

    @property
    def page_size(self):
        return self._geometry[2]

    @property
    def D(self):
        return self._geometry[3]

    @property
    def device(self):
        return self.k_codes.device


def _rows(name, t, heads, d, index):
    """The (batch, head, seq) strides of rows t [n, H_kv, D] with D contiguous."""
    if t.dim() != 3 or t.shape[1:] != (heads, d):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [n, {heads}, {d}]")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{index}")
    seq, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return 1, head if heads > 1 else d, seq if t.shape[0] > 1 else heads * d


def kv4_write(k, v, slot_map, cache):
    """Writes rows k, v [n_tokens, H_kv, D] (fp16 / bf16, any token and head
    strides of 16-byte multiples) into the cache's slots slot_map (int64
    [n_tokens]; -1 skips a row, the others must differ).  No gradient goes
    through the cache: rows that require one are refused (as by torch's out=)."""
    if k.requires_grad or v.requires_grad or forward_ad._current_level >= 0:
        _no_gradients("kv4_write", k, v)
    dt = _dtype_of("k", k)
    pages, heads, rows, d, index = cache._geometry
    n = k.shape[0]
    strides = _two_strides(*_rows("k", k, heads, d, index), *_rows("v", v, heads, d, index))
    if v.dtype is not k.dtype or v.shape[0] != n:
        raise ValueError("k and v must have the same type and shape")
    if not _is(slot_map, _I64, (n,), index):
        _check("slot_map", slot_map, _I64, (n,), index)
    lib, at = load(), cache._at
    fn, (kd, vd) = (lib.fa_kv4_write, cache._descales) if at is None else (lib.fa_kv4_write_devscale, at)
    _call("fa_kv4_write", fn, index, k.data_ptr(), v.data_ptr(), slot_map.data_ptr(),
          cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(), cache.v_scales.data_ptr(),
          kd, vd, n, heads, d, rows, pages, strides, dt)


def kv4_read(cache, slot_map, dtype=torch.bfloat16, out=None):
    """The rows k, v [n_tokens, H_kv, D] that the cache holds at slot_map, in
    `dtype` (or into `out`, a pair of dense tensors); a slot outside the cache
    reads as zeros."""
    pages, heads, rows, d, index = cache._geometry
    n = slot_map.shape[0]
    if not _is(slot_map, _I64, (n,), index):
        _check("slot_map", slot_map, _I64, (n,), index)
    given = out
    if out is None:
        out = (torch.empty((n, heads, d), dtype=dtype, device=slot_map.device),
               torch.empty((n, heads, d), dtype=dtype, device=slot_map.device))
    else:
        dtype = out[0].dtype
        for name, t in zip(("k", "v"), out):
            if not _is(t, dtype, (n, heads, d), index):
                _check(name, t, dtype, (n, heads, d), index)
    lib, at = load(), cache._at
    fn, (kd, vd) = (lib.fa_kv4_read, cache._descales) if at is None else (lib.fa_kv4_read_devscale, at)
    _call("fa_kv4_read", fn, index, cache.k_codes.data_ptr(), cache.k_scales.data_ptr(),
          cache.v_codes.data_ptr(), cache.v_scales.data_ptr(), slot_map.data_ptr(), out[0].data_ptr(),
          out[1].data_ptr(), kd, vd, n, heads, d, rows, pages, _dtype_of("out", out[0]))
    if given is not None:
        _written(given)
    return out


def paged_attention_kv4_workspace(q, cache, *, max_seqlen_q, n_seqs, total_k):
    """A workspace for paged_attention_kv4 with queries of q's shape: for any
    step with at most this many sequences, queries of one and keys in all."""
    st, nbytes = fa_fwd_paged_kv4_workspace_size(n_seqs, max_seqlen_q, total_k, q.shape[1], cache.H_kv, cache.D)
    if st != 0:
        raise FaError(st, "fa_fwd_paged_kv4_workspace_size")
    return torch.empty(nbytes, dtype=_U8, device=cache.device)


def paged_attention_kv4(q, cache, cu_seqlens_q, seqused_k, block_table, *, max_seqlen_q, total_k=None,
                        scale=None, causal="bottom_right", out=None, lse=None, workspace=None):
    """O, lse of packed queries q [total_q, H, D] over the 4-bit cache
    (fa_fwd_paged_kv4): sequence s has queries cu_seqlens_q[s] up to
    cu_seqlens_q[s + 1] and seqused_k[s] keys in the pages block_table[s].

    max_seqlen_q: at least every sequence's queries.  total_k: at least all
    sequences' keys together; it sizes the workspace of long queries (default:
    what the block table can hold).  lse is [H, total_q].  `workspace` (see
    paged_attention_kv4_workspace) saves the allocation; calls that may overlap
    need one each.  causal: "none", "top_left" or "bottom_right", as in the
    varlen calls (True says neither and is refused).  There is no gradient:
    queries that require one are refused."""
    if q.requires_grad or forward_ad._current_level >= 0:
        _no_gradients("paged_attention_kv4", q)
    if causal is True:
        raise ValueError('causal=True: say "bottom_right" (the default) or "top_left"')
    dt = _dtype_of("q", q)
    pages, heads, rows, d, index = cache._geometry
    total_q, H, _ = q.shape
    n, max_pages = block_table.shape
    if not (_is(q, q.dtype, (total_q, H, d), index) and _is(cu_seqlens_q, _I32, (n + 1,), index)
            and _is(seqused_k, _I32, (n,), index) and _is(block_table, _I32, (n, max_pages), index)):
        _check("q", q, q.dtype, (total_q, H, d), index)
        _check("cu_seqlens_q", cu_seqlens_q, _I32, (n + 1,), index)
        _check("seqused_k", seqused_k, _I32, (n,), index)
        _check("block_table", block_table, _I32, (n, max_pages), index)
    new_out, new_lse = out is None, lse is None
    if new_out:
        out = torch.empty_like(q)
    elif not _is(out, q.dtype, (total_q, H, d), index):
        _check("out", out, q.dtype, (total_q, H, d), index)
    if new_lse:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    elif not _is(lse, torch.float32, (H, total_q), index):
        _check("lse", lse, torch.float32, (H, total_q), index)
    if total_k is None:
        total_k = min(n * max_pages * rows, (1 << 31) - 256)   # (the most a call takes; short queries do not need it)
    if workspace is None:
        workspace = paged_attention_kv4_workspace(q, cache, max_seqlen_q=max_seqlen_q, n_seqs=n, total_k=total_k)
    elif workspace.dim() != 1 or not _is(workspace, _U8, workspace.shape, index):
        _check("workspace", workspace, _U8, (None,), index)
    lib, at = load(), cache._at
    fn, (kd, vd) = (lib.fa_fwd_paged_kv4, cache._descales) if at is None else (lib.fa_fwd_paged_kv4_devscale, at)
    _call("fa_fwd_paged_kv4", fn, index, q.data_ptr(), cache.k_codes.data_ptr(),
          cache.k_scales.data_ptr(), cache.v_codes.data_ptr(), cache.v_scales.data_ptr(), out.data_ptr(),
          lse.data_ptr(), cu_seqlens_q.data_ptr(), seqused_k.data_ptr(), block_table.data_ptr(), n, max_pages, rows,
          pages, total_q, max_seqlen_q, total_k, H, heads, d, 1.0 / math.sqrt(d) if scale is None else scale,
          CAUSAL[causal] if isinstance(causal, str) else int(causal), dt, kd, vd,
          workspace.data_ptr(), workspace.shape[0])
    if not (new_out and new_lse):
        _written((out, lse))
    return out, lse
