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

import contextlib
import math
from typing import NamedTuple

import torch

from .binding import CAUSAL, FA_DTYPE, FaError, fa_fwd_paged_kv4_workspace_size, load, Strides

_DTYPE = {torch.float16: FA_DTYPE["f16"], torch.bfloat16: FA_DTYPE["bf16"]}


def _on(device):
    """The device guard of a call (nothing to do on the current device)."""
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _check(name, t, dtype, shape, device):
    """A dense CUDA tensor of this type and shape on this device (None: any size)."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if len(t.shape) != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dtype_of(name, t):
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return _DTYPE[t.dtype]


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
    dev = past_k.device
    n = past_k.shape[0]
    _check("past_k", past_k, torch.int32, (n,), dev)
    _check("new_q", new_q, torch.int32, (n,), dev)
    _check("free_pages", free_pages, torch.int32, (None,), dev)
    _check("block_table", block_table, torch.int32, (n, None), dev)
    if out is None:
        i32 = {"dtype": torch.int32, "device": dev}
        out = PagedSlots(torch.empty(n + 1, **i32), torch.empty(n, **i32), torch.empty(total_q, **i32),
                         torch.empty(total_q, dtype=torch.int64, device=dev), torch.empty(1, **i32))
    else:
        _check("cu_seqlens_q", out.cu_seqlens_q, torch.int32, (n + 1,), dev)
        _check("seqused_k", out.seqused_k, torch.int32, (n,), dev)
        _check("positions", out.positions, torch.int32, (total_q,), dev)
        _check("slot_map", out.slot_map, torch.int64, (total_q,), dev)
        _check("pages_taken", out.pages_taken, torch.int32, (1,), dev)
    with _on(dev):
        st = load().fa_paged_slots(past_k.data_ptr(), new_q.data_ptr(), free_pages.data_ptr(),
                                   free_pages.shape[0], block_table.data_ptr(), n,
                                   block_table.shape[1], page_size, total_q,
                                   out.cu_seqlens_q.data_ptr(), out.seqused_k.data_ptr(),
                                   out.positions.data_ptr(), out.slot_map.data_ptr(),
                                   out.pages_taken.data_ptr(),
                                   torch.cuda.current_stream(dev).cuda_stream)
    if st != 0:
        raise FaError(st, "fa_paged_slots")
    return out


class KV4Cache:
    """A paged K/V cache of 4-bit values: value = e2m1 code * e4m3 scale of its
    16 elements * the tensor's descale.

    k_codes, v_codes: uint8 [num_pages, H_kv, page_size, D / 2]; k_scales,
    v_scales: float8_e4m3fn (or uint8) [num_pages, H_kv, page_size, D / 16].
    k_descale, v_descale: floats.  A descale of largest value / (6 * 448) uses
    the scales' whole range."""

    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "k_descale", "v_descale")

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_descale=1.0, v_descale=1.0):
        dev = k_codes.device
        if k_codes.dim() != 4:
            raise ValueError(f"k_codes: shape {tuple(k_codes.shape)}, expected [num_pages, H_kv, page_size, D / 2]")
        pages, heads, rows, half = k_codes.shape
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            _check(name, t, torch.uint8, (pages, heads, rows, half), dev)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            kind = torch.uint8 if t.dtype == torch.uint8 else torch.float8_e4m3fn
            _check(name, t, kind, (pages, heads, rows, half // 8), dev)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_descale, self.v_descale = float(k_descale), float(v_descale)

    @classmethod
    def allocate(cls, num_pages, page_size, H_kv, D, device="cuda", k_descale=1.0, v_descale=1.0):
        """A cache of zeros."""
        shape = (num_pages, H_kv, page_size)
        codes = [torch.zeros(*shape, D // 2, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(*shape, D // 16, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1], k_descale, v_descale)

    @property
    def num_pages(self):
        return self.k_codes.shape[0]

    @property
    def H_kv(self):
        return self.k_codes.shape[1]

    @property
    def page_size(self):
        return self.k_codes.shape[2]

    @property
    def D(self):
        return self.k_codes.shape[3] * 2

    @property
    def device(self):
        return self.k_codes.device


def _rows(name, t, cache):
    """Checks rows [n, H_kv, D] with D contiguous; their (batch, head, seq) strides."""
    n, h, d = t.shape
    if h != cache.H_kv or d != cache.D:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [n, {cache.H_kv}, {cache.D}]")
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")
    seq, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return Strides(1, head if h > 1 else d, seq if n > 1 else h * d)


def kv4_write(k, v, slot_map, cache):
    """Writes rows k, v [n_tokens, H_kv, D] (fp16 / bf16, any token and head
    strides of 16-byte multiples) into the cache's slots slot_map (int64
    [n_tokens]; -1 skips a row, the others must differ)."""
    dt = _dtype_of("k", k)
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must have the same type and shape")
    dev = cache.device
    _check("slot_map", slot_map, torch.int64, (k.shape[0],), dev)
    strides = (Strides * 2)(_rows("k", k, cache), _rows("v", v, cache))
    pages, heads, rows, half = cache.k_codes.shape
    with _on(dev):
        st = load().fa_kv4_write(k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), cache.k_codes.data_ptr(),
                                 cache.k_scales.data_ptr(), cache.v_codes.data_ptr(),
                                 cache.v_scales.data_ptr(), cache.k_descale, cache.v_descale,
                                 k.shape[0], heads, 2 * half, rows, pages, strides, dt,
                                 torch.cuda.current_stream(dev).cuda_stream)
    if st != 0:
        raise FaError(st, "fa_kv4_write")


def kv4_read(cache, slot_map, dtype=torch.bfloat16, out=None):
    """The rows k, v [n_tokens, H_kv, D] that the cache holds at slot_map, in
    `dtype` (or into `out`, a pair of dense tensors); a slot outside the cache
    reads as zeros."""
    dev = cache.device
    pages, heads, rows, half = cache.k_codes.shape
    n = slot_map.shape[0]
    _check("slot_map", slot_map, torch.int64, (n,), dev)
    if out is None:
        out = tuple(torch.empty(n, heads, 2 * half, dtype=dtype, device=dev) for _ in range(2))
    else:
        for name, t in zip(("k", "v"), out):
            _check(name, t, out[0].dtype, (n, heads, 2 * half), dev)
    dt = _dtype_of("out", out[0])
    with _on(dev):
        st = load().fa_kv4_read(cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(),
                                cache.v_scales.data_ptr(), slot_map.data_ptr(), out[0].data_ptr(),
                                out[1].data_ptr(), cache.k_descale, cache.v_descale, n, heads, 2 * half,
                                rows, pages, dt, torch.cuda.current_stream(dev).cuda_stream)
    if st != 0:
        raise FaError(st, "fa_kv4_read")
    return out


def paged_attention_kv4_workspace(q, cache, *, max_seqlen_q, n_seqs, total_k):
    """A workspace for paged_attention_kv4 with queries of q's shape: for any
    step with at most this many sequences, queries of one and keys in all."""
    st, nbytes = fa_fwd_paged_kv4_workspace_size(n_seqs, max_seqlen_q, total_k, q.shape[1], cache.H_kv, cache.D)
    if st != 0:
        raise FaError(st, "fa_fwd_paged_kv4_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=cache.device)


def paged_attention_kv4(q, cache, cu_seqlens_q, seqused_k, block_table, *, max_seqlen_q, total_k=None,
                        scale=None, causal="bottom_right", out=None, lse=None, workspace=None):
    """O, lse of packed queries q [total_q, H, D] over the 4-bit cache
    (fa_fwd_paged_kv4): sequence s has queries cu_seqlens_q[s] up to
    cu_seqlens_q[s + 1] and seqused_k[s] keys in the pages block_table[s].

    max_seqlen_q: at least every sequence's queries.  total_k: at least all
    sequences' keys together; it sizes the workspace of long queries (default:
    what the block table can hold).  lse is [H, total_q].  `workspace` (see
    paged_attention_kv4_workspace) saves the allocation; calls that may overlap
    need one each."""
    dt = _dtype_of("q", q)
    dev = cache.device
    pages, heads, rows, half = cache.k_codes.shape
    total_q, H, D = q.shape
    _check("q", q, q.dtype, (total_q, H, 2 * half), dev)
    n, max_pages = block_table.shape
    _check("cu_seqlens_q", cu_seqlens_q, torch.int32, (n + 1,), dev)
    _check("seqused_k", seqused_k, torch.int32, (n,), dev)
    _check("block_table", block_table, torch.int32, (n, max_pages), dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check("out", out, q.dtype, (total_q, H, D), dev)
    if lse is None:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=dev)
    else:
        _check("lse", lse, torch.float32, (H, total_q), dev)
    if total_k is None:
        total_k = n * max_pages * rows
    if workspace is None:
        workspace = paged_attention_kv4_workspace(q, cache, max_seqlen_q=max_seqlen_q, n_seqs=n, total_k=total_k)
    else:
        _check("workspace", workspace, torch.uint8, (None,), dev)
    with _on(dev):
        st = load().fa_fwd_paged_kv4(
            q.data_ptr(), cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(),
            cache.v_scales.data_ptr(), out.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(),
            seqused_k.data_ptr(), block_table.data_ptr(), n, max_pages, rows, pages, total_q,
            max_seqlen_q, total_k, H, heads, D, 1.0 / math.sqrt(D) if scale is None else scale,
            CAUSAL[causal] if isinstance(causal, str) else int(causal), dt, cache.k_descale,
            cache.v_descale, workspace.data_ptr(), workspace.shape[0],
            torch.cuda.current_stream(dev).cuda_stream)
    if st != 0:
        raise FaError(st, "fa_fwd_paged_kv4")
    return out, lse
