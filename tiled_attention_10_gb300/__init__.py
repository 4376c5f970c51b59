"""FlashAttention for one GB300 (sm_103a): Python binding of libfa_b200.

The compute path is the C-ABI library ``libfa_b200.so`` (hand-written CUDA for
sm_103a): forward (dense, grouped-query, split-KV, varlen, paged K/V, strided)
and backward, and what a serving or training step needs around it (paged
slots, query/key norm with rotation, a 4-bit K/V cache and attention over it).
This package only marshals arguments; it loads the library lazily on the first
call and raises if it is missing.
"""
from .binding import (FA_DTYPE, FA_LAYOUT, FA_STATUS, FaError, attention, attention_backward,
                      fa_bwd, fa_fwd, fa_fwd_gqa, fa_last_device_error, fa_status_string,
                      flash_attention, load)

_PAGED = ("KV4Cache", "PagedSlots", "kv4_read", "kv4_write", "paged_attention_kv4",
          "paged_attention_kv4_workspace", "paged_slots")
_ROPE = ("qk_norm_rope", "qk_norm_rope_backward")

__all__ = ["FA_DTYPE", "FA_LAYOUT", "FA_STATUS", "FaError", "attention", "attention_backward",
           "fa_bwd", "fa_fwd", "fa_fwd_gqa", "fa_last_device_error", "fa_status_string",
           "flash_attention", "load", *_PAGED, *_ROPE]


def __getattr__(name):
    """The torch-level operators, imported on first use (the binding itself does
    not need torch to load)."""
    if name in _PAGED:
        from . import paged as m
    elif name in _ROPE:
        from . import rope as m
    else:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    globals()[name] = value = getattr(m, name)
    return value
