"""The paged key-value cache of the forward step whose logits the verify reads: its tensors and
their description for the library (specdec_kv_cache_t in include/specdec.h)."""
from __future__ import annotations

import dataclasses
from typing import Optional

from . import _native

PAGE_SIZES = (16, 32, 64, 128, 256)


@dataclasses.dataclass(frozen=True, eq=False)
class PagedCache:
    """k, v: [num_pages, num_kv_heads, page_size, head_dim] CUDA tensors with the same strides and the
    elements of a head contiguous (a cache laid out slot by slot is passed as a permuted view):
    bfloat16, float16, or float8_e4m3fn (uint8 is taken as its codes) with k_exp, v_exp, the
    [num_pages, num_kv_heads, page_size] uint8 exponents, biased by 127, of each token's head."""

    k: object
    v: object
    k_exp: Optional[object] = None
    v_exp: Optional[object] = None

    def __post_init__(self):
        import torch

        types = {torch.bfloat16: _native.SPECDEC_BF16, torch.float16: _native.SPECDEC_F16,
                 torch.float8_e4m3fn: _native.SPECDEC_E4M3, torch.uint8: _native.SPECDEC_E4M3}
        if self.k.dtype not in types or self.v.dtype != self.k.dtype:
            raise _native.SpecdecError(_native.SPECDEC_ERR_UNSUPPORTED, f"cache types {self.k.dtype}, {self.v.dtype}")
        # (a stride that is never taken counts as 0)
        stride, v_stride = (tuple(s if n > 1 else 0 for n, s in zip(t.shape, t.stride())) for t in (self.k, self.v))
        if self.k.dim() != 4 or self.k.shape != self.v.shape or stride != v_stride:
            raise ValueError("k and v must be [num_pages, num_kv_heads, page_size, head_dim] of the same strides")
        if stride[3] != 1:
            raise ValueError("the elements of a head must be contiguous")
        dtype = types[self.k.dtype]
        quantised = dtype == _native.SPECDEC_E4M3
        for name, e in (("k_exp", self.k_exp), ("v_exp", self.v_exp)):
            if (e is not None) != quantised:
                raise ValueError(f"{name} goes with an e4m3 cache")
            if quantised and (e.dtype != torch.uint8 or e.shape != self.k.shape[:3] or not e.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {tuple(self.k.shape[:3])}")
        for t in (self.k, self.v, self.k_exp, self.v_exp):
            if t is not None and t.device != self.k.device:
                raise ValueError("the cache's tensors must be on one device")

        n, heads, page, dim = self.k.shape
        struct = _native.KVCacheStruct(*(None if t is None else t.data_ptr() for t in (self.k, self.v, self.k_exp, self.v_exp)),
                                       dtype, n, page, heads, dim, stride[0], stride[1], stride[2])
        # the description is made once: the fields are frozen (the tensors' contents are not)
        for name, value in (("dtype", dtype), ("num_pages", n), ("num_kv_heads", heads), ("page_size", page), ("head_dim", dim),
                            ("device", self.k.get_device()), ("_struct", struct)):
            object.__setattr__(self, name, value)

    def struct(self):
        return self._struct


def alloc(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, dtype, device="cuda") -> PagedCache:
    """A cache of `num_pages` pages, one contiguous block for each page and head."""
    import torch

    shape = (num_pages, num_kv_heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype not in (torch.float8_e4m3fn, torch.uint8):
        return PagedCache(k, v)
    return PagedCache(k, v, *(torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2)))
