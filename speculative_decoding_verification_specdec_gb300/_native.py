"""ctypes binding of libspecdec.so (include/specdec.h). Argument marshalling only:
every step of the verify runs in the CUDA library. There is no fallback; a missing
library raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libspecdec.so")

SPECDEC_OK = 0
SPECDEC_ERR_INVALID_ARG = 1
SPECDEC_ERR_UNSUPPORTED = 2
SPECDEC_ERR_CUDA = 3
SPECDEC_ERR_TIMEOUT = 4
SPECDEC_F32 = 0
SPECDEC_BF16 = 1
SPECDEC_F16 = 2
SPECDEC_E4M3 = 3
SPECDEC_KMAX = 32
TELEMETRY_SHAPE = (4, SPECDEC_KMAX + 1)   # rows: drafts, eligible, accepted-through by position; histogram

ST_BAD_DRAFT_ID = 1
ST_EMPTY_MASK_ROW = 2
ST_BAD_TEMPERATURE = 4
ST_K_TOO_LARGE = 8
ST_BAD_OFFSETS = 16
ST_DEVICE_TIMEOUT = 32
ST_BAD_TOP_P = 64
ST_BAD_LENGTH = 128
ST_BAD_PAGE = 256
ST_BAD_SCORE = 512
ST_BAD_TARGET = 1024

EXPORTED = ("specdec_verify", "specdec_verify_noalloc", "specdec_wait", "specdec_status_string",
            "specdec_launch_config", "specdec_workspace_size", "specdec_ngram_propose",
            "specdec_bitmask_scatter", "specdec_set_launch_options", "specdec_rope_frequencies",
            "specdec_rope", "specdec_kv_write", "specdec_kv_read", "specdec_paged_attention_workspace_size",
            "specdec_paged_attention", "specdec_kv_fork", "specdec_top_logits_workspace_size", "specdec_top_logits",
            "specdec_distill", "specdec_distill_backward", "specdec_beam_select_workspace_size", "specdec_beam_select")
TOP_MAX = 128                           # SPECDEC_TOP_MAX
NGRAM_MAX_N = 64                        # SPECDEC_NGRAM_MAX_N
NOALLOC_MAX_REQUESTS = 16384            # SPECDEC_NOALLOC_MAX_REQUESTS

ROPE_SCALINGS = {None: 0, "linear": 1, "by_parts": 2}      # specdec_rope_scaling_t

_lib = None


class RopeStruct(ctypes.Structure):
    """specdec_rope_t"""
    _fields_ = [("freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("amplitude", ctypes.c_float)]


class KVCacheStruct(ctypes.Structure):
    """specdec_kv_cache_t"""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
                ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64)]


class SpecdecError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library. Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.specdec_verify.restype = ctypes.c_int
    lib.specdec_verify.argtypes = [vp, ctypes.c_int, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp,
                                   vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.specdec_verify_noalloc.restype = ctypes.c_int
    lib.specdec_verify_noalloc.argtypes = [vp, ctypes.c_int, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp,
                                           vp, vp, vp, vp, vp, vp, vp, vp]
    lib.specdec_ngram_propose.restype = ctypes.c_int
    lib.specdec_ngram_propose.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
    lib.specdec_bitmask_scatter.restype = ctypes.c_int
    lib.specdec_bitmask_scatter.argtypes = [vp, ctypes.c_int64, vp, i32, vp, i32, i32, vp, vp]
    lib.specdec_workspace_size.restype = ctypes.c_size_t
    lib.specdec_workspace_size.argtypes = [i32, i32]
    lib.specdec_wait.restype = ctypes.c_int
    lib.specdec_wait.argtypes = [vp, i32]
    lib.specdec_status_string.restype = ctypes.c_char_p
    lib.specdec_status_string.argtypes = [ctypes.c_int]
    lib.specdec_launch_config.restype = ctypes.c_int
    lib.specdec_launch_config.argtypes = [i32, i32, ctypes.c_int, vp, vp, vp, vp, vp, vp]
    lib.specdec_set_launch_options.restype = ctypes.c_int
    lib.specdec_set_launch_options.argtypes = [i32, i32, i32, i32, i32]
    i64, f64 = ctypes.c_int64, ctypes.c_double
    lib.specdec_rope_frequencies.restype = ctypes.c_int
    lib.specdec_rope_frequencies.argtypes = [i32, f64, ctypes.c_int, f64, i64, f64, f64, vp, vp]
    lib.specdec_rope.restype = ctypes.c_int
    lib.specdec_rope.argtypes = [vp, vp, ctypes.c_int, i32, i32, i32, i64, i64, i64, i64, vp, i32, vp, vp, vp, i32, vp]
    lib.specdec_kv_write.restype = ctypes.c_int
    lib.specdec_kv_write.argtypes = [vp, vp, ctypes.c_int, i32, i64, i64, vp, vp, vp, vp, i32, i64, vp, vp, i32, vp, vp]
    lib.specdec_kv_read.restype = ctypes.c_int
    lib.specdec_kv_read.argtypes = [vp, vp, i32, i64, vp, vp, i32, i64, vp, vp, ctypes.c_int, i64, i64, vp, vp]
    lib.specdec_paged_attention_workspace_size.restype = ctypes.c_size_t
    lib.specdec_paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.specdec_paged_attention.restype = ctypes.c_int
    lib.specdec_paged_attention.argtypes = [vp, ctypes.c_int, i32, i32, i64, i64, vp, vp, i32, i64, vp, vp, i32, i32,
                                            ctypes.c_float, i32, vp, i64, i64, vp, vp, vp, ctypes.c_size_t, i32, vp]
    lib.specdec_kv_fork.restype = ctypes.c_int
    lib.specdec_kv_fork.argtypes = [vp, vp, i32, i64, vp, i32, vp, vp, i32, vp, i64, vp, vp, vp]
    lib.specdec_top_logits_workspace_size.restype = ctypes.c_size_t
    lib.specdec_top_logits_workspace_size.argtypes = [i32, i32, ctypes.c_int]
    lib.specdec_top_logits.restype = ctypes.c_int
    lib.specdec_top_logits.argtypes = [vp, ctypes.c_int, i32, i32, i64, vp, f64, i32, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.specdec_distill.restype = ctypes.c_int
    lib.specdec_distill.argtypes = [vp, ctypes.c_int, i32, i32, i64, vp, vp, i32, f64, i32, vp, vp, vp, vp, i64, vp, vp]
    lib.specdec_distill_backward.restype = ctypes.c_int
    lib.specdec_distill_backward.argtypes = [vp, ctypes.c_int, i32, i32, i64, vp, vp, i32, f64, i32, vp, vp, vp, i64, vp, vp]
    lib.specdec_beam_select_workspace_size.restype = ctypes.c_size_t
    lib.specdec_beam_select_workspace_size.argtypes = [i32, i32, i32, ctypes.c_int, i32]
    lib.specdec_beam_select.restype = ctypes.c_int
    lib.specdec_beam_select.argtypes = [vp, ctypes.c_int, i32, i32, i32, i64, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().specdec_status_string(int(status)).decode()


def launch_config(V: int, dtype: int, B: int = 1024) -> dict:
    c, t, s, w, k, n = (ctypes.c_int32() for _ in range(6))
    rc = load().specdec_launch_config(int(B), int(V), int(dtype), ctypes.byref(c), ctypes.byref(t),
                                      ctypes.byref(s), ctypes.byref(w), ctypes.byref(k), ctypes.byref(n))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_launch_config")
    return {"ctas_per_request": c.value, "threads_per_cta": t.value, "smem_bytes": s.value,
            "slice_ids": w.value, "kernels_with_workspace": k.value, "split_requests": n.value}


_KERNELS = {None: -1, "stream": 0, "cluster": 1}


def set_launch_options(kernel: Optional[str] = None, ctas_per_request: Optional[int] = None,
                       schedule: Optional[bool] = None, wait_limit_us: Optional[int] = None,
                       split_requests: Optional[int] = None) -> None:
    """specdec_set_launch_options: None leaves a choice to the library."""
    rc = load().specdec_set_launch_options(_KERNELS[kernel], -1 if ctas_per_request is None else int(ctas_per_request),
                                           -1 if schedule is None else int(bool(schedule)),
                                           -1 if wait_limit_us is None else int(wait_limit_us),
                                           -1 if split_requests is None else int(split_requests))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_set_launch_options")


def workspace_size(B: int, V: int) -> int:
    return int(load().specdec_workspace_size(int(B), int(V)))


def _p(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr() if hasattr(t, "data_ptr") else int(t)


def _marshal(target_logits, logits_dtype, stream, tensors):
    import torch

    if logits_dtype is None:
        if target_logits.dtype == torch.bfloat16:
            logits_dtype = SPECDEC_BF16
        elif target_logits.dtype == torch.float32:
            logits_dtype = SPECDEC_F32
        else:
            raise SpecdecError(SPECDEC_ERR_UNSUPPORTED, f"logits dtype {target_logits.dtype}")
    for name, t in tensors:
        if t is not None and hasattr(t, "is_cuda"):
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    return int(logits_dtype), stream


def specdec_verify(target_logits, draft_ids, draft_probs, has_q, cu_num_draft, B: int, V: int, max_k: int,
                   bitmask, temperature, uniforms, exp_noise, out_tokens, out_num_accepted, counters,
                   status=None, diag_accept_prob=None, diag_row_stats=None, workspace=None, stream=None,
                   logits_dtype=None, telemetry=None, top_k=None, top_p=None) -> None:
    """Queue one verify on `stream` (default: torch's current stream). Tensors are CUDA tensors
    (or raw device addresses as ints, with logits_dtype given); raises SpecdecError on a
    non-zero status."""
    dt, stream = _marshal(target_logits, logits_dtype, stream, (
        ("target_logits", target_logits), ("draft_ids", draft_ids), ("draft_probs", draft_probs),
        ("has_q", has_q), ("cu_num_draft", cu_num_draft), ("bitmask", bitmask),
        ("temperature", temperature), ("uniforms", uniforms), ("exp_noise", exp_noise),
        ("out_tokens", out_tokens), ("out_num_accepted", out_num_accepted), ("counters", counters),
        ("status", status), ("diag_accept_prob", diag_accept_prob), ("diag_row_stats", diag_row_stats),
        ("telemetry", telemetry), ("workspace", workspace), ("top_k", top_k), ("top_p", top_p)))
    rc = load().specdec_verify(
        _p(target_logits), dt, _p(draft_ids), _p(draft_probs), _p(has_q), _p(cu_num_draft),
        int(B), int(V), int(max_k), _p(bitmask), _p(temperature), _p(top_k), _p(top_p), _p(uniforms), _p(exp_noise),
        _p(out_tokens), _p(out_num_accepted), _p(counters), _p(status), _p(diag_accept_prob),
        _p(diag_row_stats), _p(telemetry), _p(workspace), 0 if workspace is None else _nbytes(workspace), stream)
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_verify")


def specdec_verify_noalloc(target_logits, draft_ids, draft_probs, has_q, cu_num_draft, B: int, V: int,
                           max_k: int, bitmask, temperature, uniforms, exp_noise, out_tokens, out_num_accepted,
                           counters, status=None, diag_accept_prob=None, diag_row_stats=None, stream=None,
                           logits_dtype=None, telemetry=None, top_k=None, top_p=None) -> None:
    """specdec_verify with the library's own schedule scratch (no workspace argument)."""
    dt, stream = _marshal(target_logits, logits_dtype, stream, (
        ("target_logits", target_logits), ("draft_ids", draft_ids), ("draft_probs", draft_probs),
        ("has_q", has_q), ("cu_num_draft", cu_num_draft), ("bitmask", bitmask),
        ("temperature", temperature), ("uniforms", uniforms), ("exp_noise", exp_noise),
        ("out_tokens", out_tokens), ("out_num_accepted", out_num_accepted), ("counters", counters),
        ("status", status), ("diag_accept_prob", diag_accept_prob), ("diag_row_stats", diag_row_stats),
        ("telemetry", telemetry), ("top_k", top_k), ("top_p", top_p)))
    rc = load().specdec_verify_noalloc(
        _p(target_logits), dt, _p(draft_ids), _p(draft_probs), _p(has_q), _p(cu_num_draft),
        int(B), int(V), int(max_k), _p(bitmask), _p(temperature), _p(top_k), _p(top_p), _p(uniforms), _p(exp_noise),
        _p(out_tokens), _p(out_num_accepted), _p(counters), _p(status), _p(diag_accept_prob),
        _p(diag_row_stats), _p(telemetry), stream)
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_verify_noalloc")


def _nbytes(t) -> int:
    return t.numel() * t.element_size() if hasattr(t, "numel") else 0


def specdec_wait(stream=None, timeout_ms: int = -1) -> None:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = load().specdec_wait(stream, int(timeout_ms))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_wait")


def ngram_propose(tokens, cu_hist, B: int, min_n: int, max_n: int, k: int, out_drafts, out_num, out_match,
                  stream=None) -> None:
    """Queue the n-gram proposer (specdec_ngram_propose) on `stream` (default: torch's current
    stream); raises SpecdecError on a non-zero status."""
    import torch

    for name, t in (("tokens", tokens), ("cu_hist", cu_hist), ("out_drafts", out_drafts), ("out_num", out_num),
                    ("out_match", out_match)):
        if t is not None and hasattr(t, "is_cuda") and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = load().specdec_ngram_propose(_p(tokens), _p(cu_hist), int(B), int(min_n), int(max_n), int(k),
                                      _p(out_drafts), _p(out_num), _p(out_match), stream)
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_ngram_propose")


def bitmask_scatter(compact, compact_rows: int, constrained, n: int, cu_num_draft, B: int, V: int, bitmask,
                    stream=None) -> None:
    """Queue specdec_bitmask_scatter on `stream` (default: torch's current stream)."""
    import torch

    for name, t in (("compact", compact), ("constrained", constrained), ("cu_num_draft", cu_num_draft),
                    ("bitmask", bitmask)):
        if t is not None and hasattr(t, "is_cuda") and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = load().specdec_bitmask_scatter(_p(compact), int(compact_rows), _p(constrained), int(n), _p(cu_num_draft),
                                        int(B), int(V), _p(bitmask), stream)
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_bitmask_scatter")


# ------------------------------------------------------------------ rotary positions, paged cache, attention
#
# These calls sit in a decode loop, where a kernel takes a few microseconds: the checks below ask each tensor
# for each property once.

_torch = None
_FLOATS: dict = {}


def _lazy_torch():
    """torch and the library's numbers of its types, looked up once."""
    global _torch
    if _torch is None:
        import torch

        _FLOATS.update({torch.float32: SPECDEC_F32, torch.bfloat16: SPECDEC_BF16, torch.float16: SPECDEC_F16})
        _torch = torch
    return _torch


def _int32(name: str, x) -> int:
    """x as it is; ctypes would take a number beyond 32 bits modulo 2^32."""
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} = {x} is beyond 32 bits")
    return x


def _stream(stream, device: int) -> int:
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _dtype_of(t) -> int:
    n = _FLOATS.get(t.dtype)
    if n is None:
        raise SpecdecError(SPECDEC_ERR_UNSUPPORTED, f"dtype {t.dtype}")
    return n


def _at(name: str, t, device: int):
    """t's address (None: none); t must be on `device`, the current one, where the library launches."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")
    return t.data_ptr()


def _ints(name: str, t, dtype, rows: int, device: int):
    """Address of an integer tensor of at least `rows` elements (None: none)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] < rows or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {rows} elements, got {t.dtype} {tuple(t.shape)}")
    return _at(name, t, device)


def _status(status, B: int, device: int):
    if status is None:
        return None
    if status.dtype not in (_torch.int32, _torch.uint32) or status.dim() != 1 or status.shape[0] < B or not status.is_contiguous():
        raise ValueError("status must be a contiguous 32-bit integer tensor of B elements")
    return _at("status", status, device)


def _heads(name: str, t):
    """(shape, strides) of t, [rows, heads, head_dim] with the elements of a head contiguous. A stride that is never taken
    (one row, one head) counts as 0."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name} must be [rows, heads, head_dim] with the elements of a head contiguous")
    if shape[0] == 1 or shape[1] == 1:
        stride = (0 if shape[0] == 1 else stride[0], 0 if shape[1] == 1 else stride[1], 1)
    return shape, stride


def _like(name: str, t, shape, dtype):
    """Strides of t, which must have that shape and type."""
    got, stride = _heads(name, t)
    if got != shape or t.dtype is not dtype:
        raise ValueError(f"{name} has shape {tuple(got)} {t.dtype}, {tuple(shape)} {dtype} is needed")
    return stride


def _table(block_table, B: int, device: int):
    """(address, max_blocks, stride between the requests' rows)"""
    shape, stride = block_table.shape, block_table.stride()
    if block_table.dtype is not _torch.int32 or len(shape) != 2 or shape[0] < B or (shape[1] > 1 and stride[1] != 1):
        raise ValueError("block_table must be int32 [B, max_blocks], a request's row contiguous")
    return _at("block_table", block_table, device), shape[1], stride[0] if shape[0] > 1 else shape[1]


def _cache_of(cache, device: int):
    if cache.device != device:
        raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{device}")
    return cache.struct()


def rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """specdec_rope_frequencies: (table, amplitude). The table is a CPU int64 tensor [rot_dim / 2] that holds
    the unsigned 64-bit units; copy it to the device once. scaling: None, "linear" or "by_parts"."""
    torch = _lazy_torch()
    if scaling not in ROPE_SCALINGS:
        raise SpecdecError(SPECDEC_ERR_INVALID_ARG, f"rope scaling {scaling!r}")
    _int32("rot_dim", rot_dim)
    if not -2 ** 63 <= original_len < 2 ** 63:
        raise ValueError(f"original_len = {original_len} is beyond 64 bits")
    table = torch.zeros(max(int(rot_dim) // 2, 1), dtype=torch.int64)
    amplitude = ctypes.c_float()
    rc = load().specdec_rope_frequencies(int(rot_dim), float(theta), ROPE_SCALINGS[scaling], float(factor), int(original_len),
                                         float(beta_fast), float(beta_slow), table.data_ptr(), ctypes.byref(amplitude))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_rope_frequencies")
    return table, amplitude.value


def _rope_struct(device: int, freqs, rot_dim: int, interleaved: bool = False, amplitude: float = 1.0) -> RopeStruct:
    return RopeStruct(_ints("freqs", freqs, _torch.int64, rot_dim // 2, device), rot_dim, 1 if interleaved else 0, amplitude)


def rope(x, out, freqs, rot_dim: int, interleaved: bool = False, amplitude: float = 1.0, inverse: bool = False,
         positions=None, cu_num_draft=None, cached_len=None, B: Optional[int] = None, stream=None) -> None:
    """Queue specdec_rope: x rotated into out (which may be x), both [rows, heads, head_dim] with any row and
    head strides. Positions are given for every row, or follow from cu_num_draft, cached_len and B."""
    torch = _lazy_torch()
    device = x.get_device()
    shape, xs = _heads("x", x)
    os_ = _like("out", out, shape, x.dtype)
    i32 = torch.int32
    if positions is None and (cu_num_draft is None or cached_len is None or B is None):
        raise ValueError("rope needs positions, or cu_num_draft, cached_len and B")
    if B is None:
        B = 0
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    r = _rope_struct(current, freqs, rot_dim, interleaved, amplitude)
    rc = load().specdec_rope(_at("x", x, current), _at("out", out, current), _dtype_of(x), shape[0], shape[1], shape[2], xs[0], xs[1],
                             os_[0], os_[1], ctypes.byref(r), 1 if inverse else 0, _ints("positions", positions, i32, shape[0], current),
                             _ints("cu_num_draft", cu_num_draft, i32, B + 1, current),
                             _ints("cached_len", cached_len, i32, B, current), B, _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_rope")


def kv_write(k, v, cache, block_table, cached_len, cu_num_draft, B: int, rope=None, positions=None, status=None,
             stream=None) -> None:
    """Queue specdec_kv_write: the rows of k and v [rows, num_kv_heads, head_dim] (same strides) into `cache`
    (kvcache.PagedCache). rope: None, or the keyword arguments of a rotation of the keys: a dict of freqs,
    rot_dim and, optionally, interleaved and amplitude."""
    torch = _lazy_torch()
    device = k.get_device()
    shape, ks = _heads("k", k)
    if _like("v", v, shape, k.dtype) != ks:
        raise ValueError("k and v must have the same strides")
    if shape[1] != cache.num_kv_heads or shape[2] != cache.head_dim:
        raise ValueError(f"rows of {tuple(shape[1:])} do not go into a cache of {(cache.num_kv_heads, cache.head_dim)}")
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    i32 = torch.int32
    table, max_blocks, block_stride = _table(block_table, B, current)
    r = None if rope is None else ctypes.byref(_rope_struct(current, **rope))
    rc = load().specdec_kv_write(_at("k", k, current), _at("v", v, current), _dtype_of(k), shape[0], ks[0], ks[1], r,
                                 _ints("positions", positions, i32, shape[0], current), ctypes.byref(_cache_of(cache, current)),
                                 table, max_blocks, block_stride, _ints("cached_len", cached_len, i32, B, current),
                                 _ints("cu_num_draft", cu_num_draft, i32, B + 1, current), B, _status(status, B, current),
                                 _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_kv_write")


def kv_read(cache, block_table, cu_len, B: int, out_k, out_v, first=None, status=None, stream=None) -> None:
    """Queue specdec_kv_read: tokens first[b] .. of every request into rows cu_len[b] .. of out_k and out_v
    ([rows, num_kv_heads, head_dim], same strides; either may be None)."""
    torch = _lazy_torch()
    out = out_k if out_k is not None else out_v
    if out is None:
        raise ValueError("kv_read needs out_k or out_v")
    device = out.get_device()
    shape, strides = _heads("out_k", out)
    if out_k is not None and out_v is not None and _like("out_v", out_v, shape, out.dtype) != strides:
        raise ValueError("out_k and out_v must have the same strides")
    if shape[1] != cache.num_kv_heads or shape[2] != cache.head_dim:
        raise ValueError(f"rows of {tuple(shape[1:])} do not hold a cache of {(cache.num_kv_heads, cache.head_dim)}")
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    table, max_blocks, block_stride = _table(block_table, B, current)
    rc = load().specdec_kv_read(ctypes.byref(_cache_of(cache, current)), table, max_blocks, block_stride,
                                _ints("first", first, torch.int32, B, current), _ints("cu_len", cu_len, torch.int64, B + 1, current), B,
                                shape[0], _at("out_k", out_k, current), _at("out_v", out_v, current), _dtype_of(out), strides[0],
                                strides[1], _status(status, B, current), _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_kv_read")


def paged_attention_workspace_size(B: int, max_k: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    sizes = dict(B=B, max_k=max_k, num_heads=num_heads, num_kv_heads=num_kv_heads, head_dim=head_dim)
    return int(load().specdec_paged_attention_workspace_size(*(int(_int32(name, x)) for name, x in sizes.items())))


def paged_attention(q, cache, block_table, cached_len, cu_num_draft, B: int, max_k: int, out, workspace,
                    scale: Optional[float] = None, window: int = 0, lse=None, status=None,
                    wait_limit_us: Optional[int] = None, stream=None) -> None:
    """Queue specdec_paged_attention: q and out [rows, num_heads, head_dim], cache a kvcache.PagedCache, workspace a
    CUDA tensor of at least paged_attention_workspace_size(...) bytes. scale: default head_dim ** -0.5."""
    torch = _lazy_torch()
    device = q.get_device()
    shape, qs = _heads("q", q)
    os_ = _like("out", out, shape, q.dtype)
    if shape[2] != cache.head_dim:
        raise ValueError(f"head_dim {shape[2]} against the cache's {cache.head_dim}")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != shape[:2] or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {tuple(shape[:2])}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _int32("max_k", max_k)
    _int32("window", window)
    if wait_limit_us is not None:
        _int32("wait_limit_us", wait_limit_us)
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    i32 = torch.int32
    table, max_blocks, block_stride = _table(block_table, B, current)
    rc = load().specdec_paged_attention(_at("q", q, current), _dtype_of(q), shape[0], shape[1], qs[0], qs[1],
                                        ctypes.byref(_cache_of(cache, current)), table, max_blocks, block_stride,
                                        _ints("cached_len", cached_len, i32, B, current),
                                        _ints("cu_num_draft", cu_num_draft, i32, B + 1, current), B, max_k,
                                        shape[2] ** -0.5 if scale is None else scale, window, _at("out", out, current), os_[0], os_[1],
                                        _at("lse", lse, current), _status(status, B, current), _at("workspace", workspace, current),
                                        workspace.numel() * workspace.element_size(), -1 if wait_limit_us is None else wait_limit_us,
                                        _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_paged_attention")


def kv_fork(cache, block_table, lengths, parent, fresh, out_table, out_lengths=None, status=None, stream=None) -> None:
    """Queue specdec_kv_fork: row i of out_table [n, max_blocks] and out_lengths [n] go on from row parent[i] of block_table
    and lengths (-1: an empty row), with the begun page copied to page fresh[i] (-1, or fresh None: shared). out_table None:
    the tokens alone, for the further caches of one table."""
    torch = _lazy_torch()
    i32 = torch.int32
    device = parent.get_device()
    n = parent.shape[0] if parent.dim() == 1 else -1
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    sources = lengths.shape[0] if lengths.dim() == 1 else -1
    table, max_blocks, block_stride = _table(block_table, max(sources, 0), current)
    to, out_stride = None, max_blocks
    if out_table is not None:
        to, width, out_stride = _table(out_table, max(n, 0), current)
        if width != max_blocks:
            raise ValueError(f"out_table has {width} pages a row, block_table {max_blocks}")
    rc = load().specdec_kv_fork(ctypes.byref(_cache_of(cache, current)), table, max_blocks, block_stride,
                                _ints("lengths", lengths, i32, sources, current), sources, _ints("parent", parent, i32, n, current),
                                _ints("fresh", fresh, i32, n, current), n, to, out_stride,
                                _ints("out_lengths", out_lengths, i32, n, current), _status(status, n, current), _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_kv_fork")


# ------------------------------------------------------------------ rows of logits beside the verify


def _row_stride(name: str, t) -> int:
    """Row stride of t [rows, V] with the elements of a row contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be [rows, V] with the elements of a row contiguous")
    return stride[0] if shape[0] > 1 else shape[1]


def _rows_of(logits):
    """(rows, V, row stride)"""
    stride = _row_stride("logits", logits)
    rows, V = logits.shape
    if rows > 0x7fffffff or V > 0x7fffffff:
        raise ValueError(f"logits of shape {tuple(logits.shape)}: a size is beyond 32 bits")
    return rows, V, stride


def _matrix(name: str, t, dtype, shape, device: int):
    """Address of a contiguous tensor of that type and shape (None: none)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")
    return t.data_ptr()


def _workspace(t, device: int):
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return _at("workspace", t, device), t.numel() * t.element_size()


def _number_of(dtype) -> int:
    _lazy_torch()
    n = _FLOATS.get(dtype)
    if n is None:
        raise SpecdecError(SPECDEC_ERR_UNSUPPORTED, f"dtype {dtype}")
    return n


def top_logits_workspace_size(rows: int, V: int, dtype) -> int:
    """Bytes of workspace for logits of that torch type."""
    return int(load().specdec_top_logits_workspace_size(_int32("rows", rows), _int32("V", V), _number_of(dtype)))


def top_logits(logits, out_ids, out_logprobs, workspace, bitmask=None, temperature: float = 1.0, lse=None, status=None,
               stream=None) -> None:
    """Queue specdec_top_logits: the n best ids of every row of logits [rows, V], into out_ids int32 and out_logprobs float32
    [rows, n]. workspace: a CUDA tensor of at least top_logits_workspace_size(...) bytes."""
    torch = _lazy_torch()
    device = logits.get_device()
    rows, V, stride = _rows_of(logits)
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    n = out_ids.shape[1] if out_ids.dim() == 2 else -1
    space, size = _workspace(workspace, current)
    rc = load().specdec_top_logits(_at("logits", logits, current), _dtype_of(logits), rows, V, stride,
                                   _matrix("bitmask", bitmask, torch.int32, (rows, (V + 31) // 32), current), temperature, n,
                                   _matrix("out_ids", out_ids, torch.int32, (rows, n), current),
                                   _matrix("out_logprobs", out_logprobs, torch.float32, (rows, n), current),
                                   _matrix("lse", lse, torch.float32, (rows,), current), _status(status, rows, current), space, size,
                                   _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_top_logits")


def distill(logits, top_ids, top_logprobs, loss, weight=None, temperature: float = 1.0, rest: bool = True, stats=None, grad=None,
            status=None, stream=None) -> None:
    """Queue specdec_distill: the loss [rows] of the drafter's logits [rows, V] against top_ids and top_logprobs [rows, n]
    (top_logits' outputs on the target's rows), with the gradient into grad [rows, V] (which may be logits) where it is given,
    and stats [rows, 2] for distill_backward. rest: whether the mass that the list leaves is a category."""
    torch = _lazy_torch()
    device = logits.get_device()
    rows, V, stride = _rows_of(logits)
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    n = top_ids.shape[1] if top_ids.dim() == 2 else -1
    to, to_stride = _gradient(logits, grad, current)
    rc = load().specdec_distill(_at("logits", logits, current), _dtype_of(logits), rows, V, stride,
                                _matrix("top_ids", top_ids, torch.int32, (rows, n), current),
                                _matrix("top_logprobs", top_logprobs, torch.float32, (rows, n), current), n, temperature,
                                1 if rest else 0, _matrix("weight", weight, torch.float32, (rows,), current),
                                _matrix("loss", loss, torch.float32, (rows,), current),
                                _matrix("stats", stats, torch.float32, (rows, 2), current), to, to_stride,
                                _status(status, rows, current), _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_distill")


def _gradient(logits, grad, device: int):
    if grad is None:
        return None, 0
    if grad.shape != logits.shape or grad.dtype is not logits.dtype:
        raise ValueError(f"grad has shape {tuple(grad.shape)} {grad.dtype}, {tuple(logits.shape)} {logits.dtype} is needed")
    return _at("grad", grad, device), _row_stride("grad", grad)


def distill_backward(logits, top_ids, top_logprobs, stats, grad_loss, grad, temperature: float = 1.0, rest: bool = True, status=None,
                     stream=None) -> None:
    """Queue specdec_distill_backward: the gradient of distill's loss alone, times grad_loss [rows] (None: 1), from its stats."""
    torch = _lazy_torch()
    device = logits.get_device()
    rows, V, stride = _rows_of(logits)
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    n = top_ids.shape[1] if top_ids.dim() == 2 else -1
    to, to_stride = _gradient(logits, grad, current)
    rc = load().specdec_distill_backward(_at("logits", logits, current), _dtype_of(logits), rows, V, stride,
                                         _matrix("top_ids", top_ids, torch.int32, (rows, n), current),
                                         _matrix("top_logprobs", top_logprobs, torch.float32, (rows, n), current), n, temperature,
                                         1 if rest else 0, _matrix("stats", stats, torch.float32, (rows, 2), current),
                                         _matrix("grad_loss", grad_loss, torch.float32, (rows,), current), to, to_stride,
                                         _status(status, rows, current), _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_distill_backward")


def beam_select_workspace_size(B: int, beams: int, V: int, dtype, n: int) -> int:
    """Bytes of workspace for logits of that torch type."""
    return int(load().specdec_beam_select_workspace_size(_int32("B", B), _int32("beams", beams), _int32("V", V), _number_of(dtype),
                                                         _int32("n", n)))


def beam_select(logits, scores, out_rows, out_tokens, out_scores, workspace, bitmask=None, finished=None, end_token: int = -1,
                out_finished=None, status=None, stream=None) -> None:
    """Queue specdec_beam_select: the n best continuations (out_rows, out_tokens, out_scores [B, n]) of the beams of every
    request: logits [B * beams, V], scores [B, beams]. workspace: a CUDA tensor of at least
    beam_select_workspace_size(...) bytes."""
    torch = _lazy_torch()
    device = logits.get_device()
    rows, V, stride = _rows_of(logits)
    if scores.dim() != 2 or out_rows.dim() != 2:
        raise ValueError("scores must be [B, beams], out_rows [B, n]")
    (B, beams), n = scores.shape, out_rows.shape[1]
    if rows != B * beams:
        raise ValueError(f"{rows} rows of logits for {B} requests of {beams} beams")
    current = torch._C._cuda_getDevice() if device >= 0 else -2
    space, size = _workspace(workspace, current)
    rc = load().specdec_beam_select(_at("logits", logits, current), _dtype_of(logits), B, beams, V, stride,
                                    _matrix("bitmask", bitmask, torch.int32, (rows, (V + 31) // 32), current),
                                    _matrix("scores", scores, torch.float32, (B, beams), current),
                                    _matrix("finished", finished, torch.uint8, (B, beams), current), _int32("end_token", end_token), n,
                                    _matrix("out_rows", out_rows, torch.int32, (B, n), current),
                                    _matrix("out_tokens", out_tokens, torch.int32, (B, n), current),
                                    _matrix("out_scores", out_scores, torch.float32, (B, n), current),
                                    _matrix("out_finished", out_finished, torch.uint8, (B, n), current), _status(status, B, current),
                                    space, size, _stream(stream, current))
    if rc != SPECDEC_OK:
        raise SpecdecError(rc, "specdec_beam_select")
