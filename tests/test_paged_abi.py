"""The paged-cache entry points refuse bad arguments on the host, before any CUDA call (no GPU needed; fake
aligned addresses, nothing is dereferenced), and the Python binding refuses tensors that do not fit."""
import ctypes

import pytest

from speculative_decoding_verification_specdec_gb300 import _native, build, kvcache

E = _native
P = 4096


@pytest.fixture(scope="module")
def lib():
    if build.needs_rebuild():
        build.build_library()
    return _native.load()


def rope_struct(**o):
    a = dict(freq=P, rot_dim=64, interleaved=0, amplitude=1.0)
    a.update(o)
    return _native.RopeStruct(*a.values())


def cache_struct(**o):
    a = dict(k=P, v=P, k_exp=None, v_exp=None, dtype=1, num_pages=8, page_size=16, num_kv_heads=2, head_dim=64,
             page_stride=2048, head_stride=1024, slot_stride=64)
    a.update(o)
    return _native.KVCacheStruct(*a.values())


def call_rope(lib, rope=(), **o):
    a = dict(x=P, out=P, dtype=1, rows=0, heads=4, dim=64, xr=256, xh=64, outr=256, outh=64, pos=P, cu=None, cached=None, B=0)
    a.update(o)
    r = rope_struct(**dict(rope))
    return lib.specdec_rope(a["x"], a["out"], a["dtype"], a["rows"], a["heads"], a["dim"], a["xr"], a["xh"], a["outr"], a["outh"],
                            ctypes.byref(r) if rope is not None else None, 0, a["pos"], a["cu"], a["cached"], a["B"], None)


def test_rope_refusals(lib):
    assert call_rope(lib) == E.SPECDEC_OK                                   # no rows: nothing launched
    for bad in (dict(rows=-1), dict(heads=0), dict(B=-1), dict(xr=-1), dict(outh=-64), dict(rows=1, x=None), dict(rows=1, out=None),
                dict(rows=1, pos=None, B=1), dict(rows=1, x=P + 1), dict(rows=1, pos=P + 2), dict(rows=1, pos=None, B=1, cu=P),
                dict(rope=dict(freq=None)), dict(rope=dict(freq=P + 4)), dict(rope=dict(rot_dim=63)), dict(rope=dict(rot_dim=0)),
                dict(rope=dict(rot_dim=66)), dict(rope=dict(interleaved=2))):
        assert call_rope(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=3), dict(dtype=9), dict(dim=63), dict(dim=0), dict(dim=258)):
        assert call_rope(lib, **bad) == E.SPECDEC_ERR_UNSUPPORTED, bad


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(k=P + 8), 1), (dict(num_pages=0), 1), (dict(num_kv_heads=0), 1),
              (dict(page_stride=-2048), 1), (dict(slot_stride=68), 1), (dict(page_stride=2 ** 39), 1), (dict(k_exp=P), 1), (dict(dtype=3), 1),
              (dict(dtype=3, k_exp=P), 1), (dict(dtype=3, k_exp=P, v_exp=P + 8), 1), (dict(dtype=0), 2), (dict(dtype=7), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
              (dict(page_size=512), 2), (dict(head_dim=8), 2), (dict(head_dim=72), 2), (dict(head_dim=144), 2)]


def call_write(lib, cache=(), rope=None, **o):
    a = dict(k=P, v=P, dtype=1, rows=0, rs=128, hs=64, pos=None, tab=P, mb=4, bs=4, cached=P, cu=P, B=2, status=None)
    a.update(o)
    c, r = cache_struct(**dict(cache)), None if rope is None else rope_struct(**rope)
    return lib.specdec_kv_write(a["k"], a["v"], a["dtype"], a["rows"], a["rs"], a["hs"], None if r is None else ctypes.byref(r), a["pos"],
                                ctypes.byref(c) if cache is not None else None, a["tab"], a["mb"], a["bs"], a["cached"], a["cu"], a["B"],
                                a["status"], None)


def test_kv_write_refusals(lib):
    assert call_write(lib) == E.SPECDEC_OK
    assert call_write(lib, rows=1, B=0) == E.SPECDEC_OK
    for bad, rc in BAD_CACHES:
        assert call_write(lib, cache=bad) == rc, bad
    assert lib.specdec_kv_write(P, P, 1, 1, 1, 1, None, None, None, P, 1, 1, P, P, 1, None, None) == E.SPECDEC_ERR_INVALID_ARG
    for bad in (dict(rows=-1), dict(B=-1), dict(mb=-1), dict(bs=-1), dict(rs=-1), dict(hs=-1), dict(rows=1, k=None), dict(rows=1, v=None),
                dict(rows=1, tab=None), dict(rows=1, cached=None), dict(rows=1, cu=None), dict(rows=1, k=P + 1), dict(rows=1, tab=P + 2),
                dict(rows=1, status=P + 2), dict(rope=dict(rot_dim=66)), dict(rope=dict(freq=None))):
        assert call_write(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    assert call_write(lib, dtype=3) == E.SPECDEC_ERR_UNSUPPORTED


def call_read(lib, cache=(), **o):
    a = dict(tab=P, mb=4, bs=4, first=None, cu=P, B=2, rows=0, ok=P, ov=P, dtype=1, r=128, h=64, status=None)
    a.update(o)
    c = cache_struct(**dict(cache))
    return lib.specdec_kv_read(ctypes.byref(c), a["tab"], a["mb"], a["bs"], a["first"], a["cu"], a["B"], a["rows"], a["ok"], a["ov"],
                               a["dtype"], a["r"], a["h"], a["status"], None)


def test_kv_read_refusals(lib):
    assert call_read(lib) == E.SPECDEC_OK
    for bad, rc in BAD_CACHES:
        assert call_read(lib, cache=bad) == rc, bad
    for bad in (dict(rows=-1), dict(B=-1), dict(mb=-1), dict(bs=-1), dict(r=-1), dict(h=-1), dict(rows=1, tab=None), dict(rows=1, cu=None),
                dict(rows=1, ok=None, ov=None), dict(rows=1, ok=P + 1), dict(rows=1, cu=P + 4), dict(rows=1, first=P + 1)):
        assert call_read(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    assert call_read(lib, dtype=3) == E.SPECDEC_ERR_UNSUPPORTED


def call_attention(lib, cache=(), **o):
    a = dict(q=P, dtype=1, rows=0, heads=8, qr=512, qh=64, tab=P, mb=4, bs=4, cached=P, cu=P, B=2, max_k=3, scale=0.125, window=0, out=P,
             outr=512, outh=64, lse=None, status=None, ws=P, wb=1 << 40, limit=-1)
    a.update(o)
    c = cache_struct(**dict(cache))
    return lib.specdec_paged_attention(a["q"], a["dtype"], a["rows"], a["heads"], a["qr"], a["qh"], ctypes.byref(c), a["tab"], a["mb"],
                                       a["bs"], a["cached"], a["cu"], a["B"], a["max_k"], a["scale"], a["window"], a["out"], a["outr"],
                                       a["outh"], a["lse"], a["status"], a["ws"], a["wb"], a["limit"], None)


def test_paged_attention_refusals(lib):
    assert call_attention(lib) == E.SPECDEC_OK
    assert call_attention(lib, rows=1, B=0) == E.SPECDEC_OK
    for bad, rc in BAD_CACHES:
        assert call_attention(lib, cache=bad) == rc, bad
    for bad in (dict(rows=-1), dict(B=-1), dict(mb=-1), dict(bs=-1), dict(max_k=-1), dict(max_k=33), dict(heads=0), dict(heads=7),
                dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(limit=-2), dict(limit=2000001), dict(qr=-8),
                dict(qr=4), dict(qh=65), dict(outh=12), dict(rows=1, q=None), dict(rows=1, out=None), dict(rows=1, tab=None),
                dict(rows=1, cached=None), dict(rows=1, cu=None), dict(rows=1, ws=None), dict(rows=1, q=P + 8), dict(rows=1, out=P + 2),
                dict(rows=1, ws=P + 8), dict(rows=1, lse=P + 2), dict(rows=1, wb=0)):
        assert call_attention(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=0), dict(dtype=3), dict(dtype=2), dict(cache=dict(dtype=2))):
        assert call_attention(lib, **bad) == E.SPECDEC_ERR_UNSUPPORTED, bad


def test_attention_workspace_size(lib):
    size = _native.paged_attention_workspace_size
    assert size(0, 3, 8, 2, 64) == 0 and size(4, -1, 8, 2, 64) == 0 and size(4, 3, 8, 0, 64) == 0
    assert 0 < size(1, 0, 8, 8, 64) <= size(1024, 8, 64, 8, 128) and size(64, 8, 64, 8, 128) % 16 == 0


def test_cache_tensors_that_do_not_fit():
    import torch

    k = torch.zeros((4, 2, 16, 32), dtype=torch.bfloat16)
    e = torch.full((4, 2, 16), 127, dtype=torch.uint8)
    c = kvcache.PagedCache(k, k.clone())
    assert (c.num_pages, c.page_size, c.dtype) == (4, 16, E.SPECDEC_BF16)
    q = torch.zeros((4, 2, 16, 32), dtype=torch.float8_e4m3fn)
    assert kvcache.PagedCache(q, q.clone(), e, e).dtype == E.SPECDEC_E4M3
    for bad in ((k, k[:3]), (k, k.half()), (k, k, e, e), (q, q), (q, q, e, e[:2]), (q, q, e.int(), e), (k[0], k[0]),
                (k, k.transpose(1, 2).contiguous().transpose(1, 2)), (k[..., ::2], k[..., ::2])):
        with pytest.raises((ValueError, E.SpecdecError)):
            kvcache.PagedCache(*bad)
    with pytest.raises(E.SpecdecError):
        kvcache.PagedCache(k.float(), k.float())


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    import torch

    x = torch.zeros((4, 2, 32), dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    table, _ = _native.rope_frequencies(32)
    c = kvcache.PagedCache(torch.zeros((4, 2, 16, 32), dtype=torch.bfloat16), torch.zeros((4, 2, 16, 32), dtype=torch.bfloat16))
    tab = torch.zeros((4, 1), dtype=torch.int32)
    for call in (lambda: _native.rope(x, x, table, 32, positions=i),                       # not on a GPU
                 lambda: _native.rope(x, x, table, 32, positions=i[:2]),
                 lambda: _native.rope(x, x, table, 32, positions=i.long()),
                 lambda: _native.rope(x, x[:3], table, 32, positions=i),
                 lambda: _native.rope(x, x, table, 32),
                 lambda: _native.kv_write(x, x[:, :, :16], c, tab, i, i, 4),
                 lambda: _native.kv_write(x[:, :1], x[:, :1], c, tab, i, i, 4),
                 lambda: _native.kv_write(x, x, c, tab[:2], i, i, 4),
                 lambda: _native.kv_write(x, x, c, tab, i, i, 4, status=i.long()),
                 lambda: _native.kv_read(c, tab, i.long(), 4, None, None),
                 lambda: _native.kv_read(c, tab, i, 4, x, x),
                 lambda: _native.paged_attention(x[..., :16], c, tab, i, i, 4, 0, x[..., :16], x),
                 lambda: _native.paged_attention(x, c, tab, i[:2], i, 4, 0, x, x),
                 lambda: _native.paged_attention(x, c, tab, i, i, 4, 0, x.float(), x),
                 lambda: _native.paged_attention(x, c, tab, i, i, 4, 0, x, x, lse=torch.zeros((4, 3)))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(E.SpecdecError):
        _native.rope_frequencies(32, scaling="by parts")


@pytest.mark.parametrize("scaling", ["linear", "by_parts"])
def test_frequencies_that_are_no_number_are_refused(scaling):
    # a factor whose reciprocal is beyond the largest double: infinite frequencies
    with pytest.raises(_native.SpecdecError):
        _native.rope_frequencies(32, scaling=scaling, factor=5e-324, original_len=1)
    _native.rope_frequencies(32, scaling=scaling, factor=1e-300, original_len=1)


def odd_strides(t, **at):
    """t with the strides of the given dimensions, all of size one, set to numbers that nothing else has."""
    s = list(t.stride())
    for d, x in at.items():
        assert t.shape[int(d[1:])] == 1
        s[int(d[1:])] = x
    return t.as_strided(t.shape, s)


def test_strides_that_are_never_taken_do_not_matter(lib):
    """Tensors of one row, one head, one page: the stride of a dimension of size one may be anything, in k and v alike. (On
    host tensors, whose device is what is refused once their shapes and strides have been taken.)"""
    import torch

    i, tab = torch.zeros(5, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32)
    for rows, heads in ((1, 2), (3, 1), (1, 1)):
        k = torch.zeros((rows, heads, 32), dtype=torch.bfloat16)
        v = odd_strides(k, **({"d0": 777} if rows == 1 else {}), **({"d1": 333} if heads == 1 else {}))
        c = kvcache.PagedCache(torch.zeros((4, heads, 16, 32), dtype=torch.bfloat16), torch.zeros((4, heads, 16, 32), dtype=torch.bfloat16))
        assert k.stride() != v.stride()
        with pytest.raises(ValueError, match="device"):
            _native.kv_write(k, v, c, tab, i, i, 1)
        with pytest.raises(ValueError, match="device"):
            _native.kv_read(c, tab, i.long(), 1, k, v)
        assert _native._heads("v", v)[1] == (0 if rows == 1 else heads * 32, 0 if heads == 1 else 32, 1)
    k = torch.zeros((1, 1, 16, 32), dtype=torch.float8_e4m3fn)
    e = torch.zeros((1, 1, 16), dtype=torch.uint8)
    s = kvcache.PagedCache(k, odd_strides(k, d0=777, d1=333), e, e).struct()
    assert (s.page_stride, s.head_stride, s.slot_stride) == (0, 0, 32)
    with pytest.raises(ValueError):                                  # a stride that is taken has to agree
        kvcache.PagedCache(torch.zeros((2, 1, 16, 32)).bfloat16(), torch.zeros((2, 2, 16, 32)).bfloat16()[:, :1])


def test_workspace_size_of_what_the_call_refuses_is_0(lib):
    size = _native.paged_attention_workspace_size
    assert size(4, 32, 8, 2, 128) > 0
    for bad in ((4, 33, 8, 2, 64), (4, 2 ** 31 - 1, 8, 2, 64), (4, 3, 7, 2, 64), (4, 3, 8, 3, 64), (4, 3, 8, 2, 8), (4, 3, 8, 2, 72), (4, 3, 8, 2, 144)):
        assert size(*bad) == 0, bad


def host_step():
    import torch

    x, i = torch.zeros((4, 2, 32), dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    c = kvcache.PagedCache(*(torch.zeros((4, 2, 16, 32), dtype=torch.bfloat16) for _ in range(2)))
    return x, c, torch.zeros((4, 1), dtype=torch.int32), i


def test_numbers_beyond_32_bits_are_refused(lib):
    """Not taken modulo 2^32 (a window of 2^32 + 5 would be one of 5)."""
    x, c, tab, i = host_step()
    for name, value in (("window", 2 ** 32), ("window", 2 ** 32 + 5), ("window", 2 ** 31), ("max_k", 2 ** 32 + 3), ("wait_limit_us", 2 ** 32 + 1)):
        kw = dict(max_k=3)
        kw[name] = value
        with pytest.raises((ValueError, E.SpecdecError), match=name):
            _native.paged_attention(x, c, tab, i, i, 4, out=x, workspace=x, **kw)
    for args in ((2 ** 32 + 4, 3, 8, 2, 64), (4, 2 ** 32 + 3, 8, 2, 64), (4, 3, 2 ** 32 + 8, 2, 64)):
        with pytest.raises(ValueError):
            _native.paged_attention_workspace_size(*args)
    for kw in (dict(rot_dim=2 ** 32 + 64), dict(rot_dim=64, scaling="by_parts", factor=8.0, original_len=2 ** 64 + 4096)):
        with pytest.raises(ValueError):
            _native.rope_frequencies(**kw)


def test_status_must_hold_whole_numbers(lib):
    """Status bits OR-ed into a tensor of another 32-bit type would read as something else."""
    import torch

    x, c, tab, i = host_step()
    for calls in (lambda st: _native.kv_write(x, x, c, tab, i, i, 4, status=st), lambda st: _native.kv_read(c, tab, i.long(), 4, x, x, status=st),
                  lambda st: _native.paged_attention(x, c, tab, i, i, 4, 0, x, x, status=st)):
        with pytest.raises(ValueError):
            calls(torch.zeros(4))
    with pytest.raises(ValueError, match="status must"):
        _native._status(torch.zeros(4), 4, -1)
    for fine in (torch.int32, torch.uint32):
        assert _native._status(torch.zeros(4, dtype=fine), 4, -1)


def test_rope_over_ragged_rows_names_their_number(lib):
    """Without B, cu_num_draft and cached_len described no request, and the call did nothing."""
    x, _, _, i = host_step()
    table, _ = _native.rope_frequencies(32)
    with pytest.raises(ValueError, match="and B"):
        _native.rope(x, x, table, 32, cu_num_draft=i, cached_len=i)
    with pytest.raises(ValueError, match="current device"):          # (a host tensor; the arguments themselves are complete)
        _native.rope(x, x, table, 32, cu_num_draft=i, cached_len=i, B=0)
