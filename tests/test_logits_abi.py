"""The entry points on rows of logits and the fork refuse bad arguments on the host, before any CUDA call (no GPU needed; fake
aligned addresses, nothing is dereferenced), and the Python binding refuses tensors that do not fit."""
import ctypes

import pytest

from speculative_decoding_verification_specdec_gb300 import _native, build, kvcache

E = _native
P = 4096
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if build.needs_rebuild():
        build.build_library()
    return _native.load()


ROWS = [dict(rows=-1), dict(V=0), dict(V=-5), dict(stride=-1), dict(rows=2, stride=99), dict(rows=1, logits=None), dict(rows=1, logits=P + 1)]
TYPES = [dict(dtype=3), dict(dtype=-1), dict(dtype=9), dict(V=2 ** 30 + 1, stride=2 ** 30 + 1)]
TEMPERATURES = [dict(temperature=t) for t in (0.0, -1.0, NAN, INF, 9e-5, 1.1e4)]


def call_top(lib, **o):
    a = dict(logits=P, dtype=1, rows=0, V=100, stride=100, mask=None, temperature=1.0, n=8, ids=P, lps=P, lse=None, status=None, ws=P, wb=1 << 40)
    a.update(o)
    return lib.specdec_top_logits(*a.values(), None)


def test_top_logits_refusals(lib):
    assert call_top(lib) == E.SPECDEC_OK
    for bad in ROWS + TEMPERATURES + [dict(n=0), dict(n=129), dict(rows=1, ids=None), dict(rows=1, lps=None), dict(rows=1, ws=None),
                                      dict(rows=1, ws=P + 8), dict(rows=1, wb=0), dict(rows=1, mask=P + 2), dict(rows=1, ids=P + 2),
                                      dict(rows=1, lps=P + 1), dict(rows=1, lse=P + 2), dict(rows=1, status=P + 2)]:
        assert call_top(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    for bad in TYPES + [dict(rows=2 ** 31 - 1, V=2 ** 20, stride=2 ** 20)]:
        assert call_top(lib, **bad) == E.SPECDEC_ERR_UNSUPPORTED, bad


def call_distill(lib, **o):
    a = dict(logits=P, dtype=1, rows=0, V=100, stride=100, ids=P, lps=P, n=8, temperature=1.0, rest=1, weight=None, loss=P, stats=None,
             grad=None, gs=0, status=None)
    a.update(o)
    return lib.specdec_distill(*a.values(), None)


def call_backward(lib, **o):
    a = dict(logits=P, dtype=1, rows=0, V=100, stride=100, ids=P, lps=P, n=8, temperature=1.0, rest=1, stats=P, weight=None, grad=P, gs=100,
             status=None)
    a.update(o)
    return lib.specdec_distill_backward(*a.values(), None)


@pytest.mark.parametrize("call", [call_distill, call_backward])
def test_distill_refusals(lib, call):
    assert call(lib) == E.SPECDEC_OK
    for bad in ROWS + TEMPERATURES + [dict(n=0), dict(n=129), dict(rest=2), dict(rest=-1), dict(gs=-1), dict(rows=1, ids=None),
                                      dict(rows=1, lps=None), dict(rows=1, ids=P + 2), dict(rows=1, lps=P + 2), dict(rows=1, weight=P + 2),
                                      dict(rows=1, stats=P + 2), dict(rows=1, grad=P + 1, gs=100), dict(rows=2, grad=P, gs=99),
                                      dict(rows=1, status=P + 2)]:
        assert call(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    for bad in TYPES:
        assert call(lib, **bad) == E.SPECDEC_ERR_UNSUPPORTED, bad
    if call is call_distill:
        assert call(lib, rows=1, loss=None) == E.SPECDEC_ERR_INVALID_ARG and call(lib, rows=1, loss=P + 2) == E.SPECDEC_ERR_INVALID_ARG
    else:
        assert call(lib, rows=1, stats=None) == E.SPECDEC_ERR_INVALID_ARG and call(lib, rows=1, grad=None) == E.SPECDEC_ERR_INVALID_ARG
    assert call(lib, rows=2 ** 31 - 1, V=2 ** 21, stride=2 ** 21, grad=P, gs=2 ** 21) == E.SPECDEC_ERR_UNSUPPORTED


def call_beam(lib, **o):
    a = dict(logits=P, dtype=1, rows=0, beams=4, V=100, stride=100, mask=None, scores=P, finished=None, end=-1, n=4, out=P, tokens=P, next=P,
             ended=None, status=None, ws=P, wb=1 << 40)
    a.update(o)
    return lib.specdec_beam_select(*a.values(), None)


def test_beam_select_refusals(lib):
    assert call_beam(lib) == E.SPECDEC_OK
    for bad in ROWS + [dict(beams=0), dict(beams=129), dict(n=0), dict(n=129), dict(end=-2), dict(end=100), dict(finished=P),
                       dict(rows=1, scores=None), dict(rows=1, out=None), dict(rows=1, tokens=None), dict(rows=1, next=None),
                       dict(rows=1, ws=None), dict(rows=1, ws=P + 8), dict(rows=1, wb=0), dict(rows=1, scores=P + 2), dict(rows=1, out=P + 2),
                       dict(rows=1, tokens=P + 2), dict(rows=1, next=P + 2), dict(rows=1, mask=P + 2), dict(rows=1, status=P + 2)]:
        assert call_beam(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    for bad in TYPES + [dict(beams=128, n=33), dict(rows=2 ** 31 - 1, beams=2)]:
        assert call_beam(lib, **bad) == E.SPECDEC_ERR_UNSUPPORTED, bad


def test_workspace_sizes(lib):
    import torch

    top, beam, f = _native.top_logits_workspace_size, _native.beam_select_workspace_size, torch.float32
    assert top(0, 5, f) == 0 and top(5, 0, f) == 0 and top(5, 2 ** 30 + 1, f) == 0 and top(2 ** 31 - 1, 2 ** 20, f) == 0
    assert beam(0, 4, 5, f, 4) == 0 and beam(2, 0, 5, f, 4) == 0 and beam(2, 129, 5, f, 1) == 0 and beam(2, 128, 5, f, 33) == 0
    assert beam(2, 4, 5, f, 0) == 0 and beam(2, 4, 0, f, 4) == 0 and beam(2 ** 31 - 1, 2, 5, f, 1) == 0
    assert 0 < top(1, 1, f) <= top(16, 151936, torch.bfloat16) and 0 < beam(1, 1, 1, f, 1) <= beam(64, 8, 151936, f, 8)
    assert top(7, 1001, f) % 16 == 0 and beam(7, 3, 1001, f, 5) % 16 == 0
    assert lib.specdec_top_logits_workspace_size(1, 1, 3) == 0
    with pytest.raises(E.SpecdecError):
        top(1, 1, torch.float64)
    with pytest.raises(ValueError):
        top(2 ** 31, 1, f)


def call_fork(lib, cache=(), **o):
    c = dict(k=P, v=P, k_exp=None, v_exp=None, dtype=1, num_pages=8, page_size=16, num_kv_heads=2, head_dim=64, page_stride=2048,
             head_stride=1024, slot_stride=64)
    c.update(dict(cache))
    a = dict(tab=P, mb=4, bs=4, lengths=P, sources=3, parent=P, fresh=P, n=0, out=P, os=4, ol=P, status=None)
    a.update(o)
    return lib.specdec_kv_fork(ctypes.byref(_native.KVCacheStruct(*c.values())), *a.values(), None)


def test_kv_fork_refusals(lib):
    assert call_fork(lib) == E.SPECDEC_OK
    for bad in (dict(n=-1), dict(sources=-1), dict(mb=-1), dict(bs=-1), dict(os=-1), dict(n=2, os=3), dict(n=1, tab=None),
                dict(n=1, lengths=None), dict(n=1, parent=None), dict(n=1, out=None, fresh=None), dict(n=1, tab=P + 2), dict(n=1, parent=P + 2),
                dict(n=1, fresh=P + 2), dict(n=1, out=P + 2), dict(n=1, ol=P + 2), dict(n=1, lengths=P + 2), dict(n=1, status=P + 2),
                dict(cache=dict(k=None)), dict(cache=dict(num_pages=0)), dict(cache=dict(slot_stride=68))):
        assert call_fork(lib, **bad) == E.SPECDEC_ERR_INVALID_ARG, bad
    for bad in (dict(cache=dict(dtype=0)), dict(cache=dict(page_size=48)), dict(cache=dict(head_dim=8))):
        assert call_fork(lib, **bad) == E.SPECDEC_ERR_UNSUPPORTED, bad
    assert lib.specdec_kv_fork(None, P, 4, 4, P, 3, P, P, 1, P, 4, P, None, None) == E.SPECDEC_ERR_INVALID_ARG


def test_binding_refuses_what_does_not_fit(lib):
    import torch

    f, i = torch.float32, torch.int32
    x, ids, lps, row, ws = (torch.zeros(s, dtype=t) for s, t in (((4, 50), f), ((4, 3), i), ((4, 3), f), (4, f), (1 << 16, torch.uint8)))
    c = kvcache.PagedCache(torch.zeros((4, 2, 16, 32), dtype=torch.bfloat16), torch.zeros((4, 2, 16, 32), dtype=torch.bfloat16))
    tab, n = torch.zeros((4, 2), dtype=i), torch.zeros(4, dtype=i)
    s = torch.zeros((2, 2), dtype=f)
    out = torch.zeros((2, 2), dtype=i)
    for call in (lambda: _native.top_logits(x, ids, lps, ws),                              # not on a GPU
                 lambda: _native.top_logits(x[:, ::2], ids, lps, ws),
                 lambda: _native.top_logits(x, ids[:3], lps, ws),
                 lambda: _native.top_logits(x, ids.long(), lps, ws),
                 lambda: _native.top_logits(x, ids, lps[:, :2], ws),
                 lambda: _native.top_logits(x, ids, lps, ws, bitmask=ids),
                 lambda: _native.top_logits(x, ids, lps, ws, lse=row[:2]),
                 lambda: _native.top_logits(x[0], ids, lps, ws),
                 lambda: _native.distill(x, ids, lps, row),
                 lambda: _native.distill(x, ids[:, :2], lps, row),
                 lambda: _native.distill(x, ids, lps, row, grad=x[:3]),
                 lambda: _native.distill(x, ids, lps, row, grad=x.half()),
                 lambda: _native.distill(x, ids, lps, row, stats=row),
                 lambda: _native.distill(x, ids, lps, row, weight=row.double()),
                 lambda: _native.distill_backward(x, ids, lps, row, None, x),
                 lambda: _native.beam_select(x, s, out, out, s, ws),
                 lambda: _native.beam_select(x[:3], s, out, out, s, ws),
                 lambda: _native.beam_select(x, s, out, out[:1], s, ws),
                 lambda: _native.beam_select(x, s, out, out, s.int(), ws),
                 lambda: _native.beam_select(x, s, out, out, s, ws, finished=s),
                 lambda: _native.kv_fork(c, tab, n, n, n, tab.clone()),
                 lambda: _native.kv_fork(c, tab, n, n.long(), n, tab.clone()),
                 lambda: _native.kv_fork(c, tab, n, n, n[:2], tab.clone()),
                 lambda: _native.kv_fork(c, tab, n, n, n, tab[:, :1]),
                 lambda: _native.kv_fork(c, tab, n, n, n, tab[:2])):
        with pytest.raises((ValueError, E.SpecdecError)):
            call()
