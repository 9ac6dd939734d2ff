"""The paged key-value cache (specdec_kv_write, specdec_kv_read) against the 64-bit definitions."""
import numpy as np
import pytest

import _paged as P
from oracle import paged_ref as ref
from speculative_decoding_verification_specdec_gb300 import _native, build, kvcache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cuda():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    if build.needs_rebuild():
        build.build_library()
    _native.load()
    torch.cuda.set_device(0)
    return "cuda:0"


def dev(a, cuda):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(cuda)


def write(cuda, ks, cached, heads, dim, kind, cache_kind, page, seed=0, rope=None, values=None, token_major=False,
          positions=None, extra_rows=2, tab=None, pages=None, inputs="packed"):
    """Writes random (or given) rows; returns the cache, host k and v rows, table and status."""
    import torch

    rng = np.random.default_rng([seed, heads, dim, page])
    cu, B = P.offsets(ks), len(ks)
    T = int(cu[-1]) + B
    total = [max(c, 0) + k + 1 for c, k in zip(cached, ks)]
    if tab is None:
        tab, pages = P.table(total, page, rng)
    kv = rng.standard_normal((T + extra_rows, 2 * heads, dim)).astype(np.float32) * 3
    if values is not None:
        kv[:T] = values
    kv = torch.from_numpy(kv).to(P.torch_type(kind)).to(cuda)
    k, v = kv[:, :heads], kv[:, heads:]
    if inputs == "odd":                                    # bases and rows off the 16-byte grid
        wide = torch.zeros((T + extra_rows, 2 * heads * dim + 1), dtype=kv.dtype, device=cuda)
        flat = wide[:, 1:]
        flat.copy_(kv.reshape(T + extra_rows, -1))
        k, v = (flat[:, i * heads * dim:(i + 1) * heads * dim].unflatten(1, (heads, dim)) for i in (0, 1))
    if token_major:
        base = kvcache.alloc(pages, page, heads, dim, P.torch_type(cache_kind), cuda)      # [pages, slot, head, dim]
        cache = kvcache.PagedCache(base.k.permute(0, 2, 1, 3), base.v.permute(0, 2, 1, 3),
                                   *(None if e is None else torch.full((pages, heads, page), 127, dtype=torch.uint8, device=cuda)
                                     for e in (base.k_exp, base.v_exp)))
    else:
        cache = kvcache.alloc(pages, heads, page, dim, P.torch_type(cache_kind), cuda)
    status = torch.zeros(B, dtype=torch.int32, device=cuda)
    _native.kv_write(k, v, cache, dev(tab, cuda), dev(np.asarray(cached, dtype=np.int32), cuda), dev(cu, cuda), B, rope=rope,
                     positions=None if positions is None else dev(positions.astype(np.int32), cuda), status=status)
    torch.cuda.synchronize()
    return cache, P.host(k)[:T], P.host(v)[:T], tab, status.cpu().numpy(), cu


def check_written(cache, k, v, tab, cu, cached, cache_kind, page, slack=0.0):
    """Every written token's values; every other place still zero. `slack`: how far a rotated key may be from
    its 64-bit value before it is rounded, relative to |a| + |b| <= 2 max |x|."""
    gk, gv = P.held(cache)
    seen = np.zeros(gk.shape[:1] + gk.shape[2:3], dtype=bool)
    for r, (b, j) in enumerate(ref.owners(cu, len(cached))):
        if cached[b] < 0:
            continue
        i = cached[b] + j
        pg, sl = tab[b, i // page], i % page
        seen[pg, sl] = True
        for got, want, s in ((gk[pg, :, sl], k[r], slack), (gv[pg, :, sl], v[r], 0.0)):
            err = s * 2 * np.abs(want).max(-1, keepdims=True)
            if cache_kind != "e4m3":
                tol = err + P.HALF[cache_kind] * (np.abs(want) + err) + (2.0 ** -25 if cache_kind == "f16" else 0.0)
                assert np.all(np.abs(got - want) <= tol)
                continue
            e = ref.e4m3_exponent(want)
            if s == 0.0:
                exact = ref.E4M3[ref.e4m3_code(want * 2.0 ** -e[..., None].astype(np.float64))] * 2.0 ** e[..., None].astype(np.float64)
                assert np.array_equal(got, exact)
            # half a step relative, or half of 2^-9 scales among subnormals (a key at the border of two scales may take the larger)
            tol = err + np.maximum(P.HALF["e4m3"] * (np.abs(want) + err), 2.0 ** -10 * 2.0 ** (e[..., None] + 1.0))
            assert np.all(np.abs(got - want) <= tol)
    for x in (gk, gv):
        assert (x.transpose(0, 2, 1, 3)[~seen] == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cache_kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("heads,dim,page", [(1, 16, 16), (8, 128, 16), (3, 80, 32), (5, 64, 64), (2, 112, 256)])
def test_write_without_rotation(cuda, kind, cache_kind, heads, dim, page):
    """Single tokens, verify steps and a prompt, at starts inside and at the ends of pages."""
    ks, cached = [0, 3, 40, 0, 8, 1], [0, page - 1, 5, page, 2 * page - 4, 1]
    cache, k, v, tab, status, cu = write(cuda, ks, cached, heads, dim, kind, cache_kind, page)
    check_written(cache, k, v, tab, cu, cached, cache_kind, page)
    assert (status == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 64), (128, 10), (48, 6), (96, 96), (80, 2)])
def test_write_rotates_keys(cuda, interleaved, cache_kind, dim, rot):
    ks, cached = [2, 0, 17], [30000, 0, 7]
    table, amp = _native.rope_frequencies(rot, scaling="by_parts", factor=8.0, original_len=4096)
    rope = dict(freqs=table.to(cuda), rot_dim=rot, interleaved=interleaved, amplitude=amp)
    cache, k, v, tab, status, cu = write(cuda, ks, cached, 3, dim, "bf16", cache_kind, 32, rope=rope)
    f, a = ref.frequencies(rot, scaling="by_parts", factor=8.0, original_len=4096)
    pos = [cached[b] + j for b, j in ref.owners(cu, 3)]
    # cosine, sine, amplitude, products and sum as in the rotation's own test, amplitude under 1.3
    check_written(cache, ref.rope(k, pos, f, interleaved, a), v, tab, cu, cached, cache_kind, 32, slack=1.3 * 8 * 2.0 ** -24)


def test_given_positions_move_the_rotation_alone(cuda):
    rope = dict(freqs=_native.rope_frequencies(32)[0].to(cuda), rot_dim=32)
    pos = np.array([9, 100000, 3, 3, 50, 60, 0, 0])
    cache, k, v, tab, status, cu = write(cuda, [1, 3], [4, 20], 2, 32, "f32", "f16", 16, rope=rope, positions=pos)
    check_written(cache, ref.rope(k, pos[:6], ref.frequencies(32)[0]), v, tab, cu, [4, 20], "f16", 16, slack=8 * 2.0 ** -24)


@pytest.mark.parametrize("inputs", ["odd", "packed"])
@pytest.mark.parametrize("token_major", [False, True])
def test_layouts(cuda, inputs, token_major):
    """Cache laid out head by head or slot by slot; inputs on and off the 16-byte grid."""
    for cache_kind in ("bf16", "e4m3"):
        cache, k, v, tab, status, cu = write(cuda, [5, 0, 31], [3, 64, 10], 3, 96, "f16", cache_kind, 64, token_major=token_major, inputs=inputs)
        check_written(cache, k, v, tab, cu, [3, 64, 10], cache_kind, 64)


def test_values_that_stress_the_scale(cuda):
    """Heads of zeros, subnormals, the border at 448, one large element among small ones, the largest fp32."""
    rng = np.random.default_rng(2)
    vals = rng.standard_normal((8, 4, 32)).astype(np.float32)
    vals[0] = 0
    vals[1] = 2.0 ** -140
    vals[2, :, 0] = 448.0 * 2.0 ** 5
    vals[3, :, 1] = np.nextafter(np.float32(448.0), np.float32(1000))
    vals[4, :, 2] = 1e30
    vals[5] *= 2.0 ** -126
    vals[6] = np.float32(3.4e38)
    vals[7] = -0.0
    cache, k, v, tab, status, cu = write(cuda, [7], [0], 2, 32, "f32", "e4m3", 16, values=vals)
    check_written(cache, k, v, tab, cu, [0], "e4m3", 16)


def test_not_finite(cuda):
    """Infinities and NaN are stored as NaN and leave the scale to the finite elements; a 16-bit cache keeps them."""
    vals = np.ones((2, 2, 16), dtype=np.float32)
    vals[0, 0, 3], vals[0, 1, 5], vals[1, 0] = np.inf, -np.inf, np.nan
    cache, k, v, tab, status, cu = write(cuda, [1], [0], 1, 16, "f32", "e4m3", 16, values=vals)
    gk, gv = P.held(cache)
    page = tab[0, 0]
    assert np.isnan(gk[page, 0, 0, 3]) and np.isnan(gv[page, 0, 0, 5]) and np.isnan(gk[page, 0, 1]).all()
    assert np.isfinite(np.delete(gk[page, 0, 0], 3)).all() and (np.delete(gk[page, 0, 0], 3) == 1).all()
    cache, _, _, tab, _, _ = write(cuda, [1], [0], 1, 16, "f32", "bf16", 16, values=vals)
    gk, gv = P.held(cache)
    assert gk[tab[0, 0], 0, 0, 3] == np.inf and gv[tab[0, 0], 0, 0, 5] == -np.inf and np.isnan(gk[tab[0, 0], 0, 1]).all()


def test_faults_are_reported_and_write_nothing(cuda):
    """A skipped request, one past its table, bad page ids, malformed offsets."""
    import torch

    rng = np.random.default_rng(0)
    tab = np.array([[0, 1], [2, 3], [4, 99], [-1, 5]], dtype=np.int32)
    cache, k, v, _, status, cu = write(cuda, [1, 3, 2, 0], [-1, 29, 15, 16], 2, 16, "f32", "bf16", 16, tab=tab, pages=6)
    assert status.tolist() == [_native.ST_BAD_LENGTH, _native.ST_BAD_LENGTH, _native.ST_BAD_PAGE, 0]
    gk, _ = P.held(cache)
    touched = [(p, s) for p in range(6) for s in range(16) if (gk[p, :, s] != 0).any()]
    assert touched == [(4, 15), (5, 0)]
    for bad in ([1, 2, 3], [0, 9, 2]):
        c = kvcache.alloc(2, 1, 16, 16, torch.bfloat16, cuda)
        st = torch.zeros(2, dtype=torch.int32, device=cuda)
        x = torch.ones((6, 1, 16), device=cuda)
        _native.kv_write(x, x, c, torch.zeros((2, 1), dtype=torch.int32, device=cuda), torch.zeros(2, dtype=torch.int32, device=cuda),
                         torch.tensor(bad, dtype=torch.int32, device=cuda), 2, status=st)
        assert (st.cpu() == _native.ST_BAD_OFFSETS).all() and (c.k == 0).all()


@pytest.mark.parametrize("out_kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cache_kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("heads,dim,page,token_major", [(1, 16, 16, False), (8, 128, 16, True), (3, 80, 64, False)])
def test_read(cuda, out_kind, cache_kind, heads, dim, page, token_major):
    """Ranges that start and end inside pages, an empty one, one token; rows behind the last stay."""
    import torch

    rng = np.random.default_rng([heads, dim, page])
    lens, first = [1, 0, 3 * page + 5, page, 70], [0, 4, 7, page, 3]
    tab, pages = P.table([f + n for f, n in zip(first, lens)], page, rng)
    cache = P.filled(pages, heads, page, dim, cache_kind, rng, cuda, token_major)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    n = int(cu[-1])
    out = torch.full((n + 2, 2 * heads, dim), 7.0, dtype=P.torch_type(out_kind), device=cuda)
    status = torch.zeros(5, dtype=torch.int32, device=cuda)
    _native.kv_read(cache, dev(tab, cuda), dev(cu, cuda), 5, out[:, :heads], out[:, heads:], first=dev(np.array(first, dtype=np.int32), cuda),
                    status=status)
    got, (gk, gv) = P.host(out), P.held(cache)
    for b in range(5):
        for x, part in ((gk, got[:, :heads]), (gv, got[:, heads:])):
            want = torch.from_numpy(P.tokens(x, tab[b], first[b] + lens[b], page)[first[b]:]).float().to(P.torch_type(out_kind)).double().numpy()
            assert np.array_equal(part[cu[b]: cu[b + 1]], want)
    assert (got[n:] == 7).all() and (status.cpu() == 0).all()


def test_read_one_of_the_two_and_off_the_grid(cuda):
    import torch

    rng = np.random.default_rng(9)
    tab, pages = P.table([20], 16, rng)
    cache = P.filled(pages, 2, 16, 48, "e4m3", rng, cuda)
    flat = torch.zeros(20 * 2 * 48 + 1, dtype=torch.bfloat16, device=cuda)
    out = flat[1:].view(20, 2, 48)
    cu = dev(np.array([0, 20], dtype=np.int64), cuda)
    for i, args in enumerate(((out, None), (None, out))):
        _native.kv_read(cache, dev(tab, cuda), cu, 1, *args)
        want = torch.from_numpy(P.tokens(P.held(cache)[i], tab[0], 20, 16)).float().to(torch.bfloat16).double().numpy()
        assert np.array_equal(P.host(out), want)


def test_read_faults(cuda):
    """A bad page reads as zeros; a range past the table, a negative start and malformed offsets write nothing."""
    import torch

    rng = np.random.default_rng(4)
    cache = P.filled(3, 1, 16, 16, "bf16", rng, cuda)
    tab = np.array([[0, 7], [1, 2], [0, 1], [-3, 1]], dtype=np.int32)
    cu = np.array([0, 20, 60, 65, 70], dtype=np.int64)
    first = np.array([0, 0, -1, 14], dtype=np.int32)
    out = torch.full((70, 1, 16), 7.0, device=cuda)
    status = torch.zeros(4, dtype=torch.int32, device=cuda)
    _native.kv_read(cache, dev(tab, cuda), dev(cu, cuda), 4, out, None, first=dev(first, cuda), status=status)
    got = P.host(out)
    assert status.tolist() == [_native.ST_BAD_PAGE, _native.ST_BAD_LENGTH, _native.ST_BAD_LENGTH, _native.ST_BAD_PAGE]
    assert (got[16:20] == 0).all() and (got[20:65] == 7).all() and (got[65:67] == 0).all()
    assert np.array_equal(got[67:70, 0], P.held(cache)[0][1, 0, :3])
    out.fill_(7.0)
    st = torch.zeros(2, dtype=torch.int32, device=cuda)
    _native.kv_read(cache, dev(tab, cuda), dev(np.array([0, 9, 4], dtype=np.int64), cuda), 2, out, None, status=st)
    assert (st.cpu() == _native.ST_BAD_OFFSETS).all() and (out == 7).all()


def test_long_cache_offsets_pass_32_bits(cuda):
    """A cache of more than 2^32 elements: the last page is written and read at its own place."""
    import torch

    pages, heads, page, dim = 2 ** 32 // (8 * 256 * 128) + 2, 8, 256, 128
    k = torch.empty((pages, heads, page, dim), dtype=torch.float8_e4m3fn, device=cuda)
    e = torch.full((pages, heads, page), 127, dtype=torch.uint8, device=cuda)
    k.view(torch.uint8)[0] = 0
    cache = kvcache.PagedCache(k, k, e, e)
    x = torch.randn((3, heads, dim), device=cuda).to(torch.bfloat16)
    tab = torch.full((1, 1), pages - 1, dtype=torch.int32, device=cuda)
    one, cu = torch.full((1,), 5, dtype=torch.int32, device=cuda), torch.tensor([0, 2], dtype=torch.int32, device=cuda)
    _native.kv_write(x, x, cache, tab, one, cu, 1)
    out = torch.empty_like(x)
    _native.kv_read(cache, tab, torch.tensor([0, 3], dtype=torch.int64, device=cuda), 1, out, None, first=one)
    xs = P.host(x)
    ex = ref.e4m3_exponent(xs)[..., None].astype(np.float64)
    assert np.array_equal(P.host(out), ref.E4M3[ref.e4m3_code(xs * 2.0 ** -ex)] * 2.0 ** ex)
    assert (k.view(torch.uint8)[0] == 0).all()


@pytest.mark.parametrize("inputs", ["odd", "packed"])
@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
def test_a_capacity_far_beyond_the_rows(cuda, cache_kind, inputs):
    """Inputs of 9000 rows of which the requests have 12: CTAs that hold some of them, and none, leave the rest."""
    rope = dict(freqs=_native.rope_frequencies(32)[0].to(cuda), rot_dim=32)
    cache, k, v, tab, status, cu = write(cuda, [4, 0, 5], [7, 0, 100], 3, 48, "bf16", cache_kind, 16, rope=rope, extra_rows=8988, inputs=inputs)
    pos = [[7, 0, 100][b] + j for b, j in ref.owners(cu, 3)]
    check_written(cache, ref.rope(k, pos, ref.frequencies(32)[0]), v, tab, cu, [7, 0, 100], cache_kind, 16, slack=8 * 2.0 ** -24)
    assert (status == 0).all()


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
def test_rows_behind_the_capacity_are_refused(cuda, cache_kind):
    """Offsets that name more rows than k and v, or the outputs, have: the request is reported and nothing of it is written."""
    import torch

    cache = kvcache.alloc(4, 2, 16, 32, P.torch_type(cache_kind), cuda)
    tab = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device=cuda)
    x = torch.ones((4, 2, 32), dtype=torch.bfloat16, device=cuda)
    status = torch.zeros(2, dtype=torch.int32, device=cuda)
    _native.kv_write(x, x, cache, tab, torch.zeros(2, dtype=torch.int32, device=cuda), torch.tensor([0, 1, 3], dtype=torch.int32, device=cuda),
                     2, status=status)                                # request 1 would end at row 5
    assert status.tolist() == [0, _native.ST_BAD_OFFSETS]
    gk, _ = P.held(cache)
    assert (gk[2, :, :2] == 1).all() and (gk[3] == 0).all() and (gk[[0, 1]] == 0).all()
    out = torch.full((5, 2, 32), 7.0, device=cuda)
    status.zero_()
    _native.kv_read(cache, tab, torch.tensor([0, 2, 6], dtype=torch.int64, device=cuda), 2, out, None, status=status)
    assert status.tolist() == [0, _native.ST_BAD_OFFSETS]
    assert (out[:2] == 1).all() and (out[2:] == 7).all()
