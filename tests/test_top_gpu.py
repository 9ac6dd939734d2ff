"""specdec_top_logits against the 64-bit definition: ids exact, log-probabilities within derived bounds."""
import numpy as np
import pytest

import _logits as L
import _paged as P
from oracle import logits_ref as ref
from speculative_decoding_verification_specdec_gb300 import _native, build

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


def top(x, n, mask=None, temperature=1.0, stream=None):
    """Runs over guarded outputs; returns host arrays."""
    import torch

    rows, V = x.shape
    ids = torch.full((rows + 2, n), -77, dtype=torch.int32, device=x.device)
    lps = torch.full((rows + 2, n), 77.0, device=x.device)
    lse = torch.full((rows + 2,), 77.0, device=x.device)
    status = torch.zeros(rows, dtype=torch.int32, device=x.device)
    size = _native.top_logits_workspace_size(rows, V, x.dtype)
    ws = torch.full((size + 64,), 0x5a, dtype=torch.uint8, device=x.device)
    _native.top_logits(x, ids[1:-1], lps[1:-1], ws[:size], bitmask=mask, temperature=temperature, lse=lse[1:-1], status=status, stream=stream)
    torch.cuda.synchronize()
    for t, g in ((ids, -77), (lps, 77.0), (lse, 77.0)):
        assert (t[0] == g).all() and (t[-1] == g).all()
    assert (ws[size:] == 0x5a).all()
    return ids[1:-1].cpu().numpy(), lps[1:-1].cpu().numpy(), lse[1:-1].cpu().numpy(), status.cpu().numpy()


def check(got, z, n, masks=None, temperature=1.0):
    ids, lps, lse, status = got
    for r in range(z.shape[0]):
        m = None if masks is None else masks[r]
        wi, wl, ws = ref.top_logits(z[r], n, temperature, m)
        assert np.array_equal(ids[r], wi), r
        assert (status[r] != 0) == (wi[0] < 0)
        if np.isnan(ws):
            assert np.isnan(lse[r]) and np.isnan(lps[r][wi >= 0]).all()
            continue
        if ws == -np.inf:
            assert lse[r] == -np.inf and (lps[r] == -np.inf).all()
            continue
        zr = z[r] if m is None else z[r][m]
        err, Z = L.lse_error(zr, temperature)
        assert abs(lse[r] - ws) <= err + L.U * abs(ws), r
        k = wi >= 0
        # z c: c's rounding; the difference to the sum's logarithm and the result's rounding
        assert np.all(np.abs(lps[r][k] - wl[k]) <= err + L.U * (Z + np.abs(wl[k]))), r
        assert (lps[r][~k] == -np.inf).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 256, 1000, 2049, 4099, 32000, 70001])
@pytest.mark.parametrize("n", [1, 8, 128])
def test_random_rows(cuda, kind, V, n):
    x, z = L.rows(np.random.default_rng([V, n]), 5, V, kind)
    check(top(x, n), z, n)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [900, 1024, 1025, 2048, 8191, 8192, 16384, 16385, 65536, 131072, 140000])
@pytest.mark.parametrize("n", [64, 127, 128])
def test_where_the_bounds_come_from(cuda, kind, V, n):
    """Sizes on both sides of every way of taking the bound, with clusters of large values beside each other."""
    rng = np.random.default_rng([V, n])
    x, _ = L.rows(rng, 3, V, kind)
    x[1, V // 3: V // 3 + 300] += 6.0
    x[2, : n + 3] = 30.0
    check(top(x, n), P.host(x), n)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("extra,shift", [(1, 0), (0, 1), (3, 5), (8, 8)])
@pytest.mark.parametrize("temperature", [0.3, 4.0])
def test_strides_and_alignments(cuda, kind, extra, shift, temperature):
    x, z = L.rows(np.random.default_rng(extra + shift), 6, 5003, kind, extra=extra, shift=shift)
    check(top(x, 20, temperature=temperature), z, 20, temperature=temperature)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [5, 33, 1000, 9001])
@pytest.mark.parametrize("shift", [0, 3])
def test_masks_hide_whatever_lies_there(cuda, kind, V, shift):
    """Forbidden places hold infinities and NaN; one row allows nothing, one a single id, one everything."""
    rng = np.random.default_rng(V)
    allowed = rng.random((6, V)) < 0.3
    allowed[0], allowed[2], allowed[1] = False, True, False
    allowed[1, V - 1] = True
    x, z = L.rows(rng, 6, V, kind, shift=shift, extra=shift)
    import torch

    bad = torch.from_numpy(np.array([np.inf, np.nan, -np.inf, 3e38], dtype=np.float32)).to(x.dtype).to(cuda)
    x.copy_(torch.where(L.dev(allowed), x, bad[L.dev(rng.integers(0, 4, (6, V)))]))
    check(top(x, 16, mask=L.dev(L.pack(allowed))), P.host(x), 16, masks=allowed)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("values", ["equal", "two", "few", "rising", "falling", "lowest", "zeros"])
def test_ties_and_orders(cuda, kind, values):
    """Equal values by the thousand (more than fit on chip), sorted rows, the type's lowest value, zeros of both signs."""
    import torch

    V = 30011
    rng = np.random.default_rng(7)
    x, _ = L.rows(rng, 3, V, kind)
    lowest = float(torch.finfo(x.dtype).min)
    rows = {"equal": np.full((3, V), 1.5), "two": rng.integers(0, 2, (3, V)), "few": rng.integers(0, 40, (3, V)),
            "rising": np.tile(np.arange(V) / 512.0, (3, 1)), "falling": np.tile(-np.arange(V) / 512.0, (3, 1)),
            "lowest": np.where(rng.random((3, V)) < 0.001, lowest, -np.inf), "zeros": np.where(rng.random((3, V)) < 0.5, 0.0, -0.0)}[values]
    x.copy_(torch.from_numpy(rows.astype(np.float32)))
    for n in (1, 100, 128):
        got = top(x, n)
        if values == "lowest" and kind != "f16":       # (the sum counts them as -infinity)
            for r in range(3):
                assert np.array_equal(got[0][r], ref.top_logits(P.host(x)[r], n)[0])
            assert (got[1] == -np.inf).all() and (got[2] == -np.inf).all()
        else:
            check(got, P.host(x), n)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_places_masked_by_the_lowest_value(cuda, kind):
    """Most of a row at its type's lowest value, whole units of it among them: the others' sum as if those were not there."""
    import torch

    x, _ = L.rows(np.random.default_rng(11), 4, 20000, kind)
    x[:, 700:19000] = float(torch.finfo(x.dtype).min)
    x[1, :] = float(torch.finfo(x.dtype).min)
    x[1, 9] = 2.0
    ids, lps, lse, status = top(x, 30)
    z = P.host(x)
    seen = np.where(z < -60000, -np.inf, z)
    for r in range(4):
        assert np.array_equal(ids[r], ref.top_logits(z[r], 30)[0])
        _, want, s = ref.top_logits(seen[r], 30)
        err, Z = L.lse_error(seen[r])
        assert abs(lse[r] - s) <= err + L.U * abs(s)
        k = want > -np.inf
        assert np.all(np.abs(lps[r][k] - want[k]) <= err + L.U * (Z + np.abs(want[k])))
    assert (status == 0).all()


def test_rows_without_a_number(cuda):
    """-infinity everywhere, NaN everywhere, NaN among numbers, +infinity among numbers."""
    x, _ = L.rows(np.random.default_rng(1), 5, 700, "f32")
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 3::7] = np.nan
    x[3, 50] = np.inf
    check(top(x, 12), P.host(x), 12)


def test_many_rows_on_a_stream_and_in_a_graph(cuda):
    """More rows than CTAs fit, on a stream of the caller's; replays read what the rows hold then."""
    import torch

    rng = np.random.default_rng(5)
    x, z = L.rows(rng, 700, 3001, "bf16")
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    check(top(x, 10, stream=other), z, 10)
    ids = torch.empty((700, 10), dtype=torch.int32, device=cuda)
    lps, lse = torch.empty((700, 10), device=cuda), torch.empty(700, device=cuda)
    ws = torch.empty(_native.top_logits_workspace_size(700, 3001, x.dtype), dtype=torch.uint8, device=cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _native.top_logits(x, ids, lps, ws, lse=lse)
    for seed in (1, 2):
        y, z = L.rows(np.random.default_rng(seed), 700, 3001, "bf16")
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        check((ids.cpu().numpy(), lps.cpu().numpy(), lse.cpu().numpy(), np.zeros(700)), z, 10)


def test_equal_rows_give_equal_bits(cuda):
    """Rows of one alignment (another one groups a row's terms differently)."""
    x, _ = L.rows(np.random.default_rng(3), 9, 20001, "f32", extra=3)
    x[:] = x[0].clone()
    ids, lps, lse, _ = top(x, 64)
    assert (ids == ids[0]).all() and (lps == lps[0]).all() and (lse == lse[0]).all()
    again = top(x, 64)
    assert all(np.array_equal(a, b) for a, b in zip((ids, lps, lse), again))
