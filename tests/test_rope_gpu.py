"""Rotary positions (specdec_rope) against the 64-bit definition: layouts, partial heads, odd sizes, strides,
far positions, the gradient, ragged rows."""
import numpy as np
import pytest

import _paged as P
from oracle import paged_ref as ref
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


def check(got, x, pos, f, kind, interleaved, amplitude, inverse=False):
    """Cosine and sine: the angle's remainder (at most pi / 4) is rounded at 2^-24, its frequency at 2^-51 of
    the whole angle, the function at 2^-23 (one unit in the last place of values up to one), amplitude
    and product at 2^-24 each; two products and a sum at 2^-24 of |a| + |b|; then the type's half step."""
    want = ref.rope(x, pos, f, interleaved, amplitude, inverse)
    rot = 2 * len(f)
    pair = np.abs(x).copy()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    both = np.abs(x[..., one]) + np.abs(x[..., two])
    pair[..., one], pair[..., two] = both, both
    angle = np.abs(np.asarray(pos, dtype=np.float64))[:, None, None] * f * 2.0 ** -51
    err = np.zeros(x.shape)
    err[..., one] = err[..., two] = amplitude * both * (angle + 0.8 * 2.0 ** -24 + 2.0 ** -23 + 4 * 2.0 ** -24)
    tol = err + P.HALF[kind] * (np.abs(want) + err) * (1.0 if kind != "f32" else 0.0)
    tol = tol + np.where(np.abs(want) < 2.0 ** -14, 2.0 ** -25, 0.0) * (kind == "f16")     # half a step among subnormals
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / np.maximum(tol, 1e-300)).max()
    assert np.array_equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot", [(1, 1, 2, 2), (3, 5, 64, 64), (17, 2, 128, 32), (40, 3, 80, 40), (5, 7, 98, 26),
                                                (33, 1, 256, 256), (2, 40, 128, 128), (7, 3, 66, 66), (300, 8, 128, 64)])
def test_given_positions(cuda, kind, interleaved, rows, heads, dim, rot):
    import torch

    rng = np.random.default_rng([rows, heads, dim, rot])
    x = torch.from_numpy(rng.standard_normal((rows, heads, dim)).astype(np.float32)).to(P.torch_type(kind)).to(cuda)
    pos = rng.integers(-5, 200000, size=rows).astype(np.int32)
    pos[0] = [0, 2 ** 31 - 1, -2 ** 31][rows % 3]
    for kw, inverse in (({}, False), (dict(scaling="by_parts", factor=8.0, original_len=4096), True)):
        table, amp = _native.rope_frequencies(rot, **kw)
        out = torch.full_like(x, 7.0)
        _native.rope(x, out, table.to(cuda), rot, interleaved, amp, inverse, positions=torch.from_numpy(pos).to(cuda))
        f, a = ref.frequencies(rot, **kw)
        check(P.host(out), P.host(x), pos, f, kind, interleaved, a, inverse)


def test_scaled_linear_and_in_place_slices(cuda):
    """The query and key heads of one packed projection, each rotated in place; what lies between stays."""
    import torch

    rng = np.random.default_rng(5)
    qkv = torch.from_numpy(rng.standard_normal((9, 16, 64)).astype(np.float32)).to(torch.bfloat16).to(cuda)
    before = P.host(qkv)
    table, amp = _native.rope_frequencies(64, scaling="linear", factor=4.0)
    pos = torch.arange(9, dtype=torch.int32, device=cuda) * 1000
    for part in (slice(0, 8), slice(10, 13)):
        _native.rope(qkv[:, part], qkv[:, part], table.to(cuda), 64, positions=pos, amplitude=amp)
    f, _ = ref.frequencies(64, scaling="linear", factor=4.0)
    got = P.host(qkv)
    for part in (slice(0, 8), slice(10, 13)):
        check(got[:, part], before[:, part], pos.cpu().numpy(), f, "bf16", False, 1.0)
    assert np.array_equal(got[:, 8:10], before[:, 8:10]) and np.array_equal(got[:, 13:], before[:, 13:])


@pytest.mark.parametrize("offset", [1, 4])
def test_unaligned_and_transposed(cuda, offset):
    """A base off the 16-byte grid, and heads laid out before rows."""
    import torch

    rng = np.random.default_rng(offset)
    flat = torch.from_numpy(rng.standard_normal(offset + 6 * 11 * 64).astype(np.float32)).to(torch.float16).to(cuda)
    x = flat[offset:].view(6, 11, 64).transpose(0, 1)                 # 11 rows, 6 heads
    out = torch.zeros((11, 6, 64), dtype=torch.float16, device=cuda)
    table, _ = _native.rope_frequencies(64)
    pos = torch.arange(11, dtype=torch.int32, device=cuda)
    _native.rope(x, out, table.to(cuda), 64, True, positions=pos)
    check(P.host(out), P.host(x), np.arange(11), ref.frequencies(64)[0], "f16", True, 1.0)


@pytest.mark.parametrize("B", [1, 5, 300, 700])
def test_ragged_rows(cuda, B):
    """Positions from cached lengths; skipped requests and rows behind the last one are left as they were."""
    import torch

    rng = np.random.default_rng(B)
    ks = rng.integers(0, 9, size=B)
    cu, cached = P.offsets(ks), rng.integers(0, 5000, size=B).astype(np.int32)
    cached[rng.integers(B)] = -1
    T = int(cu[-1]) + B
    x = torch.from_numpy(rng.standard_normal((T + 3, 2, 32)).astype(np.float32)).to(cuda)
    out = torch.full_like(x, 7.0)
    table, _ = _native.rope_frequencies(32)
    _native.rope(x, out, table.to(cuda), 32, cu_num_draft=torch.from_numpy(cu).to(cuda), cached_len=torch.from_numpy(cached).to(cuda), B=B)
    got, xs, f = P.host(out), P.host(x), ref.frequencies(32)[0]
    own = ref.owners(cu, B)
    live = np.array([cached[b] >= 0 for b, _ in own])
    pos = np.array([cached[b] + j for b, j in own])
    check(got[:T][live], xs[:T][live], pos[live], f, "f32", False, 1.0)
    assert (got[:T][~live] == 7).all() and (got[T:] == 7).all()


def test_malformed_offsets(cuda):
    """Offsets that do not start at zero or that pass the total leave every row as it was."""
    import torch

    x = torch.ones((8, 1, 16), device=cuda)
    table = _native.rope_frequencies(16)[0].to(cuda)
    for cu in ([1, 2, 3], [0, 9, 2], [0, -1, 2]):
        out = torch.full_like(x, 7.0)
        _native.rope(x, out, table, 16, cu_num_draft=torch.tensor(cu, dtype=torch.int32, device=cuda),
                     cached_len=torch.tensor([0, 0], dtype=torch.int32, device=cuda), B=2)
        assert (P.host(out) == 7).all(), cu


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(cuda, interleaved):
    """dx = rope(dout, inverse): against the formula's transpose, and against differences of the rotation
    (linear, so a difference of step one is exact up to the rounding of both values)."""
    import torch

    rng = np.random.default_rng(3)
    x, dout = (torch.from_numpy(rng.standard_normal((4, 2, 24)).astype(np.float32)).to(cuda) for _ in range(2))
    pos = torch.tensor([0, 3, 77, 123456], dtype=torch.int32, device=cuda)
    kw = dict(scaling="by_parts", factor=8.0, original_len=4096)
    table, amp = _native.rope_frequencies(16, **kw)
    args = (table.to(cuda), 16, interleaved, amp)
    dx, y0 = torch.empty_like(x), torch.empty_like(x)
    _native.rope(dout, dx, *args, inverse=True, positions=pos)
    f, a = ref.frequencies(16, **kw)
    check(P.host(dx), P.host(dout), pos.cpu().numpy(), f, "f32", interleaved, a, inverse=True)
    _native.rope(x, y0, *args, positions=pos)
    for d in (0, 7, 8, 15, 20):
        y1, xd = torch.empty_like(x), x.clone()
        xd[..., d] += 1.0
        _native.rope(xd, y1, *args, positions=pos)
        diff = ((P.host(y1) - P.host(y0)) * P.host(dout)).sum(-1)
        # each y is within 2^-20 of (|x| + 1) times the amplitude of its formula; at most two elements differ
        tol = 2.0 ** -20 * a * 8 * (np.abs(P.host(x)).max() + 1) * np.abs(P.host(dout)).max()
        assert np.all(np.abs(diff - P.host(dx)[..., d]) <= tol)


def test_another_stream_and_capture(cuda):
    """A call on a side stream, and a captured call replayed on changed positions."""
    import torch

    table = _native.rope_frequencies(32)[0].to(cuda)
    x = torch.randn((6, 3, 32), device=cuda)
    pos = torch.zeros(6, dtype=torch.int32, device=cuda)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _native.rope(x, out, table, 32, positions=pos, stream=s)
    s.synchronize()
    assert torch.equal(out, x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _native.rope(x, out, table, 32, positions=pos)
    pos.copy_(torch.arange(6, dtype=torch.int32))
    x.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    check(P.host(out), P.host(x), np.arange(6), ref.frequencies(32)[0], "f32", False, 1.0)


@pytest.mark.parametrize("kw", [dict(theta=1e6), dict(theta=1e7), dict(theta=1e7, scaling="linear", factor=1e5)])
@pytest.mark.parametrize("rot", [128, 256])
def test_small_angles_keep_their_sine(cuda, kw, rot):
    """Pairs (1, 0) become (c, s). The angle's rest goes to fp32 once (2^-24 of itself), the sine is off by a unit in the last
    place (2^-23), its products and sum by 2^-24 each, all relative to the sine, which so keeps its digits however slow
    the pair, up to the table's own 2^-64 turn a position. Angles under an eighth of a turn."""
    import torch

    pos = np.array([1, 2, 3, 100, 12345, -1, -77], dtype=np.int32)
    x = torch.zeros((len(pos), 1, rot), device=cuda)
    x[..., : rot // 2] = 1.0
    table, amp = _native.rope_frequencies(rot, **kw)
    out = torch.empty_like(x)
    _native.rope(x, out, table.to(cuda), rot, positions=torch.from_numpy(pos).to(cuda), amplitude=amp)
    f, _ = ref.frequencies(rot, **kw)
    angle = pos[:, None] * f[None, :]
    small = np.abs(angle) < np.pi / 4
    assert small.sum() > len(pos) * rot // 8 and np.abs(angle[small]).min() < 2e-6
    off = np.abs(P.host(out)[:, 0, rot // 2:] / np.sin(angle) - 1)
    tol = 5 * 2.0 ** -24 + np.broadcast_to(2.0 ** -64 * 2 * np.pi / f, angle.shape)
    assert np.all((off <= tol)[small]), (off / tol)[small].max()


@pytest.mark.parametrize("dim", [32, 34])
def test_a_capacity_far_beyond_the_rows(cuda, dim):
    """Buffers of 9000 rows of which the requests have 12: CTAs that hold some of them, and none, leave the rest."""
    import torch

    cu, cached = np.array([0, 4, 4, 9], dtype=np.int32), np.array([7, 0, 100], dtype=np.int32)
    x = torch.full((9000, 3, dim), float("nan"), device=cuda)
    x[:12] = torch.randn((12, 3, dim), generator=torch.Generator().manual_seed(dim)).to(cuda)
    out = torch.full_like(x, 7.0)
    table = _native.rope_frequencies(dim)[0].to(cuda)
    _native.rope(x, out, table, dim, cu_num_draft=torch.from_numpy(cu).to(cuda), cached_len=torch.from_numpy(cached).to(cuda), B=3)
    pos = np.array([cached[b] + j for b, j in ref.owners(cu, 3)])
    check(P.host(out)[:12], P.host(x)[:12], pos, ref.frequencies(dim)[0], "f32", False, 1.0)
    assert (out[12:] == 7).all()


def test_rows_behind_the_capacity_are_refused(cuda):
    """Offsets that name more rows than x has: the request's rows are left as they were, as a malformed one's are."""
    import torch

    x, out = torch.ones((4, 1, 16), device=cuda), torch.full((4, 1, 16), 7.0, device=cuda)
    _native.rope(x, out, _native.rope_frequencies(16)[0].to(cuda), 16, cu_num_draft=torch.tensor([0, 1, 3], dtype=torch.int32, device=cuda),
                 cached_len=torch.tensor([0, 0], dtype=torch.int32, device=cuda), B=2)           # request 1 would end at row 5
    assert (out[0] == 1).all() and not (out[1] == 7).any() and (out[2:] == 7).all()
