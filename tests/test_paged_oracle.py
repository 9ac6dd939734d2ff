"""Pins of the host definitions of rotary positions, the e4m3 cache and the attention (no GPU)."""
import numpy as np
import pytest

from oracle import paged_ref as ref
from speculative_decoding_verification_specdec_gb300 import _native, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    if build.needs_rebuild():
        build.build_library()
    return _native.load()


def test_e4m3_codes_round_to_nearest_even():
    assert ref.E4M3[126] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6
    finite = [c for c in range(256) if np.isfinite(ref.E4M3[c])]
    assert all(ref.e4m3_code(ref.E4M3[c]) == c for c in finite)
    mid = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2
    assert np.array_equal(ref.e4m3_code(mid), np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127)))
    assert ref.e4m3_code(np.inf) == 127 and ref.e4m3_code(np.nan) == 127


def test_e4m3_exponent_is_the_smallest():
    for top, e in ((448.0, 0), (448.0001, 1), (224.0, -1), (224.1, 0), (0.0, 0), (2.0 ** -140, -126), (3.4e38, 120)):
        assert ref.e4m3_exponent(np.array([0.0, -top, top / 3])) == e, top
    assert ref.e4m3_exponent(np.array([np.inf, 1.0])) == -8


@pytest.mark.parametrize("kw", [{}, dict(scaling="linear", factor=4.0),
                                dict(scaling="by_parts", factor=8.0, original_len=4096, beta_fast=32.0, beta_slow=1.0),
                                dict(theta=500000.0)])
@pytest.mark.parametrize("rot", [2, 64, 128, 256])
def test_frequency_table(kw, rot):
    """The library's host table against 64-bit frequencies: a double's 2^-52 and the table's 2^-64 turn."""
    table, amp = _native.rope_frequencies(rot, **kw)
    f, a = ref.frequencies(rot, **kw)
    turns = table.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    assert np.all(np.abs(turns - f / (2 * np.pi)) <= 2.0 ** -50 * turns + 2.0 ** -64)
    assert abs(amp - a) <= 2.0 ** -23 * a


def test_frequency_refusals(lib):
    E = _native
    ok = dict(rot_dim=64, theta=1e4, scaling=0, factor=1.0, original_len=0, fast=32.0, slow=1.0)

    def call(out=True, **o):
        import ctypes
        a = {**ok, **o}
        buf = (ctypes.c_uint64 * 256)()
        return lib.specdec_rope_frequencies(a["rot_dim"], a["theta"], a["scaling"], a["factor"], a["original_len"], a["fast"],
                                            a["slow"], ctypes.addressof(buf) if out else None, None)

    assert call() == E.SPECDEC_OK
    for bad in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=258), dict(theta=0.5), dict(theta=float("nan")), dict(theta=float("inf")),
                dict(scaling=3), dict(scaling=1, factor=0.0), dict(scaling=1, factor=float("inf")), dict(scaling=2, factor=2.0),
                dict(scaling=2, factor=2.0, original_len=4096, fast=1.0, slow=1.0), dict(out=False)):
        assert call(**bad) == E.SPECDEC_ERR_INVALID_ARG, bad


def test_rope_definition_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 12))
    pos = np.array([0, 1, -4, 1000, 2 ** 30])
    for inter in (False, True):
        f, _ = ref.frequencies(8)
        y = ref.rope(x, pos, f, inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(ref.rope(y, pos, f, inter, inverse=True), x)
        # scores depend on the distance of the positions alone
        a, b = rng.standard_normal((2, 1, 1, 12))
        s = [np.sum(ref.rope(a, [p + 7], f, inter) * ref.rope(b, [p], f, inter)) for p in (0, 1, 500)]
        assert np.allclose(s, s[0])


def test_attention_definition():
    rng = np.random.default_rng(1)
    k, v, q = rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 2, 4)), rng.standard_normal((3, 4, 4))
    out, lse, spread = ref.attention(q, k, v, 6, 0.5)
    z = 0.5 * k[:8, 1] @ q[1, 3]
    w = np.exp(z) / np.exp(z).sum()
    assert np.allclose(out[1, 3], w @ v[:8, 1]) and np.isclose(lse[1, 3], np.log(np.exp(z).sum()))
    one, _, _ = ref.attention(q, k, v, 6, 0.5, window=1)
    assert np.allclose(one[2, 0], v[8, 0])
    # values of tokens that a row does not see do not reach it
    v[8] = np.nan
    again, _, _ = ref.attention(q, k, v, 6, 0.5)
    assert np.array_equal(again[:2], out[:2]) and np.isnan(again[2]).all()
