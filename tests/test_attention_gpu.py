"""The attention of a verify step over the paged cache (specdec_paged_attention) against the 64-bit definition."""
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


class Step:
    """A random step: q, cache, table, offsets, lengths and outputs (with guard rows behind the last request)."""

    def __init__(self, cuda, ks, cached, heads, group, dim, kind="bf16", cache_kind=None, page=16, seed=0, token_major=False,
                 q_scale=1.5, max_k=None, width=0):
        import torch

        rng = np.random.default_rng([seed, heads, group, dim, page])
        self.ks, self.cached, self.group, self.kind, self.page = list(ks), list(cached), group, kind, page
        self.cache_kind = cache_kind or kind
        self.B, self.cu = len(ks), P.offsets(ks)
        self.T = int(self.cu[-1]) + self.B
        self.max_k = max(ks) if max_k is None else max_k
        self.tab, pages = P.table([max(c, 0) + k + 1 for c, k in zip(cached, ks)], page, rng, width=width)
        self.cache = P.filled(pages, heads, page, dim, self.cache_kind, rng, cuda, token_major)
        H = heads * group
        self.q = torch.from_numpy((rng.standard_normal((self.T + 2, H, dim)) * q_scale).astype(np.float32)).to(P.torch_type(kind)).to(cuda)
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((self.T + 2, H), 7.0, device=cuda)
        self.status = torch.zeros(self.B, dtype=torch.int32, device=cuda)
        self.ws = torch.full((_native.paged_attention_workspace_size(self.B, self.max_k, H, heads, dim),), 0xFF, dtype=torch.uint8, device=cuda)
        self.dtab, self.dcached, self.dcu = dev(self.tab, cuda), dev(np.array(cached, dtype=np.int32), cuda), dev(self.cu, cuda)

    def run(self, **kw):
        a = dict(lse=self.lse, status=self.status)
        a.update(kw)
        _native.paged_attention(self.q, self.cache, self.dtab, self.dcached, self.dcu, self.B, self.max_k, self.out, self.ws, **a)
        return self

    def check(self, window=0, scale=None, skip=(), zeros=()):
        """Weights are rounded by at most half a step of their 16-bit type (f16 over an e4m3 cache, where a weight
        times its token's scale may also fall under f16's smallest step, 2^-24 of the largest scale's value),
        which moves out by that share of sum p |v|; a score is off by the fp32 sum of dim products of
        |q k|, each addition 2^-23 at most, and by its scaling; exp and the sums by 2^-20; then out's half step."""
        import torch

        torch.cuda.synchronize()
        gk, gv = P.held(self.cache)
        q, out, lse = P.host(self.q), P.host(self.out), P.host(self.lse)
        D = q.shape[2]
        scale = D ** -0.5 if scale is None else scale
        step = P.HALF["f16" if self.cache_kind == "e4m3" else self.kind]
        for b in range(self.B):
            r = slice(int(self.cu[b]) + b, int(self.cu[b + 1]) + b + 1)
            if b in skip:
                assert (out[r] == 7).all() and (lse[r] == 7).all()
                continue
            if b in zeros:
                assert (out[r] == 0).all() and (lse[r] == -np.inf).all()
                continue
            n = self.cached[b] + self.ks[b] + 1
            k, v = P.tokens(gk, self.tab[b], n, self.page), P.tokens(gv, self.tab[b], n, self.page)
            want, wl, spread = ref.attention(q[r], k, v, self.cached[b], scale, window)
            fine = np.isfinite(k).all(-1).all(-1)
            big = np.abs(k[fine]).max() if fine.any() else 0.0
            score = abs(scale) * np.abs(q[r]).sum(-1) * big * (D + 4) * 2.0 ** -23        # [rows, heads]
            vmax = np.abs(v[np.isfinite(v)]).max()
            tiny = vmax * 2.0 ** -24 * min(n, 64) if self.cache_kind == "e4m3" else 0.0
            tol = (step + 2 * score[..., None] + 2.0 ** -20) * spread + tiny
            tol = tol + P.HALF[self.kind] * (np.abs(want) + tol) + 2.0 ** -25
            good = np.isfinite(want)
            assert np.array_equal(np.isnan(out[r]), np.isnan(want))
            off = np.abs(out[r] - want)[good]
            assert np.all(off <= tol[good]), (b, (off / tol[good]).max())
            ok = np.isfinite(wl)
            assert np.array_equal(wl[~ok & ~np.isnan(wl)], lse[r][~ok & ~np.isnan(wl)])
            assert np.all(np.abs(lse[r] - wl)[ok] <= (score + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl))[ok])
        assert (out[self.T:] == 7).all() and (lse[self.T:] == 7).all()
        return self


TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")]


@pytest.mark.parametrize("kind,cache_kind", TYPES)
@pytest.mark.parametrize("heads,group,dim,page", [(1, 1, 16, 16), (2, 4, 64, 16), (3, 1, 80, 32), (2, 8, 128, 64), (1, 5, 96, 128),
                                                  (2, 16, 112, 256)])
def test_types_and_heads(cuda, kind, cache_kind, heads, group, dim, page):
    """Lengths around the tile of 128 and the page, single tokens and steps, empty caches."""
    cached = [0, 1, 15, 127, 128, 129, 255, 300, 1000]
    ks = [0, 3, 0, 2, 8, 1, 0, 4, 5]
    Step(cuda, ks, cached, heads, group, dim, kind, cache_kind, page).run().check()


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 7, 128, 129, 500])
def test_window(cuda, cache_kind, window):
    Step(cuda, [0, 5, 8, 3, 1], [0, 3, 126, 1000, 129], 2, 4, 64, "bf16", cache_kind, 32).run(window=window).check(window=window)


@pytest.mark.parametrize("kind,cache_kind", TYPES)
@pytest.mark.parametrize("cached", [0, 1, 100, 4096, 20000])
def test_one_request_split_over_its_length(cuda, kind, cache_kind, cached):
    Step(cuda, [0], [cached], 1, 8, 128, kind, cache_kind, 64).run().check()
    Step(cuda, [7], [cached], 2, 2, 64, kind, cache_kind, 16).run().check()


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("k,group", [(32, 1), (32, 4), (16, 16), (8, 8), (1, 40), (32, 16)])
def test_many_rows(cuda, cache_kind, k, group):
    """More query rows a key head than one tile holds, and more draft rows than a page."""
    Step(cuda, [k, 0, k // 2], [200, 500, 17], 1, group, 64, "bf16", cache_kind, 16).run().check()


@pytest.mark.parametrize("cache_kind", ["f16", "e4m3"])
def test_many_requests(cuda, cache_kind):
    """More requests than CTAs and than threads: ragged lengths, some empty."""
    rng = np.random.default_rng(8)
    B = 700
    Step(cuda, rng.integers(0, 4, size=B), rng.integers(0, 200, size=B), 2, 2, 32, "f16", cache_kind, 16).run().check()


def test_peaked_and_shifted_scores(cuda):
    """Scores in the hundreds that grow along the cache, so that the running maximum moves in every tile."""
    s = Step(cuda, [3, 0], [2000, 700], 1, 4, 64, "bf16", "bf16", 16, q_scale=20.0)
    s.run().check()
    ramp = np.linspace(-1, 1, s.cache.num_pages)
    s.cache.k.add_(dev(ramp.astype(np.float32), cuda).to(s.cache.k.dtype)[:, None, None, None])
    s.q.abs_()
    s.run(scale=1.0).check(scale=1.0)
    s.run(scale=0.0).check(scale=0.0)
    s.run(scale=-0.5).check(scale=-0.5)


def test_scales_that_differ_widely(cuda):
    """An e4m3 cache whose tokens' scales differ by up to 2^20, for keys and values, in any order."""
    import torch

    s = Step(cuda, [2, 0], [900, 300], 2, 4, 64, "bf16", "e4m3", 16)
    g = torch.Generator(device="cpu").manual_seed(1)
    s.cache.v_exp.copy_(torch.randint(100, 121, s.cache.v_exp.shape, generator=g, dtype=torch.uint8))
    s.cache.k_exp.copy_(torch.randint(100, 121, s.cache.k_exp.shape, generator=g, dtype=torch.uint8))
    s.run().check()


@pytest.mark.parametrize("kind,cache_kind", [("bf16", "bf16"), ("f16", "e4m3")])
def test_what_a_row_does_not_see_does_not_reach_it(cuda, kind, cache_kind):
    """NaN and infinities behind the last token, in later drafts' rows, before the window, and in unused pages."""
    import torch

    for window in (0, 40):
        s = Step(cuda, [4, 0, 8], [150, 127, 260], 2, 4, 64, kind, cache_kind, 16)
        ref_out = s.run(window=window).check(window=window).out.clone()
        live = np.zeros((s.cache.num_pages, s.page), dtype=bool)
        last = []
        for b in range(3):
            n = s.cached[b] + s.ks[b] + 1
            for i in range(max(0, s.cached[b] - window + 1) if window else 0, n):
                live[s.tab[b, i // s.page], i % s.page] = True
            last.append((s.tab[b, (n - 1) // s.page], (n - 1) % s.page))
        for x in (s.cache.k, s.cache.v):
            codes = x.view(torch.uint8 if cache_kind == "e4m3" else torch.int16)
            # NaN in every place that no row sees (all bits but the sign: NaN in each of the types)
            mask = dev(~live, cuda)[:, None, :, None].expand(codes.shape)
            codes.masked_fill_(mask, 0x7F if cache_kind == "e4m3" else 0x7FFF)
        s.run(window=window).check(window=window)
        assert torch.equal(s.out, ref_out)
        # the last draft's own key and value: only the last row of each request sees them
        for (p, sl) in last:
            s.cache.v.view(torch.uint8 if cache_kind == "e4m3" else torch.int16)[p, :, sl] = 0x7F if cache_kind == "e4m3" else 0x7FFF
        s.run(window=window).check(window=window)
        for b in range(3):
            a, z = int(s.cu[b]) + b, int(s.cu[b + 1]) + b
            assert torch.equal(s.out[a:z], ref_out[a:z]) and torch.isnan(s.out[z].float()).all()


def test_infinite_and_nan_scores(cuda):
    """A NaN in one query row stays in it; keys of minus infinity for a whole row leave zeros and lse = -inf."""
    import torch

    s = Step(cuda, [2], [140], 1, 2, 32, "bf16", "bf16", 16)
    s.q[1, 0, 3] = float("nan")
    s.run().check()
    s.q.copy_(torch.ones_like(s.q))
    s.cache.k.fill_(-float("inf"))
    s.run()
    torch.cuda.synchronize()
    assert (s.out[:3] == 0).all() and (s.lse[:3] == -float("inf")).all()


def test_layouts(cuda):
    """Slot-major caches, q and out as slices and transposes, a wide table."""
    import torch

    for cache_kind in ("bf16", "e4m3"):
        s = Step(cuda, [3, 1], [77, 200], 2, 4, 64, "bf16", cache_kind, 32, token_major=True, width=40)
        s.run().check()
        want = s.out.clone()
        big = torch.zeros((s.T + 2, 12, 64), dtype=s.q.dtype, device=cuda)
        big[:, 2:10] = s.q
        s.q = big[:, 2:10]
        turned = torch.full((8, s.T + 2, 64), 7.0, dtype=s.q.dtype, device=cuda)
        s.out = turned.transpose(0, 1)
        s.run().check()
        assert torch.equal(s.out, want)


def test_faults(cuda):
    """Skipped, over-long, over-wide and malformed requests; a bad page reads as zeros; the others are exact."""
    import torch

    s = Step(cuda, [1, 2, 5, 0], [100, -1, 40, 60], 1, 4, 64, "bf16", "bf16", 16, max_k=2)
    s.run()
    assert s.status.tolist() == [0, _native.ST_BAD_LENGTH, _native.ST_K_TOO_LARGE, 0]
    s.check(zeros=(1, 2))
    s.dtab = s.dtab[:, :4].contiguous()                      # request 0 needs seven pages
    s.status.zero_()
    s.run()
    assert s.status.tolist() == [_native.ST_BAD_LENGTH, _native.ST_BAD_LENGTH, _native.ST_K_TOO_LARGE, 0]
    s.check(zeros=(0, 1, 2))
    s = Step(cuda, [1, 0], [100, 60], 1, 4, 64, "bf16", "bf16", 16)
    s.dtab[0, 2], s.dtab[1, 0] = s.cache.num_pages, -5
    s.run()
    assert s.status.tolist() == [_native.ST_BAD_PAGE] * 2
    free = [p for p in range(s.cache.num_pages) if p not in s.tab[0, :7] and p not in s.tab[1, :4]][0]
    s.cache.k[free], s.cache.v[free] = 0, 0
    s.tab[0, 2], s.tab[1, 0] = free, free
    s.check()
    for bad in ([1, 2, 3], [0, 9, 2]):
        s = Step(cuda, [1, 0], [20, 10], 1, 2, 32)
        s.dcu.copy_(torch.tensor(bad, dtype=torch.int32))
        s.run()
        assert s.status.tolist() == [_native.ST_BAD_OFFSETS] * 2
        s.check(skip=(0, 1))


def test_equal_calls_give_equal_bits_and_rows_do_not_depend_on_the_batch(cuda):
    import torch

    s = Step(cuda, [3, 0, 8, 1], [3000, 0, 777, 128], 2, 4, 128, "bf16", "bf16", 16).run()
    one = s.out.clone(), s.lse.clone()
    s.ws.fill_(0x5A)
    s.out.fill_(7.0)
    s.run()
    assert torch.equal(s.out, one[0]) and torch.equal(s.lse, one[1])


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
def test_capture_and_replay_with_other_lengths(cuda, cache_kind):
    """A captured call replayed after the lengths, the table and q changed; two graphs share the workspace one
    after the other; a call on a side stream."""
    import torch

    s = Step(cuda, [2, 2, 2], [1000, 5, 300], 2, 4, 64, "bf16", cache_kind, 16)
    s.run().check()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for cached in ([10, 700, 0], [500, 128, 127]):
        n = [c + 3 for c in cached]
        rng = np.random.default_rng(sum(cached))
        s.cached = cached
        perm = rng.permutation(s.cache.num_pages)
        s.tab[:] = -7
        at = 0
        for b in range(3):
            m = -(-n[b] // 16)
            s.tab[b, :m] = perm[at: at + m]
            at += m
        s.dtab.copy_(torch.from_numpy(s.tab))
        s.dcached.copy_(torch.tensor(cached, dtype=torch.int32))
        s.q.mul_(-0.5)
        for g in graphs:
            s.out.fill_(7.0)
            g.replay()
            s.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.out.fill_(7.0)
    side.wait_stream(torch.cuda.current_stream())
    s.run(stream=side)
    side.synchronize()
    s.check()


def test_two_streams_with_a_workspace_each(cuda):
    import torch

    steps = [Step(cuda, [3] * 40, list(range(0, 4000, 100)), 2, 4, 128, "bf16", c, 16, seed=i) for i, c in enumerate(("bf16", "e4m3"))]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s in steps:
        s.check()


def test_lse_and_status_are_optional_and_join_two_halves(cuda):
    """Results over two ranges of keys, joined by their lse, equal the whole."""
    import torch

    s = Step(cuda, [0], [599], 1, 4, 64, "f16", "f16", 16)
    s.run(status=None).check()
    whole = P.host(s.out)[0]
    parts = []
    for lo, hi in ((0, 320), (320, 600)):
        tab = s.dtab[:, lo // 16:].contiguous()
        out, lse = torch.empty_like(s.out), torch.empty_like(s.lse)
        _native.paged_attention(s.q, s.cache, tab, torch.tensor([hi - lo - 1], dtype=torch.int32, device=cuda), s.dcu, 1, 0, out, s.ws, lse=lse)
        parts.append((P.host(out)[0], P.host(lse)[0]))
    w = [np.exp(l - np.logaddexp(parts[0][1], parts[1][1]))[:, None] for _, l in parts]
    joined = w[0] * parts[0][0] + w[1] * parts[1][0]
    assert np.abs(joined - whole).max() <= 4 * 2.0 ** -11 * np.abs(whole).max() + 2.0 ** -10
    s.lse.fill_(7.0)
    s.run(lse=None, status=None)
    torch.cuda.synchronize()
    assert (s.lse == 7).all()


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("k,group", [(0, 1), (8, 8)])
def test_wait_expiry_is_reported_and_the_context_stays_usable(cuda, cache_kind, k, group):
    """With every wait inside the kernel limited to 0 us, waits expire: the requests get DEVICE_TIMEOUT, the call
    ends, rows behind the last request stay, and the same step is then exact with the default limit."""
    import torch

    s = Step(cuda, [k] * 6, [3000] * 6, 2, group, 128, "bf16", cache_kind, 16)
    s.run(wait_limit_us=0)
    torch.cuda.synchronize()
    assert ((s.status & _native.ST_DEVICE_TIMEOUT) != 0).all()
    assert (s.out[s.T:] == 7).all() and (s.lse[s.T:] == 7).all()
    s.status.zero_()
    s.run().check()
    assert (s.status == 0).all()


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_before_the_window_may_be_gone(cuda, cache_kind, page):
    """Block-table entries of pages that lie wholly before every row's window are not read."""
    import torch

    s = Step(cuda, [3, 0], [1000, 517], 2, 4, 64, "bf16", cache_kind, page)
    want = s.run(window=150).check(window=150).out.clone()
    for b in range(2):
        s.dtab[b, : (s.cached[b] - 150 + 1) // page] = -1
    s.out.fill_(7.0)
    s.run(window=150)
    assert torch.equal(s.out, want) and (s.status == 0).all()


def test_rows_behind_the_capacity_are_refused(cuda):
    """Offsets that name more rows than q and out have: the request is reported and nothing of it is read or written."""
    import torch

    s = Step(cuda, [1, 2], [40, 70], 1, 2, 64)
    s.q, s.out, s.lse = s.q[:4], s.out[:4], s.lse[:4]                 # request 1 would end at row 5
    s.T, s.B = 4, 2
    s.run()
    torch.cuda.synchronize()
    assert s.status.tolist() == [0, _native.ST_BAD_OFFSETS]
    assert (s.out[2:] == 7).all() and (s.lse[2:] == 7).all() and not (s.out[:2] == 7).any()


def test_a_scale_that_is_no_number_stays_in_the_rows_that_see_it(cuda):
    """Exponent byte 255 on the last draft's key and value: NaN in the last row alone."""
    import torch

    s = Step(cuda, [4], [200], 2, 4, 64, "bf16", "e4m3", 16)
    want = s.run().check().out.clone()
    p, sl = s.tab[0, 204 // 16], 204 % 16
    for e in (s.cache.v_exp, s.cache.k_exp):
        keep = e[p, :, sl].clone()
        e[p, :, sl] = 255
        s.run()
        torch.cuda.synchronize()
        assert torch.equal(s.out[:4], want[:4]) and torch.isnan(s.out[4].float()).all()
        e[p, :, sl] = keep


def test_no_rows_and_no_requests(cuda):
    """Empty calls launch nothing and leave everything as it was."""
    import torch

    s = Step(cuda, [0], [10], 1, 1, 32)
    args = (s.cache, s.dtab, s.dcached, s.dcu)
    _native.paged_attention(s.q, *args, 0, 0, s.out, s.ws)
    _native.paged_attention(s.q[:0], *args, 1, 0, s.out[:0], s.ws)
    torch.cuda.synchronize()
    assert (s.out == 7).all()


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("k,group", [(3, 4), (32, 1)])
def test_windows_that_hide_nothing(cuda, cache_kind, k, group):
    """A window as long as the longest request, as its row of the table, and up to the largest number equals no window,
    bit for bit; lengths whose last tile begins behind `cached`."""
    import torch

    # 50 pages of 16 a request: more than the 701 + k tokens of the longest
    s = Step(cuda, [k, k, k, 0], [125, 127, 700, 0], 2, group, 64, "bf16", cache_kind, 16, width=50)
    want = s.run().check().out.clone(), s.lse.clone()
    capacity = s.dtab.shape[1] * s.page
    for window in (700 + k + 1, capacity - 1, capacity, capacity + 1, 2 ** 31 - 200, 2 ** 31 - 130, 2 ** 31 - 129, 2 ** 31 - 2, 2 ** 31 - 1):
        s.out.fill_(7.0)
        s.lse.fill_(7.0)
        s.run(window=window)
        assert torch.equal(s.out, want[0]) and torch.equal(s.lse, want[1]), window
    assert (s.status == 0).all()


def test_a_wide_table_and_a_window_next_to_the_largest(cuda):
    """Rows of block_table that could hold 2^31 tokens, of which only the first pages are there: windows just under what 32-bit differences bear, in a tile that begins behind `cached`."""
    import torch

    s = Step(cuda, [3, 32], [125, 1000], 1, 2, 64, "bf16", "bf16", 256)
    want = s.run().check().out.clone()
    wide = torch.full((2, 2 ** 23), -1, dtype=torch.int32, device=cuda)         # 2^31 tokens a request
    wide[:, : s.dtab.shape[1]] = s.dtab
    s.dtab = wide
    for window in (2 ** 31 - 131, 2 ** 31 - 130, 2 ** 31 - 129, 2 ** 31 - 1):
        s.out.fill_(7.0)
        s.run(window=window)
        assert torch.equal(s.out, want), window
    s.run(window=60).check(window=60)
    assert (s.status == 0).all()


@pytest.mark.parametrize("kind,cache_kind", TYPES)
@pytest.mark.parametrize("k,group,dim", [(8, 8, 128), (8, 8, 80), (7, 16, 128), (32, 16, 128)])
def test_short_items_with_one_buffer_for_q(cuda, kind, cache_kind, k, group, dim):
    """Items of one or two tiles at 72 and 128 rows a key head (and several row blocks) of heads over 64: their scores wait
    for nothing but Q, which there has a single buffer that is filled again as soon as all its readers have passed."""
    import torch

    rng = np.random.default_rng([k, group, dim])
    B, cached = 90, rng.integers(0, 200, size=90)
    cached[:3] = 0, 127, 128
    s = Step(cuda, [k] * B, cached, 3, group, dim, kind, cache_kind, 16)
    want = s.run().check().out.clone()
    for _ in range(20):
        s.run()
    torch.cuda.synchronize()
    assert (s.status == 0).all() and torch.equal(s.out, want)


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("k,group,block", [(3, 16, 0), (3, 16, 1), (8, 8, 1), (8, 8, 2), (7, 16, 0), (7, 16, 3)])
@pytest.mark.parametrize("B,heads,cached", [(160, 1, 500), (1, 8, 9000)])
def test_value_scales_that_rise_where_some_columns_scores_do(cuda, kind, dim, k, group, block, B, heads, cached):
    """64, 96 and 128 rows a key head over an e4m3 cache, whose columns are dealt with 32 at a time: in every second tile the
    values' scales are 2 to 2^4 times those of the tile before, and the scores of one block of 32 columns alone are
    higher by 12 in log2, so that this block moves its reference and the others do not. Many items a CTA, and items cut
    among the CTAs with some tiles each."""
    import torch

    s = Step(cuda, [k] * B, [cached] * B, heads, group, dim, kind, "e4m3", 16)
    rng = np.random.default_rng([k, group, block, B])
    n = cached + k + 1
    odd = (np.arange(n) // 128) % 2 == 1
    lift = 12.0 * np.log(2.0) * dim ** 0.5 / 32.0            # times the block's 32 in Q, and scale: 12 in log2
    keys = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32))
    keys[..., 0] = torch.from_numpy(np.where(odd, lift, 0.0).astype(np.float32))[:, None]
    s.cache.k_exp.fill_(127)
    s.cache.v_exp.fill_(118)
    for b in range(B):
        page = torch.from_numpy(s.tab[b, np.arange(n) // s.page].astype(np.int64)).to(cuda)
        slot = torch.arange(n, device=cuda) % s.page
        s.cache.k.view(torch.uint8)[page, :, slot] = keys.to(torch.float8_e4m3fn).view(torch.uint8).to(cuda)
        s.cache.v_exp[page, :, slot] = dev(np.where(odd, 118 + rng.integers(1, 5), 118).astype(np.uint8), cuda)[:, None].expand(-1, heads)
    rows = (torch.arange((k + 1) * group) // 32 == block).view(1, k + 1, 1, group)
    s.q[: s.T, :, 0] = torch.where(rows, 32.0, 0.0).expand(B, -1, heads, -1).reshape(s.T, -1).to(s.q.dtype).to(cuda)
    s.run().check()


def test_one_row_of_one_head_with_any_strides(cuda):
    """A single row, head and request out of tensors whose row and head strides fit no alignment: they are never taken."""
    import torch

    s = Step(cuda, [0], [40], 1, 1, 32)
    want = s.run().check().out[:1].clone()
    k = torch.ones((1, 1, 32), dtype=torch.bfloat16, device=cuda)
    q, out, v = (t.as_strided((1, 1, 32), (77, 33, 1)) for t in (s.q, torch.zeros_like(want), 2 * k))
    _native.paged_attention(q, s.cache, s.dtab, s.dcached, s.dcu, 1, 0, out, s.ws)
    assert torch.equal(out, want)
    _native.kv_write(k, v, s.cache, s.dtab, s.dcached, s.dcu, 1)
    back = torch.zeros((1, 1, 32), dtype=torch.bfloat16, device=cuda), torch.zeros(200, dtype=torch.bfloat16, device=cuda).as_strided((1, 1, 32), (5, 7, 1))
    _native.kv_read(s.cache, s.dtab, torch.tensor([0, 1], dtype=torch.int64, device=cuda), 1, *back, first=s.dcached)
    assert (back[0] == 1).all() and (back[1] == 2).all()


@pytest.mark.parametrize("kind,dim,group,by", [("bf16", 64, 4, 5), ("bf16", 64, 4, 30), ("bf16", 128, 16, 12), ("bf16", 128, 16, 90),
                                               ("f16", 128, 4, 5), ("f16", 128, 4, 12)])
@pytest.mark.parametrize("cached", [0, 124, 125, 128, 130, 900])
def test_a_scale_that_is_large_stays_in_the_rows_that_see_it(cuda, kind, dim, group, by, cached):
    """The values of one of the last two drafts 2^by times the others' (f16 outputs hold 448 * 2^(121 - 127 + 12), not 2^30),
    then those of the oldest token of the first row's window: the rows that do not see them give the same bits as
    without, those that do are exact. Tiles that some or most rows see nothing of, first and later ones."""
    import torch

    s = Step(cuda, [4, 0], [cached, 3000], 2, group, dim, kind, "e4m3", 16)
    want = s.run().check().out.clone()
    for j in (4, 3):
        p, sl = s.tab[0, (cached + j) // 16], (cached + j) % 16
        keep = s.cache.v_exp[p, :, sl].clone()
        s.cache.v_exp[p, :, sl] = keep + by
        s.run().check()
        assert torch.equal(s.out[:j], want[:j]) and torch.equal(s.out[5:], want[5:])
        assert not torch.equal(s.out[j], want[j]) and (s.status == 0).all()
        s.cache.v_exp[p, :, sl] = keep
    for window in (100, 128, 700):
        if window > cached:
            continue
        want = s.run(window=window).check(window=window).out.clone()
        first = cached - window + 1                                  # the first row alone sees it
        p1, s1 = s.tab[0, first // 16], first % 16
        keep1 = s.cache.v_exp[p1, :, s1].clone()
        s.cache.v_exp[p1, :, s1] = keep1 + by
        s.run(window=window).check(window=window)
        assert torch.equal(s.out[1:], want[1:]) and not torch.equal(s.out[0], want[0])
        s.cache.v_exp[p1, :, s1] = keep1


@pytest.mark.parametrize("kind,dim,group", [("bf16", 64, 4), ("bf16", 128, 8), ("f16", 32, 16)])
@pytest.mark.parametrize("window", [1, 2, 4, 100])
@pytest.mark.parametrize("cached", [0, 121, 124, 127, 700])
def test_scales_of_rows_that_share_no_token(cuda, kind, dim, group, window, cached):
    """Windows under the step's own rows, or that begin at the end of a tile: no token of a tile may be seen by every row, and
    the rows' own scales rise or fall by up to 2^24 (f16: 2^12) from one to the next. Each row is exact by its own values."""
    import torch

    k, step = 8, 3 if kind == "bf16" else 1
    for sign in (1, -1):
        s = Step(cuda, [k, 0], [cached, 260], 2, group, dim, kind, "e4m3", 16)
        for i in range(cached + k + 1):
            s.cache.v_exp[s.tab[0, i // 16], :, i % 16] = 112 + sign * step * (i % 9 - 4)
        s.run(window=window)
        torch.cuda.synchronize()
        gk, gv = P.held(s.cache)
        kk, vv = P.tokens(gk, s.tab[0], cached + k + 1, 16), P.tokens(gv, s.tab[0], cached + k + 1, 16)
        q, out = P.host(s.q), P.host(s.out)
        for j in range(k + 1):                       # row by row: its tolerance is by what it sees itself, not by the largest scale
            n = cached + j + 1
            first = max(0, n - window)
            want, _, spread = ref.attention(q[j: j + 1], kk[:n], vv[:n], n - 1, dim ** -0.5, window)
            score = dim ** -0.5 * np.abs(q[j]).sum(-1) * np.abs(kk[:n]).max() * (dim + 4) * 2.0 ** -23
            tiny = np.abs(vv[first: n]).max() * 2.0 ** -24 * min(n - first, 64)
            tol = (2.0 ** -11 + 2 * score[:, None] + 2.0 ** -20) * spread[0] + tiny
            tol = tol + P.HALF[kind] * (np.abs(want[0]) + tol) + (2.0 ** -25 if kind == "f16" else 2.0 ** -134)
            assert np.all(np.abs(out[j] - want[0]) <= tol), (j, (np.abs(out[j] - want[0]) / tol).max())
        assert (s.status == 0).all()


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 256)])
def test_a_bad_page_of_a_quantised_cache_reads_as_zeros(cuda, dim, page):
    """Its tokens have no scale: the others' weights keep their bits, small as their values are (scales of 2^-22 and less)."""
    s = Step(cuda, [2, 0], [900, 700], 2, 4, dim, "bf16", "e4m3", page)
    s.cache.v_exp.copy_(s.cache.v_exp - 14)
    s.dtab[0, 1], s.dtab[1, 0] = s.cache.num_pages, -5
    s.run()
    assert s.status.tolist() == [_native.ST_BAD_PAGE] * 2
    free = [p for p in range(s.cache.num_pages) if p not in s.tab][0]
    s.cache.k[free], s.cache.v[free] = 0, 0
    s.tab[0, 1], s.tab[1, 0] = free, free
    s.check()
