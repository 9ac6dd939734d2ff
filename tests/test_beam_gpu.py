"""specdec_beam_select and specdec_kv_fork against the 64-bit definitions, and beam steps over one cache as they are used."""
import numpy as np
import pytest

import _logits as L
import _paged as P
from oracle import logits_ref as ref
from oracle import paged_ref
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


def select(x, scores, n, mask=None, finished=None, end_token=-1):
    import torch

    B, W = scores.shape
    d = x.device
    rows, tokens = (torch.full((B + 2, n), -77, dtype=torch.int32, device=d) for _ in range(2))
    out, ended = torch.full((B + 2, n), 77.0, device=d), torch.full((B + 2, n), 7, dtype=torch.uint8, device=d)
    status = torch.zeros(B, dtype=torch.int32, device=d)
    size = _native.beam_select_workspace_size(B, W, x.shape[1], x.dtype, n)
    ws = torch.full((size + 64,), 0x5a, dtype=torch.uint8, device=d)
    _native.beam_select(x, L.dev(scores), rows[1:-1], tokens[1:-1], out[1:-1], ws[:size], bitmask=mask,
                        finished=None if finished is None else L.dev(finished), end_token=end_token, out_finished=ended[1:-1], status=status)
    torch.cuda.synchronize()
    for t, g in ((rows, -77), (tokens, -77), (out, 77.0), (ended, 7)):
        assert (t[0] == g).all() and (t[-1] == g).all()
    assert (ws[size:] == 0x5a).all()
    return [t[1:-1].cpu().numpy() for t in (rows, tokens, out, ended)] + [status.cpu().numpy()]


def check(got, z, scores, n, masks=None, finished=None, end_token=-1):
    rows, tokens, out, ended, status = got
    B, W = scores.shape
    z = z.reshape(B, W, -1)
    for b in range(B):
        m = None if masks is None else masks.reshape(B, W, -1)[b]
        wb, wt, ws, we, found = ref.beam_select(z[b], scores[b], n, m, None if finished is None else finished[b], end_token)
        finite = z[b][np.isfinite(z[b])]
        err = L.lse_error(finite)[0]
        # candidates of different beams nearer than both sums' errors may fall either way: the seeds keep clear of that
        near = [f for f in zip(found[:n], found[1: n + 1]) if f[0][1] != f[1][1] and 0 < f[0][0] - f[1][0] <= 2 * err]
        assert not near
        assert list(rows[b]) == [b * W + w if w >= 0 else -1 for w in wb] and list(tokens[b]) == wt and list(ended[b]) == we, b
        for g, w in zip(out[b], ws):
            assert g == w or abs(g - w) <= err + L.U * abs(w)


def start(rng, B, W):
    return (-rng.uniform(0, 20, (B, 1)) - np.cumsum(rng.uniform(0, 2, (B, W)), 1)).astype(np.float32)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,W,V,n", [(1, 1, 1, 1), (3, 1, 50, 4), (2, 4, 1000, 4), (5, 3, 4099, 7), (2, 32, 600, 64), (3, 8, 33001, 16),
                                     (1, 128, 40, 32), (2, 2, 3, 128)])
def test_steps(cuda, kind, B, W, V, n):
    """Down to one id, and more survivors asked for than there are candidates."""
    rng = np.random.default_rng([B, W, V, n])
    x, z = L.rows(rng, B * W, V, kind)
    scores = start(rng, B, W)
    check(select(x, scores, n, end_token=V // 2), z, scores, n, end_token=V // 2)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_finished_and_unbegun_beams_and_masks(cuda, kind):
    """Finished beams go on at their score unread (their rows hold NaN), beams not begun have nothing, one row allows nothing."""
    rng = np.random.default_rng(6)
    B, W, V = 4, 4, 2005
    x, z = L.rows(rng, B * W, V, kind, extra=3, shift=1)
    scores = start(rng, B, W)
    finished = np.zeros((B, W), dtype=np.uint8)
    finished[0, 1] = finished[2] = finished[3, 0] = 1
    scores[1, 1:] = -np.inf
    scores[3, 0] = -np.inf
    x[1] = np.nan
    x[5:8] = np.nan
    allowed = rng.random((B * W, V)) < 0.1
    allowed[14] = False
    z[1] = z[5:8] = 0
    got = select(x, scores, 6, mask=L.dev(L.pack(allowed)), finished=finished, end_token=9)
    check(got, z, scores, 6, allowed, finished, 9)
    assert list(got[4]) == [0, 0, 0, _native.ST_EMPTY_MASK_ROW]


def test_ties_fall_to_the_lower_beam_and_id(cuda):
    x, _ = L.rows(np.random.default_rng(2), 6, 500, "f32")
    x[:] = (x[0] * 2).round() / 2
    scores = np.full((2, 3), -1.0, dtype=np.float32)
    check(select(x, scores, 40), P.host(x), scores, 40)


def test_scores_that_are_none(cuda):
    """NaN and +infinity as scores and in rows: those beams have no continuation, the others are untouched."""
    rng = np.random.default_rng(3)
    x, z = L.rows(rng, 8, 300, "f32")
    scores = start(rng, 2, 4)
    scores[0, 0], scores[0, 1] = np.nan, np.inf
    x[4, 7], x[5, 7] = np.nan, np.inf
    want = scores.copy()
    want[1, :2] = -np.inf
    got = select(x, scores, 8)
    check(got, z, want, 8)
    assert list(got[4]) == [_native.ST_BAD_SCORE] * 2


def test_scores_and_flags_in_place(cuda):
    """out_scores over scores and out_finished over finished, as a captured loop has them."""
    import torch

    rng = np.random.default_rng(4)
    B, W, V = 3, 5, 800
    x, z = L.rows(rng, B * W, V, "bf16")
    scores, finished = start(rng, B, W), (rng.random((B, W)) < 0.3).astype(np.uint8)
    s, f = L.dev(scores), L.dev(finished)
    rows, tokens = (torch.empty((B, W), dtype=torch.int32, device=cuda) for _ in range(2))
    ws = torch.empty(_native.beam_select_workspace_size(B, W, V, x.dtype, W), dtype=torch.uint8, device=cuda)
    _native.beam_select(x, s, rows, tokens, s, ws, finished=f, end_token=1, out_finished=f)
    torch.cuda.synchronize()
    check([t.cpu().numpy() for t in (rows, tokens, s, f)] + [None], z, scores, W, finished=finished, end_token=1)


def test_steps_that_follow_at_once(cuda):
    """Captured steps one behind the other over scores and flags in place, many short requests to a line of memory."""
    import torch

    rng = np.random.default_rng(9)
    B, W, V, steps = 40, 2, 300, 6
    xs = [L.rows(rng, B * W, V, "f32") for _ in range(steps)]
    scores, finished = start(rng, B, W), np.zeros((B, W), dtype=np.uint8)
    s, f = L.dev(scores), L.dev(finished)
    rows, tokens = (torch.empty((steps, B, W), dtype=torch.int32, device=cuda) for _ in range(2))
    ws = torch.empty(_native.beam_select_workspace_size(B, W, V, s.dtype, W), dtype=torch.uint8, device=cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, (x, _) in enumerate(xs):
            _native.beam_select(x, s, rows[i], tokens[i], s, ws, finished=f, end_token=5, out_finished=f)
    for _ in range(20):
        s.copy_(L.dev(scores))
        f.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, done = scores, finished
        for i, (_, z) in enumerate(xs):
            got = [ref.beam_select(z.reshape(B, W, V)[b], want[b], W, finished=done[b], end_token=5) for b in range(B)]
            assert rows[i].tolist() == [[b * W + w for w in g[0]] for b, g in enumerate(got)] and tokens[i].tolist() == [g[1] for g in got]
            want, done = np.array([g[2] for g in got]).astype(np.float32), np.array([g[3] for g in got], dtype=np.uint8)
        assert np.abs(s.cpu().numpy() - want).max() <= steps * (L.lse_error(z)[0] + 40 * L.U) and np.array_equal(f.cpu().numpy(), done)


# ---------------------------------------------------------------- forks


def raw(cache):
    import torch

    return [t.view(torch.uint8).cpu().numpy().reshape(t.shape[:3] + (-1,)) for t in (cache.k.contiguous(), cache.v.contiguous())] + \
        [e.cpu().numpy() for e in (cache.k_exp, cache.v_exp) if e is not None]


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("heads,dim,page,token_major", [(1, 16, 16, False), (3, 80, 32, False), (8, 128, 16, True), (2, 64, 256, False),
                                                        (5, 128, 256, True)])
def test_forks(cuda, kind, heads, dim, page, token_major):
    """Shared and new pages, lengths at and beside the ends of pages, several rows of one parent, empty rows."""
    import torch

    rng = np.random.default_rng([heads, dim, page])
    lengths = np.array([page - 1, page, page + 1, 1, 0, 3 * page + page // 2], dtype=np.int32)
    tab, pages = P.table(lengths, page, rng, spare=12, width=5)
    tab = np.where(tab < 0, -1, tab)
    free = np.setdiff1d(np.arange(pages), tab)
    parent = np.array([0, 0, 5, 1, -1, 3, 2, 4, 5, 5], dtype=np.int32)
    fresh = rng.permutation(free)[: len(parent)].astype(np.int32)
    fresh[1], fresh[8], fresh[9] = tab[0, 0], -1, tab[5, 3]          # (kept where it is; shared; kept)
    cache = P.filled(pages, heads, page, dim, kind, rng, cuda, token_major)
    want, table, out_lengths = raw(cache), np.full((10, 5), -9, dtype=np.int32), np.full(10, -9, dtype=np.int32)
    ref.kv_fork(want, tab, lengths, parent, fresh, page, table, out_lengths)
    wide = torch.full((12, 7), -77, dtype=torch.int32, device=cuda)
    new, n = wide[1:11, 1:6], torch.full((12,), -77, dtype=torch.int32, device=cuda)
    status = torch.zeros(10, dtype=torch.int32, device=cuda)
    args = (L.dev(tab), L.dev(lengths), L.dev(parent))
    _native.kv_fork(cache, *args, L.dev(fresh), new, n[1:-1], status=status)
    assert np.array_equal(new.cpu().numpy(), table) and np.array_equal(n[1:-1].cpu().numpy(), out_lengths)
    assert all(np.array_equal(a, b) for a, b in zip(raw(cache), want)) and (status == 0).all()
    wide[1:11, 1:6] = -77
    assert (wide == -77).all() and (n[[0, -1]] == -77).all()
    # without fresh pages nothing is copied
    _native.kv_fork(cache, *args, None, new)
    ref.kv_fork(want, tab, lengths, parent, None, page, table, out_lengths)
    assert np.array_equal(new.cpu().numpy(), table) and all(np.array_equal(a, b) for a, b in zip(raw(cache), want))


def test_forks_that_are_malformed(cuda):
    """Parents, lengths and pages outside their ranges: empty rows, or the parent's page kept; nothing else is touched."""
    import torch

    rng = np.random.default_rng(1)
    page = 16
    lengths = np.array([20, -1, 100, 20, 64, 33], dtype=np.int32)
    tab = np.array([[0, 1, -1, -1], [0, -1, -1, -1], [0, 1, 2, 3], [4, 99, -1, -1], [5, 6, 7, 8], [9, 10, -1, -1]], dtype=np.int32)
    cache = P.filled(16, 2, page, 32, "bf16", rng, cuda)
    before = raw(cache)
    parent = np.array([6, -2, 1, 2, 3, 0, 4, 5], dtype=np.int32)
    fresh = np.array([11, 11, 11, 11, 11, 16, 11, 11], dtype=np.int32)
    new, n = torch.full((8, 4), -9, dtype=torch.int32, device=cuda), torch.full((8,), -9, dtype=torch.int32, device=cuda)
    status = torch.zeros(8, dtype=torch.int32, device=cuda)
    _native.kv_fork(cache, L.dev(tab), L.dev(lengths), L.dev(parent), L.dev(fresh), new, n, status=status)
    E = _native
    assert list(status.cpu().numpy()) == [E.ST_BAD_OFFSETS] * 2 + [E.ST_BAD_LENGTH] * 2 + [E.ST_BAD_PAGE] * 2 + [0, E.ST_BAD_PAGE]
    none = [-1] * 4
    assert new.cpu().tolist() == [none] * 4 + [[4, 99, -1, -1], [0, 1, -1, -1], [5, 6, 7, 8], [9, 10, -1, -1]]
    assert n.cpu().tolist() == [0, 0, 0, 0, 20, 20, 64, 33]
    assert all(np.array_equal(a, b) for a, b in zip(raw(cache), before))


# ---------------------------------------------------------------- as they are used


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
def test_beam_decoding_over_one_cache(cuda, cache_kind):
    """Prompts enter the cache once; every step selects, forks, writes the survivors' tokens and attends over what each beam
    descends from. The expected cache is kept beam by beam on the host. One captured step is replayed throughout."""
    import torch

    rng = np.random.default_rng(21)
    B, W, H, G, D, V, page, steps, end = 3, 4, 2, 2, 32, 300, 16, 20, 7
    R = B * W
    prompt = np.array([13, 1, 32], dtype=np.int32)
    blocks = (int(prompt.max()) + steps) // page + 2
    shared = [-(-int(p) // page) for p in prompt]
    cache = kvcache.alloc(sum(shared) + 2 * R * blocks, H, page, D, P.torch_type(cache_kind), cuda)
    tab = np.full((B, blocks), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        tab[b, : shared[b]] = np.arange(at, at + shared[b])
        at += shared[b]
    kv = torch.from_numpy(rng.standard_normal((int(prompt.sum()), 2 * H, D)).astype(np.float32)).to(torch.bfloat16).to(cuda)
    cu = P.offsets(prompt - 1)
    _native.kv_write(kv[:, :H], kv[:, H:], cache, L.dev(tab), torch.zeros(B, dtype=torch.int32, device=cuda), L.dev(cu), B)
    first = np.concatenate([[0], np.cumsum(prompt)])
    history = [[P.host(kv[first[b]: first[b + 1]])[i] for i in range(prompt[b])] for b in range(B) for _ in range(W)]
    head = torch.randn((H * G * D, V), generator=torch.Generator().manual_seed(1)).to(cuda)

    # the beams start on their request's prompt: one begun, the others at -infinity
    table = L.dev(np.repeat(tab, W, 0))
    lengths = L.dev(np.repeat(prompt, W))
    scores = torch.full((B, W), -torch.inf, device=cuda)
    scores[:, 0] = 0
    finished = torch.zeros((B, W), dtype=torch.uint8, device=cuda)
    logits = torch.randn((R, V), generator=torch.Generator().manual_seed(2)).to(cuda).to(torch.bfloat16)
    rows, tokens = (torch.empty((B, W), dtype=torch.int32, device=cuda) for _ in range(2))
    ws = torch.empty(_native.beam_select_workspace_size(B, W, V, logits.dtype, W), dtype=torch.uint8, device=cuda)
    aws = torch.empty(_native.paged_attention_workspace_size(R, 0, H * G, H, D), dtype=torch.uint8, device=cuda)
    new_table, new_lengths, fresh = torch.empty_like(table), torch.empty_like(lengths), torch.empty_like(lengths)
    one = torch.zeros(R + 1, dtype=torch.int32, device=cuda)
    qkv = torch.empty((R, H * G + 2 * H, D), dtype=torch.bfloat16, device=cuda)
    out = torch.empty((R, H * G, D), dtype=torch.bfloat16, device=cuda)
    status = torch.zeros(R, dtype=torch.int32, device=cuda)

    def step():
        _native.beam_select(logits, scores, rows, tokens, scores, ws, finished=finished, end_token=end, out_finished=finished, status=status)
        _native.kv_fork(cache, table, lengths, rows.view(-1), fresh, new_table, new_lengths, status=status)
        _native.kv_write(qkv[:, H * G: H * G + H], qkv[:, H * G + H:], cache, new_table, new_lengths, one, R, status=status)
        _native.paged_attention(qkv[:, : H * G], cache, new_table, new_lengths, one, R, 0, out, aws, status=status)
        table.copy_(new_table)
        torch.add(new_lengths, 1, out=lengths)

    graph = None
    for i in range(steps):
        z, s, f = P.host(logits), scores.cpu().numpy(), finished.cpu().numpy()
        qkv.copy_(torch.from_numpy(rng.standard_normal(qkv.shape).astype(np.float32)))
        # every beam owns two sets of pages, used in turn (a page lives on in the tables of those that share it)
        fresh.copy_(L.dev((at + (np.arange(R) * 2 + i % 2) * blocks + (np.repeat(prompt, W) + i) // page).astype(np.int32)))
        if i == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        assert (status == 0).all()
        check([t.cpu().numpy() for t in (rows, tokens, scores, finished)] + [None], z, s, W, finished=f, end_token=end)
        q, k, v = (P.host(x) for x in (qkv[:, : H * G], qkv[:, H * G: H * G + H], qkv[:, H * G + H:]))
        history = [list(history[p]) + [np.concatenate([k[r], v[r]])] for r, p in enumerate(rows.view(-1).cpu().tolist())]
        held_k, held_v = P.held(cache)
        now, n = table.cpu().numpy(), lengths.cpu().numpy()
        for r in range(R):
            assert n[r] == len(history[r])
            keys, values = (P.tokens(x, now[r], n[r], page) for x in (held_k, held_v))
            seen = np.array(history[r])
            for got, want in ((keys, seen[:, :H]), (values, seen[:, H:])):
                if cache_kind == "e4m3":
                    e = paged_ref.e4m3_exponent(want)[..., None].astype(np.float64)
                    want = paged_ref.E4M3[paged_ref.e4m3_code(want * 2.0 ** -e)] * 2.0 ** e
                assert np.array_equal(got, want), (i, r)
            want, _, spread = paged_ref.attention(q[r:r + 1], keys, values, n[r] - 1, D ** -0.5)
            assert np.all(np.abs(P.host(out[r:r + 1]) - want) <= 2.0 ** -8 * (np.abs(want) + 2 * spread)), (i, r)
        logits.copy_((out.float().reshape(R, -1) @ head) * 0.5)
