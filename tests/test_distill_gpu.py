"""specdec_distill and specdec_distill_backward against the 64-bit definition and against differences."""
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


def lists(rng, z, n, temperature, noise=1.0):
    """A teacher's record near the student's rows: ids int32, log-probabilities float32 (-1 where the row has fewer ids)."""
    rows, V = z.shape
    ids, lps = np.full((rows, n), -1, dtype=np.int32), np.zeros((rows, n), dtype=np.float32)
    for r in range(rows):
        t = np.where(np.isfinite(z[r]), z[r], 0.0) + noise * rng.standard_normal(V)
        i, lp, _ = ref.top_logits(t, min(n, V), temperature)
        p = rng.permutation(len(i))
        ids[r, : len(i)], lps[r, : len(i)] = i[p], lp[p]
    return ids, lps


TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}


def rounded(stats):
    """What the two sums' rounding to fp32 makes of an exponential, relative (-infinity is exact)."""
    return 2 * L.U * float(stats[stats.isfinite()].abs().max())


class Case:
    def __init__(self, x, ids, lps, temperature=1.0, rest=True, weight=None, cuda="cuda:0"):
        import torch

        self.x, self.z, self.rows, self.V = x, P.host(x), x.shape[0], x.shape[1]
        self.ids, self.lps, self.temperature, self.rest = ids, lps, temperature, rest
        self.weight = np.ones(self.rows, dtype=np.float32) if weight is None else np.asarray(weight, dtype=np.float32)
        self.given = None if weight is None else L.dev(self.weight)
        self.dids, self.dlps = L.dev(ids), L.dev(lps)
        self.kw = dict(temperature=temperature, rest=rest)
        self.torch = torch
        self.want = [ref.distill(self.z[r], ids[r], lps[r], temperature, rest, float(self.weight[r])) for r in range(self.rows)]

    def forward(self, grad=None, stream=None):
        torch = self.torch
        loss = torch.full((self.rows + 2,), 77.0, device=self.x.device)
        stats = torch.full((self.rows + 2, 2), 77.0, device=self.x.device)
        status = torch.zeros(self.rows, dtype=torch.int32, device=self.x.device)
        _native.distill(self.x, self.dids, self.dlps, loss[1:-1], weight=self.given, stats=stats[1:-1], grad=grad, status=status, stream=stream,
                        **self.kw)
        torch.cuda.synchronize()
        assert (loss[[0, -1]] == 77.0).all() and (stats[[0, -1]] == 77.0).all()
        return loss[1:-1], stats[1:-1].clone(), status.cpu().numpy()

    def check_loss(self, loss, stats):
        for r, (want, (every, others), _, _) in enumerate(self.want):
            got, (a, b) = float(loss[r]), (float(y) for y in stats[r])
            err = L.loss_error(self.z[r], self.temperature, self.weight[r], 2.0)
            if not np.isfinite(want):
                assert got == want or (np.isnan(got) and np.isnan(want)), r
                continue
            assert abs(got - want) <= err + L.U * abs(want), (r, got, want)
            one = L.loss_error(self.z[r], self.temperature, 1.0) / 3
            for g, e in ((a, every), (b, others)):
                assert g == e or abs(g - e) <= one + L.U * abs(e), (r, g, e)

    def check_grad(self, grad, kind, more=0.0):
        """An element is off by an exponential's error and its factor's, relative to each of the two products whose difference it is,
        and by its rounding. `more`: a further relative error of both products."""
        g = P.host(grad)
        for r, (_, (every, others), want, ratio) in enumerate(self.want):
            w, tau = abs(float(self.weight[r])), self.temperature
            rel = 2 * L.loss_error(self.z[r], tau, 1.0) / 3 + 4 * L.U + more
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.exp(self.z[r] / tau - every) if np.isfinite(every) else np.zeros(self.V)
            ids, lps, _ = ref.entries(self.ids[r], self.lps[r], self.V, self.rest)
            size = s * (2 + ratio)
            size[ids] += np.exp(lps) if self.rest or not lps.size else np.exp(lps - ref.log_sum(lps))
            err = rel * size * w / tau
            assert np.all(np.abs(g[r] - want) <= err + P.HALF[kind] * (np.abs(want) + err) + TINY[kind]), r


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,n", [(1, 1), (2, 2), (9, 3), (130, 128), (1000, 8), (4099, 64), (33001, 20)])
@pytest.mark.parametrize("rest", [False, True])
def test_loss_and_gradient(cuda, kind, V, n, rest):
    import torch

    rng = np.random.default_rng([V, n])
    x, z = L.rows(rng, 4, V, kind)
    ids, lps = lists(rng, z, n, 1.3)
    c = Case(x, ids, lps, 1.3, rest, weight=[0.5, 0.0, 2.0, 1.0])
    loss, stats, status = c.forward()
    c.check_loss(loss, stats)
    grad = torch.full((4, V), 7.0, dtype=x.dtype, device=cuda)
    again = c.forward(grad=grad)
    c.check_loss(again[0], again[1])
    assert (status == 0).all()
    c.check_grad(grad, kind)
    # a backward pass of its own, from the sums in fp32: their rounding is a relative error of the exponentials
    back = torch.full((4, V), 7.0, dtype=x.dtype, device=cuda)
    kept = stats.clone()
    _native.distill_backward(x, c.dids, c.dlps, kept, c.given, back, **c.kw)
    torch.cuda.synchronize()
    c.check_grad(back, kind, more=rounded(kept))
    assert torch.equal(kept, stats)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("extra,shift,grad_extra", [(1, 0, 1), (0, 3, 0), (5, 2, 0), (0, 0, 3)])
def test_strides_and_alignments(cuda, kind, extra, shift, grad_extra):
    """Rows on and off the 16-byte grid, the gradient's on the same one or another; what lies between rows stays."""
    import torch

    rng = np.random.default_rng(extra)
    V = 6007
    x, z = L.rows(rng, 5, V, kind, extra=extra, shift=shift)
    ids, lps = lists(rng, z, 12, 1.0)
    c = Case(x, ids, lps)
    for backward in (False, True):
        wide = torch.full((5, V + grad_extra), 7.0, dtype=x.dtype, device=cuda)
        grad = wide[:, :V]
        loss, stats, _ = c.forward(grad=None if backward else grad)
        if backward:
            _native.distill_backward(x, c.dids, c.dlps, stats, None, grad, **c.kw)
            torch.cuda.synchronize()
        c.check_loss(loss, stats)
        c.check_grad(grad, kind, more=rounded(stats))
        assert (wide[:, V:] == 7.0).all()


@pytest.mark.parametrize("kind,V", [("bf16", 128256), ("f32", 151936), ("f32", 400003)])
@pytest.mark.parametrize("rows", [2, 330])
def test_whole_vocabularies_in_place(cuda, kind, V, rows):
    """Rows over several CTAs (the last size: longer than they hold at once), few and many; the gradient over the logits. Three
    rows are compared in full."""
    import torch

    rng = np.random.default_rng(V)
    g = torch.Generator(device=cuda)
    g.manual_seed(V)
    x = (torch.randn((rows, V), generator=g, device=cuda) * 3).to(P.torch_type(kind))
    some = sorted({0, rows // 2, rows - 1})
    ids, lps = np.tile(np.arange(40, dtype=np.int32) * (V // 41), (rows, 1)), np.full((rows, 40), -5.0, dtype=np.float32)
    ids[some], lps[some] = lists(rng, P.host(x[some]), 40, 1.0)
    part = Case(x[some].clone(), ids[some], lps[some])
    loss, stats = torch.empty(rows, device=cuda), torch.empty((rows, 2), device=cuda)
    back = x.clone()
    _native.distill(x, L.dev(ids), L.dev(lps), loss, stats=stats, grad=x)
    _native.distill_backward(back, L.dev(ids), L.dev(lps), stats, None, back)
    torch.cuda.synchronize()
    for r, (want, _, _, _) in enumerate(part.want):
        # (a thread adds up to 80 vectors here)
        assert abs(float(loss[some[r]]) - want) <= 3 * L.U * (2.1 * 16 + 110) + L.U * want
    part.check_grad(x[some], kind, more=80 * L.U)
    part.check_grad(back[some], kind, more=80 * L.U + 2 * L.U * 20)


@pytest.mark.parametrize("share", [0.0, 0.2, 0.9, 1.0])
@pytest.mark.parametrize("V", [700, 40003])
def test_rows_without_weight_are_not_read(cuda, share, V):
    """More rows than are in flight at once, that share of them with a weight; the others hold NaN, their lists anything."""
    import torch

    rng = np.random.default_rng([V, int(10 * share)])
    rows = 2500 if V < 1000 else 600
    some = np.sort(rng.permutation(rows)[:6])
    weight = np.where(rng.random(rows) < share, 0.25, 0.0).astype(np.float32)
    x, _ = L.rows(rng, rows, V, "bf16")
    x[L.dev(weight) == 0] = torch.nan
    ids, lps = rng.integers(-5, V + 5, (rows, 9)).astype(np.int32), np.full((rows, 9), -3.0, dtype=np.float32)
    ids[some] = np.stack([rng.permutation(V)[:9] for _ in some])
    loss, stats, grad = torch.full((rows,), 7.0, device=cuda), torch.full((rows, 2), 7.0, device=cuda), torch.full_like(x, 7.0)
    _native.distill(x, L.dev(ids), L.dev(lps), loss, weight=L.dev(weight), stats=stats, grad=grad)
    alone = torch.full((rows,), 7.0, device=cuda)
    _native.distill(x, L.dev(ids), L.dev(lps), alone, weight=L.dev(weight))
    back = torch.full_like(x, 7.0)
    _native.distill_backward(x, L.dev(ids), L.dev(lps), stats, L.dev(weight), back)
    none = torch.from_numpy(weight == 0).to(cuda)
    for t in (loss, stats, grad, alone, back):
        assert (t[none] == 0).all() and torch.isfinite(t[~none].float()).all()
    part = Case(x[torch.from_numpy(some).to(cuda)], ids[some], lps[some], weight=weight[some])
    for r, (want, _, _, _) in enumerate(part.want):
        err = 0 if weight[some[r]] == 0 else L.loss_error(part.z[r], 1.0, weight[some[r]], 2.0)
        assert abs(float(loss[some[r]]) - want) <= err + L.U * abs(want) and abs(float(alone[some[r]]) - want) <= err + L.U * abs(want)
    keep = weight[some] != 0
    if keep.any():
        sub = Case(x[torch.from_numpy(some[keep]).to(cuda)], ids[some[keep]], lps[some[keep]], weight=weight[some[keep]])
        sub.check_grad(grad[torch.from_numpy(some[keep]).to(cuda)], "bf16")
        sub.check_grad(back[torch.from_numpy(some[keep]).to(cuda)], "bf16", more=2 * L.U * 20)


def test_gradient_against_differences(cuda):
    """Along a direction of at most 1 an element: a central difference of step h is off by both losses' errors over 2 h and by
    h^2 / 6 times a third derivative, which is at most 16 for a softmax and its part (third moments of what lies in [-1, 1])."""
    import torch

    rng = np.random.default_rng(4)
    x, z = L.rows(rng, 6, 901, "f32")
    ids, lps = lists(rng, z, 15, 1.0)
    h = 2.0 ** -5
    d = torch.from_numpy(rng.uniform(-1, 1, (6, 901)).astype(np.float32)).to(cuda)
    for rest in (False, True):
        grad = torch.empty_like(x)
        Case(x, ids, lps, 1.0, rest).forward(grad=grad)
        up, down = Case(x + h * d, ids, lps, 1.0, rest), Case(x - h * d, ids, lps, 1.0, rest)
        diff = (up.forward()[0] - down.forward()[0]).double() / (2 * h)
        dot = (grad.double() * d.double()).sum(1)
        err = 2 * L.loss_error(z, 1.0, 1.0, 2.0) / (2 * h) + h * h / 6 * 16 + 901 * 2.0 ** -22
        assert (diff - dot).abs().max() <= err


def test_sure_students(cuda):
    """One listed logit far above the rest: what is left for the others is far under one ulp of the sum, and still counted."""
    import torch

    rng = np.random.default_rng(8)
    x, z = L.rows(rng, 3, 2000, "f32", sigma=1.0)
    x[0, 5], x[1, 5], x[2, 5] = 20.0, 60.0, 200.0
    ids = np.tile(np.array([5, 9], dtype=np.int32), (3, 1))
    lps = np.tile(np.log(np.array([0.7, 0.2])).astype(np.float32), (3, 1))
    c = Case(x, ids, lps)
    grad = torch.empty_like(x)
    loss, stats, _ = c.forward(grad=grad)
    c.check_loss(loss, stats)
    c.check_grad(grad, "f32")
    assert (loss[1:] - loss[:-1] > 1.0).all()


def test_small_targets_keep_their_shares(cuda):
    """A renormalised list whose log-probabilities are all far below fp32's smallest exponential, in every warp that holds one."""
    import torch

    rng = np.random.default_rng(14)
    x, z = L.rows(rng, 2, 800, "f32")
    ids = np.stack([rng.permutation(800)[:100] for _ in range(2)]).astype(np.int32)
    lps = (-300 - rng.uniform(0, 4, (2, 100))).astype(np.float32)
    lps[1, 50:] -= 2000
    c = Case(x, ids, lps, 1.0, False)
    grad = torch.empty_like(x)
    loss, stats, _ = c.forward(grad=grad)
    c.check_loss(loss, stats)
    _, _, want, _ = zip(*c.want)
    # the targets' exponents are below 2050 in size: fp32 holds their differences to 2^-13 at worst, in the second row's last ones
    assert np.all(np.abs(P.host(grad) - np.array(want)) <= 2.0 ** -14)
    _native.distill_backward(x, c.dids, c.dlps, stats, None, grad, rest=False)
    assert np.all(np.abs(P.host(grad) - np.array(want)) <= 2.0 ** -14)


@pytest.mark.parametrize("V", [400, 60001])
@pytest.mark.parametrize("rest", [False, True])
def test_long_lists_with_repeated_ids(cuda, V, rest):
    """Full lists of which many entries repeat, within 32 of each other and further apart, in one part of the row and in several."""
    import torch

    rng = np.random.default_rng(V)
    x, _ = L.rows(rng, 4, V, "f32")
    ids = rng.integers(0, V, (4, 128)).astype(np.int32)
    ids[0] = rng.integers(0, 90, 128)
    ids[1, 64:] = ids[1, :64]
    ids[2, 1::2] = ids[2, ::2]
    lps = (-5 - rng.uniform(0, 2, (4, 128))).astype(np.float32)
    lps[3, ::5] = np.nan
    c = Case(x, ids, lps, 1.0, rest)
    grad, back = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    loss, stats, status = c.forward(grad=grad)
    _native.distill_backward(x, c.dids, c.dlps, stats, None, back, rest=rest)
    c.check_loss(loss, stats)
    c.check_grad(grad, "f32")
    c.check_grad(back, "f32", more=rounded(stats))
    assert (status == _native.ST_BAD_TARGET).all()


def test_entries_that_do_not_count(cuda):
    """Padding, repeated ids, ids outside the vocabulary, log-probabilities that are none, an empty list."""
    import torch

    x, _ = L.rows(np.random.default_rng(9), 7, 50, "f32")
    ids = np.array([[3, -1, 7, -1], [3, 3, 7, 3], [50, 3, -2, 7], [3, 7, 9, 11], [-1, -1, -1, -1], [3, 7, 9, 2 ** 31 - 1], [3, 7, 9, 11]],
                   dtype=np.int32)
    lps = np.full((7, 4), -1.5, dtype=np.float32)
    lps[0, 1] = np.nan
    lps[6] = [0.25, 3.0, -4.0, 80.0]              # (no log-probabilities but the first and third, unless they are renormalised)
    lps[3] = [-1.0, np.nan, np.inf, -np.inf]
    for rest in (False, True):
        c = Case(x, ids, lps, 1.0, rest)
        grad = torch.full_like(x, 7.0)
        loss, stats, status = c.forward(grad=grad)
        c.check_loss(loss, stats)
        c.check_grad(grad, "f32")
        bad = _native.ST_BAD_TARGET
        assert list(status) == [0, bad, bad, bad, 0, bad, bad if rest else 0]
        status = torch.zeros(7, dtype=torch.int32, device=cuda)
        _native.distill_backward(x, c.dids, c.dlps, stats, None, grad, rest=rest, status=status)
        c.check_grad(grad, "f32", more=16 * L.U)
        assert list(status.cpu().numpy()) == [0, bad, bad, bad, 0, bad, bad if rest else 0]


def test_rows_without_a_number_and_infinities(cuda):
    """No finite logit; only listed ones; listed ones at -infinity; NaN; +infinity; the lowest value; weight 0 over NaN."""
    import torch

    x, _ = L.rows(np.random.default_rng(10), 7, 300, "f32")
    ids = np.tile(np.array([3, 70], dtype=np.int32), (7, 1))
    lps = np.full((7, 2), -1.5, dtype=np.float32)
    keep = x[1, [3, 70]].clone()
    x[0], x[1] = -np.inf, -np.inf
    x[1, [3, 70]] = keep
    x[2, 3] = -np.inf
    x[3, 200], x[4, 100] = np.nan, np.inf
    x[5, 100:] = float(torch.finfo(torch.float32).min)
    x[6] = np.nan
    c = Case(x, ids, lps, weight=[1, 1, 1, 1, 1, 1, 0])
    grad = torch.full_like(x, 7.0)
    loss, stats, status = c.forward(grad=grad)
    got = loss.cpu().numpy()
    assert got[0] == np.inf and got[2] == np.inf and np.isnan(got[3]) and np.isnan(got[4]) and got[6] == 0
    assert abs(got[1] - c.want[1][0]) <= L.loss_error(c.z[1], 1.0, 1.0) and abs(got[5] - c.want[5][0]) <= 3 * L.U * (2.1 * 16 + 57)
    g = P.host(grad)
    assert (g[0] == 0).all() and (g[6] == 0).all() and np.isnan(g[3]).all() and np.isnan(g[4]).all()
    for r in (1, 2, 5):
        assert np.all(np.abs(g[r] - c.want[r][2]) <= 1e-5)
    assert status[0] == _native.ST_EMPTY_MASK_ROW and (status[1:] == 0).all()


def test_graph_and_stream(cuda):
    """A captured step (record, loss with gradient) replayed over new rows, on a stream of the caller's."""
    import torch

    rng = np.random.default_rng(12)
    teacher, _ = L.rows(rng, 40, 5000, "bf16")
    x, _ = L.rows(rng, 40, 5000, "bf16")
    ids, lps = torch.empty((40, 16), dtype=torch.int32, device=cuda), torch.empty((40, 16), device=cuda)
    ws = torch.empty(_native.top_logits_workspace_size(40, 5000, x.dtype), dtype=torch.uint8, device=cuda)
    loss, stats, grad = torch.empty(40, device=cuda), torch.empty((40, 2), device=cuda), torch.empty_like(x)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        _native.top_logits(teacher, ids, lps, ws, temperature=2.0)
        _native.distill(x, ids, lps, loss, stats=stats, grad=grad, temperature=2.0)
    for seed in (1, 2):
        teacher.copy_(L.rows(np.random.default_rng(seed), 40, 5000, "bf16")[0])
        x.copy_(teacher + 0.5 * torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        c = Case(x, ids.cpu().numpy(), lps.cpu().numpy(), 2.0)
        c.check_loss(loss, stats)
        c.check_grad(grad, "bf16")


def test_calls_at_the_same_time(cuda):
    """Records and losses of different rows on two streams at once, each with its own workspace, equal the same calls alone."""
    import torch

    streams, work = [torch.cuda.Stream() for _ in range(2)], []
    for i, (rows, V, kind) in enumerate(((300, 70001, "bf16"), (700, 9000, "f32"))):
        x, _ = L.rows(np.random.default_rng(20 + i), rows, V, kind)
        ids, lps = torch.empty((rows, 32), dtype=torch.int32, device=cuda), torch.empty((rows, 32), device=cuda)
        ws = torch.empty(_native.top_logits_workspace_size(rows, V, x.dtype), dtype=torch.uint8, device=cuda)
        work.append((x, ids, lps, ws, torch.empty(rows, device=cuda), torch.empty_like(x)))

    def call(w, stream=None):
        x, ids, lps, ws, loss, grad = w
        _native.top_logits(x, ids, lps, ws, temperature=2.0, stream=stream)
        _native.distill(x, ids, lps, loss, temperature=1.5, grad=grad, stream=stream)

    alone = []
    for w in work:
        call(w)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in (w[1], w[2], w[4], w[5])])
    for _ in range(5):
        for w in work:
            for t in (w[1], w[2], w[4], w[5]):
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for w, s in zip(work, streams):
                call(w, s)
        torch.cuda.synchronize()
        for w, a in zip(work, alone):
            assert all(torch.equal(t, u) for t, u in zip((w[1], w[2], w[4], w[5]), a))


def test_offsets_beyond_32_bits(cuda):
    """More than 2^31 elements: the record, the loss with its gradient in place and the backward pass of the last rows."""
    import torch

    rows, V, n = 15000, 151936, 8
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device=cuda)
    last = slice(rows - 3, rows)
    x[last] = L.rows(np.random.default_rng(15), 3, V, "bf16")[0]
    z = P.host(x[last])
    ids, lps = torch.empty((rows, n), dtype=torch.int32, device=cuda), torch.empty((rows, n), device=cuda)
    ws = torch.empty(_native.top_logits_workspace_size(rows, V, x.dtype), dtype=torch.uint8, device=cuda)
    _native.top_logits(x, ids, lps, ws)
    want = [ref.top_logits(r, n)[0] for r in z]
    assert np.array_equal(ids[last].cpu().numpy(), want) and (ids[:-3] == torch.arange(n, device=cuda)).all()
    loss, stats = torch.empty(rows, device=cuda), torch.empty((rows, 2), device=cuda)
    lps -= 0.5
    c = Case(x[last].clone(), ids[last].cpu().numpy(), lps[last].cpu().numpy())
    back = x.clone()
    _native.distill(x, ids, lps, loss, stats=stats, grad=x)
    _native.distill_backward(back, ids, lps, stats, None, back)
    torch.cuda.synchronize()
    c.check_loss(loss[last], stats[last])
    c.check_grad(x[last], "bf16", more=40 * L.U)
    c.check_grad(back[last], "bf16", more=40 * L.U + rounded(stats))
