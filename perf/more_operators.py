"""The cases by which the operators on rows of logits beside the verify are measured: the top logits of every
row with their log-probabilities (a teacher's record, a server's log-probabilities), the distillation of a
drafter from such a record (loss, gradient, backward pass), the selection of a beam step over beams and
vocabulary, and the fork of the beams' paged caches.

Rows are [rows, V]; a bitmask row has one bit an id. ``run`` with ``own`` false computes the operators in
elementary torch operations in 32 bits (in 64: a distillation's sums and targets, and the scores by which beams compete),
with ``own`` true through the library. ``exact`` states the same in 64 bits, some rows at a time."""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
DEV = "cuda"
LIMIT = 2 * 10 ** 9          # bytes that a drawn case may move


def listed():
    return [
        # the best ids of every row
        # the alternatives shown beside the tokens of a four-request step over a small vocabulary
        dict(name="top_rows_small", op="top", rows=16, V=1000, dtype="f32", n=8, masked=False, temperature=1.0),
        # log-probabilities of a structured-output batch's rows, 5 % of the ids allowed
        dict(name="top_step_masked", op="top", rows=768, V=151936, dtype="f32", n=20, masked=True, temperature=0.8),
        # the record of a teacher over a batch of training rows
        dict(name="top_teacher", op="top", rows=2048, V=128256, dtype="bf16", n=64, masked=False, temperature=1.0),
        # distillation from such a record
        # the validation loss of a few rows, targets renormalised over their list
        dict(name="distill_rows_small", op="distill", part="loss", rows=16, V=1000, dtype="f32", n=8, rest=False, temperature=1.0),
        # a validation batch over an odd vocabulary, a tenth of the rows padding
        dict(name="distill_loss_odd", op="distill", part="loss", rows=500, V=100003, dtype="f16", n=20, rest=True, temperature=2.0),
        # a training step's loss with its gradient
        dict(name="distill_train", op="distill", part="train", rows=2048, V=151936, dtype="bf16", n=64, rest=True, temperature=1.0),
        # the gradient alone, from the sums that a forward pass kept
        dict(name="distill_backward_f32", op="distill", part="backward", rows=700, V=128256, dtype="f32", n=32, rest=True, temperature=1.0),
        # a beam step
        # four requests of four beams over a small vocabulary
        dict(name="beam_step_small", op="beam", B=4, beams=4, V=1000, dtype="f32", n=4, masked=False),
        # the structured-output batch with beams in place of samples
        dict(name="beam_step_masked", op="beam", B=64, beams=8, V=151936, dtype="bf16", n=8, masked=True),
        # the largest: twice as many survivors as beams, for a caller that ends hypotheses itself
        dict(name="beam_step_large", op="beam", B=128, beams=8, V=128256, dtype="f32", n=16, masked=False),
        # the survivors' caches
        # the small step's
        dict(name="fork_step_small", op="fork", B=4, beams=4, len_lo=1, len_hi=300, heads=2, dim=64, page=16, cache="e4m3"),
        # long conversations over large pages
        dict(name="fork_step_long", op="fork", B=64, beams=8, len_lo=100, len_hi=4000, heads=8, dim=128, page=64, cache="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges; its work is kept under the largest listed case's."""
    op = rng.choice(["top", "distill", "distill", "beam", "beam", "fork"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    V = rng.choice([1000, 32000, 128256, 151936]) if rng.random() < 0.3 else _log(rng, 200, 260000)
    most = lambda parts: max(1, min(4096, LIMIT // 3 // (V * SIZES[dtype] * parts)))  # noqa: E731
    if op == "top":
        return dict(op=op, rows=_log(rng, 1, most(1)), V=V, dtype=dtype, n=_log(rng, 1, 128), masked=rng.random() < 0.4,
                    temperature=rng.choice([1.0, round(rng.uniform(0.5, 3.0), 2)]))
    if op == "distill":
        part = rng.choice(["loss", "train", "train", "backward"])
        return dict(op=op, part=part, rows=_log(rng, 1, most(1 if part == "loss" else 2)), V=V, dtype=dtype, n=_log(rng, 1, 128),
                    rest=rng.random() < 0.6, temperature=rng.choice([1.0, round(rng.uniform(0.5, 3.0), 2)]))
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
        return dict(op=op, B=_log(rng, 1, max(1, most(1) // beams)), beams=beams, V=V, dtype=dtype, n=min(64, rng.choice([1, beams, 2 * beams])),
                    masked=rng.random() < 0.4)
    heads, dim, page = rng.randint(1, 8), 16 * rng.randint(1, 8), rng.choice([16, 32, 64, 128, 256])
    beams = rng.randint(1, 12)
    B = _log(rng, 1, max(1, min(128, 100_000_000 // (beams * heads * dim * page * 4))))
    hi = _log(rng, 2, max(3, min(8000, 200_000_000 // (B * heads * dim * 4))))
    return dict(op=op, B=B, beams=beams, len_lo=rng.randint(1, hi), len_hi=hi, heads=heads, dim=dim, page=page,
                cache=rng.choice(["bf16", "f16", "e4m3"]))


# ---------------------------------------------------------------- inputs


def _rows(case, g, rows, more=None):
    """Logits N(0, 3) with three favoured ids a row, made some rows at a time. more(first, part): called with every part
    in 32 bits before it is rounded."""
    x = torch.empty((rows, case["V"]), dtype=DTYPES[case["dtype"]], device=DEV)
    step = max(1, (1 << 26) // case["V"])
    for i in range(0, rows, step):
        m = min(step, rows - i)
        part = torch.randn((m, case["V"]), generator=g, device=DEV) * 3.0
        third = case["V"] // 3
        at = torch.randint(0, third, (m, 3), generator=g, device=DEV) + third * torch.arange(3, device=DEV)
        part.scatter_(1, at, 6.0 + 8.0 * torch.rand((m, 3), generator=g, device=DEV))
        if more is not None:
            more(i, part)
        x[i: i + m] = part.to(x.dtype)
    return x


def _mask(case, g, rows):
    """Packed words: about 4 % of the ids in runs of 64, 1 % one by one; one id of every row is allowed in any case."""
    V, words = case["V"], (case["V"] + 31) // 32
    out = torch.empty((rows, words), dtype=torch.int32, device=DEV)
    shift = torch.arange(32, device=DEV)
    step = max(1, (1 << 26) // V)
    for i in range(0, rows, step):
        m = min(step, rows - i)
        runs = (torch.rand((m, (words + 1) // 2), generator=g, device=DEV) < 0.04).repeat_interleave(64, 1)[:, : words * 32]
        bits = runs | (torch.rand((m, words * 32), generator=g, device=DEV) < 0.01)
        bits.scatter_(1, torch.randint(0, V, (m, 1), generator=g, device=DEV), True)
        packed = (bits.view(m, words, 32).long() << shift).sum(-1)
        out[i: i + m] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).int()
    return out


def _lengths(case):
    """Cached tokens of every request (host): the case's own, whatever the seed."""
    rng = np.random.default_rng([case["B"], case["heads"], case["dim"], case["page"]])
    n = rng.integers(case["len_lo"], case["len_hi"] + 1, size=case["B"])
    n[rng.integers(case["B"])] = case["len_hi"]
    return n


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=case)
    op = case["op"]
    if op == "top":
        s["logits"] = _rows(case, g, case["rows"])
        s["mask"] = _mask(case, g, case["rows"]) if case["masked"] else None
        s["ids"] = torch.empty((case["rows"], case["n"]), dtype=torch.int32, device=DEV)
        s["logprobs"] = torch.empty((case["rows"], case["n"]), device=DEV)
        s["lse"] = torch.empty(case["rows"], device=DEV)
    elif op == "distill":
        rows, n = case["rows"], case["n"]
        s["ids"] = torch.empty((rows, n), dtype=torch.int32, device=DEV)
        s["logprobs"] = torch.empty((rows, n), device=DEV)

        def teach(first, part):
            teacher = (part + torch.randn(part.shape, generator=g, device=DEV)) / case["temperature"]
            top = torch.topk(teacher, min(n, case["V"]), dim=1)
            s["ids"][first: first + len(part)] = top.indices.int()
            s["logprobs"][first: first + len(part)] = top.values - torch.logsumexp(teacher, 1, keepdim=True)

        s["logits"] = _rows(case, g, rows, teach)
        # padding, and the mean's share (an f16 gradient is scaled by 256 rows, or its small elements would be lost)
        s["weight"] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.1, 0.0, 256.0 if case["dtype"] == "f16" else 1.0 / rows)
        s["loss"] = torch.empty(rows, device=DEV)
        s["stats"] = torch.empty((rows, 2), device=DEV)
        s["grad"] = torch.empty_like(s["logits"]) if case["part"] != "loss" else None
        if case["part"] == "backward":
            for r in range(0, rows, 128):
                z = s["logits"][r: r + 128].double() / case["temperature"]
                s["stats"][r: r + 128, 0] = torch.logsumexp(z, 1)
                s["stats"][r: r + 128, 1] = torch.logsumexp(z.scatter_(1, s["ids"][r: r + 128].long(), -torch.inf), 1)
    elif op == "beam":
        B, W, n = case["B"], case["beams"], case["n"]
        s["logits"] = _rows(case, g, B * W)
        s["mask"] = _mask(case, g, B * W) if case["masked"] else None
        # beams of one request lie within a few units of each other, best first
        s["scores"] = -(torch.rand((B, 1), generator=g, device=DEV) * 60.0 + torch.rand((B, W), generator=g, device=DEV).mul(4.0).cumsum(1))
        s["finished"] = (torch.rand((B, W), generator=g, device=DEV) < 0.1).to(torch.uint8)
        s["rows"], s["tokens"] = (torch.empty((B, n), dtype=torch.int32, device=DEV) for _ in range(2))
        s["next"] = torch.empty((B, n), device=DEV)
        s["ended"] = torch.empty((B, n), dtype=torch.uint8, device=DEV)
    else:
        B, W, page = case["B"], case["beams"], case["page"]
        length = _lengths(case)
        full = length // page                                # pages that the beams of a request share
        width = int(full.max()) + 1
        n = int(full.sum()) + 2 * B * W + 3
        perm = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        start = torch.from_numpy(np.concatenate([[0], np.cumsum(full)[:-1]])).to(DEV)
        L, F = (torch.from_numpy(x).to(DEV).repeat_interleave(W) for x in (length, full))
        at = torch.arange(width, device=DEV)
        table = perm[(start.repeat_interleave(W)[:, None] + at).clamp(max=n - 1)]
        last = perm[int(full.sum()) + torch.arange(B * W, device=DEV)]
        s["table"] = torch.where(at < F[:, None], table, torch.where(at == F[:, None], last[:, None], -1)).int().contiguous()
        s["lengths"] = L.int()
        s["fresh"] = perm[int(full.sum()) + B * W + torch.arange(B * W, device=DEV)].contiguous()
        # survivors descend from few of the beams
        s["parent"] = ((torch.rand((B, W), generator=g, device=DEV) ** 2 * W).int() + W * torch.arange(B, device=DEV, dtype=torch.int32)[:, None]).view(-1)
        shape = (n, case["heads"], page, case["dim"])
        for x in ("k", "v"):
            s[x] = torch.empty(shape, dtype=DTYPES[case["cache"]], device=DEV)
            step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
            for i in range(0, n, step):
                part = torch.randn((min(step, n - i),) + shape[1:], generator=g, device=DEV)
                s[x][i: i + step] = ((part * 90.0).clamp(-448.0, 448.0) if case["cache"] == "e4m3" else part).to(s[x].dtype)
            s[x + "_exp"] = (torch.randint(119, 122, shape[:3], generator=g, device=DEV, dtype=torch.uint8)
                             if case["cache"] == "e4m3" else None)
        s["new_table"], s["new_lengths"] = torch.empty_like(s["table"]), torch.empty_like(s["lengths"])
    if own:
        from speculative_decoding_verification_specdec_gb300 import _native, kvcache

        if op == "top":
            size = _native.top_logits_workspace_size(case["rows"], case["V"], s["logits"].dtype)
        elif op == "beam":
            size = _native.beam_select_workspace_size(case["B"], case["beams"], case["V"], s["logits"].dtype, case["n"])
        else:
            size = 0
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        if op == "fork":
            s["cache"] = kvcache.PagedCache(s["k"], s["v"], s["k_exp"], s["v_exp"])
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from speculative_decoding_verification_specdec_gb300 import _native

    c = s["case"]
    if c["op"] == "top":
        _native.top_logits(s["logits"], s["ids"], s["logprobs"], s["workspace"], bitmask=s["mask"], temperature=c["temperature"], lse=s["lse"])
        return s["ids"], s["logprobs"], s["lse"]
    if c["op"] == "distill":
        given = dict(temperature=c["temperature"], rest=c["rest"])
        if c["part"] == "backward":
            _native.distill_backward(s["logits"], s["ids"], s["logprobs"], s["stats"], s["weight"], s["grad"], **given)
            return s["grad"]
        _native.distill(s["logits"], s["ids"], s["logprobs"], s["loss"], weight=s["weight"], stats=s["stats"], grad=s["grad"], **given)
        return (s["loss"], s["stats"]) + ((s["grad"],) if c["part"] == "train" else ())
    if c["op"] == "beam":
        _native.beam_select(s["logits"], s["scores"], s["rows"], s["tokens"], s["next"], s["workspace"], bitmask=s["mask"],
                            finished=s["finished"], end_token=2, out_finished=s["ended"])
        return s["rows"], s["tokens"], s["next"], s["ended"]
    _native.kv_fork(s["cache"], s["table"], s["lengths"], s["parent"], s["fresh"], s["new_table"], s["new_lengths"])
    return _forked(s)


def _forked(s):
    """The new tables and lengths, and the cache as it stands; e4m3 codes and power-of-two scales by their own 8-bit types."""
    if s["k_exp"] is None:
        return s["new_table"], s["new_lengths"], s["k"], s["v"]
    return s["new_table"], s["new_lengths"], s["k"], s["v"], s["k_exp"].view(torch.float8_e8m0fnu), s["v_exp"].view(torch.float8_e8m0fnu)


def _allowed(words, V):
    """Truth value of every id, from packed words."""
    return ((words[:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).bool().view(words.shape[0], -1)[:, :V]


def _log_sum(z):
    """ln of the sum of exp over the last axis, kept."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    return m + torch.log(torch.exp(z - m).sum(-1, keepdim=True))


def _best(x, n):
    """The n largest of every row of x above -inf, lowest index first among equals: (values, indices), -inf and -1 behind them."""
    least = torch.topk(x, min(n, x.shape[1]), dim=1).values[:, -1:]
    row, at = torch.nonzero((x >= least) & (x > -torch.inf), as_tuple=True)
    found = x[row, at]
    by = torch.sort(found, descending=True, stable=True).indices
    by = by[torch.sort(row[by], stable=True).indices]
    row, at, found = row[by], at[by], found[by]
    first = torch.searchsorted(row, torch.arange(x.shape[0], device=DEV))
    place = torch.arange(row.shape[0], device=DEV) - first[row]
    keep = place < n
    values = torch.full((x.shape[0], n), -torch.inf, dtype=x.dtype, device=DEV)
    indices = torch.full((x.shape[0], n), -1, dtype=torch.int64, device=DEV)
    values[row[keep], place[keep]], indices[row[keep], place[keep]] = found[keep], at[keep]
    return values, indices


def _run_plain(s):
    return {"top": _top_plain, "distill": _distill_plain, "beam": _beam_plain, "fork": _fork_plain}[s["case"]["op"]](s)


def _top_plain(s):
    c = s["case"]
    z = s["logits"].float()
    if s["mask"] is not None:
        z = z.masked_fill(~_allowed(s["mask"], c["V"]), -torch.inf)
    values, ids = _best(z, c["n"])
    lse = _log_sum(z / c["temperature"])
    return ids.int(), values / c["temperature"] - lse, lse[:, 0]


def _distill_plain(s):
    c = s["case"]
    tau, ids = c["temperature"], s["ids"].long()
    w = s["weight"][:, None].double()
    z = s["logits"].float()
    top, lp = z.gather(1, ids).double() / tau, s["logprobs"].double()
    if not c["rest"]:
        lp = lp - torch.log(torch.exp(lp).sum(1, keepdim=True))
    t = torch.exp(lp)
    r = (1.0 - t.sum(1, keepdim=True)).clamp(min=0.0) if c["rest"] else torch.zeros_like(t[:, :1])
    mass = t.sum(1, keepdim=True) + r
    if c["part"] == "backward":
        lse, lse_rest = s["stats"][:, :1].double(), s["stats"][:, 1:].double()
    else:  # the loss is a small difference of logarithms: in 64 bits
        lse_rest = _log_sum(z.scatter(1, ids, -torch.inf).double() / tau)
        lse = _log_sum(torch.cat([top, lse_rest], 1))
        share = torch.where(r > 0, r * (torch.log(r) - (lse_rest - lse)), 0.0)
        loss = (w * ((t * (lp - (top - lse))).sum(1, keepdim=True) + share))[:, 0].float()
        stats = torch.where(w == 0, 0.0, torch.cat([lse, lse_rest], 1)).float()
        if c["part"] == "loss":
            return loss, stats
    grad = (torch.exp(z / tau - lse.float()) * mass.float()).sub_(torch.exp(z / tau - lse_rest.float()) * r.float())
    grad.scatter_(1, ids, (torch.exp(top - lse) * mass - t).float())
    grad = (grad * (w / tau).float()).to(s["logits"].dtype)
    return grad if c["part"] == "backward" else (loss, stats, grad)


def _beam_plain(s):
    c = s["case"]
    B, W, V = c["B"], c["beams"], c["V"]
    z = s["logits"].double()
    if s["mask"] is not None:
        z = z.masked_fill(~_allowed(s["mask"], V), -torch.inf)
    total = s["scores"].view(-1, 1).double() + (z - _log_sum(z))
    done = s["finished"].view(-1, 1) != 0
    stay = torch.where(torch.arange(V, device=DEV) == 2, s["scores"].view(-1, 1).double(), -torch.inf)
    total = torch.where(done, stay, total)
    values, at = _best(total.view(B, W * V), c["n"])
    none = at < 0
    rows = torch.where(none, -1, at // V + W * torch.arange(B, device=DEV)[:, None])
    tokens = torch.where(none, -1, at % V)
    ended = ~none & (done[rows.clamp(min=0), 0] | (tokens == 2))
    return rows.int(), tokens.int(), values.float(), ended.to(torch.uint8)


def _fork_plain(s):
    page = s["case"]["page"]
    parent, length = s["parent"].long(), s["lengths"][s["parent"].long()].long()
    at = torch.arange(s["table"].shape[1], device=DEV)
    last = (length // page)[:, None]
    old = s["table"][parent]
    s["new_table"].copy_(torch.where(at < last, old, torch.where(at == last, s["fresh"][:, None], -1)))
    s["new_lengths"].copy_(length)
    row, slot = torch.nonzero(torch.arange(page, device=DEV) < (length % page)[:, None], as_tuple=True)
    src, dst = old.gather(1, last)[row, 0].long(), s["fresh"][row].long()
    for x in ("k", "v", "k_exp", "v_exp"):
        if s[x] is not None:
            codes = s[x].view(torch.uint8) if s[x].dtype == torch.float8_e4m3fn else s[x]
            codes[dst, :, slot] = codes[src, :, slot]
    return _forked(s)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    """Inputs read once and outputs written once. Of a masked row, the whole row counts, and its mask words."""
    c = case
    if c["op"] == "fork":
        length = _lengths(c)
        held = c["dim"] * SIZES[c["cache"]] + (c["cache"] == "e4m3")
        copied = float((length % c["page"]).sum()) * c["beams"] * 2 * c["heads"] * held
        return {"bytes": 2 * copied + 8.0 * c["beams"] * float((length // c["page"] + 1).sum()), "flops": 0}
    rows = c["rows"] if c["op"] != "beam" else c["B"] * c["beams"]
    row = c["V"] * SIZES[c["dtype"]]
    if c["op"] == "distill":
        each = {"loss": 1, "train": 2, "backward": 2}[c["part"]]
        return {"bytes": float(rows) * (each * row + 8 * c["n"] + 16), "flops": float(rows) * c["V"] * 3 * each}
    out = rows * (8 * c["n"] + 4) if c["op"] == "top" else c["B"] * 13 * c["n"] + 5 * rows
    return {"bytes": float(rows) * (row + (c["V"] / 8 if c["masked"] else 0)) + out, "flops": float(rows) * c["V"] * 3}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"top": _top64, "distill": _distill64, "beam": _beam64, "fork": _fork64}[case["op"]](s, case)


def _row64(s, r, c):
    """Row r in 64 bits, ids that its mask forbids at -inf."""
    z = s["logits"][r].double()
    if s.get("mask") is not None:
        bits = np.unpackbits(s["mask"][r].cpu().numpy().view(np.uint8), bitorder="little")[: c["V"]]
        z[torch.from_numpy(bits == 0).to(DEV)] = -torch.inf
    return z


def _top64(s, c):
    ids = torch.full((c["rows"], c["n"]), -1, dtype=torch.int32, device=DEV)
    logprobs = torch.full((c["rows"], c["n"]), -torch.inf, dtype=torch.float64, device=DEV)
    lse = torch.empty(c["rows"], dtype=torch.float64, device=DEV)
    for r in range(c["rows"]):
        z = _row64(s, r, c)
        lse[r] = torch.logsumexp(z / c["temperature"], 0)
        order = torch.sort(z, descending=True, stable=True)
        m = min(c["n"], int((z > -torch.inf).sum()))
        ids[r, :m] = order.indices[:m].int()
        logprobs[r, :m] = order.values[:m] / c["temperature"] - lse[r]
    return ids, logprobs, lse


def _distill64(s, c):
    tau, V = c["temperature"], c["V"]
    loss = torch.zeros(c["rows"], dtype=torch.float64, device=DEV)
    stats = torch.zeros((c["rows"], 2), dtype=torch.float64, device=DEV)
    grad = torch.zeros((c["rows"], V), dtype=torch.float64, device=DEV) if c["part"] != "loss" else None
    weights = s["weight"].double().tolist()
    for r, w in enumerate(weights):
        if w == 0.0:
            continue
        z = s["logits"][r].double() / tau
        ids = s["ids"][r].long()
        inside = torch.zeros(V, dtype=torch.bool, device=DEV)
        inside[ids] = True
        target = torch.exp(s["logprobs"][r].double())
        if not c["rest"]:
            target = target / target.sum()
        left = max(0.0, 1.0 - float(target.sum())) if c["rest"] else 0.0
        logs = z - torch.logsumexp(z, 0)
        stats[r, 0], stats[r, 1] = torch.logsumexp(z, 0), torch.logsumexp(z[~inside], 0)
        tail = torch.logsumexp(logs[~inside], 0)
        total = (target * (torch.log(target) - logs[ids])).sum()
        if left > 0.0:
            total = total + left * (math.log(left) - tail)
        loss[r] = w * total
        if grad is not None:  # the student's share of each category against the teacher's, by the chain rule
            share = torch.exp(logs)
            d = share * (target.sum() + left)
            d[ids] -= target
            d[~inside] -= left * torch.exp(logs[~inside] - tail)
            grad[r] = d * (w / tau)
    return grad if c["part"] == "backward" else (loss, stats) + ((grad,) if grad is not None else ())


def _beam64(s, c):
    B, W, V, n = c["B"], c["beams"], c["V"], c["n"]
    rows, tokens = (torch.full((B, n), -1, dtype=torch.int32, device=DEV) for _ in range(2))
    scores = torch.full((B, n), -torch.inf, dtype=torch.float64, device=DEV)
    ended = torch.zeros((B, n), dtype=torch.uint8, device=DEV)
    given, done = s["scores"].double().tolist(), s["finished"].tolist()
    for b in range(B):
        found = []
        for w in range(W):
            if done[b][w]:
                found.append((given[b][w], w, 2, 1))
                continue
            z = _row64(s, b * W + w, c)
            lse = torch.logsumexp(z, 0)
            # the beam's own best: nothing else of it can survive
            order = torch.sort(z, descending=True, stable=True)
            m = min(n, int((z > -torch.inf).sum()))
            for x, i in zip((given[b][w] + (order.values[:m] - lse)).tolist(), order.indices[:m].tolist()):
                found.append((x, w, i, int(i == 2)))
        found.sort(key=lambda f: (-f[0], f[1], f[2]))
        for i, (x, w, token, end) in enumerate(found[:n]):
            rows[b, i], tokens[b, i], scores[b, i], ended[b, i] = b * W + w, token, x, end
    return rows, tokens, scores, ended


def _fork64(s, c):
    page = c["page"]
    table, lengths, fresh = (s[x].cpu().numpy() for x in ("table", "lengths", "fresh"))
    new, length = np.full_like(table, -1), np.zeros_like(lengths)
    held = {x: s[x].double() if s[x].dtype != torch.uint8 else torch.exp2(s[x].double() - 127.0)
            for x in ("k", "v", "k_exp", "v_exp") if s[x] is not None}
    for i, p in enumerate(s["parent"].cpu().numpy()):
        n = int(lengths[p])
        length[i] = n
        new[i, : n // page] = table[p, : n // page]
        new[i, n // page] = fresh[i]
        for x in held.values():
            x[int(fresh[i]), :, : n % page] = x[int(table[p, n // page]), :, : n % page]
    return (torch.from_numpy(new).to(DEV), torch.from_numpy(length).to(DEV)) + tuple(held.values())
