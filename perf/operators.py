"""The cases by which the paged-cache operators are measured: rotary positions, the paged cache's
write (with quantisation) and read-back, and the attention of a verify step's rows over it.

Every case is in the library's row layout: request b owns the k_b + 1 rows cu[b] + b + j. ``run`` with
``own`` false computes the operators in elementary torch operations in 32 bits (angles in 64), with
``own`` true through the library. ``exact`` states the same in 64 bits, request by request."""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
DEV = "cuda"


def listed():
    return [
        # rotary positions
        # a four-request verify step of a small fp32 model, a quarter of the head rotated, adjacent pairs
        dict(name="rope_step_small", op="rope", B=4, k_lo=3, k_hi=3, past=1000, heads=8, dim=64, rot=16, style="interleaved",
             dtype="f32", scaling="none", inverse=False, packed=False),
        # the query heads of a 256-request step, taken out of the packed projection's output
        dict(name="rope_step_queries", op="rope", B=256, k_lo=4, k_hi=4, past=32000, heads=32, dim=128, rot=128, style="half",
             dtype="bf16", scaling="none", inverse=False, packed=True),
        # the gradient over prompts at far positions of a context extended by parts
        dict(name="rope_prompt_gradient", op="rope", B=3, k_lo=2500, k_hi=4999, past=900000, heads=32, dim=128, rot=128, style="half",
             dtype="bf16", scaling="by_parts", inverse=True, packed=False),
        # writing the cache
        # the keys and values of a 64-request verify step, quantised
        dict(name="write_step_e4m3", op="write", B=64, k_lo=3, k_hi=5, past=4000, heads=8, dim=128, rot=128, style="half",
             dtype="bf16", cache="e4m3", page=16, scaling="linear"),
        # four prompts entering an unquantised cache
        dict(name="write_prompt_bf16", op="write", B=4, k_lo=5001, k_hi=8191, past=0, heads=8, dim=128, rot=64, style="interleaved",
             dtype="bf16", cache="bf16", page=64, scaling="none"),
        # reading it back
        # a few short prefixes with an odd head of 80, to fp32
        dict(name="read_prefix_small", op="read", B=4, len_lo=1, len_hi=300, heads=4, dim=80, cache="f16", page=32, dtype="f32"),
        # the long quantised prefixes of a 64-request batch, for another worker
        dict(name="read_prefixes_e4m3", op="read", B=64, len_lo=100, len_hi=4000, heads=8, dim=128, cache="e4m3", page=16, dtype="bf16"),
        # attention
        # a small verify step, where latency counts
        dict(name="attend_step_small", op="attend", B=4, k_lo=3, k_hi=3, past_lo=100, past_hi=1000, heads=2, group=4, dim=64,
             dtype="bf16", cache="bf16", page=16, window=0),
        # one new token of one long conversation over a quantised cache
        dict(name="attend_token_long_e4m3", op="attend", B=1, k_lo=0, k_hi=0, past_lo=130001, past_hi=130001, heads=8, group=4, dim=128,
             dtype="bf16", cache="e4m3", page=64, window=0),
        # single tokens of a 256-request batch, one query head a key head, a sliding window, a head of 80
        dict(name="attend_tokens_window", op="attend", B=256, k_lo=0, k_hi=0, past_lo=1, past_hi=4000, heads=8, group=1, dim=80,
             dtype="f16", cache="f16", page=32, window=1000),
        # the structured-output batch's verify step over a quantised cache
        dict(name="attend_step_e4m3", op="attend", B=128, k_lo=5, k_hi=5, past_lo=500, past_hi=8000, heads=8, group=4, dim=128,
             dtype="bf16", cache="e4m3", page=16, window=0),
        # a ragged verify step over long caches, the largest
        dict(name="attend_step_long", op="attend", B=64, k_lo=1, k_hi=8, past_lo=1000, past_hi=32000, heads=8, group=8, dim=128,
             dtype="bf16", cache="bf16", page=16, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges; its work is kept under the largest listed case's."""
    op = rng.choice(["rope", "write", "read", "attend", "attend", "attend"])
    style, scaling = rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "by_parts"])
    if op == "rope":
        B = _log(rng, 1, 256)
        dim = 2 * rng.randint(16, 128) if rng.random() < 0.4 else rng.choice([64, 128, 192, 256])
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
        heads = rng.randint(1, 40)
        k = _log(rng, 1, max(2, min(5000, 200_000_000 // (B * dim * heads))))
        return dict(op=op, B=B, k_lo=k // 2, k_hi=k, past=_log(rng, 1, 1_000_000), heads=heads, dim=dim, rot=rot, style=style,
                    dtype=rng.choice(["f32", "bf16", "f16"]), scaling=scaling, inverse=rng.random() < 0.3, packed=rng.random() < 0.5)
    cache, page = rng.choice(["bf16", "f16", "e4m3", "e4m3"]), rng.choice([16, 32, 64, 128, 256])
    dim = rng.choice([64, 128, 128, 16 * rng.randint(1, 8)])
    heads = rng.randint(1, 12)
    if op == "write":
        B = _log(rng, 1, 256)
        k = _log(rng, 1, max(2, min(8000, 40_000_000 // (B * dim * heads))))
        return dict(op=op, B=B, k_lo=k // 2, k_hi=k, past=_log(rng, 1, 4000), heads=heads, dim=dim,
                    rot=dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2), style=style, dtype=rng.choice(["f32", "bf16", "f16"]),
                    cache=cache, page=page, scaling=scaling)
    if op == "read":
        B = _log(rng, 1, 128)
        hi = _log(rng, 2, max(3, min(30000, 200_000_000 // (B * dim * heads))))
        return dict(op=op, B=B, len_lo=rng.randint(1, hi), len_hi=hi, heads=heads, dim=dim, cache=cache, page=page,
                    dtype=rng.choice(["f32", "bf16", "f16"]))
    B, group, k_hi = _log(rng, 1, 256), rng.choice([1, 2, 4, 5, 8]), rng.choice([0, rng.randint(0, 8), rng.randint(0, 16)])
    hi = _log(rng, 1, max(2, min(130000, 600_000_000 // (B * heads * max(dim, (k_hi + 1) * group)))))
    dtype = rng.choice(["bf16", "f16"])
    return dict(op=op, B=B, k_lo=rng.randint(0, k_hi), k_hi=k_hi, past_lo=rng.randint(0, hi), past_hi=hi, heads=heads, group=group,
                dim=dim, dtype=dtype, cache="e4m3" if cache == "e4m3" else dtype, page=page,
                window=0 if rng.random() < 0.7 else _log(rng, 1, 4000))


# ---------------------------------------------------------------- inputs


def _ragged(case):
    """Draft counts, their offsets and cached lengths of the batch (host arrays): the case's own, whatever the seed."""
    B = case["B"]
    rng = np.random.default_rng([B, case["heads"], case["dim"]])
    if case["op"] == "read":
        k = rng.integers(case["len_lo"], case["len_hi"] + 1, size=B) - 1
        past = np.zeros(B, dtype=np.int64)
        k[rng.integers(B)] = case["len_hi"] - 1
    else:
        k = rng.integers(case["k_lo"], case["k_hi"] + 1, size=B)
        if case["op"] == "attend":
            past = rng.integers(case["past_lo"], case["past_hi"] + 1, size=B)
            past[rng.integers(B)] = case["past_hi"]
        else:
            past = rng.integers(0, case["past"] + 1, size=B)
    cu = np.zeros(B + 1, dtype=np.int64)
    cu[1:] = np.cumsum(k)
    return k, cu, past


def _inv_freq(case):
    """Angle per token of each rotated pair, and the amplitude, in 64 bits."""
    f = 10000.0 ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "by_parts":  # turns over the 4096 trained positions: over 32 kept, under 1 divided by 8, a ramp between
        keep = np.clip((4096.0 * f / (2 * np.pi) - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * (keep + (1.0 - keep) / 8.0), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _frequencies(case):
    from speculative_decoding_verification_specdec_gb300 import _native

    more = {"none": {}, "linear": dict(scaling="linear", factor=4.0),
            "by_parts": dict(scaling="by_parts", factor=8.0, original_len=4096, beta_fast=32.0, beta_slow=1.0)}[case["scaling"]]
    freqs, amplitude = _native.rope_frequencies(case["rot"], 10000.0, **more)
    return dict(freqs=freqs.to(DEV), rot_dim=case["rot"], interleaved=case["style"] == "interleaved", amplitude=amplitude)


def _pages(case, total, g):
    """A block table over shuffled pages, with spare ones: (table, number of pages)."""
    need = -(-total // case["page"])
    n = int(need.sum()) + 3
    perm = torch.randperm(n, generator=g, device=DEV).to(torch.int32).cpu().numpy()
    table = np.full((len(total), int(need.max())), -1, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(len(total)):
        table[b, : need[b]] = perm[at[b]: at[b + 1]]
    return torch.from_numpy(table).to(DEV), n


def _cache(case, n, g, filled):
    """k, v [pages, heads, page, dim] and, for e4m3, one power-of-two exponent (biased by 127) a token and head."""
    shape = (n, case["heads"], case["page"], case["dim"])
    got = []
    for _ in range(2):
        if not filled:
            x, e = torch.zeros(shape, dtype=DTYPES[case["cache"]], device=DEV), None
            e = torch.full(shape[:3], 127, dtype=torch.uint8, device=DEV)
        else:
            x = torch.empty(shape, dtype=DTYPES[case["cache"]], device=DEV)
            step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
            for i in range(0, n, step):
                part = torch.randn((min(step, n - i),) + shape[1:], generator=g, device=DEV)
                x[i: i + step] = ((part * 90.0).clamp(-448.0, 448.0) if case["cache"] == "e4m3" else part).to(x.dtype)
            # tokens differ in size by up to 8 times
            e = torch.randint(119, 122, shape[:3], generator=g, device=DEV, dtype=torch.uint8)
        got.append((x, e if case["cache"] == "e4m3" else None))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    k, cu, past = _ragged(case)
    B, T = case["B"], int(cu[-1]) + case["B"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case, T=T, cu=torch.from_numpy(cu.astype(np.int32)).to(DEV), past=torch.from_numpy(past.astype(np.int32)).to(DEV))
    rows = lambda heads: torch.randn((T, heads, case["dim"]), generator=g, device=DEV).to(dt)  # noqa: E731
    if op in ("rope", "write"):
        s["inv_freq"], s["amp"] = torch.from_numpy(_inv_freq(case)[0]).to(DEV), _inv_freq(case)[1]
        if own:
            s["rope"] = _frequencies(case)
    if op == "rope":
        # packed: the heads are a slice of a row that holds two more heads on either side
        s["x"] = rows(case["heads"] + 4)[:, 2:-2] if case["packed"] else rows(case["heads"])
        s["out"] = torch.empty((T, case["heads"], case["dim"]), dtype=dt, device=DEV)
        return s
    total = past + k + 1
    s["table"], n = _pages(case, total, g)
    s["k"], s["v"], s["k_exp"], s["v_exp"] = _cache(case, n, g, op != "write")
    if own:
        from speculative_decoding_verification_specdec_gb300 import _native, kvcache

        s["cache"] = kvcache.PagedCache(s["k"], s["v"], s["k_exp"], s["v_exp"])
    if op == "write":
        qkv = rows(2 * case["heads"])  # keys and values as the projection leaves them, side by side
        s["new_k"], s["new_v"] = qkv[:, : case["heads"]], qkv[:, case["heads"]:]
    elif op == "read":
        first = np.concatenate([[0], np.cumsum(total)])
        s["cu_len"], s["rows"] = torch.from_numpy(first.astype(np.int64)).to(DEV), int(first[-1])
        s["out_k"], s["out_v"] = (torch.empty((s["rows"], case["heads"], case["dim"]), dtype=dt, device=DEV) for _ in range(2))
    else:
        s["max_len"], s["scale"] = int(total.max()), case["dim"] ** -0.5
        heads = case["heads"] * case["group"]
        s["q"] = (torch.randn((T, heads, case["dim"]), generator=g, device=DEV) * 1.5).to(dt)
        s["out"] = torch.empty((T, heads, case["dim"]), dtype=dt, device=DEV)
        s["lse"] = torch.empty((T, heads), dtype=torch.float32, device=DEV)
        if own:
            size = _native.paged_attention_workspace_size(B, case["k_hi"], heads, case["heads"], case["dim"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from speculative_decoding_verification_specdec_gb300 import _native

    c = s["case"]
    op, B = c["op"], c["B"]
    if op == "rope":
        _native.rope(s["x"], s["out"], cu_num_draft=s["cu"], cached_len=s["past"], B=B, inverse=c["inverse"], **s["rope"])
        return s["out"]
    if op == "write":
        _native.kv_write(s["new_k"], s["new_v"], s["cache"], s["table"], s["past"], s["cu"], B, rope=s["rope"])
        return _held(s)
    if op == "read":
        _native.kv_read(s["cache"], s["table"], s["cu_len"], B, s["out_k"], s["out_v"])
        return s["out_k"], s["out_v"]
    _native.paged_attention(s["q"], s["cache"], s["table"], s["past"], s["cu"], B, c["k_hi"], s["out"], s["workspace"],
                            scale=s["scale"], window=c["window"], lse=s["lse"])
    return s["out"], s["lse"]


def _held(s):
    """The cache as it stands; e4m3 codes and power-of-two scales by their own 8-bit types."""
    if s["k_exp"] is None:
        return s["k"], s["v"]
    return s["k"], s["v"], s["k_exp"].view(torch.float8_e8m0fnu), s["v_exp"].view(torch.float8_e8m0fnu)


def _owners(s):
    """Request and index within it of every row."""
    B = s["case"]["B"]
    t = torch.arange(s["T"], device=DEV)
    ends = s["cu"][1:].long() + torch.arange(1, B + 1, device=DEV)
    b = torch.searchsorted(ends, t, right=True)
    return b, t - s["cu"].long()[b] - b


def _rotate(x, pos, s):
    """x in 32 bits with its first `rot` elements of every head turned by pos times their frequencies."""
    c = s["case"]
    angle = pos.double()[:, None] * s["inv_freq"]
    if c.get("inverse"):
        angle = -angle
    cos, sin = ((f(angle) * s["amp"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    x = x.float()
    head, rest = x[..., : c["rot"]], x[..., c["rot"]:]
    if c["style"] == "half":
        a, b = head[..., : c["rot"] // 2], head[..., c["rot"] // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _quantised(x):
    """e4m3 codes of x, and the biased exponent of the smallest power of two that brings each head under 448."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, 0, e - 8 - (m <= 0.875).int()).clamp(min=-126)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rope":
        b, j = _owners(s)
        return _rotate(s["x"], s["past"].long()[b] + j, s).to(s["x"].dtype)
    page = c["page"]
    if c["op"] == "write":
        b, j = _owners(s)
        i = s["past"].long()[b] + j
        at = s["table"].long()[b, i // page], slice(None), i % page
        rotated = _rotate(s["new_k"], i, s)
        if s["k_exp"] is None:
            s["k"][at], s["v"][at] = rotated.to(s["k"].dtype), s["new_v"].to(s["v"].dtype)
        else:
            (kq, ke), (vq, ve) = _quantised(rotated), _quantised(s["new_v"].float())
            s["k"].view(torch.uint8)[at], s["v"].view(torch.uint8)[at] = kq.view(torch.uint8), vq.view(torch.uint8)
            s["k_exp"][at], s["v_exp"][at] = ke, ve
        return _held(s)
    if c["op"] == "read":
        row = torch.arange(s["rows"], device=DEV)
        b = torch.searchsorted(s["cu_len"][1:], row, right=True)
        i = row - s["cu_len"][b]
        at = s["table"].long()[b, i // page], slice(None), i % page
        return tuple(_values(s, x, at).to(DTYPES[c["dtype"]]) for x in ("k", "v"))
    return _attend_plain(s)


def _values(s, x, at):
    """What the cache holds at those tokens, in 32 bits."""
    if s["k_exp"] is None:
        return s[x][at].float()
    codes = s[x].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return torch.ldexp(codes, (s[x + "_exp"][at].int() - 127)[..., None])


def _attend_plain(s):
    c = s["case"]
    B, G, J, L, D = c["B"], c["group"], c["k_hi"] + 1, s["max_len"], c["dim"]
    i = torch.arange(L, device=DEV)
    at = s["table"].long()[:, i // c["page"]].clamp(min=0), slice(None), (i % c["page"])[None, :].expand(B, L)
    K, V = _values(s, "k", at), _values(s, "v", at)  # [B, L, heads, D]
    b, j = _owners(s)
    q = torch.zeros((B, J, c["heads"], G, D), device=DEV)
    q[b, j] = s["q"].float().view(-1, c["heads"], G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, c["heads"], J * G, D)
    z = torch.matmul(q, K.permute(0, 2, 3, 1)) * s["scale"]  # [B, heads, J G, L]
    pos = (s["past"].long()[:, None] + torch.arange(J, device=DEV)).repeat_interleave(G, 1)[:, None, :, None]
    seen = i <= pos
    if c["window"]:
        seen = seen & (i > pos - c["window"])
    z = z.masked_fill(~seen, -torch.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    V = V.permute(0, 2, 1, 3)
    o = torch.matmul(p, V) / total
    lse = m + torch.log(total)
    o = o.view(B, c["heads"], J, G, D).permute(0, 2, 1, 3, 4)[b, j].reshape(s["T"], c["heads"] * G, D)
    lse = lse.view(B, c["heads"], J, G).permute(0, 2, 1, 3)[b, j].reshape(s["T"], c["heads"] * G)
    return o.to(s["q"].dtype), lse


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    """Inputs read once and outputs written once, over the case's own ragged lengths."""
    c = case
    k, cu, past = (x.astype(float) for x in _ragged(c))
    held, value = c["dim"] * SIZES.get(c.get("cache"), 0) + (c.get("cache") == "e4m3"), c["dim"] * SIZES[c["dtype"]]
    n = float((k + 1).sum()) * c["heads"]
    if c["op"] == "read":
        return {"bytes": 2 * n * (held + value), "flops": 2 * n * c["dim"]}
    if c["op"] == "rope":
        return {"bytes": 2 * n * value, "flops": 3 * n * c["rot"]}
    if c["op"] == "write":
        return {"bytes": 2 * n * (held + value), "flops": 3 * n * c["rot"]}
    window = c["window"] or 1 << 40
    read = float((np.minimum(past + 1, window) + k).sum())  # tokens that some row of the request sees
    seen = sum(float(np.minimum(p + 1 + np.arange(m + 1), window).sum()) for p, m in zip(past, k))
    heads = c["heads"] * c["group"]
    return {"bytes": 2 * read * c["heads"] * held + float((k + 1).sum()) * heads * (2 * value + 4), "flops": 4 * seen * heads * c["dim"]}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    k, cu, past = _ragged(case)
    rows = [slice(int(cu[b]) + b, int(cu[b + 1]) + b + 1) for b in range(c["B"])]
    if c["op"] == "rope":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
        for b, r in enumerate(rows):
            out[r] = _turn64(s["x"][r], int(past[b]), case)
        return out
    if c["op"] == "write":
        held = []
        for x, new in (("k", "new_k"), ("v", "new_v")):
            if c["cache"] == "e4m3" and x == "k":  # a rotated value next to a border between two codes falls by its last bit
                held.append(None)
                continue
            full = s[x].double()
            for b, r in enumerate(rows):
                y = _turn64(s[new][r], int(past[b]), case) if x == "k" else s[new][r].double()
                i = int(past[b]) + np.arange(y.shape[0])
                page = s["table"][b].cpu().numpy()[i // c["page"]]
                if c["cache"] == "e4m3":
                    y = (y / _scale64(y)).float().to(torch.float8_e4m3fn).double()
                full[torch.from_numpy(page).long().to(DEV), :, torch.from_numpy(i % c["page"]).to(DEV)] = y
            held.append(full)
        if c["cache"] == "e4m3":
            e = torch.ones(s["v_exp"].shape, dtype=torch.float64, device=DEV)
            for b, r in enumerate(rows):
                y = s["new_v"][r].double()
                i = int(past[b]) + np.arange(y.shape[0])
                page = s["table"][b].cpu().numpy()[i // c["page"]]
                e[torch.from_numpy(page).long().to(DEV), :, torch.from_numpy(i % c["page"]).to(DEV)] = _scale64(y)[..., 0]
            held += [None, e]
        return tuple(held)
    if c["op"] == "read":
        got = []
        for x in ("k", "v"):
            got.append(torch.cat([_sequence64(s, x, b, int(k[b]) + 1) for b in range(c["B"])]))
        return tuple(got)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    G = c["group"]
    for b, r in enumerate(rows):
        n = int(past[b] + k[b]) + 1
        first = max(0, int(past[b]) - c["window"] + 1) if c["window"] else 0
        K, V = (_sequence64(s, x, b, n, first) for x in ("k", "v"))
        at = torch.arange(first, n, device=DEV)
        q = s["q"][r].double()
        for j in range(q.shape[0]):
            low = max(0, int(past[b]) + j - c["window"] + 1) if c["window"] else 0
            keep = (at <= int(past[b]) + j) & (at >= low)
            z = torch.einsum("hgd,lhd->hgl", q[j].view(c["heads"], G, -1), K[keep]) * s["scale"]
            lse[r.start + j] = torch.logsumexp(z, -1).view(-1)
            out[r.start + j] = torch.einsum("hgl,lhd->hgd", torch.softmax(z, -1), V[keep]).reshape(-1, c["dim"])
    return out, lse


def _turn64(x, first, case):
    """Complex rotation of the pairs of x [n, heads, dim], at positions first, first + 1, ..."""
    f, amp = _inv_freq(case)
    pos = first + np.arange(x.shape[0], dtype=np.float64)
    angle = np.outer(pos, f) * (-1.0 if case.get("inverse") else 1.0)
    turn = torch.from_numpy(amp * np.exp(1j * angle)).to(DEV)[:, None, :]
    y = x.double().clone()
    h = case["rot"] // 2
    one, two = (slice(0, h), slice(h, 2 * h)) if case["style"] == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    z = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _scale64(y):
    """The smallest power of two that brings the largest of each head to 448 or less (1 for a head of zeros)."""
    top = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448.0).clamp(min=-126.0))
    two = torch.exp2(e)
    two = torch.where(top / two > 448.0, two * 2, torch.where(top / (two / 2) <= 448.0, two / 2, two))
    return torch.where(top == 0, torch.ones_like(top), two)


def _sequence64(s, x, b, n, first=0):
    """Tokens first .. n-1 of request b in the cache, page by page: [n - first, heads, dim]."""
    page = s["case"]["page"]
    ids = s["table"][b, first // page: -(-n // page)].long()
    y = s[x].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() if s["k_exp"] is not None else s[x][ids].double()
    if s["k_exp"] is not None:
        y = y * torch.exp2(s[x + "_exp"][ids].double() - 127.0)[..., None]
    y = y.permute(0, 2, 1, 3).reshape(-1, y.shape[1], y.shape[3])
    return y[first % page: first % page + n - first]
