"""Batches for the tests of the paged-cache operators: ragged rows, shuffled pages, host copies."""
import numpy as np

from oracle import paged_ref as ref

F = {"f32": "float32", "bf16": "bfloat16", "f16": "float16", "e4m3": "float8_e4m3fn"}
# half a rounding step relative to the value
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}


def torch_type(name):
    import torch

    return getattr(torch, F[name])


def offsets(ks):
    cu = np.zeros(len(ks) + 1, dtype=np.int32)
    cu[1:] = np.cumsum(ks)
    return cu


def table(total, page, rng, spare=2, width=0):
    """Block table over shuffled pages (unused entries -7) and the number of pages."""
    need = [max(0, -(-int(t) // page)) for t in total]
    n = sum(need) + spare
    perm = rng.permutation(n)
    out = np.full((len(need), max(max(need), width, 1)), -7, dtype=np.int32)
    at = 0
    for b, m in enumerate(need):
        out[b, :m] = perm[at: at + m]
        at += m
    return out, n


def host(t):
    """A tensor's values as float64."""
    import torch

    if t.dtype == torch.float8_e4m3fn:
        return ref.E4M3[t.view(torch.uint8).cpu().numpy()]
    return t.double().cpu().numpy()


def held(cache):
    """What a kvcache.PagedCache holds, [num_pages, heads, page, dim] float64: (k, v)."""
    k, v = host(cache.k), host(cache.v)
    if cache.k_exp is not None:
        k = k * 2.0 ** (cache.k_exp.cpu().numpy().astype(np.float64) - 127)[..., None]
        v = v * 2.0 ** (cache.v_exp.cpu().numpy().astype(np.float64) - 127)[..., None]
    return k, v


def tokens(x, row, n, page):
    """Tokens 0 .. n - 1 through block-table row `row` of x [pages, heads, page, dim]: [n, heads, dim]."""
    i = np.arange(n)
    return x[row[i // page], :, i % page]


def filled(pages, heads, page, dim, kind, rng, device, token_major=False, spread=3):
    """A cache of random contents: values of order one, e4m3 heads with exponents that differ by up to
    2^spread."""
    import torch

    from speculative_decoding_verification_specdec_gb300 import kvcache

    shape = (pages, page, heads, dim) if token_major else (pages, heads, page, dim)
    got = []
    for _ in range(2):
        x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
        if kind == "e4m3":
            x = (x * 100).clamp(-448, 448)
        x = x.to(torch_type(kind)).to(device)
        got.append(x.permute(0, 2, 1, 3) if token_major else x)
    if kind != "e4m3":
        return kvcache.PagedCache(*got)
    exps = [torch.from_numpy(rng.integers(121 - spread, 121, size=(pages, heads, page)).astype(np.uint8)).to(device) for _ in range(2)]
    return kvcache.PagedCache(*got, *exps)
