"""Rows of logits for the tests of the operators beside the verify."""
import numpy as np

import _paged as P

U = 2.0 ** -24


def rows(rng, n, V, kind="f32", sigma=3.0, cuda="cuda:0", extra=0, shift=0):
    """Random rows of that type as a view of rows `extra` elements longer, `shift` elements off the allocation's start:
    (tensor, float64)."""
    import torch

    wide = torch.zeros(n * (V + extra) + shift, dtype=P.torch_type(kind), device=cuda)
    view = wide[shift:].view(n, V + extra)[:, :V]
    view.copy_(torch.from_numpy((rng.standard_normal((n, V)) * sigma).astype(np.float32)))
    return view, P.host(view)


def pack(allowed):
    """Packed words of truth values [rows, V]; the bits behind V are ones."""
    n, V = allowed.shape
    bits = np.ones((n, (V + 31) // 32 * 32), dtype=bool)
    bits[:, :V] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def dev(a, cuda="cuda:0"):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(cuda)


def lse_error(z, temperature=1.0):
    """How far the top logits' ln of the sum may be off, Z the largest |z / temperature|. An exponent of 2 in size 1.45 Z is off by
    c's rounding and the product's (2^-24 each) and its reference's (as large): 3 * 1.45 * ln 2 Z < 3.1 Z; exp2's 2^-22 is 4;
    8 + 8 additions by a thread and 5 across the lanes are 21; the rest is in 64 bits but for the result's own rounding."""
    Z = np.abs(z[np.isfinite(z)]).max(initial=0.0) / temperature
    return U * (3.1 * Z + 4 + 21), Z


def loss_error(z, temperature, weight, mass=1.0):
    """How far a distillation's loss may be off. The exponents have no error of c's own: 1.45 * 2 * ln 2 Z < 2.1 Z; exp2's 4; a
    thread adds 8 and then its vectors one by one (under 40 in these tests), 5 across lanes: 53. The loss holds the
    logarithms of both sums, of all and of the rest, the latter twice at most: 3 times; and it is rounded once."""
    Z = np.abs(z[np.isfinite(z)]).max(initial=0.0) / temperature
    return 3 * mass * abs(weight) * U * (2.1 * Z + 57)
