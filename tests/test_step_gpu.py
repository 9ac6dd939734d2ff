"""A verify step as it is used: keys and values rotated, quantised and written, queries rotated, attention, the
verify on logits from its output, and the next step at the accepted length."""
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


@pytest.mark.parametrize("cache_kind", ["bf16", "e4m3"])
def test_steps_over_one_cache(cuda, cache_kind):
    import torch

    rng = np.random.default_rng(11)
    B, H, G, D, V, page = 5, 2, 4, 64, 500, 16
    table, amp = _native.rope_frequencies(D, 10000.0)
    rope = dict(freqs=table.to(cuda), rot_dim=D, amplitude=amp)
    f, _ = ref.frequencies(D)
    prompt = np.array([1, 40, 7, 130, 16])
    tab, pages = P.table(prompt + 40, page, rng)
    cache = kvcache.alloc(pages, H, page, D, P.torch_type(cache_kind), cuda)
    dtab = torch.from_numpy(tab).to(cuda)
    cached = torch.zeros(B, dtype=torch.int32, device=cuda)
    status = torch.zeros(B, dtype=torch.int32, device=cuda)
    head = torch.randn((H * G * D, V), generator=torch.Generator().manual_seed(1)).to(cuda)

    def rows(ks):
        cu = P.offsets(ks)
        T = int(cu[-1]) + B
        qkv = torch.from_numpy(rng.standard_normal((T, H * G + 2 * H, D)).astype(np.float32)).to(torch.bfloat16).to(cuda)
        return torch.from_numpy(cu).to(cuda), qkv[:, : H * G], qkv[:, H * G: H * G + H], qkv[:, H * G + H:]

    # the prompts enter the cache
    cu, _, k, v = rows(prompt - 1)
    keys, values = ([list(P.host(x[int(a) + b: int(z) + b + 1])) for b, (a, z) in enumerate(zip(cu, cu[1:]))] for x in (k, v))
    _native.kv_write(k, v, cache, dtab, cached, cu, B, rope=rope, status=status)
    cached += torch.from_numpy(prompt.astype(np.int32)).to(cuda)

    for step in range(4):
        ks = rng.integers(0, 5, size=B)
        cu, q, k, v = rows(ks)
        T = q.shape[0]
        before, past = P.host(q), cached.cpu().numpy()
        _native.kv_write(k, v, cache, dtab, cached, cu, B, rope=rope, status=status)
        _native.rope(q, q, cu_num_draft=cu, cached_len=cached, B=B, **rope)
        out = torch.empty((T, H * G, D), dtype=torch.bfloat16, device=cuda)
        ws = torch.empty(_native.paged_attention_workspace_size(B, 4, H * G, H, D), dtype=torch.uint8, device=cuda)
        _native.paged_attention(q, cache, dtab, cached, cu, B, 4, out, ws, status=status)
        logits = out.reshape(T, -1).float() @ head
        tokens, acc = (torch.empty(n, dtype=torch.int32, device=cuda) for n in (T, B))
        ids = torch.from_numpy(rng.integers(0, V, size=max(int(ks.sum()), 1)).astype(np.int32)).to(cuda)
        counters = torch.zeros(4, dtype=torch.int64, device=cuda)
        _native.specdec_verify(logits, ids, None, None, cu, B, V, 4, None, torch.zeros(B, device=cuda),
                               torch.rand(T, device=cuda), torch.ones((T, V), device=cuda), tokens, acc, counters)
        cached += acc + 1
        torch.cuda.synchronize()
        # every row against its history: rotated and quantised keys, the step's own rows among them
        a = acc.cpu().numpy()
        for b in range(B):
            r = slice(int(cu[b]) + b, int(cu[b + 1]) + b + 1)
            K = np.array(keys[b] + [x for x in P.host(k[r])])
            Vv = np.array(values[b] + [x for x in P.host(v[r])])
            n = K.shape[0]
            assert n == past[b] + ks[b] + 1
            K = ref.rope(K, np.arange(n), f)
            qr = ref.rope(before[r], past[b] + np.arange(ks[b] + 1), f)
            if cache_kind == "e4m3":
                e = [2.0 ** ref.e4m3_exponent(x)[..., None].astype(np.float64) for x in (K, Vv)]
                K, Vv = (ref.E4M3[ref.e4m3_code(x / s)] * s for x, s in zip((K, Vv), e))
            want, _, spread = ref.attention(qr, K, Vv, int(past[b]), D ** -0.5)
            # keys and queries rounded to bf16 (2^-8 each; e4m3 keys are exact but for a code at a border), so a
            # score of |q||k| moves by 2 * 2^-8 of it in the worst case; weights and output 2^-8
            score = 2 * 2.0 ** -8 * D ** -0.5 * np.sqrt((qr ** 2).sum(-1)) * np.sqrt((K ** 2).sum(-1)).max()
            tol = (2 * score[..., None] + 2.0 ** -8) * spread + 2.0 ** -7 * np.abs(want)
            assert np.all(np.abs(P.host(out[r]) - want) <= tol)
            keep = int(a[b]) + 1
            keys[b] += [x for x in P.host(k[r])[:keep]]
            values[b] += [x for x in P.host(v[r])[:keep]]
    assert (status.cpu() == 0).all()


def test_a_captured_step(cuda):
    """Write, rotate and attend in one graph, replayed as the lengths grow, equal the same calls made eagerly."""
    import torch

    B, H, G, D, page = 3, 2, 4, 128, 32
    rng = np.random.default_rng(3)
    tab, pages = P.table([300] * B, page, rng)
    dtab = torch.from_numpy(tab).to(cuda)
    caches = [kvcache.alloc(pages, H, page, D, torch.float8_e4m3fn, cuda) for _ in range(2)]
    cu = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device=cuda)
    T = 8
    qkv = torch.randn((T, H * G + 2 * H, D), device=cuda).to(torch.bfloat16)
    rope = dict(freqs=_native.rope_frequencies(64)[0].to(cuda), rot_dim=64, interleaved=True)
    cached = torch.zeros(B, dtype=torch.int32, device=cuda)
    ws = torch.empty(_native.paged_attention_workspace_size(B, 3, H * G, H, D), dtype=torch.uint8, device=cuda)
    q, outs = torch.empty((T, H * G, D), dtype=torch.bfloat16, device=cuda), [torch.empty((T, H * G, D), dtype=torch.bfloat16, device=cuda) for _ in range(2)]

    def step(i):
        _native.kv_write(qkv[:, H * G: H * G + H], qkv[:, H * G + H:], caches[i], dtab, cached, cu, B, rope=rope)
        _native.rope(qkv[:, : H * G], q, cu_num_draft=cu, cached_len=cached, B=B, **rope)
        _native.paged_attention(q, caches[i], dtab, cached, cu, B, 3, outs[i], ws)

    step(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(1)
    for _ in range(60):
        step(0)
        g.replay()
        cached += torch.tensor([3, 1, 4], dtype=torch.int32, device=cuda)
        qkv.copy_(torch.randn(qkv.shape, device=cuda))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(caches[0].k.view(torch.uint8), caches[1].k.view(torch.uint8))
