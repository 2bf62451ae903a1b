"""Speculative steps in a loop that keeps its buffers: the drafts' k and v of each
layer stay where they are, and the layers' array is built once."""
import pytest
import torch

from long_context_decode_flash_b200 import flint, speculative

from spec_helpers import quantise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_kept_buffers_give_what_new_ones_give(fp8):
    g = torch.Generator().manual_seed(71)
    tree = speculative.DraftTree([[-1, 0, 1, 0], [-1, -1, 1]])
    B, N, V = 2, 4, 61
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    scale = [6.0 / 448.0] * 4 if fp8 else None
    w = (1 + 0.1 * torch.randn(2, 128, generator=g)).to(torch.bfloat16).cuda()
    sinks, ws = torch.randn(32, generator=g).cuda(), flint.tree_workspace()
    windows = (513, 0)
    caches, bufs, twins = [], [], []
    for window in windows:
        shape = (B, 513, 4, 128) if window else (B, 700, 4, 128)
        both = [rnd(*shape) for _ in range(2)]
        both = [quantise(t.cpu(), scale).cuda() if fp8 else t for t in both]
        twin = [t.clone() for t in both]
        kw = dict(layout=flint.RING if window else flint.CONTIGUOUS, capacity=shape[1], k_scale=scale, v_scale=scale)
        caches.append((flint.kv_cache(*both, **kw), flint.kv_cache(*twin, **kw)))
        bufs.append(both)
        twins.append(twin)
    ks, vs = ([torch.full((B, N, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in windows] for _ in range(2))
    outs = [torch.full((B, N, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in windows]
    kept = flint.path_layers([(k, v, c[0]) for k, v, c in zip(ks, vs, caches)])
    lens = [600, 77]
    for _ in range(3):
        pos, new = tree.positions(lens), []
        for i, window in enumerate(windows):
            qkv = rnd(B, N, 40, 128)
            args = lambda v, c: (tree, pos, qkv[:, :, :32], qkv[:, :, 32:36], v, w[0], w[1], flint.rope() if window else None, c, lens,  # noqa: E731
                                 sinks, window, ws)
            vs[i].copy_(qkv[:, :, 36:])
            out, k = speculative.attend_layer(*args(vs[i], caches[i][0]), k=ks[i], out=outs[i])
            assert out is outs[i] and k is ks[i]
            v = qkv[:, :, 36:].contiguous()
            fresh, fresh_k = speculative.attend_layer(*args(v, caches[i][1]))
            for b, n in enumerate(tree.n_draft):
                assert torch.equal(out[b, :n], fresh[b, :n]) and (out[b, n:] == 7.0).all() and (fresh[b, n:] == 0).all()
                assert torch.equal(k[b, :n], fresh_k[b, :n])
            new.append((fresh_k, v, caches[i][1]))
        target = torch.softmax(torch.randn(B, N + 1, V, generator=g), -1).cuda()
        tokens = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32).cuda()
        ua, us = torch.rand(B, N, generator=g).cuda() * 0.02, torch.rand(B, generator=g).cuda()
        a = speculative.verify_and_append(tree, target, None, tokens, ua, us, kept, lens)
        b = speculative.verify_and_append(tree, target, None, tokens, ua, us, new, lens)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        for x, y in zip(bufs, twins):
            for s, t in zip(x, y):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
        lens = [n + int(m) for n, m in zip(lens, a[1])]
    assert lens != [600, 77]


def test_a_buffer_of_another_shape_is_refused():
    tree = speculative.DraftTree([[-1, 0]])
    pos = tree.positions([5])
    x = torch.zeros((1, 2, 40, 128), dtype=torch.bfloat16, device="cuda")
    buf = torch.zeros((2, 1, 8, 4, 128), dtype=torch.bfloat16, device="cuda")
    cache = flint.kv_cache(buf[0], buf[1], flint.CONTIGUOUS, capacity=8)
    v, ws, sinks = x[:, :, 36:].contiguous(), flint.tree_workspace(), torch.zeros(32, device="cuda")
    call = lambda **kw: speculative.attend_layer(tree, pos, x[:, :, :32], x[:, :, 32:36], v, None, None, None, cache, [5], sinks, 0, ws, **kw)  # noqa: E731
    call(k=torch.empty_like(v))
    for k in (v[:, :1], v.repeat(1, 2, 1, 1)[:, ::2], v.view(2, 1, 4, 128)):
        with pytest.raises(ValueError):
            call(k=k)
    for bad in (dict(k=v.float()), dict(out=torch.empty((1, 2, 32, 64), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(flint.FlintError):
            call(**bad)
