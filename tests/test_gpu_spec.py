"""The other calls of a speculative step on the GPU: verification, norm and
rotary at given positions, append of the accepted path, and a whole step."""
import math
import random

import numpy as np
import pytest
import torch

from long_context_decode_flash_b200 import flint, speculative

from spec_helpers import quantise, random_tree, verify_reference

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ verification --

def _probs(g, *shape, peak=2.0):
    return torch.softmax(torch.randn(shape, generator=g) * peak, -1)


def _run_verify(target, draft, tokens, parent, n, ua, us):
    B, N = tokens.shape
    path = torch.full((B, N), 99, dtype=torch.int32, device="cuda")
    acc, nxt = (torch.full((B,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    flint.flint_verify_tree(target, draft, tokens.cuda(), parent.cuda(), n, ua.cuda(), us.cuda(), path, acc, nxt, dev_err=err)
    torch.cuda.synchronize()
    return path.cpu(), acc.cpu(), nxt.cpu(), int(err)


def _check_verify(target, draft, tokens, parents, n, ua, us, got):
    path, acc, nxt, _ = got
    for b in range(len(n)):
        want, token = verify_reference(target[b].numpy(), None if draft is None else draft[b].numpy(), tokens[b, :n[b]].tolist(),
                                       parents[b], ua[b].numpy(), us[b].numpy())
        assert int(acc[b]) == len(want) and int(nxt[b]) == token, (b, want, path[b].tolist(), token, int(nxt[b]))
        assert path[b].tolist() == want + [-1] * (path.shape[1] - len(want))


@pytest.mark.parametrize("dists", [True, False])
@pytest.mark.parametrize("kind", ["chain", "tree", "star"])
@pytest.mark.parametrize("N,V", [(1, 1), (1, 31), (5, 33), (4, 1000), (16, 4097), (64, 515), (7, 50001)])
def test_verify(N, V, kind, dists):
    B, rng, g = 9, random.Random(N * V), torch.Generator().manual_seed(N + V)
    n = [rng.randint(0, N) for _ in range(B - 1)] + [N]
    parents = [random_tree(k, rng, kind) for k in n]
    parent = torch.full((B, N), 4321, dtype=torch.int32)
    target, draft = _probs(g, B, N + 1, V), _probs(g, B, N, V)
    draft = torch.softmax(target[:, :N].log() + 0.5 * torch.randn(B, N, V, generator=g), -1) if V > 1 else draft
    tokens = torch.full((B, N), -7, dtype=torch.int32)
    for b in range(B):
        parent[b, :n[b]] = torch.tensor(parents[b], dtype=torch.int32)
        for i, p in enumerate(parents[b]):
            tokens[b, i] = torch.multinomial(draft[b, p + 1], 1, generator=g)
    ua, us = torch.rand((B, N), generator=g), torch.rand((B,), generator=g)
    d = draft if dists else None
    got = _run_verify(target.cuda(), None if d is None else d.cuda(), tokens, parent, n, ua, us)
    assert got[3] == 0
    _check_verify(target, d, tokens, parents, n, ua, us, got)


def test_verify_at_the_ends_of_the_random_numbers():
    g = torch.Generator().manual_seed(5)
    target, draft = _probs(g, 4, 3, 100), _probs(g, 4, 2, 100)
    target[:, :, :7] = 0.0  # tokens that the target never gives
    target[:, :, 93:] = 0.0
    tokens = torch.tensor([[3, 50], [50, 3], [95, 95], [20, 20]], dtype=torch.int32)
    parents = [[-1, 0], [-1, 0], [-1, -1], [-1, -1]]
    parent = torch.tensor(parents, dtype=torch.int32)
    below = float(np.nextafter(np.float32(1), np.float32(0)))
    for u, v in ((0.0, 0.0), (below, below), (0.0, below), (below, 0.0)):
        ua, us = torch.full((4, 2), u), torch.full((4,), v)
        for d in (draft, None):
            got = _run_verify(target.cuda(), None if d is None else d.cuda(), tokens, parent, [2] * 4, ua, us)
            _check_verify(target, d, tokens, parents, [2] * 4, ua, us, got)
            assert ((got[2] >= 7) & (got[2] < 93)).all()


def test_verify_where_draft_and_target_are_one():
    # u < 1 always accepts; and a row with nothing in it gives token 0
    g = torch.Generator().manual_seed(6)
    target = _probs(g, 2, 5, 300)
    draft = target[:, :4].clone()
    tokens = torch.randint(0, 300, (2, 4), generator=g, dtype=torch.int32)
    parent = torch.tensor([[-1, 0, 1, 2]] * 2, dtype=torch.int32)
    ua, us = torch.rand((2, 4), generator=g), torch.rand((2,), generator=g)
    got = _run_verify(target.cuda(), draft.cuda(), tokens, parent, [4, 4], ua, us)
    assert got[1].tolist() == [4, 4]
    _check_verify(target, draft, tokens, [[-1, 0, 1, 2]] * 2, [4, 4], ua, us, got)
    target[1] = 0.0
    got = _run_verify(target.cuda(), draft.cuda(), tokens, parent, [4, 4], ua, us)
    assert int(got[2][1]) == 0 and int(got[1][1]) == 0


def test_verify_rows_apart_and_bad_entries():
    g = torch.Generator().manual_seed(7)
    wide_t, wide_d = _probs(g, 3, 4, 200), _probs(g, 3, 3, 208)
    target, draft = wide_t[..., :199], wide_d[..., :199]
    tokens = torch.tensor([[5, 6, 7], [198, 0, 199], [1, -1, 2]], dtype=torch.int32)  # 199 and -1: no tokens
    parents = [[-1, 0, 1], [-1, -1, -1], [-1, 0, 0]]
    ua, us = torch.rand((3, 3), generator=g), torch.rand((3,), generator=g)
    got = _run_verify(wide_t.cuda()[..., :199], wide_d.cuda()[..., :199], tokens,
                      torch.tensor(parents, dtype=torch.int32), [3, 3, 3], ua, us)
    assert got[3] == flint.FLINT_ERR_INVALID_ARG
    _check_verify(target, draft, tokens, parents, [3, 3, 3], ua, us, got)
    # a parent that is no earlier node counts as the context
    parent = torch.tensor([[-1, 1, 0], [-1, -5, 70], [-1, 0, 0]], dtype=torch.int32)
    tokens = tokens.clamp(0, 198)
    got = _run_verify(wide_t.cuda()[..., :199], wide_d.cuda()[..., :199], tokens, parent, [3, 3, 3], ua, us)
    assert got[3] == flint.FLINT_ERR_INVALID_ARG
    _check_verify(target, draft, tokens, [[-1, -1, 0], [-1, -1, -1], [-1, 0, 0]], [3, 3, 3], ua, us, got)


# ------------------------------------------------------ norm and rotation --

def _rope_reference(x, w, pos, r, eps=1e-6):
    """(values, bound) in float64 for bf16 x [T, heads, 128]: float32 arithmetic (a
    norm of 128 terms, cos and sin within 2^-22, two products) and one rounding
    to bf16."""
    y = x.double()
    if w is not None:
        y = y * w.double() / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    z, size = y.clone(), y.abs()
    if r is not None and r.rotary_dim:
        half = r.rotary_dim // 2
        i = torch.arange(half)
        f = r.theta ** (-2.0 * i.double() / r.rotary_dim)
        if r.scaling == flint.ROPE_LINEAR:
            f = f / r.factor
        if r.scaling == flint.ROPE_BY_PARTS:
            turns = r.original_context * f / (2 * math.pi)
            keep = ((turns - r.beta_slow) / (r.beta_fast - r.beta_slow)).clamp(0, 1)
            f = keep * f + (1 - keep) * f / r.factor
        a, b = (2 * i, 2 * i + 1) if r.layout == flint.ROPE_INTERLEAVED else (i, i + half)
        t = pos.double()[:, None, None] * f
        c, s = torch.cos(t) * r.attn_factor, torch.sin(t) * r.attn_factor
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        both = (y[..., a].abs() + y[..., b].abs()) * r.attn_factor
        size = size.clone()
        size[..., a], size[..., b] = both, both
    return z, z.abs() * 2.0 ** -8 * 1.01 + size * 2.0 ** -18


ROPES = [dict(), dict(interleaved=True), dict(rotary_dim=64), dict(rotary_dim=96, interleaved=True), dict(rotary_dim=2),
         dict(rotary_dim=80), dict(rotary_dim=126), dict(rotary_dim=0), dict(scaling="linear", factor=4.0),
         dict(scaling="yarn", factor=8.0, theta=5e5), dict(scaling="yarn", factor=16.0, rotary_dim=112, interleaved=True,
                                                            original_context=4096.0, attn_factor=1.0)]


@pytest.mark.parametrize("kwargs", ROPES)
@pytest.mark.parametrize("T,fused", [(1, False), (1, True), (7, True), (300, False)])
def test_norm_and_rotation_at_given_positions(kwargs, T, fused):
    g = torch.Generator().manual_seed(T)
    qkv = torch.randn(T, 41, 128, generator=g).to(torch.bfloat16)
    dev = qkv.cuda()
    q, k = (qkv[:, :32], qkv[:, 33:37]) if fused else (qkv[:, :32].contiguous(), qkv[:, 33:37].contiguous())
    qd, kd = (dev[:, :32], dev[:, 33:37]) if fused else (q.cuda(), k.cuda())
    w = (1 + 0.1 * torch.randn(2, 128, generator=g)).to(torch.bfloat16)
    pos = torch.randint(0, 262144, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0 if T > 1 else 262143
    r = flint.rope(**kwargs)
    for norm in (True, False):
        qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format).cuda(), torch.empty_like(k, memory_format=torch.contiguous_format).cuda()
        flint.flint_qk_norm_rope_at(qd, kd, w[0].cuda() if norm else None, w[1].cuda() if norm else None, pos.cuda(), r,
                                    q_out=qo, k_out=ko)
        for x, wx, got in ((q, w[0], qo), (k, w[1], ko)):
            want, bound = _rope_reference(x, wx if norm else None, pos, r)
            assert ((got.cpu().double() - want).abs() <= bound).all()


def test_rotation_is_the_models_own_form():
    # flint_qk_norm_rope, one token per request, bit for bit up to the rounding
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn(5, 32, 128, generator=g).to(torch.bfloat16).cuda(), torch.randn(5, 4, 128, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.1 * torch.randn(2, 128, generator=g)).to(torch.bfloat16).cuda()
    pos = [0, 1, 777, 100000, 262143]
    k1 = torch.empty_like(k)
    flint.flint_qk_norm_rope(q, k, w[0], w[1], pos, k_out=k1)
    k2 = torch.empty_like(k)
    flint.flint_qk_norm_rope_at(None, k, w[0], w[1], torch.tensor(pos, dtype=torch.int32, device="cuda"), flint.rope(), k_out=k2)
    a, b = k1.cpu().double(), k2.cpu().double()
    assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 1e-5).all() and (a != b).double().mean() < 0.01


def test_rotation_in_place_and_nothing():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(50, 32, 128, generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    for r in (flint.rope(), flint.rope(rotary_dim=36), flint.rope(interleaved=True)):
        out, own = torch.empty_like(q), q.clone()
        flint.flint_qk_norm_rope_at(q, None, w, w, pos, r, q_out=out)
        flint.flint_qk_norm_rope_at(own, None, w, w, pos, r, q_out=own)
        assert torch.equal(out.view(torch.int16), own.view(torch.int16))
    empty = torch.empty((0, 32, 128), dtype=torch.bfloat16, device="cuda")
    flint.flint_qk_norm_rope_at(empty, None, w, w, pos[:0], flint.rope(), q_out=empty)


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", [flint.CONTIGUOUS, flint.RING, flint.PAGED])
@pytest.mark.parametrize("n_layers", [1, 3])
def test_append_path(layout, fp8, n_layers):
    B, N, rng, g = 4, 6, random.Random(1), torch.Generator().manual_seed(4)
    lens = [0, 62, 510, 700]
    paths = [[0, 2, 5], [], [1, 2, 3, 4, 5], [4, 4]]  # the same node twice is two tokens
    path = torch.full((B, N), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    n = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    scale = [0.01, 0.02, 0.03, 0.05] if fp8 else None
    table = torch.tensor([[b * 13 + j for j in range(13)] for b in range(B)], dtype=torch.int32)
    rows, wants = [], []
    for _ in range(n_layers):
        shape = (52, 64, 4, 128) if layout == flint.PAGED else (B, 513 if layout == flint.RING else 720, 4, 128)
        bufs = [torch.randint(0, 126, shape, generator=g, dtype=torch.uint8) if fp8 else
                torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2)]
        drafts = [torch.randn(B, N, 4, 128, generator=g).mul_(3).to(torch.bfloat16) for _ in range(2)]
        want = [t.clone() for t in bufs]
        for t, d in zip(want, drafts):
            for b, p in enumerate(paths):
                for j, node in enumerate(p):
                    at = lens[b] + j
                    where = ((int(table[b, at // 64]), at % 64) if layout == flint.PAGED else
                             (b, at % 513) if layout == flint.RING else (b, at))
                    t[where] = quantise(d[b, node], scale) if fp8 else d[b, node]
        dev = [t.cuda() for t in bufs]
        cache = flint.kv_cache(dev[0], dev[1], layout, capacity=0 if layout == flint.PAGED else shape[1],
                               block_table=table.cuda() if layout == flint.PAGED else None,
                               num_blocks=52 if layout == flint.PAGED else 0, k_scale=scale, v_scale=scale)
        rows.append((drafts[0].cuda(), drafts[1].cuda(), cache))
        wants.append((dev, want))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    flint.flint_kv_append_path(rows, path.cuda(), n.cuda(), lens, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for dev, want in wants:
        for a, b in zip(dev, want):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def test_append_path_refuses_bad_entries_on_the_device():
    k = torch.zeros(1, 4, 4, 128, dtype=torch.bfloat16, device="cuda") + 1
    buf = torch.zeros(2, 8, 4, 128, dtype=torch.bfloat16, device="cuda")
    cache = flint.kv_cache(buf[0], buf[1], flint.CONTIGUOUS, capacity=8)
    for path, n, L, written in (([0, 9, 1, -1], 3, 0, [0, 2]), ([0, 1, 2, 3], 4, 6, [6, 7]), ([0, 1, 2, 3], 5, 0, []),
                                ([0, 1, 2, 3], -1, 0, []), ([0, -1, -1, -1], 2, 0, [0])):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        buf.zero_()
        flint.flint_kv_append_path([(k, k, cache)], torch.tensor([path], dtype=torch.int32, device="cuda"),
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), [L], dev_err=err)
        torch.cuda.synchronize()
        assert int(err) == flint.FLINT_ERR_INVALID_ARG
        assert [j for j in range(8) if bool((buf[:, j] == 1).all())] == written
        assert float(buf.sum()) == len(written) * 2 * 512
    pool = torch.zeros(2, 2, 64, 4, 128, dtype=torch.bfloat16, device="cuda")
    for table in ([[0, 2]], [[0, -1]], [[0]]):
        cache = flint.kv_cache(pool[0], pool[1], flint.PAGED, num_blocks=2,
                               block_table=torch.tensor(table, dtype=torch.int32, device="cuda"))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pool.zero_()
        flint.flint_kv_append_path([(k, k, cache)], torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device="cuda"),
                                   torch.tensor([4], dtype=torch.int32, device="cuda"), [62], dev_err=err)
        torch.cuda.synchronize()
        assert int(err) == flint.FLINT_ERR_INVALID_ARG and float(pool.sum()) == 2 * 2 * 512


# -------------------------------------------------------------- whole step --

@pytest.mark.parametrize("fp8", [False, True])
def test_a_whole_step_continues_as_decoding_does(fp8):
    """Two layers (a ring window with rotation, a full one), a batch of two trees:
    attend, verify, append; then the caches hold what decoding the accepted
    tokens one by one leaves."""
    g = torch.Generator().manual_seed(21)
    lens, parents = [600, 70], [[-1, 0, 0, 2, 3], [-1, 0, 1]]
    tree = speculative.DraftTree(parents)
    B, N, V = 2, 5, 97
    pos = tree.positions(lens)
    assert pos.tolist() == [[600, 601, 601, 602, 603], [70, 71, 72, 70, 70]]
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    scale = [6.0 / 448.0] * 4 if fp8 else None
    err = torch.zeros(8, dtype=torch.int32, device="cuda")
    ws, layers, plain = flint.tree_workspace(), [], []
    for window in (513, 0):
        shape = (B, 513, 4, 128) if window else (B, 720, 4, 128)
        bufs = [rnd(*shape) for _ in range(2)]
        bufs = [quantise(t.cpu(), scale).cuda() if fp8 else t for t in bufs]
        twin = [t.clone() for t in bufs]
        kw = dict(layout=flint.RING if window else flint.CONTIGUOUS, capacity=shape[1], k_scale=scale, v_scale=scale)
        qkv = rnd(B, N, 40, 128)
        w = (1 + 0.1 * torch.randn(2, 128, generator=g)).to(torch.bfloat16).cuda()
        v = qkv[:, :, 36:].contiguous()
        out, k = speculative.attend_layer(tree, pos, qkv[:, :, :32], qkv[:, :, 32:36], v, w[0], w[1],
                                          flint.rope() if window else None, flint.kv_cache(*bufs, **kw), lens,
                                          torch.randn(32, generator=g).cuda(), window, ws, dev_err=err)
        assert torch.isfinite(out.float()).all() and (out[1, 3:] == 0).all() and (out[1, :3] != 0).any()
        layers.append((k, v, flint.kv_cache(*bufs, **kw)))
        plain.append((bufs, twin, flint.kv_cache(*twin, **kw)))
    target, draft = _probs(g, B, N + 1, V), _probs(g, B, N, V)
    tokens = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32)
    ua, us = torch.zeros(B, N), torch.rand(B, generator=g)  # u = 0 takes the first child everywhere
    path, n, token = speculative.verify_and_append(tree, target.cuda(), draft.cuda(), tokens.cuda(), ua.cuda(), us.cuda(),
                                                   layers, lens, dev_err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    assert path.tolist() == [[0, 1, -1, -1, -1], [0, 1, 2, -1, -1]] and n.tolist() == [2, 3]
    want = [verify_reference(target[b].numpy(), draft[b].numpy(), tokens[b].tolist()[:len(parents[b])], parents[b],
                             ua[b].numpy(), us[b].numpy())[1] for b in range(B)]
    assert token.tolist() == want
    for (k, v, _), (bufs, twin, cache) in zip(layers, plain):
        for b, nodes in enumerate(([0, 1], [0, 1, 2])):
            for j, node in enumerate(nodes):
                # the append takes requests from the first on: give both, change one
                both = [lens[0], lens[1]]
                both[b] += j
                keep = [t.clone() for t in twin]
                flint.flint_kv_append(k[:, node].contiguous(), v[:, node].contiguous(), both, cache)
                for t, o in zip(twin, keep):
                    t[1 - b] = o[1 - b]
        for a, t in zip(bufs, twin):
            assert torch.equal(a.view(torch.uint8), t.view(torch.uint8))
