"""The speculative-decode calls at their limits: values that are no numbers where
some nodes do not look, far offsets, full batches, every bf16 value through the
quantisation, two calls at once, a wait that runs out."""
import ctypes
import random
import time

import pytest
import torch

from long_context_decode_flash_b200 import build as cuda_build
from long_context_decode_flash_b200 import flint

from spec_helpers import TreeCase, lines, quantise

pytestmark = pytest.mark.gpu


def attend(c, q=None, out=None, ws=None, num_ctas=0, stream=None):
    q = c.q.cuda() if q is None else q
    out = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    flint.flint_attn_tree(q, c.kd.cuda(), c.vd.cuda(), c.parent.cuda(), c.device_cache(), c.lens, c.n_draft, c.sinks.cuda(),
                          513 if c.window else 0, out, flint.tree_workspace(num_ctas) if ws is None else ws, num_ctas=num_ctas)
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["vd", "kd"])
def test_a_siblings_value_that_is_no_number(what, bad, fp8):
    """Node 2's k or v is NaN or infinite: its descendants see it, nobody else."""
    c = TreeCase(flint.PAGED, fp8, False, [200], [6], 6, seed=31)
    c.parents = [[-1, 0, 0, 2, 1, -1]]
    c.parent[0] = torch.tensor(c.parents[0])
    want, bound = c.reference()
    clean = getattr(c, what).clone()
    getattr(c, what)[0, 2, :, 5] = bad
    got = attend(c).cpu().double()
    setattr(c, what, clean)
    seen = [2 in line for line in lines(c.parents[0])]
    for i in range(6):
        if not seen[i]:
            assert ((got[0, i] - want[0, i]).abs() <= bound[0, i]).all()
        elif bad != bad:
            assert not torch.isfinite(got[0, i]).all()


@pytest.mark.parametrize("layout", [flint.CONTIGUOUS, flint.PAGED, flint.RING])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_cached_value_that_only_shallow_nodes_attend(layout, fp8):
    """The oldest token of the first node's window holds NaN in v: nodes one
    position on do not attend it."""
    L = 700
    c = TreeCase(layout, fp8, True, [L], [4], 4, kind="chain", seed=32)
    want, bound = c.reference()
    p = L - 512
    where = (int(c.table[0, p // 64]), p % 64) if layout == flint.PAGED else (0, p % 513) if layout == flint.RING else (0, p)
    c.v[where] = 0x7F if fp8 else float("nan")
    got = attend(c).cpu().double()
    assert torch.isnan(got[0, 0]).all()
    assert ((got[0, 1:] - want[0, 1:]).abs() <= bound[0, 1:]).all()


def test_q_of_every_size():
    """Rows of q from tiny to large against an E4M3 cache (each row has its own
    scale there), and rows of zeros."""
    for scale in (2.0 ** -120, 2.0 ** -30, 1.0, 30.0):
        c = TreeCase(flint.CONTIGUOUS, True, False, [150], [3], 3, seed=33)
        c.q = (c.q.float() * scale).to(torch.bfloat16)
        c.q[0, 1, 3] = 0
        c.check(attend(c).cpu())


def test_pages_beyond_32_bit_offsets():
    """Page ids whose element offsets pass 2^31 (4.6 GB per buffer)."""
    n_pages = 70_000
    c = TreeCase(flint.PAGED, False, False, [150, 70], [5, 2], 5, seed=34)
    want = attend(c)
    k, v = (torch.zeros((n_pages, 64, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moved = c.table.clone()
    used = sorted({int(x) for b, L in enumerate(c.lens) for x in c.table[b, :-(-L // 64)]})
    to = {p: n_pages - 1 - 3 * i for i, p in enumerate(used)}
    for p in used:
        k[to[p]], v[to[p]] = c.k[p].cuda(), c.v[p].cuda()
    for b, L in enumerate(c.lens):
        for j in range(-(-L // 64)):
            moved[b, j] = to[int(c.table[b, j])]
    cache = flint.kv_cache(k, v, flint.PAGED, block_table=moved.cuda(), num_blocks=n_pages)
    out = torch.full_like(want, 77.0)
    kd, vd = c.kd.cuda(), c.vd.cuda()
    flint.flint_attn_tree(c.q.cuda(), kd, vd, c.parent.cuda(), cache, c.lens, c.n_draft, c.sinks.cuda(), 0, out, flint.tree_workspace())
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    # the append writes there too
    path = torch.tensor([[0, 1, 2, -1, -1], [1, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    n = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    flint.flint_kv_append_path([(kd, vd, cache)], path, n, c.lens)
    for b, nodes in enumerate(([0, 1, 2], [1])):
        for j, node in enumerate(nodes):
            at = c.lens[b] + j
            assert torch.equal(k[to[int(c.table[b, at // 64])], at % 64], kd[b, node])


def test_a_full_batch_of_full_trees():
    B, N = 64, 64
    c = TreeCase(flint.PAGED, True, False, [(37 * b) % 150 for b in range(B)], [N] * B, N, kind="tree", seed=35)
    c.lens_check = None
    got = attend(c).cpu().double()
    assert torch.isfinite(got).all()
    for b in (0, 31, 63):  # whole requests alone give the same values
        one = TreeCase(flint.PAGED, True, False, [c.lens[b]], [N], N, seed=35)
        one.q, one.kd, one.vd, one.parent, one.sinks = c.q[b:b + 1], c.kd[b:b + 1], c.vd[b:b + 1], c.parent[b:b + 1], c.sinks
        one.parents, one.hist, one.k, one.v, one.table, one.num_blocks = [c.parents[b]], [c.hist[b]], c.k, c.v, c.table[b:b + 1].contiguous(), c.num_blocks
        want, bound = one.reference()
        assert ((got[b:b + 1] - want).abs() <= bound).all()


def test_two_calls_at_once():
    cases = [TreeCase(flint.CONTIGUOUS, fp8, False, [3000, 500], [12, 3], 12, seed=36 + fp8) for fp8 in (False, True)]
    alone = [attend(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs, ws = [torch.full_like(a, 77.0) for a in alone], [flint.tree_workspace() for _ in cases]
    args = [[x.cuda() for x in (c.q, c.kd, c.vd, c.parent)] + [c.device_cache(), c.lens, c.n_draft, c.sinks.cuda()] for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            flint.flint_attn_tree(*args[i], 0, outs[i], ws[i], stream=s)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a.view(torch.int16), o.view(torch.int16))


def every_bf16():
    """All 2^16 bf16 values but NaN (0 in their place)."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    return torch.where(torch.isnan(x), torch.zeros_like(x), x)


@pytest.mark.parametrize("scale", [[1.0, 0.5, 2.0 ** -9, 3.0], [6.0 / 448, 0.0133, 0.7, 1e-3], [1e30, 1e-30, 2e38, 1e-38],
                                   [0.1, 0.3333333, 17.0, 1.0000001]])
def test_every_value_through_the_quantisation(scale):
    """Append: the codes are those of the float32 quotient, bit for bit."""
    x = every_bf16().view(1, 32, 4, 4, 128)  # [.., head]: each head sees a quarter
    for turn in range(4):  # ... and every quarter in turn
        y = x.roll(turn, 3).reshape(1, 128, 4, 128)
        halves = [y[:, :64].contiguous(), y[:, 64:].contiguous()]
        buf = torch.zeros((2, 1, 64, 4, 128), dtype=torch.uint8, device="cuda")
        cache = flint.kv_cache(buf[0], buf[1], flint.CONTIGUOUS, capacity=64, k_scale=scale, v_scale=scale)
        path = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
        flint.flint_kv_append_path([(halves[0].cuda(), halves[1].cuda(), cache)], path,
                                   torch.tensor([64], dtype=torch.int32, device="cuda"), [0])
        for got, h in zip(buf.cpu(), halves):
            want = quantise(h, scale)
            assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("scale", [[1.0, 0.5, 2.0 ** -9, 3.0], [6.0 / 448, 0.0133, 0.7, 1e-3]])
def test_drafts_are_attended_as_the_cache_holds_them(scale):
    """A node alone (no context, no sink) gives its own v: every finite bf16 value
    comes back as code * scale."""
    x = every_bf16()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).view(32, 4, 4, 128)
    for turn in range(4):
        v = x.roll(turn, 2).reshape(128, 4, 128).view(2, 64, 4, 128).contiguous()
        B, N = 2, 64
        parent = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
        zero = torch.zeros((B, N, 4, 128), dtype=torch.bfloat16, device="cuda")
        q = torch.zeros((B, N, 32, 128), dtype=torch.bfloat16, device="cuda")
        pool = torch.zeros((2, 1, 8, 4, 128), dtype=torch.uint8, device="cuda").expand(2, B, 8, 4, 128).contiguous()
        cache = flint.kv_cache(pool[0], pool[1], flint.CONTIGUOUS, capacity=8, k_scale=scale, v_scale=scale)
        out = torch.empty((B, N, 32, 128), dtype=torch.bfloat16, device="cuda")
        flint.flint_attn_tree(q, zero, v.cuda(), parent, cache, [0, 0], [N, N], torch.full((32,), float("-inf"), device="cuda"), 0,
                              out, flint.tree_workspace())
        code = quantise(v, scale).view(torch.float8_e4m3fn).float() * torch.tensor(scale).view(4, 1)
        want = code.double().repeat_interleave(8, 2)
        # one key: the probability over the sum is 1 to a few units of fp32, then bf16
        assert ((out.cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 * 1.01).all()


def test_verify_strides_beyond_32_bits():
    """Rows 2^27 values apart (a view of one large buffer): the offsets of the
    last rows pass 2^31 bytes and elements."""
    V, N, B, apart = 1000, 3, 4, 1 << 27
    g = torch.Generator().manual_seed(41)
    big = torch.zeros(B * (N + 1) * apart, dtype=torch.float32, device="cuda")  # 8.6 GB
    rows = torch.softmax(torch.randn(B, N + 1, V, generator=g) * 2, -1).cuda()
    view = big.view(B, N + 1, apart)[..., :V]
    view.copy_(rows)
    tokens = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32).cuda()
    parent = torch.tensor([[-1, -1, 1]] * B, dtype=torch.int32, device="cuda")
    ua, us = torch.zeros(B, N, device="cuda"), torch.rand(B, generator=g).cuda()
    outs = []
    for t in (rows, view):
        path, n, token = torch.empty_like(tokens), torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        flint.flint_verify_tree(t, None, tokens, parent, [N] * B, ua, us, path, n, token)
        outs.append((path, n, token))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_bindings_refuse_other_tensors():
    c = TreeCase(flint.CONTIGUOUS, False, False, [20], [2], 2, seed=42)
    args = [x.cuda() for x in (c.q, c.kd, c.vd, c.parent)]
    cache, ws, out, sinks = c.device_cache(), flint.tree_workspace(), torch.empty_like(args[0]), c.sinks.cuda()
    ok = lambda a, **kw: flint.flint_attn_tree(*a, cache, kw.get("lens", [20]), kw.get("n", [2]), kw.get("sinks", sinks), 0,  # noqa: E731
                                               kw.get("out", out), kw.get("ws", ws), dev_err=kw.get("err"))
    ok(args)
    for k in range(4):
        for bad in (args[k].cpu(), args[k].float(), args[k].repeat(1, 2, *[1] * (args[k].dim() - 2))[:, ::2]):
            with pytest.raises(flint.FlintError):
                ok(args[:k] + [bad] + args[k + 1:])
    for kw in (dict(lens=[20, 20]), dict(n=[]), dict(sinks=sinks.cpu()), dict(out=out[:, :1]), dict(ws=ws.cpu()), dict(ws=ws[:100]),
               dict(err=torch.zeros(1, dtype=torch.int64, device="cuda"))):
        with pytest.raises(flint.FlintError):
            ok(args, **kw)


def test_a_stalled_tile_times_out_then_recovers():
    hooks, limit = flint.open_library(cuda_build.build_hooks()), cuda_build.HOOKS_WAIT_LIMIT_NS * 1e-9
    saved, flint._lib = flint._lib, hooks
    try:
        for fp8 in (False, True):
            c = TreeCase(flint.PAGED, fp8, False, [3000, 900], [20, 5], 20, seed=43)
            args = [x.cuda() for x in (c.q, c.kd, c.vd, c.parent)]
            cache, ws, sinks = c.device_cache(), flint.tree_workspace(), c.sinks.cuda()
            out = torch.full(c.q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
            err = torch.zeros(8, dtype=torch.int32, device="cuda")

            def call():
                flint.flint_attn_tree(*args, cache, c.lens, c.n_draft, sinks, 0, out, ws, num_ctas=8, dev_err=err)
                torch.cuda.synchronize()
            assert hooks.flint_test_stall_tree(-1, -1) == 0
            call()
            assert int(err[0]) == 0
            assert hooks.flint_test_stall_tree(2, 3) == 0  # CTA 2 never loads its fourth K tile
            t0 = time.perf_counter()
            call()
            assert int(err[0]) == flint.FLINT_ERR_TIMEOUT
            assert time.perf_counter() - t0 < 8 * limit + 0.25
            assert hooks.flint_test_stall_tree(-1, -1) == 0
            err.zero_()
            out.fill_(77.0)
            call()
            assert int(err[0]) == 0
            c.check(out.cpu())
    finally:
        flint._lib = saved
