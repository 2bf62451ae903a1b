"""flint_attn_tree over the whole range of bf16 values v: sizes far from 1, sizes
that change along a context, infinite ones and NaN, and the same beside
flint_attn_decode."""
import math

import pytest
import torch

from long_context_decode_flash_b200 import flint

from spec_helpers import TreeCase, lines

pytestmark = pytest.mark.gpu


def scale_v(c, f):
    """Every v of the case times f, a power of two."""
    by = lambda x: (x.double() * f).to(torch.bfloat16)  # noqa: E731
    c.vd, c.v = by(c.vd), by(c.v)
    c.hist = [(first, k, by(v)) for first, k, v in c.hist]


def bounds(c):
    """The reference and its bound, plus what v loses: where a share of the keys holds
    a v of 2^-12 and none beyond 65504, all of its v enter the product in fp16, below
    2^-14 to 2^-25 (and the probabilities sum to at most 1); else in fp32."""
    want, bound = c.reference()
    for b, n in enumerate(c.n_draft):
        top = torch.cat([c.hist[b][2], c.vd[b, :n]]).double().abs().amax((0, 2))  # per KV head
        bound[b] += torch.where(top >= 2.0 ** -12, 2.0 ** -25, 0.0).repeat_interleave(8)[None, :, None]
    return want, bound


def check(c, got):
    want, bound = bounds(c)
    for b, n in enumerate(c.n_draft):
        g = got[b, :n].double()
        over = (g - want[b, :n]).abs() - bound[b, :n]
        assert n == 0 or float(over.max()) <= 0, f"request {b}: {float(over.max()):.3e} above the bound"


@pytest.mark.parametrize("power", [-70, -30, -20, -9, 12, 17, 40, 100])
@pytest.mark.parametrize("layout,window,N", [(flint.CONTIGUOUS, False, 5), (flint.PAGED, False, 12), (flint.RING, True, 20)])
def test_values_of_every_size(layout, window, N, power):
    c = TreeCase(layout, False, window, [900, 0, 70, 300], [N, N, 3, N - 1], N, seed=61)
    scale_v(c, 2.0 ** power)
    for ctas in (0, 4):
        check(c, c.run(num_ctas=ctas))


def test_the_largest_values():
    """All v are the largest bf16 or its negative, in half of the dims the largest:
    the mean is no larger."""
    c = TreeCase(flint.CONTIGUOUS, False, False, [700], [4], 4, seed=62)
    top = torch.finfo(torch.bfloat16).max
    sign = lambda x: torch.where(x < 0, -top, top).to(torch.bfloat16)  # noqa: E731
    c.vd, c.hist = sign(c.vd), [(0, c.hist[0][1], sign(c.hist[0][2]))]
    c.vd[..., :64], c.hist[0][2][..., :64] = top, top
    c.v[0, :700] = c.hist[0][2]
    check(c, c.run())


@pytest.mark.parametrize("at", [[0, 1], [200], [699], [150, 640], []])
@pytest.mark.parametrize("N", [6, 11, 18])
def test_sizes_that_change_along_the_context(N, at):
    """Tokens with v of 2^20 and a score lower by ln 2^18 among tokens with v of 1:
    both count, wherever the larger ones stand (none: only the drafts are large)."""
    c = TreeCase(flint.CONTIGUOUS, False, False, [700], [N], N, seed=63)
    first, k, v = c.hist[0]
    # dim 0 of q and k carries the difference: 8 * 18 ln 2 sqrt(128) / 8
    c.q[..., 0] = 8.0
    lift = 18 * math.log(2) * math.sqrt(128) / 8
    k[..., 0], c.kd[..., 0] = lift, lift
    if at:
        k[at, :, 0], v[at] = 0.0, (v[at].float() * 2.0 ** 20).to(torch.bfloat16)
    else:
        c.kd[..., 0], c.vd = 0.0, (c.vd.float() * 2.0 ** 20).to(torch.bfloat16)
    c.k[0, :700], c.v[0, :700] = k, v
    for ctas in (0, 4, 12):
        check(c, c.run(num_ctas=ctas))


def test_small_values_before_and_after_large_ones():
    """Sizes along a context: 2^-40, then 0, then 2^-12, then 1, and drafts of 2^-60."""
    c = TreeCase(flint.CONTIGUOUS, False, False, [1000], [3], 3, seed=64)
    _, _, v = c.hist[0]
    for a, e, f in ((0, 300, 2.0 ** -40), (300, 450, 0.0), (450, 800, 2.0 ** -12)):
        v[a:e] = (v[a:e].float() * f).to(torch.bfloat16)
    c.vd = (c.vd.float() * 2.0 ** -60).to(torch.bfloat16)
    c.v[0, :1000] = v
    for ctas in (0, 4):
        check(c, c.run(num_ctas=ctas))


@pytest.mark.parametrize("power", [-20, 0, 30])
def test_a_chain_is_decoding_at_every_size(power):
    c = TreeCase(flint.CONTIGUOUS, False, False, [450], [5], 5, kind="chain", seed=65)
    scale_v(c, 2.0 ** power)
    got = c.run()
    cache, ws = c.device_cache(), flint.workspace(1)
    c.kdev[0, 450:], c.vdev[0, 450:] = 0, 0
    q, kd, vd = c.q.cuda(), c.kd.cuda(), c.vd.cuda()
    _, bound = bounds(c)
    for i in range(5):
        flint.flint_kv_append(kd[:, i].contiguous(), vd[:, i].contiguous(), [450 + i], cache)
        one = torch.empty((1, 32, 128), dtype=torch.float32, device="cuda")
        flint.flint_attn_decode(q[:, i].contiguous(), cache, [451 + i], c.sinks.cuda(), 0, one, ws)
        # the decode call's own error is far below the bound's 2^-10 share
        over = (one.cpu().double()[0] - got[0, i].double()).abs() - bound[0, i] * 1.1
        assert float(over.max()) <= 0, f"node {i}: {float(over.max()):.3e} above the bound"


def sibling_case(fp8, N=6, seed=66):
    c = TreeCase(flint.PAGED, fp8, False, [200, 90], [N, 3], N, seed=seed)
    c.parents[0] = [-1, 0, 0, 2, 1, -1] + [2] * (N - 6)
    c.parent[0] = torch.tensor(c.parents[0])
    return c, [2 in line for line in lines(c.parents[0])]


@pytest.mark.parametrize("N", [6, 20])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_draft_with_a_value_that_is_no_number(value, N):
    """bf16: dim 5 of node 2's v.  Its descendants have it in dim 5 of every head and
    nothing of it elsewhere (NaN may take the row); nobody else sees it."""
    c, seen = sibling_case(False, N)
    want, bound = bounds(c)
    c.vd[0, 2, :, 5] = value
    for ctas in (0, 4):
        got = c.run(num_ctas=ctas).double()
        for b, n in enumerate(c.n_draft):
            for i in range(n):
                if b == 0 and seen[i]:
                    assert (got[b, i, :, 5].isnan() if value != value else got[b, i, :, 5] == value).all()
                    if value != value:
                        continue
                    rest = [d for d in range(128) if d != 5]
                else:
                    rest = list(range(128))
                assert ((got[b, i][:, rest] - want[b, i][:, rest]).abs() <= bound[b, i][:, rest]).all()


def test_a_draft_beyond_the_codes_saturates():
    """E4M3: an infinite v is attended as the append writes it (448 times its scale),
    NaN as NaN in every head of every descendant."""
    for value in (float("inf"), float("-inf"), float("nan")):
        c, seen = sibling_case(True)
        clean = c.reference()
        c.vd[0, 2, :, 5] = value
        want, bound = clean if value != value else c.reference()
        got = c.run().double()
        for i in range(6):
            if seen[i] and value != value:
                assert got[0, i, :, 5].isnan().all()
            else:
                assert ((got[0, i] - want[0, i]).abs() <= bound[0, i]).all()


@pytest.mark.parametrize("value", [float("inf"), 3e38, -1e30])
@pytest.mark.parametrize("layout", [flint.CONTIGUOUS, flint.PAGED, flint.RING])
def test_a_cached_value_beyond_fp16(layout, value):
    """One token of the window, attended by all nodes or only by the first: those that
    attend it have it in its dim, in proportion; the others do not see it."""
    for at, first in ((600, False), (188, True)):
        c = TreeCase(layout, False, True, [700], [4], 4, kind="chain", seed=67)
        lo, k, v = c.hist[0]
        v[at - lo, :, 9] = value
        where = (int(c.table[0, at // 64]), at % 64) if layout == flint.PAGED else (0, at % 513) if layout == flint.RING else (0, at)
        c.v[where] = v[at - lo]
        want, bound = c.reference()
        for ctas in (0, 4):
            got = c.run(num_ctas=ctas).double()
            attends = [0] if first else [0, 1, 2, 3]
            for i in range(4):
                fine = ~torch.isinf(want[0, i])
                assert bool(torch.isinf(want[0, i, :, 9]).all()) == (value == float("inf") and i in attends)
                assert (got[0, i][~fine] == want[0, i][~fine]).all()
                assert ((got[0, i] - want[0, i]).abs()[fine] <= bound[0, i][fine]).all()
