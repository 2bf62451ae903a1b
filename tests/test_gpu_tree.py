"""flint_attn_tree against a float64 reference: layouts, cache types, windows,
trees, lengths from none to several splits, and what must not be read."""
import pytest
import torch

from long_context_decode_flash_b200 import flint

from spec_helpers import TreeCase

pytestmark = pytest.mark.gpu

CONFIGS = [(flint.CONTIGUOUS, False), (flint.CONTIGUOUS, True), (flint.PAGED, False), (flint.PAGED, True),
           (flint.RING, True)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout,window", CONFIGS)
def test_lengths_around_every_boundary(layout, window, fp8):
    lens = [0, 1, 2, 63, 64, 65, 127, 128, 129, 511, 512, 513, 514, 700, 1027]
    n = [1, 2, 3, 4, 5, 6, 7, 8, 5, 4, 3, 8, 7, 6, 1]
    c = TreeCase(layout, fp8, window, lens, n, 8, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout,window", CONFIGS)
@pytest.mark.parametrize("N", [1, 9, 16, 17, 33, 64])
def test_tree_sizes(layout, window, fp8, N):
    c = TreeCase(layout, fp8, window, [301, 77, 640], [N, max(0, N - 3), (N + 1) // 2], N, seed=N)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["chain", "star"])
@pytest.mark.parametrize("layout,window", [(flint.RING, True), (flint.PAGED, False)])
def test_shapes_of_tree(kind, layout, window):
    # a chain of 64 reaches 63 positions past the context: its last nodes'
    # windows begin 63 tokens later than the first node's
    c = TreeCase(layout, False, window, [530], [64], 64, kind=kind, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_split_over_few_and_many_ctas(fp8):
    c = TreeCase(flint.CONTIGUOUS, fp8, False, [3001, 40], [7, 3], 7, seed=5)
    outs = [c.run(num_ctas=n) for n in (0, 1, 2, 5, 37, 296)]
    for o in outs:
        c.check(o)


def test_the_same_bits_every_run():
    c = TreeCase(flint.PAGED, False, False, [2500, 900, 64], [16, 5, 1], 16, seed=6)
    ws = flint.tree_workspace()
    ws.fill_(0xFF)  # nothing of an earlier call is read
    first = c.run(ws=ws)
    for _ in range(3):
        assert torch.equal(first.view(torch.int16), c.run(ws=ws).view(torch.int16))


def test_requests_apart_and_value_sizes():
    # requests further apart than their slots, by whole rows and by less
    for extra in (512, 2048 + 16):
        for fp8 in (False, True):
            c = TreeCase(flint.CONTIGUOUS, fp8, False, [100, 200], [5, 9], 9, seed=8, stride_extra=extra)
            c.check(c.run())
    c = TreeCase(flint.CONTIGUOUS, False, False, [300], [4], 4, seed=9, value_scale=6.0)
    c.check(c.run())  # scores in the hundreds: one key takes it all


def test_no_nodes_anywhere_writes_nothing():
    c = TreeCase(flint.CONTIGUOUS, False, False, [10, 0], [0, 0], 4, seed=10)
    assert (c.run() == 77.0).all()


def test_sink_of_minus_infinity_and_of_much():
    c = TreeCase(flint.PAGED, False, False, [90], [3], 3, seed=11)
    c.sinks[:8] = float("-inf")
    c.sinks[8:12] = 300.0  # takes all of the softmax
    got = c.run()
    c.check(got)


def test_bad_parents_and_pages_are_reported():
    c = TreeCase(flint.CONTIGUOUS, False, False, [70], [4], 4, seed=12)
    err = torch.zeros(8, dtype=torch.int32, device="cuda")
    out = torch.zeros((1, 4, 32, 128), dtype=torch.bfloat16, device="cuda")
    args = [x.cuda() for x in (c.q, c.kd, c.vd)]
    parent = torch.tensor([[-1, 0, 2, 1]], dtype=torch.int32, device="cuda")  # node 2 names itself
    flint.flint_attn_tree(*args, parent, c.device_cache(), c.lens, c.n_draft, c.sinks.cuda(), 0, out,
                          flint.tree_workspace(), dev_err=err)
    torch.cuda.synchronize()
    assert int(err[0]) == flint.FLINT_ERR_INVALID_ARG
    c.parents = [[-1, 0, -1, 1]]  # what such a parent counts as
    want, bound = c.reference()
    assert ((out.cpu().double() - want).abs() <= bound).all()
    c = TreeCase(flint.PAGED, False, False, [200], [2], 2, seed=13)
    for bad in (-1, 10 ** 6):
        c.table[0, 1] = bad
        err.zero_()
        flint.flint_attn_tree(c.q.cuda(), c.kd.cuda(), c.vd.cuda(), c.parent.cuda(), c.device_cache(), c.lens, c.n_draft,
                              c.sinks.cuda(), 0, out[:, :2].contiguous(), flint.tree_workspace(), dev_err=err)
        torch.cuda.synchronize()
        assert int(err[0]) == flint.FLINT_ERR_INVALID_ARG


def test_captured_and_replayed_on_another_stream():
    c = TreeCase(flint.PAGED, False, False, [1500, 33], [6, 2], 6, seed=14)
    q, kd, vd, parent, sinks = (x.cuda() for x in (c.q, c.kd, c.vd, c.parent, c.sinks))
    cache, ws = c.device_cache(), flint.tree_workspace()
    out = torch.full((2, 6, 32, 128), 77.0, dtype=torch.bfloat16, device="cuda")
    call = lambda: flint.flint_attn_tree(q, kd, vd, parent, cache, c.lens, c.n_draft, sinks, 0, out, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
        call()
    out.fill_(77.0)
    graph.replay()
    torch.cuda.synchronize()
    c.check(out.cpu())


def test_a_chain_is_decoding_one_by_one():
    """The tree call on a chain against flint_kv_append and flint_attn_decode in turn."""
    for fp8 in (False, True):
        c = TreeCase(flint.CONTIGUOUS, fp8, False, [450], [5], 5, kind="chain", seed=15)
        got = c.run()
        cache, ws = c.device_cache(), flint.workspace(1)
        c.kdev[0, 450:], c.vdev[0, 450:] = 0, 0
        q, kd, vd = c.q.cuda(), c.kd.cuda(), c.vd.cuda()
        _, bound = c.reference()
        for i in range(5):
            flint.flint_kv_append(kd[:, i].contiguous(), vd[:, i].contiguous(), [450 + i], cache)
            one = torch.empty((1, 32, 128), dtype=torch.float32, device="cuda")
            flint.flint_attn_decode(q[:, i].contiguous(), cache, [451 + i], c.sinks.cuda(), 0, one, ws)
            d = (one.cpu().double()[0] - got[0, i].double()).abs()
            # the decode call's own error is far below the bound's 2^-10 share
            assert (d <= bound[0, i] * 1.1).all()
