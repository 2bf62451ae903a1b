"""flint_attn_tree where a CTA works through many small units one after another."""
import pytest
import torch

from long_context_decode_flash_b200 import flint

from spec_helpers import TreeCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("top", [64, 192, 450])
@pytest.mark.parametrize("N", [5, 20])
def test_short_contexts_one_after_another(N, top, fp8):
    """One group of CTAs takes the units of 48 requests in turn, most of one to four
    key tiles; scores of very different sizes, so that another item's maximum or
    sum would show."""
    lens = [(23 * b) % (top + 1) for b in range(48)]
    n = [1 + (7 * b) % N for b in range(48)]
    c = TreeCase(flint.PAGED, fp8, False, lens, n, N, seed=51)
    for b in range(48):
        c.q[b] *= (0.05, 8.0, 1.0, 3.0, 0.3)[b % 5]
    first = c.run(num_ctas=4)
    c.check(first)
    for ctas in (4, 12, 0):
        got = c.run(num_ctas=ctas)
        c.check(got)
        if ctas == 4:
            assert torch.equal(first.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,N", [([100_000], 40), ([60_000, 40_000, 70_001], 12), ([30_000] * 4, 33), ([100_000], 8)])
def test_many_calls_back_to_back(lens, N, fp8):
    """Captured calls that follow one another without a pause, all SMs loading at
    once: every one gives the bits of a call alone, and no wait runs out."""
    B, L = len(lens), max(lens)
    g = torch.Generator(device="cuda").manual_seed(52)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    k, v = rnd(B, L, 4, 128), rnd(B, L, 4, 128)
    if fp8:
        k, v = ((x * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    scale = [1 / 64] * 4 if fp8 else None
    cache = flint.kv_cache(k, v, flint.CONTIGUOUS, capacity=L, k_scale=scale, v_scale=scale)
    q, kd, vd = rnd(B, N, 32, 128), rnd(B, N, 4, 128), rnd(B, N, 4, 128)
    parent = torch.tensor([[i // 2 - 1 for i in range(N)]] * B, dtype=torch.int32, device="cuda")
    sinks, ws = torch.zeros(32, device="cuda"), flint.tree_workspace()
    err = torch.zeros(8, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q) for _ in range(10)]
    call = lambda out: flint.flint_attn_tree(q, kd, vd, parent, cache, lens, [N] * B, sinks, 0, out, ws, dev_err=err)  # noqa: E731
    call(outs[0])
    torch.cuda.synchronize()
    alone = outs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in outs:
            call(out)
    for _ in range(20):
        for out in outs:
            out.fill_(77.0)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err[0]) == 0, err.tolist()
        for out in outs:
            assert torch.equal(out.view(torch.int16), alone.view(torch.int16))
