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
