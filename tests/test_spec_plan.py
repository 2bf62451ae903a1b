"""The plan of the tree attention (pure host code): every tile of every unit
belongs to exactly one group, and what the kernel relies on."""
import random

import pytest

from long_context_decode_flash_b200 import flint

LAYOUTS = (flint.CONTIGUOUS, flint.RING, flint.PAGED)


def tiles_of(L, window, layout):
    """Tiles of 128 keys: a half of 64 for the drafts, and the cache's in halves."""
    lo = max(0, L - 512) if window else 0
    if layout == flint.RING:
        base, hi = 0, min(L, 513)
    else:
        base, hi = (lo // 64 * 64 if layout == flint.PAGED else lo), L
    return (1 + -(-(hi - base) // 64) + 1) // 2


@pytest.mark.parametrize("seed", range(300))
def test_every_tile_once(seed):
    rng = random.Random(seed)
    B = rng.choice([1, 2, 5, 33, 64])
    layout = rng.choice(LAYOUTS)
    window = 513 if layout == flint.RING or rng.random() < 0.3 else 0
    top = rng.choice([1, 200, 3000, 262144])
    lens = [rng.randint(0, top) for _ in range(B)]
    n = [rng.randint(0, rng.choice([1, 8, 17, 64])) for _ in range(B)]
    ctas = rng.choice([1, 4, 7, 60, 148, 296])
    units, cuts = flint.flint_plan_tree(lens, n, window, layout, rng.random() < 0.5, ctas)
    want = [(b, r, tiles_of(lens[b], window, layout), 2 if n[b] - 32 * r > 16 else 1) for b in range(B) for r in range(-(-n[b] // 32))]
    assert sorted(units) == want  # (units that stay whole are dealt by size)
    if not units:
        assert cuts == [(0, 0)] and len(cuts) == 1
        return
    assert len(cuts) - 1 <= max(1, ctas // 4)
    assert cuts[0] == (0, 0) and cuts[-1] == (len(units), 0)
    for (u, t), (v, s) in zip(cuts, cuts[1:]):
        assert (u, t) < (v, s)  # no empty group
        assert t < units[u][2] and (v == len(units) or s < units[v][2])
        # items: only the first and the last may be parts of their unit (two
        # places for partials a CTA)
        items = [(x, t if x == u else 0, units[x][2] if x < v else s) for x in range(u, v + 1) if x < v or s > 0]
        assert all(a == 0 and e == units[x][2] for x, a, e in items[1:-1])
        assert all(a < e for _, a, e in items)


def test_shares_are_even():
    units, cuts = flint.flint_plan_tree([100000], [8])
    at = [t for _, t in cuts[:-1]] + [units[0][2]]
    shares = [b - a for a, b in zip(at, at[1:])]
    assert len(shares) == 37 and max(shares) - min(shares) <= 5


def test_refusals():
    for kw in (dict(seq_lens=[-1], n_draft=[1]), dict(seq_lens=[1], n_draft=[65]), dict(seq_lens=[1], n_draft=[1], window=5),
               dict(seq_lens=[1], n_draft=[1], num_ctas=0), dict(seq_lens=[1], n_draft=[1], num_ctas=297),
               dict(seq_lens=[1], n_draft=[1], layout=3), dict(seq_lens=[1] * 65, n_draft=[1] * 65)):
        with pytest.raises(flint.FlintError):
            flint.flint_plan_tree(**kw)
