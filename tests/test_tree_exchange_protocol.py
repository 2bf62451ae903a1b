"""Model check, on the CPU, of how the tree attention's two softmax warpgroups
exchange their rows' maximum and sum at the end of an item with one row tile.

A CTA works through items (a unit's share of key tiles).  With one row tile the
key tiles of parity w are stream w's; at the item's end warpgroup w writes its
state to slot w of one shared buffer, both read both slots, and the MMA warp
starts the next item's first S without waiting for any of it.  So a warpgroup
whose stream has no or one step in the next item can reach its next write while
the other still reads, unless it waits for that item's end (o_free) first.

Three agents (the MMA warp, a warp of each warpgroup) run fixed programs of
waits, arrivals, writes and reads; every interleaving is visited.  Checked: each
read finds its own item's state; no wait is two phases behind (a parity would
mislead it); every state goes on until all agents have ended.  The writer's wait
is in the model where the kernel's source has it."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "long_context_decode_flash_b200", "csrc", "flint_tree.cu")
COUNT = {"s0": 1, "s1": 1, "p0": 1, "p1": 1, "ex": 2, "o_full": 1, "o_free": 2}


def steps_of(item):
    """Steps of stream 0, 1: an item is (row tiles, key tiles)."""
    mt, tiles = item
    return (tiles, tiles) if mt == 2 else ((tiles + 1) // 2, tiles // 2)


def programs(items, guarded):
    mma, soft = [], ([], [])
    done, x = [0, 0], 0
    for i, item in enumerate(items):
        mt, tiles = item
        steps = mt * tiles
        for s in range(-2, steps):
            w = s & 1
            if s >= 0:
                mma.append(("wait", f"p{w}", done[w] + (s >> 1)))
                if s == 0 and i > 0:
                    mma.append(("wait", "o_free", i - 1))
                if s == steps - 1:
                    mma.append(("arrive", "o_full"))
            if s + 2 < steps:
                mma.append(("arrive", f"s{w}"))
        for w, run in enumerate(soft):
            for s in range(steps_of(item)[w]):
                run += [("wait", f"s{w}", done[w] + s), ("arrive", f"p{w}")]
            if mt == 1:
                if guarded and i > 0:
                    run.append(("wait", "o_free", i - 1))
                run += [("write", w, i), ("arrive", "ex"), ("wait", "ex", x), ("read", 0, i), ("read", 1, i)]
            run += [("wait", "o_full", i), ("arrive", "o_free")]
        done = [done[w] + steps_of(item)[w] for w in range(2)]
        x += mt == 1
    return [mma, *soft]


def violations(items, guarded):
    """What goes wrong in some interleaving: a set of texts."""
    runs = programs(items, guarded)
    # per agent and position: arrivals so far, and the last value written
    arrived = [[{}] for _ in runs]
    written = [[None] for _ in runs]
    for a, run in enumerate(runs):
        for op in run:
            n = dict(arrived[a][-1])
            if op[0] == "arrive":
                n[op[1]] = n.get(op[1], 0) + 1
            arrived[a].append(n)
            written[a].append(op[2] if op[0] == "write" else written[a][-1])
    wrong, seen, todo = set(), {(0, 0, 0)}, [(0, 0, 0)]
    while todo:
        at = todo.pop()
        moved = False
        for a, run in enumerate(runs):
            if at[a] == len(run):
                continue
            op = run[at[a]]
            if op[0] == "wait":
                complete = sum(arrived[k][at[k]].get(op[1], 0) for k in range(3)) // COUNT[op[1]]
                if complete <= op[2]:
                    continue
                if complete > op[2] + 1:
                    wrong.add(f"a wait for {op[1]} is {complete - op[2]} phases behind")
            if op[0] == "read" and written[1 + op[1]][at[1 + op[1]]] != op[2]:
                wrong.add(f"slot {op[1]} read for item {op[2]} holds another's")
            moved = True
            nxt = at[:a] + (at[a] + 1,) + at[a + 1:]
            if nxt not in seen:
                seen.add(nxt)
                todo.append(nxt)
        if not moved and any(at[a] < len(run) for a, run in enumerate(runs)):
            wrong.add(f"nobody can go on at {at}")
    return wrong


def kernel_waits():
    """The kernel's writer waits for the end of the item before."""
    text = open(SOURCE).read()
    end = text.index("ex[w * kTrRows + r] = ")
    begin = text.rindex("if (!two) {", 0, end)
    return re.search(r"it\.i > 0 && !warp_wait\(smem_u32\(&B->o_free\), static_cast<uint32_t>\(it\.i - 1\) & 1u, B\)\) return false;",
                     text[begin:end]) is not None


# short contexts one after another, longer ones between, and units of two row tiles
LISTS = [[(1, 1)] * 4, [(1, 2)] * 4, [(1, 3), (1, 1), (1, 2), (1, 1)], [(1, 5), (1, 1), (1, 4), (1, 3)],
         [(2, 2), (1, 1), (2, 1), (1, 2), (1, 1)], [(1, 1), (2, 3), (1, 3), (1, 1)]]


@pytest.mark.parametrize("items", LISTS)
def test_every_read_finds_its_own_item(items):
    assert violations(items, kernel_waits()) == set()


@pytest.mark.parametrize("items", LISTS[:4])
def test_the_model_sees_a_writer_that_does_not_wait(items):
    assert any("another's" in x for x in violations(items, False))
