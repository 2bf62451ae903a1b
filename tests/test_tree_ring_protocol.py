"""Model check, on the CPU, of the tree attention's rings of key and value tiles.

Two producer warps load K and V tiles into stages, the converter warps make
operands of V (and, against E4M3, of the drafts in an item's first K tile), the
MMA warp consumes both.  With a bf16 cache K and V share one ring of 6 or 5
stages in the order of their use; with E4M3, K has 3 stages, V's codes 3 and
fp16 V 3 or 2.  Loads land in any order.

A wait names a phase by its parity, so it tells phase n from phase n - 2 only
once phase n - 1 is complete.  The converters do not wait for K tiles: where V
tiles landed on the same barriers, a wait for one could pass while the stage's K
tile before it was in flight.  So each stage of the shared ring has a barrier for
either kind.  (With E4M3 the converters meet K tiles only at an item's start, where
the tile before is known to have landed.)

Every interleaving of the agents and of the loads' landings is visited.  Checked:
no wait passes before its own phase is complete, none finds a later one
complete, and every state goes on until all agents have ended.  The barriers are
apart in the model where they are in the kernel's source."""
import os

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "long_context_decode_flash_b200", "csrc", "flint_tree.cu")


def seq_of(v, j, n, mt):
    if mt == 2:
        return 2 * j + v
    return (2 * n - 1 if j == n - 1 else 2 * j + 2) if v else (0 if j == 0 else 2 * j - 1)


def mma_steps(mt, n):
    """("s" | "pv", tile, whether it is the tile's last use) of an item."""
    out = []
    for s in range(-2, mt * n):
        tile = lambda x: x >> 1 if mt == 2 else x  # noqa: E731
        last = mt == 1 or s & 1
        if s >= 0:
            out.append(("pv", tile(s), last))
        if s + 2 < mt * n:
            out.append(("s", tile(s + 2), last))
    return out


def shared_ring(items, size, apart):
    """bf16: agents' programs; items: (row tiles, key tiles).  apart: a stage has a
    barrier for K tiles and one for V tiles, else one for both."""
    kp, vp, conv, mma = [], [], [], []
    T, phases, phase_of = 0, {}, {}
    # phases in the order in which a stage's tiles land
    order = sorted((2 * U + seq_of(v, j, n, mt), v) for U, (mt, n) in zip(starts(items), items) for j in range(n) for v in (0, 1))
    for c, v in order:
        bar = ("full", c % size, v if apart else 0)
        phase_of[c] = bar, phases.get(bar, 0)
        phases[bar] = phases.get(bar, 0) + 1
    for mt, n in items:
        for j in range(n):
            for run, v in ((kp, 0), (vp, 1)):
                c = 2 * T + seq_of(v, j, n, mt)
                if c >= size:
                    run.append(("wait", ("empty", c % size), c // size - 1))
                run.append(("load", phase_of[c][0]))
            c = 2 * T + seq_of(1, j, n, mt)
            conv += [("wait", *phase_of[c]), ("arrive", ("v_ready", (T + j) % 4))]
        for kind, j, last in mma_steps(mt, n):
            c = 2 * T + seq_of(kind == "pv", j, n, mt)
            mma.append(("wait", ("v_ready", (T + j) % 4), (T + j) // 4) if kind == "pv" else ("wait", *phase_of[c]))
            if last:
                mma.append(("arrive", ("empty", c % size)))
        T += n
    return [kp, vp, conv, mma], {}


def starts(items):
    return [sum(n for _, n in items[:i]) for i in range(len(items))]


def split_rings(items, v_tiles):
    """E4M3; an item that begins its unit (all here) has drafts in its first tile.
    Two of the converter warps: the one that also loads Q waits for the item before."""
    kp, vp, mma = [], [], []
    convs = ([], [])
    T = raw_in = raw_out = 0
    for i, (mt, n) in enumerate(items):
        for w, conv in enumerate(convs):
            raw = raw_out
            if w == 0 and i > 0:
                conv.append(("wait", ("q_empty", 0), i - 1))

            def take(bar, size):
                nonlocal raw
                conv.extend([("wait", (bar, raw % size), raw // size), ("arrive", ("raw_free", raw % size))])
                raw += 1
            conv.append(("wait", ("raw", raw % 3), raw // 3))
            conv += [("wait", ("full", T % 3), T // 3), ("arrive", ("raw_free", raw % 3)), ("arrive", ("kd", 0))]
            raw += 1
            for j in range(n):
                if T + j >= v_tiles:
                    conv.append(("wait", ("v_empty", (T + j) % v_tiles), (T + j) // v_tiles - 1))
                if j == 0:
                    take("raw", 3)
                take("raw", 3)
                conv.append(("arrive", ("v_ready", (T + j) % 4)))
        raw_out = raw
        for j in range(n):
            if T + j >= 3:
                kp.append(("wait", ("empty", (T + j) % 3), (T + j) // 3 - 1))
            kp.append(("load", ("full", (T + j) % 3)))
            for _ in range(3 if j == 0 else 1):
                if raw_in >= 3:
                    vp.append(("wait", ("raw_free", raw_in % 3), raw_in // 3 - 1))
                vp.append(("load", ("raw", raw_in % 3)))
                raw_in += 1
        mma.append(("wait", ("kd", 0), i))
        steps = mma_steps(mt, n)
        for k, (kind, j, last) in enumerate(steps):
            t = T + j
            if kind == "pv":
                mma.append(("wait", ("v_ready", t % 4), t // 4))
                if last:
                    mma.append(("arrive", ("v_empty", t % v_tiles)))
            else:
                mma.append(("wait", ("full", t % 3), t // 3))
                if last:
                    mma.append(("arrive", ("empty", t % 3)))
                if all(x[0] == "pv" for x in steps[k + 1:]):
                    mma.append(("arrive", ("q_empty", 0)))
        T += n
    both = {b: 2 for b in [("raw_free", k) for k in range(3)] + [("v_ready", k) for k in range(4)] + [("kd", 0)]}
    return [kp, vp, *convs, mma], both


def violations(model):
    runs, counts = model
    # every arrival by position: agents', and loads (which land later)
    loads = [(a, k, op[1]) for a, run in enumerate(runs) for k, op in enumerate(run) if op[0] == "load"]
    by_agent = [{} for _ in runs]
    for a, run in enumerate(runs):
        for k, op in enumerate(run):
            if op[0] == "arrive":
                by_agent[a].setdefault(op[1], []).append(k)
    load_of = {}
    for x, (_, _, bar) in enumerate(loads):
        load_of.setdefault(bar, []).append(x)

    def complete(bar, at, landed):
        n = sum(sum(k < at[a] for k in by_agent[a].get(bar, ())) for a in range(len(runs)))
        n += sum(landed >> x & 1 for x in load_of.get(bar, ()))
        return n // counts.get(bar, 1)
    start = (tuple(0 for _ in runs), 0)
    wrong, seen, todo = set(), {start}, [start]
    while todo:
        at, landed = todo.pop()
        nexts = []
        for x, (a, k, _) in enumerate(loads):
            if at[a] > k and not landed >> x & 1:
                nexts.append((at, landed | 1 << x))
        for a, run in enumerate(runs):
            if at[a] == len(run):
                continue
            op = run[at[a]]
            if op[0] == "wait":
                done = complete(op[1], at, landed)
                if (done + op[2]) % 2 == 0:  # the phase of this parity is the one in progress
                    continue
                if done != op[2] + 1:
                    wrong.add(f"a wait for phase {op[2]} of {op[1]} passes with {done} complete")
                    continue
            nexts.append((at[:a] + (at[a] + 1,) + at[a + 1:], landed))
        if not nexts and any(at[a] < len(run) for a, run in enumerate(runs)):
            wrong.add(f"nobody can go on at {at}")
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
        if len(wrong) > 3:
            break
    return wrong


def barriers_apart():
    """The kernel's K and V tiles of the shared ring land on barriers of their own."""
    text = open(SOURCE).read()
    producer = text[text.index("bool run_tma("):text.index("// Byte offset of chunk")]
    conv = text[text.index("bool run_conv("):text.index("// The MMA warp, over its items' steps")]
    return ("kV ? B->full_v : B->full" in producer and conv.count("&B->full_v[") == 1 and "phases ^= 1u <<" in conv and
            conv.count("&B->full[") == 1)  # (that one: an item's first K tile, against E4M3)


SHARED = [(6, [(1, 7)]), (6, [(1, 2), (1, 1), (1, 3), (1, 2)]), (5, [(1, 6)]), (5, [(2, 5)]), (5, [(2, 2), (1, 3), (1, 1), (2, 2)])]
SPLIT = [(3, [(1, 4), (1, 2)]), (3, [(1, 1), (1, 1), (1, 1), (1, 1)]), (2, [(2, 3), (2, 2)]), (2, [(1, 3), (2, 2)])]


@pytest.mark.parametrize("size,items", SHARED)
def test_one_ring_for_both(size, items):
    assert violations(shared_ring(items, size, barriers_apart())) == set()


@pytest.mark.parametrize("v_tiles,items", SPLIT)
def test_rings_of_their_own(v_tiles, items):
    assert violations(split_rings(items, v_tiles)) == set()


@pytest.mark.parametrize("size,items", [SHARED[0], SHARED[2], SHARED[3]])
def test_the_model_sees_a_wait_that_passes_early(size, items):
    assert any("passes with" in x for x in violations(shared_ring(items, size, False)))
