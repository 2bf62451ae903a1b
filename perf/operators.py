"""The operators of one speculative decode step, measured: drafted tokens are
normed and rotated at their positions (`rope`), attend the committed cache and
their own ancestors (`attend`), are verified against the target's
probabilities (`verify`), and the accepted ones are written to every layer's
cache (`append`).

Geometry throughout: 32 query heads over 4 KV heads of 128 dims, a learned sink
logit per query head, full layers or 513-token windows, 64-token pages.
"""
import math
import random

import torch

own = False

HEADS, KV_HEADS, DIM, GROUP = 32, 4, 128, 8
WINDOW, PAGE, LAYERS = 513, 64, 49
CONTIGUOUS, RING, PAGED = 0, 1, 2


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # A chain of five drafts behind one 513-token window layer of one
        # request: the smallest step, where only latency counts.
        dict(name="attend window ring B1 N5", op="attend", layout="ring", kv="bf16", window=True, B=1, N=5,
             lo=100000, hi=100000, tree="chain"),
        # The batch-1 long-context step this framework is built for, with a
        # tree of eight drafts on a full layer.
        dict(name="attend 100k B1 N8", op="attend", layout="contiguous", kv="bf16", window=False, B=1, N=8,
             lo=100000, hi=100000, tree="tree"),
        # A wide tree on the same layer with the 8-bit cache.
        dict(name="attend 100k e4m3 B1 N30", op="attend", layout="contiguous", kv="e4m3", window=False, B=1, N=30,
             lo=100000, hi=100000, tree="tree"),
        # The paged serving batch, ragged lengths and ragged trees.
        dict(name="attend paged B32 N16", op="attend", layout="paged", kv="bf16", window=False, B=32, N=16,
             lo=4096, hi=131072, tree="tree"),
        # The largest trees on a middle context: work bound by arithmetic.
        dict(name="attend paged e4m3 B4 N64", op="attend", layout="paged", kv="e4m3", window=False, B=4, N=64,
             lo=20011, hi=40009, tree="tree"),
        # One request, a chain of four, a small vocabulary.
        dict(name="verify B1 N4 V32000", op="verify", B=1, N=4, V=32000, tree="chain", dists=True),
        # A full batch of chains with a large vocabulary.
        dict(name="verify B64 N6 V150001", op="verify", B=64, N=6, V=150001, tree="chain", dists=True),
        # Trees of fixed candidates (no draft distribution).
        dict(name="verify B16 N31 V131072", op="verify", B=16, N=31, V=131072, tree="tree", dists=False),
        # The drafted tokens of a small batch, the model's own rotary form,
        # q and k as slices of one fused projection.
        dict(name="rope T40 half", op="rope", T=40, fused=True, dim=128, interleaved=False, scaling="none",
             factor=1.0, far=100000),
        # A prompt's worth of tokens of a long-context checkpoint: part of the
        # head, interleaved pairs, scaled frequencies.
        dict(name="rope T8191 part interleaved", op="rope", T=8191, fused=False, dim=96, interleaved=True,
             scaling="yarn", factor=8.0, far=262000),
        # The accepted path of one request into 14 full layers.
        dict(name="append B1 N5 bf16", op="append", B=1, N=5, layers=14, kv="bf16", pages=4),
        # A full batch into all 49 layers, quantised as it is written.
        dict(name="append B64 N8 e4m3", op="append", B=64, N=8, layers=LAYERS, kv="e4m3", pages=2),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "verify", "verify", "rope", "append"])
    if op == "attend":
        layout = rng.choice(["contiguous", "paged", "ring"])
        B, N = _log_uniform(rng, 1, 48), _log_uniform(rng, 1, 64)
        # at most ~1.1 M cached tokens over the batch, at most 16 times fewer
        # with 64 drafts than with 4
        top = max(300, min(131072, 1_100_000 // B, 8_000_000 // (B * max(4, N))))
        hi = _log_uniform(rng, 1, top)
        lo = max(0, int(hi * rng.random()))
        window = layout == "ring" or rng.random() < 0.25
        return dict(op=op, layout=layout, kv=rng.choice(["bf16", "e4m3"]), window=window, B=B, N=N, lo=lo, hi=hi,
                    tree=rng.choice(["chain", "tree", "tree"]))
    if op == "verify":
        N = _log_uniform(rng, 1, 64)
        V = _log_uniform(rng, 500, 200000)
        B = min(64, max(1, _log_uniform(rng, 1, max(1, 60_000_000 // (V * N)))))
        return dict(op=op, B=B, N=N, V=V, tree=rng.choice(["chain", "tree"]), dists=rng.random() < 0.6)
    if op == "rope":
        scaling = rng.choice(["none", "linear", "yarn"])
        return dict(op=op, T=_log_uniform(rng, 1, 8191), fused=rng.random() < 0.5, dim=2 * rng.randint(1, 64),
                    interleaved=rng.random() < 0.5, scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 3.5]),
                    far=_log_uniform(rng, 10, 262000))
    return dict(op=op, B=_log_uniform(rng, 1, 64), N=rng.randint(1, 12), layers=rng.randint(1, LAYERS),
                kv=rng.choice(["bf16", "e4m3"]), pages=rng.randint(1, 2))


def _lengths(case):
    """Committed tokens of each request: log-uniform in [lo, hi], fixed by the case."""
    rng = random.Random("lengths %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    lo, hi = case["lo"], case["hi"]
    return [lo if lo == hi else max(lo, min(hi, _log_uniform(rng, max(1, lo), hi))) for _ in range(case["B"])]


def _counts(case):
    """Drafted tokens of each request: all N, or ragged below it in a batch."""
    rng = random.Random("counts %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    return [case["N"] if case["B"] == 1 or rng.random() < 0.5 else rng.randint(1, case["N"]) for _ in range(case["B"])]


def _parents(case, rng):
    """parent[b][i] in [-1, i): a chain, or a tree of a few children a node."""
    B, N = case["B"], case["N"]
    if case["tree"] == "chain":
        return [[i - 1 for i in range(N)] for _ in range(B)]
    return [[rng.randint(max(-1, i // 2 - 3), max(-1, i // 2 - 1)) for i in range(N)] for _ in range(B)]


# ---------------------------------------------------------------- prepare --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)


def _randn(g, *shape):
    """bf16 N(0, 1)."""
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _cache_values(g, kv, *shape):
    """A cache buffer of history: bf16 values, or E4M3 codes of values / scale."""
    if kv == "bf16":
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return (x.mul_(448.0 / 6.0).clamp_(-448.0, 448.0)).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(kv, seed):
    rng = random.Random("scales %d" % seed)
    return [[6.0 / 448.0 * rng.uniform(0.9, 1.1) for _ in range(KV_HEADS)] for _ in range(2)] if kv == "e4m3" else [None, None]


def prepare(case, seed):
    return {"attend": _prepare_attend, "verify": _prepare_verify, "rope": _prepare_rope,
            "append": _prepare_append}[case["op"]](case, seed)


def _prepare_attend(case, seed):
    g, rng = _gen(seed), random.Random("tree %d" % seed)
    B, N, kv = case["B"], case["N"], case["kv"]
    lens, counts = _lengths(case), _counts(case)
    s = dict(case=case, lens=lens, counts=counts)
    if case["layout"] == "paged":
        used = [max(1, -(-n // PAGE)) for n in lens]
        order = torch.randperm(sum(used), generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((B, max(used)), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = order[at:at + n]
            at += n
        shape, s["table"] = (sum(used), PAGE, KV_HEADS, DIM), table
    else:
        slots = WINDOW if case["layout"] == "ring" else max(1, max(lens))
        shape, s["table"] = (B, slots, KV_HEADS, DIM), None
    s["k"], s["v"] = _cache_values(g, kv, *shape), _cache_values(g, kv, *shape)
    s["k_scale"], s["v_scale"] = _scales(kv, seed)
    s["q"] = _randn(g, B, N, HEADS, DIM)
    s["k_draft"], s["v_draft"] = _randn(g, B, N, KV_HEADS, DIM), _randn(g, B, N, KV_HEADS, DIM)
    s["sinks"] = torch.randn(HEADS, generator=g, device="cuda", dtype=torch.float32)
    s["parents"] = _parents(case, rng)
    s["parent"] = torch.tensor(s["parents"], dtype=torch.int32, device="cuda")
    s["out"] = torch.zeros((B, N, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
    if own:  # the cache handle and the workspace that a serving loop keeps
        from long_context_decode_flash_b200 import flint
        layout = {"contiguous": flint.CONTIGUOUS, "ring": flint.RING, "paged": flint.PAGED}[case["layout"]]
        s["cache"] = flint.kv_cache(s["k"], s["v"], layout, capacity=0 if layout == flint.PAGED else shape[1],
                                    block_table=s["table"], num_blocks=shape[0] if layout == flint.PAGED else 0,
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["ws"] = flint.tree_workspace()
    return s


def _prepare_verify(case, seed):
    g, rng = _gen(seed), random.Random("tree %d" % seed)
    B, N, V = case["B"], case["N"], case["V"]
    parents = _parents(case, rng)
    s = dict(case=case, counts=_counts(case), parents=parents)
    s["parent"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    target = torch.empty((B, N + 1, V), dtype=torch.float32, device="cuda")
    draft = torch.empty((B, N, V), dtype=torch.float32, device="cuda")
    tokens = torch.empty((B, N), dtype=torch.int64, device="cuda")
    row = s["parent"].long() + 1
    for b in range(B):
        logits = torch.randn((N + 1, V), generator=g, device="cuda").mul_(3.0)
        target[b] = torch.softmax(logits, -1)
        logits.add_(torch.randn((N + 1, V), generator=g, device="cuda").mul_(0.7))
        draft[b] = torch.softmax(logits[:N], -1)
        # each drafted token is a draw from the draft's distribution at its parent
        noise = torch.empty((N, V), device="cuda").exponential_(generator=g)
        tokens[b] = (draft[b][row[b]] / noise).argmax(-1)
    s["target"], s["draft"] = target, draft if case["dists"] else None
    s["tokens"] = tokens.to(torch.int32)
    s["u_accept"] = torch.rand((B, N), generator=g, device="cuda")
    s["u_sample"] = torch.rand((B,), generator=g, device="cuda")
    s["path"] = torch.empty((B, N), dtype=torch.int32, device="cuda")
    s["n_accepted"] = torch.empty((B,), dtype=torch.int32, device="cuda")
    s["next_token"] = torch.empty((B,), dtype=torch.int32, device="cuda")
    return s


def _prepare_rope(case, seed):
    g = _gen(seed)
    T = case["T"]
    if case["fused"]:  # q, k and v side by side in one projection's output
        qkv = _randn(g, T, HEADS + 2 * KV_HEADS, DIM)
        q, k = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS]
    else:
        q, k = _randn(g, T, HEADS, DIM), _randn(g, T, KV_HEADS, DIM)
    s = dict(case=case, q_raw=q, k_raw=k)
    s["w_q"], s["w_k"] = ((1.0 + 0.1 * torch.randn(DIM, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
    s["q_out"] = torch.empty((T, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
    s["k_out"] = torch.empty((T, KV_HEADS, DIM), dtype=torch.bfloat16, device="cuda")
    if own:  # the rotary description that a model keeps
        from long_context_decode_flash_b200 import flint
        s["rope"] = flint.rope(rotary_dim=case["dim"], interleaved=case["interleaved"], theta=10000.0,
                               scaling=case["scaling"], factor=case["factor"], original_context=8192)
    return s


def _prepare_append(case, seed):
    g, rng = _gen(seed), random.Random("path %d" % seed)
    B, N, n, kv = case["B"], case["N"], case["layers"], case["kv"]
    pages = case["pages"]
    s = dict(case=case, lens=[rng.randint(0, pages * PAGE - N) for _ in range(B)])
    s["k_draft"], s["v_draft"] = _randn(g, n, B, N, KV_HEADS, DIM), _randn(g, n, B, N, KV_HEADS, DIM)
    s["k"], s["v"] = (_cache_values(g, kv, n, B * pages, PAGE, KV_HEADS, DIM) for _ in range(2))
    s["k_scale"], s["v_scale"] = _scales(kv, seed)
    s["table"] = torch.randperm(B * pages, generator=g, device="cuda").to(torch.int32).view(B, pages)
    # accepted paths: increasing node indices, a ragged number of them
    accepted = [rng.randint(0, N) if B > 1 else max(1, N - 1) for _ in range(B)]
    paths = [sorted(rng.sample(range(N), a)) + [-1] * (N - a) for a in accepted]
    s["path"] = torch.tensor(paths, dtype=torch.int32, device="cuda")
    s["n_accepted"] = torch.tensor(accepted, dtype=torch.int32, device="cuda")
    s["lens_dev"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    if own:  # the layers' handles that a serving loop keeps
        from long_context_decode_flash_b200 import flint
        caches = [flint.kv_cache(s["k"][i], s["v"][i], flint.PAGED, block_table=s["table"], num_blocks=B * pages,
                                 k_scale=s["k_scale"], v_scale=s["v_scale"]) for i in range(n)]
        s["layers"] = flint.path_layers([(s["k_draft"][i], s["v_draft"][i], caches[i]) for i in range(n)])
    return s


# -------------------------------------------------------------------- run --

def run(state):
    return {"attend": _run_attend, "verify": _run_verify, "rope": _run_rope, "append": _run_append}[state["case"]["op"]](state)


def _dequantised(x, scale):
    """fp32 values of a cache buffer [..., 4, 128]."""
    if scale is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * torch.tensor(scale, dtype=torch.float32, device=x.device)[:, None]


def _codes(x, scale):
    """E4M3 codes of bf16 values [..., 4, 128]: value / scale in fp32, nearest even, saturating."""
    y = x.float() / torch.tensor(scale, dtype=torch.float32, device=x.device)[:, None]
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _ancestors(parents):
    """[N, N] truth values: node i attends node j (its ancestors and itself)."""
    rows = []
    for i, p in enumerate(parents):
        rows.append([j == i or (p >= 0 and rows[p][j]) for j in range(len(parents))])
    return rows


def _run_attend(s):
    case = s["case"]
    if own:
        from long_context_decode_flash_b200 import flint
        return flint.flint_attn_tree(s["q"], s["k_draft"], s["v_draft"], s["parent"], s["cache"], s["lens"], s["counts"],
                                     s["sinks"], WINDOW if case["window"] else 0, s["out"], s["ws"])
    out, quant = s["out"], case["kv"] == "e4m3"
    k_draft = _dequantised(_codes(s["k_draft"], s["k_scale"]), s["k_scale"]) if quant else s["k_draft"].float()
    v_draft = _dequantised(_codes(s["v_draft"], s["v_scale"]), s["v_scale"]) if quant else s["v_draft"].float()
    for b, (L, n) in enumerate(zip(s["lens"], s["counts"])):
        first = max(0, L - WINDOW + 1) if case["window"] else 0
        pos = torch.arange(first, L, device="cuda")
        if case["layout"] == "paged":
            take = lambda x: x[s["table"][b].long()].flatten(0, 1)[first:L]  # noqa: E731
        elif case["layout"] == "ring":
            take = lambda x: x[b][pos % WINDOW]  # noqa: E731
        else:
            take = lambda x: x[b, first:L]  # noqa: E731
        k = torch.cat([_dequantised(take(s["k"]), s["k_scale"]), k_draft[b, :n]])
        v = torch.cat([_dequantised(take(s["v"]), s["v_scale"]), v_draft[b, :n]])
        tree = torch.tensor(_ancestors(s["parents"][b][:n]), device="cuda")
        depth = tree.sum(-1) - 1
        near = pos[None] > (L + depth)[:, None] - WINDOW if case["window"] else pos.new_ones((n, L - first), dtype=torch.bool)
        seen = torch.cat([near, tree], -1)  # [n, keys]
        q = s["q"][b, :n].float().view(n, KV_HEADS, GROUP, DIM).permute(1, 2, 0, 3).reshape(KV_HEADS, GROUP * n, DIM)
        score = torch.bmm(q, k.permute(1, 2, 0)).view(KV_HEADS, GROUP, n, -1) / math.sqrt(DIM)
        score = score.masked_fill(~seen, -math.inf)
        sink = s["sinks"].view(KV_HEADS, GROUP, 1, 1)
        top = torch.maximum(score.amax(-1, keepdim=True), sink)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True) + torch.exp(sink - top)
        o = torch.bmm(p.view(KV_HEADS, GROUP * n, -1), v.permute(1, 0, 2)).view(KV_HEADS, GROUP, n, DIM) / total
        out[b, :n] = o.permute(2, 0, 1, 3).reshape(n, HEADS, DIM).to(torch.bfloat16)
    return out


def _run_verify(s):
    case = s["case"]
    if own:
        from long_context_decode_flash_b200 import flint
        flint.flint_verify_tree(s["target"], s["draft"], s["tokens"], s["parent"], s["counts"], s["u_accept"],
                                s["u_sample"], s["path"], s["n_accepted"], s["next_token"])
        return s["path"], s["n_accepted"], s["next_token"]
    # 64 bits throughout: a draw decides at a border.  w, Z: the residual
    # distribution at the current node and its total.
    B, N = case["B"], case["N"]
    at = torch.arange(B, device="cuda")
    count = torch.tensor(s["counts"], device="cuda")
    cur = torch.full((B,), -1, device="cuda")
    taken = torch.zeros((B,), dtype=torch.int64, device="cuda")
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    w = s["target"][:, 0].double()
    Z = torch.ones((B,), dtype=torch.float64, device="cuda")
    for i in range(N):
        x = s["tokens"][:, i].long()
        q = s["draft"][at, (s["parent"][:, i] + 1).long()].double() if case["dists"] else None
        qx = q[at, x] if case["dists"] else 1.0
        asked = (s["parent"][:, i] == cur) & (i < count)
        yes = asked & (s["u_accept"][:, i].double() * qx * Z < w[at, x])
        no = asked & ~yes
        # a rejection leaves what the draft did not offer
        if case["dists"]:
            left = (w - Z[:, None] * q).clamp(min=0)
            sum_left = left.sum(-1)
        else:
            left = w.clone()
            left[at, x] = 0
            sum_left = Z - w[at, x]
        keep = no & (sum_left > 0)
        w = torch.where(keep[:, None], left, w)
        Z = torch.where(keep, sum_left, Z)
        # an acceptance moves on to the node
        w = torch.where(yes[:, None], s["target"][:, i + 1].double(), w)
        Z = torch.where(yes, 1.0, Z)
        path[at, taken.clamp(max=N - 1)] = torch.where(yes, i, path[at, taken.clamp(max=N - 1)].long()).to(torch.int32)
        taken = taken + yes
        cur = torch.where(yes, i, cur)
    c = w.cumsum(-1)
    over = c > s["u_sample"].double()[:, None] * c[:, -1:]
    held = torch.where(w > 0, torch.arange(case["V"], device="cuda"), 0).amax(-1)
    token = torch.where(over.any(-1), over.to(torch.uint8).argmax(-1), held)
    return path, taken.to(torch.int32), token.to(torch.int32)


def _frequencies(case):
    """The rotary frequencies of the pairs, in 64 bits, and the factor on cos and sin."""
    dim, factor = case["dim"], case["factor"]
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "yarn":  # by parts: fast pairs keep their frequency, slow ones are stretched
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _run_rope(s):
    case = s["case"]
    if own:
        from long_context_decode_flash_b200 import flint
        return flint.flint_qk_norm_rope_at(s["q_raw"], s["k_raw"], s["w_q"], s["w_k"], s["pos"], s["rope"],
                                           q_out=s["q_out"], k_out=s["k_out"])
    f, factor = _frequencies(case)
    angle = s["pos"].double()[:, None, None] * f
    cos, sin = (torch.cos(angle) * factor).float(), (torch.sin(angle) * factor).float()
    outs = []
    for x, w in ((s["q_raw"], s["w_q"]), (s["k_raw"], s["w_k"])):
        y = x.float()
        y = y * (1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6)) * w.float()
        r, rest = y[..., :case["dim"]], y[..., case["dim"]:]
        if case["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r.chunk(2, -1)
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        outs.append(torch.cat([r, rest], -1).to(torch.bfloat16))
    return outs[0], outs[1]


def _as_values(x, kv):
    return x if kv == "bf16" else x.view(torch.float8_e4m3fn)


def _run_append(s):
    case = s["case"]
    B, N = case["B"], case["N"]
    if own:
        from long_context_decode_flash_b200 import flint
        flint.flint_kv_append_path(s["layers"], s["path"], s["n_accepted"], s["lens"])
    else:
        step = torch.arange(N, device="cuda")
        b, j = torch.nonzero(step[None] < s["n_accepted"][:, None], as_tuple=True)
        node, pos = s["path"][b, j].long(), s["lens_dev"][b].long() + j
        page, row = s["table"][b, pos // PAGE].long(), pos % PAGE
        for name, scale in (("k", s["k_scale"]), ("v", s["v_scale"])):
            x = s[name + "_draft"][:, b, node]
            s[name][:, page, row] = x if scale is None else _codes(x, scale)
    return _as_values(s["k"], case["kv"]), _as_values(s["v"], case["kv"])


# ------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op == "attend":
        element = 2 if case["kv"] == "bf16" else 1
        tokens, pairs = 0, 0
        for L, n in zip(_lengths(case), _counts(case)):
            kept = min(L, WINDOW - 1) if case["window"] else L
            tokens += kept
            pairs += n * (kept + (n + 1) / 2)
        rows = sum(_counts(case))
        return dict(bytes=tokens * 2 * KV_HEADS * DIM * element + rows * DIM * 2 * (2 * HEADS + 2 * KV_HEADS),
                    flops=4 * DIM * HEADS * pairs)
    if op == "verify":  # the row that the next token comes from, and the draft's where one was rejected
        rows = 2 if case["dists"] else 1
        return dict(bytes=case["B"] * case["V"] * 4 * rows, flops=case["B"] * case["V"] * 3)
    if op == "rope":
        values = case["T"] * (HEADS + KV_HEADS) * DIM
        return dict(bytes=4 * values, flops=8 * values)
    half = case["N"] / 2 if case["B"] > 1 else max(1, case["N"] - 1)
    values = case["layers"] * case["B"] * half * 2 * KV_HEADS * DIM
    return dict(bytes=values * (4 if case["kv"] == "bf16" else 3), flops=values)


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    return None  # whole numbers


def _value64(code, scale):
    """fp64 [..., 128] of one KV head's cache values."""
    if scale is None:
        return code.to(torch.float64)
    e, m = ((code >> 3) & 15).to(torch.float64), (code & 7).to(torch.float64)
    size = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))
    return torch.where(code >= 128, -size, size) * float(torch.tensor(scale, dtype=torch.float32))


def _quantised64(x, scale):
    """What an E4M3 cache holds for the bf16 values x, as fp64."""
    if scale is None:
        return x.to(torch.float64)
    f = float(torch.tensor(scale, dtype=torch.float32))
    y = (x.to(torch.float64) / f).float().double()  # the quotient is a float32
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0) * f  # torch.round: half to even


def _exact_attend(case, s):
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    for b in range(case["B"]):
        L, n, parents = s["lens"][b], s["counts"][b], s["parents"][b]
        first = max(0, L - (WINDOW - 1)) if case["window"] else 0
        p = torch.arange(first, L, device="cuda")
        if case["layout"] == "paged":
            at = s["table"][b].long()[p // PAGE] * PAGE + p % PAGE
            flat = [x.view(-1, KV_HEADS, DIM) for x in (s["k"], s["v"])]
        else:
            at = p % WINDOW if case["layout"] == "ring" else p
            flat = [x[b] for x in (s["k"], s["v"])]
        hide = torch.ones((n, L - first + n), dtype=torch.bool, device="cuda")
        for i in range(n):
            line, j = [], i
            while j >= 0:
                line.append(j)
                j = parents[j]
            begin = max(0, L + len(line) - 1 - (WINDOW - 1)) if case["window"] else 0
            hide[i, max(0, begin - first):L - first] = False
            hide[i, [L - first + j for j in line]] = False
        for g in range(KV_HEADS):
            ks, vs = (s[x] and s[x][g] for x in ("k_scale", "v_scale"))
            k = torch.cat([_value64(flat[0][at, g], ks), _quantised64(s["k_draft"][b, :n, g], ks)])
            v = torch.cat([_value64(flat[1][at, g], vs), _quantised64(s["v_draft"][b, :n, g], vs)])
            for h in range(g * GROUP, (g + 1) * GROUP):
                a = s["q"][b, :n, h].to(torch.float64) @ k.T / DIM ** 0.5
                a[hide] = -math.inf
                sink = s["sinks"][h].to(torch.float64)
                norm = torch.logaddexp(torch.logsumexp(a, -1), sink)
                out[b, :n, h] = torch.exp(a - norm[:, None]) @ v
    return out


def _exact_rope(case, s):
    dim, factor = case["dim"], case["factor"]
    pairs = dim // 2
    freq, gain = [], 1.0
    for i in range(pairs):
        f = math.exp(-math.log(10000.0) * 2 * i / dim)
        if case["scaling"] == "linear":
            f /= factor
        elif case["scaling"] == "yarn":
            r = 8192 * f / (2 * math.pi)
            gamma = min(1.0, max(0.0, (r - 1) / 31))
            f = (1 - gamma) * f / factor + gamma * f
            gain = 0.1 * math.log(factor) + 1
        freq.append(f)
    turn = torch.polar(torch.full((case["T"], pairs), gain, dtype=torch.float64, device="cuda"),
                       s["pos"].to(torch.float64)[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))[:, None]
    outs = []
    for x, w in ((s["q_raw"], s["w_q"]), (s["k_raw"], s["w_k"])):
        x = x.to(torch.float64)
        y = w.to(torch.float64) * x / (x.square().sum(-1, keepdim=True) / DIM + 1e-6).sqrt()
        i = torch.arange(pairs, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y)
    return outs[0], outs[1]


def _exact_append(case, s):
    outs = []
    for name in ("k", "v"):
        scale, draft = s[name + "_scale"], s[name + "_draft"]
        x = s[name].to(torch.float64) if scale is None else _value64(s[name], 1.0)
        lens, path, n, table = s["lens"], s["path"].tolist(), s["n_accepted"].tolist(), s["table"].tolist()
        for b in range(case["B"]):
            for j in range(n[b]):
                p = lens[b] + j
                for g in range(KV_HEADS):
                    value = _quantised64(draft[:, b, path[b][j], g], scale and scale[g])
                    if scale is not None:
                        value = value / float(torch.tensor(scale[g], dtype=torch.float32))
                    x[:, table[b][p // PAGE], p % PAGE, g] = value
        outs.append(x)
    return outs[0], outs[1]
