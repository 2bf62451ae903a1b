"""References in float64 for the speculative-decode calls, written from their
definitions: plain loops over requests and nodes."""
import math
import random

import numpy as np
import torch

from long_context_decode_flash_b200 import flint

W = 513


def lines(parents):
    """Per node: the node and its ancestors."""
    out = []
    for i, p in enumerate(parents):
        out.append(([] if p < 0 else out[p]) + [i])
    return out


def random_tree(n, rng, kind):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] * n
    return [rng.randint(-1, i - 1) for i in range(n)]


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float64)


def quantise(x, scale):
    """uint8 codes of bf16 [..., 4, 128] by per-KV-head scales."""
    y = x.to(torch.float32) / torch.tensor(scale, dtype=torch.float32).view(4, 1)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


class TreeCase:
    """Seeded inputs of one flint_attn_tree call on the CPU, in any layout and
    type.  Everything that must not be read as data holds NaN."""

    def __init__(self, layout, fp8, window, lens, n_draft, N, kind="tree", seed=0, stride_extra=0, value_scale=1.0):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.layout, self.fp8, self.window, self.lens, self.n_draft, self.N, self.B = layout, fp8, window, lens, n_draft, N, B
        rnd = lambda *s: torch.randn(s, generator=g).mul_(value_scale).to(torch.bfloat16)  # noqa: E731
        nan = float("nan")
        self.k_scale = [0.01 * (1 + 0.3 * h) for h in range(4)] if fp8 else None
        self.v_scale = [0.02 * (1 + 0.2 * h) for h in range(4)] if fp8 else None
        self.parents = [random_tree(n, rng, kind) for n in n_draft]
        self.q, self.kd, self.vd = rnd(B, N, 32, 128), rnd(B, N, 4, 128), rnd(B, N, 4, 128)
        self.sinks = torch.randn(32, generator=g)
        self.parent = torch.full((B, N), 12345, dtype=torch.int32)
        for b, n in enumerate(n_draft):
            self.parent[b, :n] = torch.tensor(self.parents[b], dtype=torch.int32)
            for t in (self.q, self.kd, self.vd):
                t[b, n:] = nan
        # the attended history per request, and where it lies
        hist = []
        for L in lens:
            first = max(0, L - W + 1) if window else 0
            k, v = rnd(L - first, 4, 128), rnd(L - first, 4, 128)
            if fp8:
                k, v = quantise(k, self.k_scale), quantise(v, self.v_scale)
            hist.append((first, k, v))
        self.table = None
        if layout == flint.PAGED:
            used = [max(1, -(-L // 64)) for L in lens]
            pool = sum(used) + 3
            order = list(range(pool))
            rng.shuffle(order)
            self.table = torch.zeros((B, max(used) + 1), dtype=torch.int32)
            shape, at = (pool, 64, 4, 128), 0
            for b, n in enumerate(used):
                self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
                at += n
            self.capacity, self.num_blocks = 0, pool
        else:
            self.capacity = W if layout == flint.RING else max(1, max(lens) + 5)
            shape, self.num_blocks = (B, self.capacity, 4, 128), 0
        fill = lambda: torch.full(shape, 0x7F, dtype=torch.uint8) if fp8 else torch.full(shape, nan, dtype=torch.bfloat16)  # noqa: E731
        self.k, self.v = fill(), fill()
        for b, (first, k, v) in enumerate(hist):
            for j in range(k.shape[0]):
                p = first + j
                where = ((int(self.table[b, p // 64]), p % 64) if layout == flint.PAGED
                         else (b, p % W) if layout == flint.RING else (b, p))
                self.k[where], self.v[where] = k[j], v[j]
        self.stride_extra = stride_extra if layout != flint.PAGED else 0
        if self.stride_extra:  # requests further apart than their slots
            flat = lambda t: torch.cat([t.reshape(B, -1), t.new_full((B, self.stride_extra), 0x7F if fp8 else nan)], 1)  # noqa: E731
            self.k, self.v = flat(self.k), flat(self.v)
        self.hist = hist

    def values(self, x, scale):
        return e4m3(x) * torch.tensor(scale, dtype=torch.float32).double().view(4, 1) if self.fp8 else x.double()

    def reference(self):
        """(out, bound) in float64.  bound: the kernel's arithmetic is fp32 (scores
        of 128 products, ~1e-5 relative in e^s), the probabilities are rounded to
        fp16 (2^-11 relative) and the result to bf16 (2^-8): per value
        2^-8 |out| + 2^-10 sum_j p_j |v_j|, with the second-order terms.  Small
        probabilities are off by an absolute amount: the kernel holds
        2^(x - m + 7) in fp16, whose subnormals lie 2^-24 apart, so each is off by
        at most 2^-25; the row's largest is at least 2^7 (the reference m is at most
        the maximum), and so is their sum, which divides: 2^-32 |v_j| per key.
        (float32's own smallest numbers are far below that.)"""
        out = torch.zeros(self.B, self.N, 32, 128, dtype=torch.float64)
        spread, lost = torch.zeros_like(out), torch.zeros_like(out)
        for b, L in enumerate(self.lens):
            n = self.n_draft[b]
            if n == 0:
                continue
            first, hk, hv = self.hist[b]
            kd, vd = self.kd[b, :n], self.vd[b, :n]
            if self.fp8:
                kd, vd = quantise(kd, self.k_scale), quantise(vd, self.v_scale)
            k = torch.cat([self.values(hk, self.k_scale), self.values(kd, self.k_scale)])
            v = torch.cat([self.values(hv, self.v_scale), self.values(vd, self.v_scale)])
            for i, line in enumerate(lines(self.parents[b])):
                lo = max(0, L + len(line) - 1 - W + 1) if self.window else 0
                keys = list(range(lo - first, L - first)) + [L - first + j for j in line]
                kk, vv = k[keys], v[keys]
                for h in range(32):
                    s = kk[:, h // 8] @ self.q[b, i, h].double() / math.sqrt(128)
                    sink = float(self.sinks[h])
                    top = max(float(s.max()), sink)
                    e = torch.exp(s - top)
                    p = e / (e.sum() + math.exp(sink - top))
                    out[b, i, h] = p @ vv[:, h // 8]
                    spread[b, i, h] = p @ vv[:, h // 8].abs()
                    lost[b, i, h] = vv[:, h // 8].abs().sum(0)
        return out, out.abs() * 2.0 ** -8 * 1.01 + spread * 2.0 ** -10 * 1.01 + lost * 2.0 ** -32

    def device_cache(self):
        self.kdev, self.vdev = self.k.cuda(), self.v.cuda()
        table = None if self.table is None else self.table.cuda()
        stride = self.capacity * 512 + self.stride_extra if self.stride_extra else 0
        return flint.kv_cache(self.kdev, self.vdev, self.layout, capacity=self.capacity, req_stride=stride,
                              block_table=table, num_blocks=self.num_blocks, k_scale=self.k_scale, v_scale=self.v_scale)

    def run(self, num_ctas=0, ws=None, out=None):
        err = torch.zeros(8, dtype=torch.int32, device="cuda")
        if out is None:
            out = torch.full((self.B, self.N, 32, 128), 77.0, dtype=torch.bfloat16, device="cuda")
        ws = flint.tree_workspace(num_ctas) if ws is None else ws
        flint.flint_attn_tree(self.q.cuda(), self.kd.cuda(), self.vd.cuda(), self.parent.cuda(), self.device_cache(),
                              self.lens, self.n_draft, self.sinks.cuda(), W if self.window else 0, out, ws,
                              num_ctas=num_ctas, dev_err=err)
        torch.cuda.synchronize()
        assert int(err[0]) == 0, err.tolist()
        return out.cpu()

    def check(self, got):
        want, bound = self.reference()
        for b, n in enumerate(self.n_draft):
            g = got[b, :n].double()
            assert torch.isfinite(g).all(), f"request {b}: non-finite output"
            over = (g - want[b, :n]).abs() - bound[b, :n]
            assert n == 0 or over.max() <= 0, f"request {b}: {float(over.max()):.3e} above the bound"
            assert (got[b, n:] == 77.0).all(), f"request {b}: rows behind its nodes were written"


def verify_reference(target, draft, tokens, parents, u_accept, u_sample):
    """One request of flint_verify_tree, literally, in float64 with whole rows:
    target [N + 1, V], draft [N, V] or None; (path, next_token)."""
    cur, path = -1, []
    w, Z = target[0].astype(np.float64), 1.0
    for i, x in enumerate(tokens):
        if parents[i] != cur or not 0 <= x < w.size:
            continue
        q = draft[cur + 1].astype(np.float64) if draft is not None else np.where(np.arange(w.size) == x, 1.0, 0.0)
        if float(u_accept[i]) * q[x] * Z < w[x]:
            cur = i
            path.append(i)
            w, Z = target[i + 1].astype(np.float64), 1.0
            continue
        if draft is not None:
            left = np.maximum(w - Z * q, 0.0)
            total = left.sum()
        else:
            left = np.where(q > 0, 0.0, w)
            total = Z - w[x]
        if total > 0:
            w, Z = left, total
    c = np.cumsum(w)
    over = np.nonzero(c > float(u_sample) * c[-1])[0]
    held = np.nonzero(w > 0)[0]
    return path, int(over[0]) if over.size else int(held[-1]) if held.size else 0
