"""One speculative decode step on the library's calls: the drafted tokens of a
batch stand as a tree on each request's committed context; every layer norms
and rotates them at their positions and attends the cache and the tree
(attend_layer), and once the target's probabilities are known the accepted
path is found and written to every layer's cache (verify_and_append).

From the first layer to the append nothing waits for the GPU: the accepted
counts stay on the device.  Lengths and node counts are host values that go into
the launches, so the next step has to read n_accepted, and a captured step holds
for the lengths that it was captured with.  A loop that keeps the drafted k and v
of its layers in buffers of its own (attend_layer's k) builds the layers' array,
flint.path_layers, once.

This module only marshals: the compute steps run in the CUDA library."""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch

from . import flint


class DraftTree:
    """The drafted tokens of B requests: parents[b][i] in [-1, i) for the nodes
    of request b (-1: the node continues the context).  Requests may hold
    different numbers of nodes; N is the largest."""

    def __init__(self, parents: Sequence[Sequence[int]], device=None):
        self.n_draft: List[int] = [len(p) for p in parents]
        self.N = max(self.n_draft, default=0)
        if not 1 <= self.N <= flint.MAX_TREE:
            raise ValueError(f"a tree holds 1 to {flint.MAX_TREE} nodes, not {self.N}")
        depth = [[0] * self.N for _ in parents]
        full = [[-1] * self.N for _ in parents]
        for b, row in enumerate(parents):
            for i, p in enumerate(row):
                if not -1 <= p < i:
                    raise ValueError(f"request {b}: the parent of node {i} must be -1 or an earlier node, not {p}")
                full[b][i] = p
                depth[b][i] = 0 if p < 0 else depth[b][p] + 1
        device = device or "cuda"
        self.parent = torch.tensor(full, dtype=torch.int32, device=device)
        self.depth = torch.tensor(depth, dtype=torch.int32, device=device)

    def positions(self, seq_lens: Sequence[int]) -> torch.Tensor:
        """int32 [B, N]: node i of request b stands at seq_lens[b] + its depth."""
        lens = torch.tensor(list(seq_lens), dtype=torch.int32, device=self.depth.device)
        return self.depth + lens[:, None]


def attend_layer(tree: DraftTree, pos: torch.Tensor, q_raw: torch.Tensor, k_raw: torch.Tensor, v: torch.Tensor,
                 w_q, w_k, rope: Optional[flint.Rope], cache: flint.KVCache, seq_lens: Sequence[int], sinks, window: int,
                 ws: torch.Tensor, eps: float = 1e-6, dev_err=None, k: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One layer of the step: q_raw [B, N, 32, 128], k_raw and v [B, N, 4, 128] in
    bf16 (q_raw and k_raw may be slices of a fused projection's rows).  Returns
    (out bf16 [B, N, 32, 128], the drafted k after norm and rotation bf16
    [B, N, 4, 128]), in the caller's dense buffers where these are given.  Rows of
    out behind a request's nodes are 0, in a given buffer as they were."""
    B, N = pos.shape
    q = torch.empty((B, N, flint.NUM_Q_HEADS, flint.HEAD_DIM), dtype=torch.bfloat16, device=pos.device)
    if k is None:
        k = torch.empty((B, N, flint.NUM_KV_HEADS, flint.HEAD_DIM), dtype=torch.bfloat16, device=pos.device)
    elif k.shape != (B, N, flint.NUM_KV_HEADS, flint.HEAD_DIM) or not k.is_contiguous():
        raise ValueError(f"k must be a dense tensor [{B}, {N}, {flint.NUM_KV_HEADS}, {flint.HEAD_DIM}]")
    flint.flint_qk_norm_rope_at(q_raw.flatten(0, 1), k_raw.flatten(0, 1), w_q, w_k, pos.reshape(-1), rope, eps,
                                q_out=q.view(B * N, flint.NUM_Q_HEADS, flint.HEAD_DIM),
                                k_out=k.view(B * N, flint.NUM_KV_HEADS, flint.HEAD_DIM))
    if out is None:
        out = torch.zeros_like(q)
    flint.flint_attn_tree(q, k, v, tree.parent, cache, seq_lens, tree.n_draft, sinks, window, out, ws, dev_err=dev_err)
    return out, k


def verify_and_append(tree: DraftTree, target, draft, tokens, u_accept, u_sample, layers, seq_lens: Sequence[int],
                      dev_err=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The end of the step: find the accepted path of every request and append its
    k and v to every layer's cache at positions seq_lens[b] ..; layers as for
    flint.flint_kv_append_path.  Returns (path, n_accepted, next_token) on the
    device: request b then holds seq_lens[b] + n_accepted[b] committed tokens,
    and next_token[b] follows them."""
    B, N = tokens.shape
    path = torch.empty((B, N), dtype=torch.int32, device=tokens.device)
    n_accepted = torch.empty((B,), dtype=torch.int32, device=tokens.device)
    next_token = torch.empty((B,), dtype=torch.int32, device=tokens.device)
    flint.flint_verify_tree(target, draft, tokens, tree.parent, tree.n_draft, u_accept, u_sample, path, n_accepted,
                            next_token, dev_err=dev_err)
    flint.flint_kv_append_path(layers, path, n_accepted, seq_lens, dev_err=dev_err)
    return path, n_accepted, next_token
