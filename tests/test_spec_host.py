"""Host-side checks of the speculative-decode calls that need no GPU: argument
validation before any CUDA call, and the draft tree's positions."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_decode_flash_b200 import flint, speculative

from spec_helpers import verify_reference

E, U = flint.FLINT_ERR_INVALID_ARG, flint.FLINT_ERR_UNSUPPORTED
P = ctypes.c_void_p(0x10000)


def _cache(layout=flint.CONTIGUOUS, capacity=4096):
    c = flint.KVCache()
    c.k, c.v, c.layout, c.capacity = 0x10000, 0x20000, layout, capacity
    return c


def _i32(*v):
    return (ctypes.c_int32 * len(v))(*v)


def _tree(cache=None, N=4, lens=(100,), n=(4,), window=0, q=P, out=P, ws=1 << 30, num_ctas=148, B=None):
    return flint.load_library().flint_attn_tree(q, P, P, P, N, ctypes.byref(cache or _cache()), _i32(*lens), _i32(*n),
                                                len(lens) if B is None else B, P, window, out, P, ws, num_ctas, None, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(N=0), E), (dict(N=65), E), (dict(B=0), E), (dict(lens=(5,) * 65, n=(1,) * 65), E),
    (dict(lens=(-1,)), E), (dict(lens=(4097,)), E), (dict(lens=(300000,)), E), (dict(n=(5,)), E), (dict(n=(-1,)), E),
    (dict(window=100), U), (dict(q=None), E), (dict(out=ctypes.c_void_p(0x10008)), E), (dict(num_ctas=297), E),
    (dict(num_ctas=-1), E), (dict(ws=4 * 148 * 66560 - 1), flint.FLINT_ERR_WORKSPACE),
])
def test_tree_attention_refuses(kwargs, status):
    assert _tree(**kwargs) == status
    assert flint.flint_last_error() != ""


def test_tree_attention_refuses_caches():
    assert _tree(_cache(flint.RING, 512), window=513) == U
    assert _tree(_cache(flint.RING, 513), window=0) == U
    paged = _cache(flint.PAGED, 0)
    assert _tree(paged) == E
    paged.block_table, paged.block_size, paged.max_blocks_per_req, paged.num_blocks = 0x70000, 64, 4, 8
    assert _tree(paged, lens=(257,)) == E
    paged.block_size = 32
    assert _tree(paged) == U
    bad = _cache()
    bad.dtype = flint.KV_FP8_E4M3  # no scales
    assert _tree(bad) == E


def test_tree_workspace_bytes():
    assert flint.flint_tree_workspace_bytes(148) == 4 * 148 * 66560
    assert flint.flint_tree_workspace_bytes(1) == flint.flint_tree_workspace_bytes(7) == 16 * 66560
    assert flint.flint_tree_workspace_bytes(-1) == 0 and flint.flint_tree_workspace_bytes(297) == 0


def test_verify_refuses():
    lib = flint.load_library()

    def call(B=1, N=2, V=10, n=(2,), ts=0, ds=0, target=P, path=P):
        return lib.flint_verify_tree(target, ts, P, ds, P, P, _i32(*n), B, N, V, P, P, path, P, P, None, None)
    for kwargs in (dict(B=0), dict(B=65, n=(1,) * 65), dict(N=0), dict(N=65), dict(V=0), dict(V=(1 << 24) + 1), dict(n=(3,)),
                   dict(n=(-1,)), dict(ts=9), dict(ds=9), dict(target=None), dict(path=None), dict(path=ctypes.c_void_p(0x10002))):
        assert call(**kwargs) == E, kwargs


def test_rope_refuses():
    lib = flint.load_library()

    def call(rope=None, q=P, k=P, wq=P, wk=P, pos=P, T=4, qs=0, ks=0, qo=P, ko=ctypes.c_void_p(0x90000), eps=1e-6):
        return lib.flint_qk_norm_rope_at(q, qs, k, ks, wq, wk, pos, T, eps, ctypes.byref(rope) if rope else None, qo, ko, None)
    for kwargs in (dict(qo=None, ko=None), dict(q=None), dict(k=None), dict(wq=None), dict(wk=None), dict(pos=None), dict(T=-1),
                   dict(T=262145), dict(qs=4095), dict(qs=4100), dict(ks=504), dict(qs=5120, qo=P), dict(eps=-1.0),
                   dict(q=ctypes.c_void_p(0x10008))):
        assert call(**kwargs) == E, kwargs
    for kwargs in (dict(rotary_dim=130), dict(rotary_dim=-2), dict(rotary_dim=7), dict(theta=0.0), dict(theta=float("inf")),
                   dict(factor=0.5), dict(attn_factor=0.0), dict(attn_factor=float("nan")),
                   dict(scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=1.0),
                   dict(scaling="yarn", factor=2.0, original_context=0.0)):
        assert call(flint.rope(**kwargs)) == E, kwargs
    with pytest.raises(flint.FlintError):
        flint.rope(scaling="cubic")
    r = flint.rope()
    r.layout = 2
    assert call(r) == E
    r = flint.rope()
    r.scaling = 9
    assert call(r) == E


def test_append_path_refuses():
    lib = flint.load_library()
    layer = (flint.PathLayer * 1)()
    layer[0].k, layer[0].v, layer[0].cache = 0x10000, 0x20000, _cache()

    def call(n_layers=1, N=2, lens=(0,), B=1, arr=layer, path=P):
        return lib.flint_kv_append_path(arr, n_layers, path, P, N, _i32(*lens), B, None, None)
    for kwargs in (dict(n_layers=0), dict(n_layers=50), dict(N=0), dict(N=65), dict(B=0), dict(B=65, lens=(0,) * 65),
                   dict(lens=(-1,)), dict(lens=(262145,)), dict(path=None), dict(arr=(flint.PathLayer * 1)())):
        assert call(**kwargs) == E, kwargs


def test_draft_tree():
    t = speculative.DraftTree([[-1, 0, 0, 2], [], [-1]], device="cpu")
    assert t.N == 4 and t.n_draft == [4, 0, 1]
    assert t.positions([10, 20, 30]).tolist() == [[10, 11, 11, 12], [20] * 4, [30] * 4]
    for bad in ([[0]], [[-1, 1]], [[-2]], [[]], [[-1] * 65]):
        with pytest.raises(ValueError):
            speculative.DraftTree(bad, device="cpu")


@pytest.mark.parametrize("fixed", [False, True])
def test_the_verified_token_follows_the_target(fixed):
    """The definition's point, on its reference: over the draft's and the test's
    random numbers the first token of the result is distributed as the target's
    row.  Two candidates, five tokens; 20,000 draws give a standard error of at
    most sqrt(0.25 / 20000) = 0.0036 per token, and 5 of them are allowed."""
    rng = np.random.default_rng(3)
    p, q = np.array([0.5, 0.2, 0.15, 0.1, 0.05]), np.array([0.1, 0.4, 0.2, 0.2, 0.1])
    target, draft = np.stack([p, p, p]), np.stack([q, q])
    seen = np.zeros(5)
    for _ in range(20000):
        tokens = [3, 0] if fixed else rng.choice(5, size=2, p=q).tolist()
        path, token = verify_reference(target, None if fixed else draft, tokens, [-1, -1], rng.random(2), rng.random())
        seen[tokens[path[0]] if path else token] += 1
    assert np.abs(seen / 20000 - p).max() < 5 * 0.0036
