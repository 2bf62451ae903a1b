"""ctypes binding of libflint.so (include/flint.h), argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
device pointers (``tensor.data_ptr()``) and the current CUDA stream.  There is
no fallback: if libflint.so is missing or a call fails, FlintError is raised.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from array import array
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflint.so")

FLINT_OK = 0
FLINT_ERR_INVALID_ARG = 1
FLINT_ERR_UNSUPPORTED = 2
FLINT_ERR_WORKSPACE = 3
FLINT_ERR_CUDA = 4
FLINT_ERR_TIMEOUT = 5

CONTIGUOUS, RING, PAGED = 0, 1, 2
KV_BF16, KV_FP8_E4M3 = 0, 1
NUM_Q_HEADS, NUM_KV_HEADS, HEAD_DIM = 32, 4, 128
WINDOW, BLOCK_SIZE, MAX_CONTEXT = 513, 64, 262144
MAX_BATCH, MAX_LAYERS = 64, 49

EXPORTED = (
    "flint_status_string", "flint_last_error", "flint_kv_bytes", "flint_qk_norm_rope",
    "flint_kv_append", "flint_attn_workspace_bytes", "flint_attn_decode", "flint_attn_stack",
    "flint_attn_stack_noalloc", "flint_attn_layers_serial", "flint_plan_items", "flint_plan_split",
    "flint_prefill_qk_norm_rope", "flint_prefill_attn", "flint_attn_decode_partial",
    "flint_merge_partials", "flint_qk_norm_rope_at", "flint_tree_workspace_bytes", "flint_attn_tree",
    "flint_verify_tree", "flint_kv_append_path", "flint_plan_tree",
)
MAX_TREE = 64
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_UNSCALED, ROPE_LINEAR, ROPE_BY_PARTS = 0, 1, 2
CP_PARTIAL_FLOATS = 32 * 128 + 2 * 32


class FlintError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"flint status {status}: {detail}")
        self.status = status


class KVCache(ctypes.Structure):
    """flint_kv_cache.  Build with kv_cache(); it keeps its tensors alive."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layout", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("req_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("max_blocks_per_req", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float * 4),
                ("v_scale", ctypes.c_float * 4)]


class StackLayer(ctypes.Structure):
    """flint_layer."""
    _fields_ = [("q_raw", ctypes.c_void_p), ("k_raw", ctypes.c_void_p), ("v_raw", ctypes.c_void_p),
                ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p), ("sinks", ctypes.c_void_p),
                ("cache", KVCache), ("window", ctypes.c_int32), ("rope", ctypes.c_int32)]


class Rope(ctypes.Structure):
    """flint_rope.  Build with rope()."""
    _fields_ = [("theta", ctypes.c_double), ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("attn_factor", ctypes.c_double),
                ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class PathLayer(ctypes.Structure):
    """flint_path_layer."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("cache", KVCache)]


_lock = threading.Lock()
_lib = None


def open_library(path: str) -> ctypes.CDLL:
    """Load a build of the library from `path` with its signatures declared
    (load_library() does this for the package's libflint.so; tests use it for
    the test builds)."""
    if not os.path.exists(path):
        raise FlintError(FLINT_ERR_CUDA, f"{path} is not built "
                         "(python -m long_context_decode_flash_b200.build)")
    lib = ctypes.CDLL(path)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.flint_status_string.argtypes = [ctypes.c_int]
    lib.flint_status_string.restype = ctypes.c_char_p
    lib.flint_last_error.restype = ctypes.c_char_p
    lib.flint_kv_bytes.argtypes = [I64, I32, I32, I32, I32]
    lib.flint_kv_bytes.restype = ctypes.c_uint64
    lib.flint_qk_norm_rope.argtypes = [P, P, P, P, P, P, I32, ctypes.c_float, ctypes.c_double,
                                       I32, P, P, P, P, P]
    lib.flint_kv_append.argtypes = [P, P, P, I32, P, P, P]
    lib.flint_attn_workspace_bytes.argtypes = [I32, I32]
    lib.flint_attn_workspace_bytes.restype = ctypes.c_size_t
    lib.flint_attn_decode.argtypes = [P, I32, P, P, I32, P, I32, P, P, ctypes.c_size_t,
                                      I32, P, P]
    lib.flint_attn_stack.argtypes = [P, I32, I32, ctypes.c_float, ctypes.c_double, P, P,
                                     ctypes.c_size_t, I32, P, P]
    lib.flint_attn_layers_serial.argtypes = [P, I32, I32, ctypes.c_float, ctypes.c_double, P, P,
                                             ctypes.c_size_t, I32, P, P]
    lib.flint_attn_stack_noalloc.argtypes = [P, I32, I32, ctypes.c_float, ctypes.c_double,
                                             P, I32, P, P]
    lib.flint_prefill_qk_norm_rope.argtypes = [P, P, P, P, P, I32, ctypes.c_float,
                                               ctypes.c_double, I32, P, P, P, P, P, P]
    lib.flint_prefill_attn.argtypes = [P, P, P, I32, P, I32, P, P, P]
    lib.flint_attn_decode_partial.argtypes = [P, I32, P, P, I32, P, P, ctypes.c_size_t, I32, P, P]
    lib.flint_merge_partials.argtypes = [P, I32, I32, P, P, P]
    lib.flint_qk_norm_rope_at.argtypes = [P, I64, P, I64, P, P, P, I32, ctypes.c_float, P, P, P, P]
    lib.flint_tree_workspace_bytes.argtypes = [I32]
    lib.flint_tree_workspace_bytes.restype = ctypes.c_size_t
    lib.flint_attn_tree.argtypes = [P, P, P, P, I32, P, P, P, I32, P, I32, P, P, ctypes.c_size_t, I32, P, P]
    lib.flint_verify_tree.argtypes = [P, I64, P, I64, P, P, P, I32, I32, I32, P, P, P, P, P, P, P]
    lib.flint_kv_append_path.argtypes = [P, I32, P, P, I32, P, I32, P, P]
    lib.flint_plan_tree.argtypes = [P, P, I32, I32, I32, I32, I32, P, I32, P, P, I32]
    lib.flint_plan_tree.restype = I32
    lib.flint_plan_items.argtypes = [P, I32, I32, I32, P, P, P, P, I32]
    lib.flint_plan_items.restype = I32
    lib.flint_plan_split.argtypes = [P, I32, I32, I32, I32, P, P, P, P, P]
    lib.flint_plan_split.restype = I32
    for name in ("flint_qk_norm_rope", "flint_kv_append", "flint_attn_decode",
                 "flint_attn_stack", "flint_attn_stack_noalloc", "flint_attn_layers_serial",
                 "flint_prefill_qk_norm_rope", "flint_prefill_attn", "flint_attn_decode_partial",
                 "flint_merge_partials", "flint_qk_norm_rope_at", "flint_attn_tree", "flint_verify_tree",
                 "flint_kv_append_path"):
        getattr(lib, name).restype = ctypes.c_int
    # test builds only (libflint_hooks.so): leave one pipeline stage unarmed
    for name in ("flint_test_stall_decode", "flint_test_stall_prefill", "flint_test_stall_prefill_prep",
                 "flint_test_stall_tree"):
        if hasattr(lib, name):
            getattr(lib, name).argtypes = [ctypes.c_int, ctypes.c_int]
            getattr(lib, name).restype = ctypes.c_int
    if hasattr(lib, "flint_test_ex2"):  # the prefill softmax's two exponentials, side by side
        lib.flint_test_ex2.argtypes = [P, P, P, I32, P]
        lib.flint_test_ex2.restype = ctypes.c_int
    return lib


def load_library() -> ctypes.CDLL:
    global _lib
    with _lock:
        if _lib is None:
            _lib = open_library(LIB_PATH)
    return _lib


def _check(status: int) -> None:
    if status != FLINT_OK:
        lib = load_library()
        raise FlintError(status, lib.flint_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _i32_host(values: Sequence[int]):
    arr = (ctypes.c_int32 * len(values))(*[int(v) for v in values])
    return arr


def flint_status_string(status: int) -> str:
    return load_library().flint_status_string(int(status)).decode()


def flint_last_error() -> str:
    return load_library().flint_last_error().decode()


def flint_kv_bytes(ctx_len: int, n_full: int = 14, n_window: int = 35, window: int = WINDOW,
                   elem_bytes: int = 2) -> int:
    return int(load_library().flint_kv_bytes(ctx_len, n_full, n_window, window, elem_bytes))


def kv_cache(k: torch.Tensor, v: torch.Tensor, layout: int, capacity: int = 0,
             req_stride: int = 0, block_table: Optional[torch.Tensor] = None,
             num_blocks: int = 0, k_scale: Optional[Sequence[float]] = None,
             v_scale: Optional[Sequence[float]] = None) -> KVCache:
    """A flint_kv_cache over tensors k, v (CONTIGUOUS/RING: [B, cap, 4, 128]
    or [cap, 4, 128]; PAGED: [num_blocks, 64, 4, 128] with an int32 table):
    bf16 tensors, or uint8 tensors of E4M3 codes with k_scale and v_scale
    (4 floats each, one per KV head)."""
    c = KVCache()
    if k.dtype == torch.uint8:
        if k_scale is None or v_scale is None or len(k_scale) != 4 or len(v_scale) != 4:
            raise FlintError(FLINT_ERR_INVALID_ARG, "an E4M3 cache needs 4 k_scale and 4 v_scale values")
        c.dtype = KV_FP8_E4M3
        c.k_scale[:] = [float(x) for x in k_scale]
        c.v_scale[:] = [float(x) for x in v_scale]
    elif k.dtype != torch.bfloat16:
        raise FlintError(FLINT_ERR_INVALID_ARG, f"cache tensors must be bf16 or uint8, not {k.dtype}")
    c.k, c.v = k.data_ptr(), v.data_ptr()
    c.layout = int(layout)
    c.capacity = int(capacity)
    c.req_stride = int(req_stride)
    c.block_table = block_table.data_ptr() if block_table is not None else None
    c.max_blocks_per_req = int(block_table.shape[-1]) if block_table is not None else 0
    c.block_size = BLOCK_SIZE if layout == PAGED else 0
    c.num_blocks = int(num_blocks)
    c._keep = (k, v, block_table)  # keep the tensors alive with the struct
    return c


def flint_attn_workspace_bytes(n_problems: int, num_ctas: int = 0) -> int:
    return int(load_library().flint_attn_workspace_bytes(n_problems, num_ctas))


def workspace(n_problems: int, num_ctas: int = 0, device=None) -> torch.Tensor:
    """A zero-filled workspace of the required size (the library keeps it zeroed)."""
    n = flint_attn_workspace_bytes(n_problems, num_ctas)
    if n == 0:
        raise FlintError(FLINT_ERR_INVALID_ARG, "invalid workspace request")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def flint_qk_norm_rope(q_raw, k_raw, w_q, w_k, pos: Sequence[int], eps: float = 1e-6,
                       theta: float = 10000.0, apply_rope: bool = True, q_out=None, k_out=None,
                       v_raw=None, cache: Optional[KVCache] = None, dev_err=None, stream=None):
    B = len(pos)
    lib = load_library()
    _check(lib.flint_qk_norm_rope(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(w_q), _ptr(w_k),
                                  _i32_host(pos), B, eps, theta, int(bool(apply_rope)),
                                  _ptr(q_out), _ptr(k_out),
                                  ctypes.byref(cache) if cache is not None else None,
                                  _ptr(dev_err), _stream(stream)))
    return q_out, k_out


def flint_kv_append(k, v, pos: Sequence[int], cache: KVCache, dev_err=None, stream=None) -> None:
    lib = load_library()
    _check(lib.flint_kv_append(_ptr(k), _ptr(v), _i32_host(pos), len(pos), ctypes.byref(cache),
                               _ptr(dev_err), _stream(stream)))


def flint_prefill_qk_norm_rope(q_raw, k_raw, w_q, w_k, eps: float = 1e-6, theta: float = 10000.0,
                               apply_rope: bool = True, q_out=None, k_out=None, v_raw=None, v_out=None,
                               cache: Optional[KVCache] = None, dev_err=None, stream=None):
    """Norm (+RoPE) of the T tokens of one prompt at positions 0..T-1: q and k
    out in bf16, v out in fp16 (the attention's v operand), optional cache
    write (request 0 of `cache`)."""
    T = int(q_raw.shape[0])
    lib = load_library()
    _check(lib.flint_prefill_qk_norm_rope(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(w_q), _ptr(w_k),
                                          T, eps, theta, int(bool(apply_rope)), _ptr(q_out),
                                          _ptr(k_out), _ptr(v_out),
                                          ctypes.byref(cache) if cache is not None else None,
                                          _ptr(dev_err), _stream(stream)))
    return q_out, k_out, v_out


def flint_prefill_attn(q, k, v, sinks, window: int, out, dev_err=None, stream=None):
    """Causal attention (with sinks) of a T-token prompt over itself:
    q bf16 [T, 32, 128], k bf16 [T, 4, 128], v fp16 [T, 4, 128],
    out fp32 [T, 32, 128]."""
    lib = load_library()
    _check(lib.flint_prefill_attn(_ptr(q), _ptr(k), _ptr(v), int(q.shape[0]), _ptr(sinks), int(window),
                                  _ptr(out), _ptr(dev_err), _stream(stream)))
    return out


def flint_attn_decode(q, cache: KVCache, seq_lens: Sequence[int], sinks, window: int, out,
                      ws: torch.Tensor, num_ctas: int = 0, dev_err=None, stream=None):
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise FlintError(FLINT_ERR_INVALID_ARG, "q must be bf16 or fp32")
    lib = load_library()
    _check(lib.flint_attn_decode(_ptr(q), int(q.dtype == torch.float32), ctypes.byref(cache),
                                 _i32_host(seq_lens), len(seq_lens), _ptr(sinks), int(window),
                                 _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), int(num_ctas),
                                 _ptr(dev_err), _stream(stream)))
    return out


def flint_attn_decode_partial(q, cache: KVCache, seq_lens: Sequence[int], partials, ws: torch.Tensor,
                              num_ctas: int = 0, dev_err=None, stream=None):
    """This rank's unnormalised attention over tokens [0, seq_lens[b]) of its
    cache: partials fp32 [B, CP_PARTIAL_FLOATS] (O [32,128], m [32], l [32])."""
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise FlintError(FLINT_ERR_INVALID_ARG, "q must be bf16 or fp32")
    lib = load_library()
    _check(lib.flint_attn_decode_partial(_ptr(q), int(q.dtype == torch.float32), ctypes.byref(cache),
                                         _i32_host(seq_lens), len(seq_lens), _ptr(partials), _ptr(ws),
                                         ws.numel() * ws.element_size(), int(num_ctas), _ptr(dev_err),
                                         _stream(stream)))
    return partials


def flint_merge_partials(partials, sinks, out, stream=None):
    """Merge partials fp32 [n_parts, B, CP_PARTIAL_FLOATS] with the sinks into
    out fp32 [B, 32, 128]."""
    n, B = int(partials.shape[0]), int(partials.shape[1])
    lib = load_library()
    _check(lib.flint_merge_partials(_ptr(partials), n, B, _ptr(sinks), _ptr(out), _stream(stream)))
    return out


def stack_layers(layers) -> ctypes.Array:
    """A flint_layer array from objects with q_raw, k_raw, v_raw, w_q, w_k, sinks
    (device tensors), cache (KVCache), window and rope."""
    arr = (StackLayer * len(layers))()
    keep = []
    for i, ly in enumerate(layers):
        s = arr[i]
        s.q_raw, s.k_raw, s.v_raw = ly.q_raw.data_ptr(), ly.k_raw.data_ptr(), ly.v_raw.data_ptr()
        s.w_q, s.w_k, s.sinks = ly.w_q.data_ptr(), ly.w_k.data_ptr(), ly.sinks.data_ptr()
        s.cache = ly.cache
        s.window = int(ly.window)
        s.rope = int(bool(ly.rope))
        keep.append(ly)
    arr._keep = keep
    return arr


def flint_attn_stack(layers, pos: int, out, ws: torch.Tensor, eps: float = 1e-6,
                     theta: float = 10000.0, num_ctas: int = 0, dev_err=None, stream=None):
    """layers: a ctypes array from stack_layers() (or a list, converted here)."""
    arr = layers if isinstance(layers, ctypes.Array) else stack_layers(layers)
    lib = load_library()
    _check(lib.flint_attn_stack(arr, len(arr), int(pos), eps, theta, _ptr(out), _ptr(ws),
                                ws.numel() * ws.element_size(), int(num_ctas), _ptr(dev_err),
                                _stream(stream)))
    return out


def flint_attn_layers_serial(layers, pos: int, out, ws: torch.Tensor, eps: float = 1e-6,
                             theta: float = 10000.0, num_ctas: int = 0, dev_err=None, stream=None):
    """flint_attn_stack as one dependent launch per layer (programmatic
    dependent launch); layers: a ctypes array from stack_layers() or a list."""
    arr = layers if isinstance(layers, ctypes.Array) else stack_layers(layers)
    lib = load_library()
    _check(lib.flint_attn_layers_serial(arr, len(arr), int(pos), eps, theta, _ptr(out), _ptr(ws),
                                        ws.numel() * ws.element_size(), int(num_ctas), _ptr(dev_err),
                                        _stream(stream)))
    return out


def flint_attn_stack_noalloc(layers, pos: int, out, eps: float = 1e-6, theta: float = 10000.0,
                             num_ctas: int = 0, dev_err=None, stream=None):
    """flint_attn_stack on the library's own fixed device scratch (no workspace)."""
    arr = layers if isinstance(layers, ctypes.Array) else stack_layers(layers)
    lib = load_library()
    _check(lib.flint_attn_stack_noalloc(arr, len(arr), int(pos), eps, theta, _ptr(out),
                                        int(num_ctas), _ptr(dev_err), _stream(stream)))
    return out


# ---- speculative decode ------------------------------------------------------


def _need(cond: bool, what: str) -> None:
    if not cond:
        raise FlintError(FLINT_ERR_INVALID_ARG, what)


def _dense(t, dtype, shape, name: str, dev: int) -> int:
    """The address of a dense tensor of this type and shape on the CUDA device dev."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise FlintError(FLINT_ERR_INVALID_ARG, f"{name} must be a dense {dtype} tensor {list(shape)}, "
                         f"not {t.dtype} {list(t.shape)}")
    if t.get_device() != dev:
        raise FlintError(FLINT_ERR_INVALID_ARG, f"{name} is on {t.device}, not on the current CUDA device")
    return t.data_ptr()


def _error_word(dev_err, dev: int) -> Optional[int]:
    """The address of dev_err (int32, at least one value), or None."""
    if dev_err is None:
        return None
    _need(dev_err.dtype is torch.int32 and dev_err.numel() > 0, "dev_err must be an int32 tensor")
    return _dense(dev_err, torch.int32, dev_err.shape, "dev_err", dev)


def _stream_of(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _host_i32(values: Sequence[int], n: int, name: str) -> array:
    """Host int32 values; .buffer_info()[0] is their address."""
    _need(len(values) == n, f"{name} must hold {n} values")
    return array("i", values)


def rope(rotary_dim: int = HEAD_DIM, interleaved: bool = False, theta: float = 10000.0, scaling: str = "none",
         factor: float = 1.0, original_context: float = 8192.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
         attn_factor: Optional[float] = None) -> Rope:
    """A flint_rope: the first `rotary_dim` dims turn, in pairs (i, i + rotary_dim/2)
    or (2i, 2i + 1) (interleaved); scaling "none", "linear" (every frequency over
    `factor`) or "yarn" (by parts).  attn_factor multiplies cos and sin; by
    default 1, with "yarn" 0.1 ln(factor) + 1."""
    kinds = {"none": ROPE_UNSCALED, "linear": ROPE_LINEAR, "yarn": ROPE_BY_PARTS}
    _need(scaling in kinds, f"unknown rotary scaling {scaling!r}")
    if attn_factor is None:
        attn_factor = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor >= 1.0 else 1.0
    return Rope(theta, factor, original_context, beta_fast, beta_slow, attn_factor, int(rotary_dim),
                ROPE_INTERLEAVED if interleaved else ROPE_HALF, kinds[scaling], 0)


def _token_rows(t, heads: int, T: int, name: str, dev: int) -> int:
    """The token stride (elements) of bf16 [T, heads, 128] with dense heads."""
    if t.dtype is not torch.bfloat16 or t.shape != (T, heads, HEAD_DIM) or t.get_device() != dev:
        raise FlintError(FLINT_ERR_INVALID_ARG, f"{name} must be bf16 [{T}, {heads}, 128] on the current CUDA device")
    st = t.stride()
    _need(T == 0 or st[2] == 1 and st[1] == HEAD_DIM and (T == 1 or st[0] >= heads * HEAD_DIM),
          f"{name}: the heads of a token must be dense, and the tokens apart")
    return st[0] if T > 1 else 0


def flint_qk_norm_rope_at(q_raw, k_raw, w_q, w_k, pos, rope: Optional[Rope] = None, eps: float = 1e-6, q_out=None,
                          k_out=None, stream=None):
    """RMSNorm (unless w_q and w_k are None) and rotary positions of T tokens at
    the positions pos (device int32 [T]): q_raw [T, 32, 128] and k_raw
    [T, 4, 128] in bf16, dense or slices of wider token rows, to the dense
    q_out and k_out.  An input without its output is not read, and may be None."""
    T, dev, bf16 = int(pos.shape[0]), torch.cuda.current_device(), torch.bfloat16
    at_pos = _dense(pos, torch.int32, (T,), "pos", dev)
    qi = ki = qo = ko = wq = wk = None
    qs = ks = 0
    if q_out is not None:
        qs, qi = _token_rows(q_raw, NUM_Q_HEADS, T, "q_raw", dev), q_raw.data_ptr()
        qo = _dense(q_out, bf16, (T, NUM_Q_HEADS, HEAD_DIM), "q_out", dev)
    if k_out is not None:
        ks, ki = _token_rows(k_raw, NUM_KV_HEADS, T, "k_raw", dev), k_raw.data_ptr()
        ko = _dense(k_out, bf16, (T, NUM_KV_HEADS, HEAD_DIM), "k_out", dev)
    if w_q is not None:
        wq = _dense(w_q, bf16, (HEAD_DIM,), "w_q", dev)
    if w_k is not None:
        wk = _dense(w_k, bf16, (HEAD_DIM,), "w_k", dev)
    _check(load_library().flint_qk_norm_rope_at(qi, qs, ki, ks, wq, wk, at_pos, T, eps, None if rope is None else ctypes.byref(rope),
                                                qo, ko, _stream_of(stream, dev)))
    return q_out, k_out


def flint_tree_workspace_bytes(num_ctas: int = 0) -> int:
    return int(load_library().flint_tree_workspace_bytes(num_ctas))


def tree_workspace(num_ctas: int = 0, device=None) -> torch.Tensor:
    """A workspace for flint_attn_tree (uninitialised: it needs no zeroing)."""
    n = flint_tree_workspace_bytes(num_ctas)
    _need(n > 0, "invalid workspace request")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def flint_attn_tree(q, k_draft, v_draft, parent, cache: KVCache, seq_lens: Sequence[int], n_draft: Sequence[int], sinks,
                    window: int, out, ws: torch.Tensor, num_ctas: int = 0, dev_err=None, stream=None):
    """Attention of drafted tokens [B, N] over the cache and their own tree: q and
    out bf16 [B, N, 32, 128], k_draft and v_draft bf16 [B, N, 4, 128], parent
    int32 [B, N]; seq_lens and n_draft are host values per request."""
    _need(q.dim() == 4, "q must be [B, N, 32, 128]")
    B, N = q.shape[0], q.shape[1]
    dev, bf16, heads, kv = torch.cuda.current_device(), torch.bfloat16, (B, N, NUM_Q_HEADS, HEAD_DIM), (B, N, NUM_KV_HEADS, HEAD_DIM)
    lens, counts = _host_i32(seq_lens, B, "seq_lens"), _host_i32(n_draft, B, "n_draft")
    _need(ws.is_contiguous() and ws.get_device() == dev, "ws must be a dense tensor on the current CUDA device")
    _check(load_library().flint_attn_tree(
        _dense(q, bf16, heads, "q", dev), _dense(k_draft, bf16, kv, "k_draft", dev), _dense(v_draft, bf16, kv, "v_draft", dev),
        _dense(parent, torch.int32, (B, N), "parent", dev), N, ctypes.byref(cache), lens.buffer_info()[0],
        counts.buffer_info()[0], B, _dense(sinks, torch.float32, (NUM_Q_HEADS,), "sinks", dev), int(window),
        _dense(out, bf16, heads, "out", dev), ws.data_ptr(), ws.nbytes, int(num_ctas), _error_word(dev_err, dev),
        _stream_of(stream, dev)))
    return out


def _prob_rows(t, B: int, rows: int, name: str, dev: int) -> int:
    """The row stride (elements) of fp32 [B, rows, V] whose rows are evenly spaced."""
    if t.dtype is not torch.float32 or t.dim() != 3 or t.shape[0] != B or t.shape[1] != rows or t.get_device() != dev:
        raise FlintError(FLINT_ERR_INVALID_ARG, f"{name} must be fp32 [{B}, {rows}, V] on the current CUDA device")
    b, r, v = t.stride()
    if rows == 1:
        r = b if B > 1 else t.shape[2]
    _need((v == 1 or t.shape[2] == 1) and (B == 1 or b == rows * r) and r >= t.shape[2],
          f"{name}: rows must be dense, apart and evenly spaced over the batch")
    return r


def flint_verify_tree(target, draft, tokens, parent, n_draft: Sequence[int], u_accept, u_sample, path, n_accepted,
                      next_token, dev_err=None, stream=None):
    """Verification of drafted tokens [B, N] against the target's probabilities
    fp32 [B, N + 1, V] (row 0 after the context, row i + 1 after node i), from
    the uniforms u_accept [B, N] and u_sample [B]; draft fp32 [B, N, V] holds the
    distributions that the children of each row's node were drawn from, None:
    fixed candidates.  Writes path int32 [B, N], n_accepted and next_token int32 [B]."""
    _need(tokens.dim() == 2, "tokens must be [B, N]")
    B, N = tokens.shape
    dev, i32, f32 = torch.cuda.current_device(), torch.int32, torch.float32
    ts = _prob_rows(target, B, N + 1, "target", dev)
    V = target.shape[2]
    ds, at_draft = 0, None
    if draft is not None:
        ds, at_draft = _prob_rows(draft, B, N, "draft", dev), draft.data_ptr()
        _need(draft.shape[2] == V, "target and draft must have rows of one length")
    counts = _host_i32(n_draft, B, "n_draft")
    _check(load_library().flint_verify_tree(
        target.data_ptr(), ts, at_draft, ds, _dense(tokens, i32, (B, N), "tokens", dev), _dense(parent, i32, (B, N), "parent", dev),
        counts.buffer_info()[0], B, N, V, _dense(u_accept, f32, (B, N), "u_accept", dev),
        _dense(u_sample, f32, (B,), "u_sample", dev), _dense(path, i32, (B, N), "path", dev),
        _dense(n_accepted, i32, (B,), "n_accepted", dev), _dense(next_token, i32, (B,), "next_token", dev),
        _error_word(dev_err, dev), _stream_of(stream, dev)))
    return path, n_accepted, next_token


def path_layers(layers) -> ctypes.Array:
    """A flint_path_layer array from (k_draft, v_draft, cache) per layer: bf16
    [B, N, 4, 128] tensors and the layer's KVCache."""
    arr = (PathLayer * len(layers))()
    shape, dev = tuple(layers[0][0].shape) if len(layers) else (), torch.cuda.current_device()
    for i, (k, v, cache) in enumerate(layers):
        _need(len(shape) == 4, "the drafts must be [B, N, 4, 128]")
        full = shape[:2] + (NUM_KV_HEADS, HEAD_DIM)
        arr[i].k = _dense(k, torch.bfloat16, full, f"layer {i}: k", dev)
        arr[i].v = _dense(v, torch.bfloat16, full, f"layer {i}: v", dev)
        arr[i].cache = cache
    arr._keep, arr._shape, arr._dev = list(layers), shape[:2], dev
    return arr


def flint_kv_append_path(layers, path, n_accepted, seq_lens: Sequence[int], dev_err=None, stream=None) -> None:
    """Append the drafted k and v of the accepted nodes path[b, :n_accepted[b]]
    (device int32) at positions seq_lens[b] .. of every layer's cache; layers:
    an array from path_layers() or a list for it."""
    arr, dev = layers if isinstance(layers, ctypes.Array) else path_layers(layers), torch.cuda.current_device()
    _need(len(arr) > 0 and path.shape == arr._shape, "path must be [B, N] as the layers' drafts are")
    _need(arr._dev == dev, "the layers are not on the current CUDA device")
    B, N = path.shape
    lens = _host_i32(seq_lens, B, "seq_lens")
    _check(load_library().flint_kv_append_path(
        arr, len(arr), _dense(path, torch.int32, (B, N), "path", dev), _dense(n_accepted, torch.int32, (B,), "n_accepted", dev), N,
        lens.buffer_info()[0], B, _error_word(dev_err, dev), _stream_of(stream, dev)))


def flint_plan_tree(seq_lens: Sequence[int], n_draft: Sequence[int], window: int = 0, layout: int = CONTIGUOUS, fp8: bool = False,
                    num_ctas: int = 148):
    """The plan of a flint_attn_tree call: (units [(request, node block, tiles, row
    tiles)], cuts [(unit, tile)] of the groups and the end)."""
    B, max_units, max_groups = len(seq_lens), 128, 74
    lens, counts = _host_i32(seq_lens, B, "seq_lens"), _host_i32(n_draft, B, "n_draft")
    units, cuts, n = (ctypes.c_int32 * (4 * max_units))(), (ctypes.c_int32 * (2 * max_groups + 2))(), ctypes.c_int32()
    groups = load_library().flint_plan_tree(lens.buffer_info()[0], counts.buffer_info()[0], B, int(window), int(layout), int(fp8),
                                            int(num_ctas), units, max_units, ctypes.byref(n), cuts, max_groups)
    _need(groups >= 0, "flint_plan_tree: invalid arguments")
    return ([tuple(units[4 * u:4 * u + 4]) for u in range(n.value)],
            [tuple(cuts[2 * q:2 * q + 2]) for q in range(groups + 1)])


def flint_plan_items(seg_tiles: Sequence[int], num_ctas: int, item_cost: int = 2,
                     max_items: int = 512):
    """Returns (items [(seg, t0, t1)], cta_begin list) from the C planner."""
    n = len(seg_tiles)
    st = _i32_host(seg_tiles)
    seg = (ctypes.c_int32 * max_items)()
    t0 = (ctypes.c_int32 * max_items)()
    t1 = (ctypes.c_int32 * max_items)()
    cb = (ctypes.c_int32 * (num_ctas + 1))()
    k = load_library().flint_plan_items(st, n, num_ctas, item_cost, seg, t0, t1, cb, max_items)
    if k < 0:
        raise FlintError(FLINT_ERR_INVALID_ARG, "planner rejected the arguments")
    return [(seg[i], t0[i], t1[i]) for i in range(k)], list(cb)


def flint_plan_split(seg_tiles: Sequence[int], num_ctas: int, item_cost: int = 2,
                     max_items: int = 768):
    """Returns (items [(seg, t0, t1)] sorted by segment, static lists [[item
    index, ...] per CTA], queue [item index, ...]) from the C planner."""
    n = len(seg_tiles)
    st = _i32_host(seg_tiles)
    seg = (ctypes.c_int32 * max_items)()
    t0 = (ctypes.c_int32 * max_items)()
    t1 = (ctypes.c_int32 * max_items)()
    order = (ctypes.c_int32 * max_items)()
    cb = (ctypes.c_int32 * (num_ctas + 1))()
    k = load_library().flint_plan_split(st, n, num_ctas, item_cost, max_items, seg, t0, t1, order, cb)
    if k < 0:
        raise FlintError(FLINT_ERR_INVALID_ARG, "planner rejected the arguments")
    items = [(seg[i], t0[i], t1[i]) for i in range(k)]
    lists = [[order[j] for j in range(cb[c], cb[c + 1])] for c in range(num_ctas)]
    queue = [order[j] for j in range(cb[num_ctas], k)]
    return items, lists, queue
