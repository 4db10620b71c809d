"""Thin ctypes binding of libbkv (include/bkv.h), same names as the C ABI.

Argument marshalling only: tensors become device pointers, a torch stream
becomes its cudaStream_t, status codes become exceptions. Every step of the
eviction runs in the library's CUDA kernels. The library must be built
(`kv_cache_eviction_head_gb300.build.build()`); importing this module without
it raises ImportError.
"""

from __future__ import annotations

import ctypes
import os
from array import array
from dataclasses import dataclass

import numpy as np

# BKV_LIBRARY=checked loads the bounds-checked build (libbkv_checked.so)
_VARIANTS = {"": "libbkv.so", "checked": "libbkv_checked.so"}
_variant = os.environ.get("BKV_LIBRARY", "")
if _variant not in _VARIANTS:
    raise ImportError(f"BKV_LIBRARY={_variant!r}: expected one of {sorted(_VARIANTS)}")
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), _VARIANTS[_variant])
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with kv_cache_eviction_head_gb300.build.build()"
                      + (" (checked=True)" if _variant else ""))
_lib = ctypes.CDLL(_LIB_PATH)

BKV_OK = 0
BKV_ERR_INVALID_ARG = 1
BKV_ERR_STATE = 2
BKV_ERR_WORKSPACE = 3
BKV_ERR_CUDA = 4
BKV_ERR_NONFINITE = 5
BKV_ERR_TIMEOUT = 6
BKV_ERR_UNSUPPORTED = 7
BKV_ERR_INTERNAL = 8
BKV_FLAG_KEEP_SCORES = 1
BKV_FLAG_ORDER_FREE = 2
BKV_FLAG_MEAN_POOL = 4

EXPORTED = ["bkv_workspace_bytes", "bkv_create", "bkv_set_stream", "bkv_append_queries",
            "bkv_evict", "bkv_prefill", "bkv_coverage", "bkv_selftest_wait", "bkv_sync",
            "bkv_get_fps_trace", "bkv_get_scores", "bkv_get_head_state",
            "bkv_profile", "bkv_profile_read", "bkv_score_select_noalloc", "bkv_get_stats",
            "bkv_store_kv", "bkv_attend_prompt", "bkv_attend_tree", "bkv_commit_tree",
            "bkv_make_rope", "bkv_store_paged", "bkv_attend_paged_bytes", "bkv_attend_paged", "bkv_weigh_prompt",
            "bkv_evict_weight",
            "bkv_destroy", "bkv_status_str"]
KERNELS = ["append", "rope", "score_select", "fps", "coverage", "prefill"]


class BkvConfig(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("d", ctypes.c_int32),
                ("budget", ctypes.c_int32), ("period", ctypes.c_int32), ("prefix", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("fps_cap", ctypes.c_int32), ("fps_keep", ctypes.c_int32),
                ("layers", ctypes.c_int32), ("batch", ctypes.c_int32), ("max_cache", ctypes.c_int32),
                ("rope_theta", ctypes.c_double), ("flags", ctypes.c_int32)]


class BkvStats(ctypes.Structure):
    _fields_ = [("evictions", ctypes.c_uint64), ("fps_calls", ctypes.c_uint64),
                ("rows_moved", ctypes.c_uint64), ("beacons", ctypes.c_int32),
                ("recents", ctypes.c_int32), ("cache_len", ctypes.c_int32),
                ("last_step", ctypes.c_int64)]


class BkvKernelTimes(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * 6), ("launches", ctypes.c_uint64 * 6)]


class BkvPages(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("per_seq", ctypes.c_int32),
                ("table", ctypes.c_void_p)]


class BkvRope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scale", ctypes.c_double),
                ("inv_freq", ctypes.c_double * 64)]


ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

_vp, _sz, _i32, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
_lib.bkv_workspace_bytes.argtypes = [ctypes.POINTER(BkvConfig), ctypes.POINTER(_sz)]
_lib.bkv_create.argtypes = [ctypes.POINTER(BkvConfig), _vp, _sz, _vp, ctypes.POINTER(_vp)]
_lib.bkv_set_stream.argtypes = [_vp, _vp]
_lib.bkv_append_queries.argtypes = [_vp, _vp, _i64]
_lib.bkv_evict.argtypes = [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), _i32, _i64, _vp]
_lib.bkv_coverage.argtypes = [_vp, _vp, _i32, _vp]
_lib.bkv_prefill.argtypes = [_vp, _vp, _i32, _i64, _vp]
_lib.bkv_sync.argtypes = [_vp]
_lib.bkv_selftest_wait.argtypes = [_vp, _i64]
_lib.bkv_get_fps_trace.argtypes = [_vp, _vp, _sz]
_lib.bkv_get_scores.argtypes = [_vp, _vp, _sz]
_lib.bkv_get_head_state.argtypes = [_vp, _i32, _i32, _i32, _vp, _sz]
_lib.bkv_get_stats.argtypes = [_vp, ctypes.POINTER(BkvStats)]
_lib.bkv_profile.argtypes = [_vp, _i32]
_lib.bkv_profile_read.argtypes = [_vp, ctypes.POINTER(BkvKernelTimes)]
_lib.bkv_score_select_noalloc.argtypes = [ctypes.POINTER(BkvConfig), _vp, _vp, _i32, _i32,
                                          ctypes.POINTER(_vp), _i32, _i64, _vp, _vp, _vp]
_lib.bkv_store_kv.argtypes = [ctypes.POINTER(BkvConfig), _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _vp,
                              _vp, _vp, _vp, _vp, _vp, _vp]
_lib.bkv_attend_prompt.argtypes = [ctypes.POINTER(BkvConfig), _vp, _i64, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.bkv_attend_tree.argtypes = [ctypes.POINTER(BkvConfig), _vp, _i64, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                 _vp]
_lib.bkv_commit_tree.argtypes = [ctypes.POINTER(BkvConfig), ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp, _vp, _vp,
                                 _i32, _vp, _vp]
_cfgp, _pagesp, _f32 = ctypes.POINTER(BkvConfig), ctypes.POINTER(BkvPages), ctypes.c_float
_lib.bkv_make_rope.argtypes = [ctypes.POINTER(BkvRope), ctypes.c_double, _i32, _i32, _i32, ctypes.c_double,
                               ctypes.c_double]
_lib.bkv_store_paged.argtypes = [_cfgp, _pagesp, ctypes.POINTER(BkvRope), _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp,
                                 _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.bkv_attend_paged_bytes.argtypes = [_cfgp, _pagesp, _i32, ctypes.POINTER(_sz)]
_lib.bkv_attend_paged.argtypes = [_cfgp, _pagesp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _sz, _vp, _vp]
_lib.bkv_weigh_prompt.argtypes = [_cfgp, _pagesp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _vp, _f32, _vp, _vp]
_lib.bkv_evict_weight.argtypes = [_cfgp, _pagesp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp,
                                  _vp, _vp, _vp, _vp]
_lib.bkv_destroy.argtypes = [_vp]
_lib.bkv_destroy.restype = None
_lib.bkv_status_str.argtypes = [_i32]
_lib.bkv_status_str.restype = ctypes.c_char_p
for _n in EXPORTED[:-2]:
    getattr(_lib, _n).restype = ctypes.c_int


class BkvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {bkv_status_str(code)}")


def bkv_status_str(code: int) -> str:
    return _lib.bkv_status_str(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != BKV_OK:
        raise BkvError(code, where)


def _check_tensor(t, name: str, dtype, shape) -> None:
    """Raises ValueError unless t is a contiguous CUDA tensor of this dtype and shape."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def _check_layers(ts, name: str, cfg) -> None:
    """`layers` bf16 caches [batch][kv_heads][max_cache][d], one per layer."""
    import torch
    if len(ts) != cfg.layers:
        raise ValueError(f"{name}: expected {cfg.layers} per-layer tensors, got {len(ts)}")
    for l, t in enumerate(ts):
        _check_tensor(t, f"{name}[{l}]", torch.bfloat16, (cfg.batch, cfg.kv_heads, cfg.max_cache, cfg.d))


def _stream_ptr(stream) -> int:
    if stream is None:
        return 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def make_config(*, heads, kv_heads, d, budget, period, prefix, recent, fps_cap=32, fps_keep=16,
                layers, batch, max_cache, rope_theta, flags=0) -> BkvConfig:
    return BkvConfig(heads, kv_heads, d, budget, period, prefix, recent, fps_cap, fps_keep, layers,
                     batch, max_cache, float(rope_theta), flags)


def bkv_workspace_bytes(cfg: BkvConfig) -> int:
    n = _sz(0)
    _check(_lib.bkv_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n)), "bkv_workspace_bytes")
    return n.value


@dataclass
class Handle:
    ptr: int
    cfg: BkvConfig
    workspace: object  # keeps the caller's workspace tensor alive


def bkv_create(cfg: BkvConfig, workspace, stream=None) -> Handle:
    """workspace: a uint8 CUDA tensor of at least bkv_workspace_bytes(cfg) bytes."""
    out = _vp(0)
    _check(_lib.bkv_create(ctypes.byref(cfg), _vp(workspace.data_ptr()), _sz(workspace.numel() * workspace.element_size()),
                           _vp(_stream_ptr(stream)), ctypes.byref(out)), "bkv_create")
    return Handle(out.value, cfg, workspace)


def bkv_set_stream(h: Handle, stream) -> None:
    _check(_lib.bkv_set_stream(_vp(h.ptr), _vp(_stream_ptr(stream))), "bkv_set_stream")


def bkv_append_queries(h: Handle, q_pre, step: int) -> None:
    """q_pre: bf16 CUDA tensor [layers][batch][heads][d], contiguous."""
    import torch
    c = h.cfg
    _check_tensor(q_pre, "q_pre", torch.bfloat16, (c.layers, c.batch, c.heads, c.d))
    _check(_lib.bkv_append_queries(_vp(h.ptr), _vp(q_pre.data_ptr()), _i64(step)), "bkv_append_queries")


def bkv_evict(h: Handle, K, V, cache_len: int, step: int, kept) -> None:
    """K, V: sequences of `layers` bf16 CUDA tensors [batch][kv_heads][max_cache][d];
    kept: int32 CUDA tensor [layers][batch][kv_heads][budget]."""
    import torch
    c = h.cfg
    _check_layers(K, "K", c)
    _check_layers(V, "V", c)
    _check_tensor(kept, "kept", torch.int32, (c.layers, c.batch, c.kv_heads, c.budget))
    n = len(K)
    kp = (_vp * n)(*[t.data_ptr() for t in K])
    vp = (_vp * n)(*[t.data_ptr() for t in V])
    _check(_lib.bkv_evict(_vp(h.ptr), kp, vp, _i32(cache_len), _i64(step), _vp(kept.data_ptr())),
           "bkv_evict")


def bkv_evict_ptrs(h: Handle, kptrs, vptrs, cache_len: int, step: int, kept_ptr: int) -> None:
    """bkv_evict with raw device pointers (pre-marshalled pointer arrays allowed)."""
    _check(_lib.bkv_evict(_vp(h.ptr), kptrs, vptrs, _i32(cache_len), _i64(step), _vp(kept_ptr)),
           "bkv_evict")


def bkv_prefill(h: Handle, q_prompt, first_step: int, trace_out=None) -> None:
    """q_prompt: bf16 CUDA tensor [P][layers][batch][heads][d]; trace_out: optional
    int32 CUDA tensor [layers][batch][heads][min(fps_keep, P - recents)]."""
    import torch
    c = h.cfg
    P = q_prompt.shape[0] if q_prompt.dim() == 5 else -1
    _check_tensor(q_prompt, "q_prompt", torch.bfloat16, (P, c.layers, c.batch, c.heads, c.d))
    if trace_out is not None:
        n_rq = c.fps_cap - c.fps_keep
        m = min(c.fps_keep, P - min(n_rq, P))
        _check_tensor(trace_out, "trace_out", torch.int32, (c.layers, c.batch, c.heads, m))
    _check(_lib.bkv_prefill(_vp(h.ptr), _vp(q_prompt.data_ptr()), _i32(q_prompt.shape[0]),
                            _i64(first_step), _vp(trace_out.data_ptr() if trace_out is not None else 0)),
           "bkv_prefill")


def bkv_coverage(h: Handle, q_future, out) -> None:
    """q_future: bf16 CUDA tensor [n_future][layers][batch][heads][d];
    out: float64 CUDA tensor [layers][batch][heads][n_future]."""
    import torch
    c = h.cfg
    n = q_future.shape[0] if q_future.dim() == 5 else -1
    _check_tensor(q_future, "q_future", torch.bfloat16, (n, c.layers, c.batch, c.heads, c.d))
    _check_tensor(out, "out", torch.float64, (c.layers, c.batch, c.heads, n))
    _check(_lib.bkv_coverage(_vp(h.ptr), _vp(q_future.data_ptr()), _i32(q_future.shape[0]),
                             _vp(out.data_ptr())), "bkv_coverage")


def bkv_sync(h: Handle) -> None:
    _check(_lib.bkv_sync(_vp(h.ptr)), "bkv_sync")


def bkv_selftest_wait(h: Handle, wait_cycles: int) -> None:
    """Enqueues the bounded-wait self-test; the next bkv_sync raises BKV_ERR_TIMEOUT."""
    _check(_lib.bkv_selftest_wait(_vp(h.ptr), _i64(wait_cycles)), "bkv_selftest_wait")


def bkv_get_fps_trace(h: Handle) -> np.ndarray:
    c = h.cfg
    out = np.empty((c.layers, c.batch, c.heads, c.fps_keep), dtype=np.int8)
    _check(_lib.bkv_get_fps_trace(_vp(h.ptr), _vp(out.ctypes.data), _sz(out.nbytes)), "bkv_get_fps_trace")
    return out


def bkv_get_scores(h: Handle) -> np.ndarray:
    c = h.cfg
    out = np.empty((c.layers, c.batch, c.kv_heads, c.max_cache), dtype=np.float32)
    _check(_lib.bkv_get_scores(_vp(h.ptr), _vp(out.ctypes.data), _sz(out.size)), "bkv_get_scores")
    return out


def bkv_get_head_state(h: Handle, layer: int, seq: int, head: int) -> np.ndarray:
    """uint16 [fps_cap + n_rq][d]: beacon rows, then the recent ring slots."""
    c = h.cfg
    out = np.empty((c.fps_cap + c.fps_cap - c.fps_keep, c.d), dtype=np.uint16)
    _check(_lib.bkv_get_head_state(_vp(h.ptr), layer, seq, head, _vp(out.ctypes.data), _sz(out.size)),
           "bkv_get_head_state")
    return out


def bkv_profile(h: Handle, enable: bool) -> None:
    _check(_lib.bkv_profile(_vp(h.ptr), _i32(1 if enable else 0)), "bkv_profile")


def bkv_profile_read(h: Handle) -> dict:
    """{kernel name: (summed ms, launches)} since profiling was enabled."""
    t = BkvKernelTimes()
    _check(_lib.bkv_profile_read(_vp(h.ptr), ctypes.byref(t)), "bkv_profile_read")
    return {k: (t.ms[i], int(t.launches[i])) for i, k in enumerate(KERNELS)}


def bkv_score_select_noalloc(cfg: BkvConfig, bq, rq, beacons: int, recents: int, K,
                             cache_len: int, step: int, kept, status=None, stream=None) -> None:
    """Score + keep-set selection without a handle or workspace (see include/bkv.h).
    bq: bf16 CUDA tensor [layers][batch][heads][fps_cap][d]; rq: bf16 CUDA tensor
    [layers][batch][heads][fps_cap - fps_keep][d]; K: `layers` bf16 CUDA tensors
    [batch][kv_heads][max_cache][d]; kept: int32 CUDA tensor
    [layers][batch][kv_heads][budget]; status: optional uint32-sized CUDA tensor
    (int32, one element) receiving the device-side status."""
    import torch
    c = cfg
    n_rq = c.fps_cap - c.fps_keep
    _check_tensor(bq, "bq", torch.bfloat16, (c.layers, c.batch, c.heads, c.fps_cap, c.d))
    _check_tensor(rq, "rq", torch.bfloat16, (c.layers, c.batch, c.heads, n_rq, c.d))
    _check_layers(K, "K", c)
    _check_tensor(kept, "kept", torch.int32, (c.layers, c.batch, c.kv_heads, c.budget))
    if status is not None:
        _check_tensor(status, "status", torch.int32, (1,))
    n = len(K)
    kp = (_vp * n)(*[t.data_ptr() for t in K])
    _check(_lib.bkv_score_select_noalloc(ctypes.byref(cfg), _vp(bq.data_ptr()), _vp(rq.data_ptr()),
                                         _i32(beacons), _i32(recents), kp, _i32(cache_len),
                                         _i64(step), _vp(kept.data_ptr()),
                                         _vp(status.data_ptr() if status is not None else 0),
                                         _vp(_stream_ptr(stream))),
           "bkv_score_select_noalloc")


class _Lazy:
    """torch and what the short calls below use of it, looked up once: their host time is
    most of a decode step's, and an import statement or a chain of attributes per argument
    is a good part of that."""
    torch = None


def _load():
    import torch
    _Lazy.bf16, _Lazy.i32, _Lazy.i64, _Lazy.f32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
    _Lazy.Tensor, _Lazy.torch = torch.Tensor, torch
    return _Lazy


def _device():
    return (_Lazy if _Lazy.torch is not None else _load()).torch.cuda.current_device()


def _check_on_device(t, name: str, dtype, shape, device):
    """_check_tensor, and that t lives on the current device (kernels launch there).
    Returns its address. The first test passes without building a message."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _check_tensor(t, name, dtype, shape)
    raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{device}")


def _check_caches(ts, name: str, n: int, shape, device, dtype=None):
    """A _vp array of n per-layer caches (bf16 unless said) of this shape on this device. The attributes of
    all layers are gathered by C-level maps; on a mismatch the layers are looked at one by
    one for the message."""
    T = _Lazy.Tensor
    dtype = dtype or _Lazy.bf16
    if len(ts) != n:
        raise ValueError(f"{name}: expected {n} per-layer tensors, got {len(ts)}")
    try:
        if (list(map(T.size, ts)) == [shape] * n and list(map(T.get_device, ts)) == [device] * n
                and all(map(T.is_contiguous, ts)) and {t.dtype for t in ts} == {dtype}):
            return (_vp * n).from_buffer(array("Q", map(T.data_ptr, ts)))
    except (TypeError, AttributeError):
        pass
    return (_vp * n)(*[_check_on_device(t, f"{name}[{l}]", dtype, shape, device) for l, t in enumerate(ts)])


def _check_packed(t, name: str, shape, device):
    """Raises ValueError unless t is a bf16 tensor of this shape on this device whose heads
    and elements are contiguous and whose tokens are evenly spaced; returns its address and
    the elements between two tokens."""
    try:
        ok = t.dtype is _Lazy.bf16 and t.shape == shape and t.get_device() == device
        if ok and t.is_contiguous():
            return t.data_ptr(), shape[-2] * shape[-1]
    except AttributeError:
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}") from None
    stride = shape[-2] * shape[-1]
    if ok:
        s = t.stride()
        # a dimension of one element may have any stride
        ok = s[-1] == 1 and (s[-2] == shape[-1] or shape[-2] == 1)
        if shape[-3] != 1:
            stride = s[-3]
        elif len(shape) == 4 and shape[0] != 1:
            stride = s[0]
        if len(shape) == 4 and shape[0] != 1 and shape[1] != 1:
            ok = ok and s[0] == shape[1] * stride
    if not ok:
        if t.is_cuda and t.get_device() != device:
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{device}")
        raise ValueError(f"{name}: expected a CUDA torch.bfloat16 tensor of shape {tuple(shape)} with contiguous "
                         f"heads and evenly spaced tokens, got {t.dtype} {tuple(t.shape)} {t.stride()} on {t.device}")
    return t.data_ptr(), stride


def _dims(t, name: str, shape: str, n: int):
    """t's shape, if it has n dimensions."""
    s = getattr(t, "shape", ())
    if len(s) != n:
        raise ValueError(f"{name}: expected a tensor {shape}")
    return s


def bkv_store_kv(cfg: BkvConfig, q_pre, k_pre, v, cu_seqlens, first_slot, first_pos, q_rot, K, V, *,
                 depth=None, status=None, stream=None) -> None:
    """RoPE and the write to the cache slots (see include/bkv.h). q_pre [total][heads][d],
    k_pre, v [total][kv_heads][d]: bf16, tokens any multiple of 8 elements apart; q_rot bf16
    [total][heads][d]; cu_seqlens int32 [batch + 1]; first_slot, first_pos int32 [batch];
    depth: optional int32 [total]; K, V: one layer's bf16 caches
    [batch][kv_heads][max_cache][d]; status: optional int32 of one element."""
    dev = _device()
    bf16, i32 = _Lazy.bf16, _Lazy.i32
    batch, heads, kv, d = cfg.batch, cfg.heads, cfg.kv_heads, cfg.d
    total = _dims(q_pre, "q_pre", "[tokens][heads][d]", 3)[0]
    cache, rows, one = (batch, kv, cfg.max_cache, d), (total, kv, d), (batch,)
    q, qs = _check_packed(q_pre, "q_pre", (total, heads, d), dev)
    k, ks = _check_packed(k_pre, "k_pre", rows, dev)
    vv, vs = _check_packed(v, "v", rows, dev)
    _check(_lib.bkv_store_kv(
        cfg, q, qs, k, ks, vv, vs, total, _check_on_device(cu_seqlens, "cu_seqlens", i32, (batch + 1,), dev),
        _check_on_device(first_slot, "first_slot", i32, one, dev),
        _check_on_device(first_pos, "first_pos", i32, one, dev),
        None if depth is None else _check_on_device(depth, "depth", i32, (total,), dev),
        _check_on_device(q_rot, "q_rot", bf16, (total, heads, d), dev), _check_on_device(K, "K", bf16, cache, dev),
        _check_on_device(V, "V", bf16, cache, dev),
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_store_kv")


def bkv_attend_prompt(cfg: BkvConfig, q, K, V, cu_seqlens, first_slot, out, *, lse=None, status=None,
                      stream=None) -> None:
    """Causal attention of packed prompts over one layer's caches (see include/bkv.h).
    q [total][heads][d]: rotated queries, bf16, tokens any multiple of 8 elements apart;
    out bf16 [total][heads][d]; lse: optional float32 [total][heads]; the others as
    bkv_store_kv."""
    dev = _device()
    bf16, i32 = _Lazy.bf16, _Lazy.i32
    batch, heads, d = cfg.batch, cfg.heads, cfg.d
    total = _dims(q, "q", "[tokens][heads][d]", 3)[0]
    cache, rows = (batch, cfg.kv_heads, cfg.max_cache, d), (total, heads, d)
    qp, qs = _check_packed(q, "q", rows, dev)
    _check(_lib.bkv_attend_prompt(
        cfg, qp, qs, _check_on_device(K, "K", bf16, cache, dev), _check_on_device(V, "V", bf16, cache, dev),
        _check_on_device(cu_seqlens, "cu_seqlens", i32, (batch + 1,), dev),
        _check_on_device(first_slot, "first_slot", i32, (batch,), dev), total,
        _check_on_device(out, "out", bf16, rows, dev),
        None if lse is None else _check_on_device(lse, "lse", _Lazy.f32, (total, heads), dev),
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_attend_prompt")


def bkv_attend_tree(cfg: BkvConfig, q, K, V, cache_lens, out, *, mask=None, nodes=None, lse=None, status=None,
                    stream=None) -> None:
    """Attention of a tree of drafted tokens (n = 1: a decode step) over one layer's
    caches (see include/bkv.h). q: rotated queries, bf16 [batch][n][heads][d]; cache_lens
    int32 [batch]; mask: optional int64 [batch][n]; nodes: optional int32 [batch]; out bf16
    [batch][n][heads][d]; lse: optional float32 [batch][n][heads]."""
    dev = _device()
    bf16, i32 = _Lazy.bf16, _Lazy.i32
    batch, heads, d = cfg.batch, cfg.heads, cfg.d
    n = _dims(q, "q", "[batch][n][heads][d]", 4)[1]
    cache, rows = (batch, cfg.kv_heads, cfg.max_cache, d), (batch, n, heads, d)
    qp, qs = _check_packed(q, "q", rows, dev)
    _check(_lib.bkv_attend_tree(
        cfg, qp, qs, _check_on_device(K, "K", bf16, cache, dev), _check_on_device(V, "V", bf16, cache, dev),
        _check_on_device(cache_lens, "cache_lens", i32, (batch,), dev), n,
        None if mask is None else _check_on_device(mask, "mask", _Lazy.i64, (batch, n), dev),
        None if nodes is None else _check_on_device(nodes, "nodes", i32, (batch,), dev),
        _check_on_device(out, "out", bf16, rows, dev),
        None if lse is None else _check_on_device(lse, "lse", _Lazy.f32, (batch, n, heads), dev),
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_attend_tree")


def bkv_commit_tree(cfg: BkvConfig, K, V, cache_lens, path, count, *, status=None, stream=None) -> None:
    """Keeps an accepted path in every layer (see include/bkv.h). K, V: `layers` bf16
    caches [batch][kv_heads][max_cache][d]; cache_lens, count int32 [batch]; path int32
    [batch][n]."""
    dev = _device()
    i32, batch, layers = _Lazy.i32, cfg.batch, cfg.layers
    n = _dims(path, "path", "[batch][n]", 2)[1]
    cache = (batch, cfg.kv_heads, cfg.max_cache, cfg.d)
    kp, vp = _check_caches(K, "K", layers, cache, dev), _check_caches(V, "V", layers, cache, dev)
    _check(_lib.bkv_commit_tree(
        cfg, kp, vp, _check_on_device(cache_lens, "cache_lens", i32, (batch,), dev),
        _check_on_device(path, "path", i32, (batch, n), dev), _check_on_device(count, "count", i32, (batch,), dev), n,
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_commit_tree")


def make_rope(*, theta=1e4, rotary_dim=128, interleaved=False, scaling="none", factor=1.0, original_len=0,
              inv_freq=None, scale=1.0) -> BkvRope:
    """Rotary positions (see bkv_make_rope in include/bkv.h); scaling: one of ROPE_SCALINGS.
    inv_freq: the caller's own rotary_dim / 2 frequencies, with `scale`, instead of theta
    and a scaling."""
    r = BkvRope()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling: expected one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    if inv_freq is not None and (scaling != "none" or len(inv_freq) != rotary_dim // 2):
        raise ValueError(f"inv_freq: expected {rotary_dim // 2} frequencies and no scaling, got {len(inv_freq)} and {scaling!r}")
    _check(_lib.bkv_make_rope(ctypes.byref(r), theta, rotary_dim, 1 if interleaved else 0, ROPE_SCALINGS[scaling], factor,
                              original_len), "bkv_make_rope")
    if inv_freq is not None:
        r.inv_freq[:rotary_dim // 2] = [float(f) for f in inv_freq]
        r.scale = float(scale)
    return r


def _check_pool(cfg, K, table, device, name="K"):
    """The pool's pages as the library takes them (None: the dense caches), and the shape that
    goes with them without d."""
    if table is None:
        return None, (cfg.batch, cfg.kv_heads, cfg.max_cache)
    s = _dims(K, name, "[pages][kv_heads][page_size][d]", 4)
    t = _dims(table, "table", "[batch][per_seq]", 2)
    p = BkvPages(s[0], s[2], t[1], _check_on_device(table, "table", _Lazy.i32, (cfg.batch, t[1]), device))
    return p, (s[0], cfg.kv_heads, s[2])


def bkv_store_paged(cfg: BkvConfig, rope: BkvRope, q_pre, k_pre, v, cu_seqlens, first_slot, first_pos, q_rot, K, V, *,
                    table=None, depth=None, status=None, stream=None) -> None:
    """Rotary positions and the write to the pages (see include/bkv.h). K, V: one layer's bf16
    pools [pages][kv_heads][page_size][d] with table int32 [batch][per_seq], or without a
    table the dense caches [batch][kv_heads][max_cache][d]; the others as bkv_store_kv."""
    dev = _device()
    bf16, i32 = _Lazy.bf16, _Lazy.i32
    batch, heads, kv, d = cfg.batch, cfg.heads, cfg.kv_heads, cfg.d
    pages, shape = _check_pool(cfg, K, table, dev)
    total = _dims(q_pre, "q_pre", "[tokens][heads][d]", 3)[0]
    pool, rows, one = shape + (d,), (total, kv, d), (batch,)
    q, qs = _check_packed(q_pre, "q_pre", (total, heads, d), dev)
    k, ks = _check_packed(k_pre, "k_pre", rows, dev)
    vv, vs = _check_packed(v, "v", rows, dev)
    _check(_lib.bkv_store_paged(
        cfg, pages, rope, q, qs, k, ks, vv, vs, total, _check_on_device(cu_seqlens, "cu_seqlens", i32, (batch + 1,), dev),
        _check_on_device(first_slot, "first_slot", i32, one, dev),
        _check_on_device(first_pos, "first_pos", i32, one, dev),
        None if depth is None else _check_on_device(depth, "depth", i32, (total,), dev),
        _check_on_device(q_rot, "q_rot", bf16, (total, heads, d), dev), _check_on_device(K, "K", bf16, pool, dev),
        _check_on_device(V, "V", bf16, pool, dev),
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_store_paged")


def bkv_attend_paged_bytes(cfg: BkvConfig, K, table=None, *, weighed=False) -> int:
    """Bytes of bkv_attend_paged's workspace for these pools."""
    pages, _ = _check_pool(cfg, K, table, _device())
    n = _sz(0)
    _check(_lib.bkv_attend_paged_bytes(cfg, pages, 1 if weighed else 0, ctypes.byref(n)), "bkv_attend_paged_bytes")
    return n.value


def bkv_attend_paged(cfg: BkvConfig, q, K, V, lens, out, workspace, *, table=None, lse=None, weights=None, decay=1.0,
                     status=None, stream=None) -> None:
    """Attention of one new token per sequence over pages or dense caches (see include/bkv.h).
    q, out: bf16 [batch][heads][d]; lens int32 [batch]; workspace: uint8, at least
    bkv_attend_paged_bytes; lse: optional float32 [batch][heads]; weights: optional float32
    [pages][kv_heads][page_size], updated with `decay`."""
    dev = _device()
    bf16, i32, f32 = _Lazy.bf16, _Lazy.i32, _Lazy.f32
    batch, heads, d = cfg.batch, cfg.heads, cfg.d
    pages, shape = _check_pool(cfg, K, table, dev)
    pool, rows = shape + (d,), (batch, heads, d)
    qp, qs = _check_packed(q, "q", rows, dev)
    size = _dims(workspace, "workspace", "[bytes]", 1)[0]
    _check(_lib.bkv_attend_paged(
        cfg, pages, qp, qs, _check_on_device(K, "K", bf16, pool, dev), _check_on_device(V, "V", bf16, pool, dev),
        _check_on_device(lens, "lens", i32, (batch,), dev), _check_on_device(out, "out", bf16, rows, dev),
        None if lse is None else _check_on_device(lse, "lse", f32, (batch, heads), dev),
        None if weights is None else _check_on_device(weights, "weights", f32, shape, dev), decay,
        _check_on_device(workspace, "workspace", _Lazy.torch.uint8, (size,), dev), size,
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_attend_paged")


def bkv_weigh_prompt(cfg: BkvConfig, q, lse, K, cu_seqlens, first_slot, weights, *, table=None, decay=1.0, status=None,
                     stream=None) -> None:
    """The attention weight of packed prompts' queries, summed per slot (see include/bkv.h).
    q: rotated queries, bf16 [total][heads][d]; lse float32 [total][heads] as
    bkv_attend_prompt left it; weights float32 [pages][kv_heads][page_size] beside K."""
    dev = _device()
    i32, f32 = _Lazy.i32, _Lazy.f32
    batch, heads, d = cfg.batch, cfg.heads, cfg.d
    pages, shape = _check_pool(cfg, K, table, dev)
    total = _dims(q, "q", "[tokens][heads][d]", 3)[0]
    qp, qs = _check_packed(q, "q", (total, heads, d), dev)
    _check(_lib.bkv_weigh_prompt(
        cfg, pages, qp, qs, _check_on_device(lse, "lse", f32, (total, heads), dev),
        _check_on_device(K, "K", _Lazy.bf16, shape + (d,), dev),
        _check_on_device(cu_seqlens, "cu_seqlens", i32, (batch + 1,), dev),
        _check_on_device(first_slot, "first_slot", i32, (batch,), dev), total,
        _check_on_device(weights, "weights", f32, shape, dev), decay,
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_weigh_prompt")


def bkv_evict_weight(cfg: BkvConfig, K, V, weights, cache_lens, kept, *, table=None, new_lens=None, status=None,
                     stream=None) -> None:
    """Eviction by accumulated weight, in every layer (see include/bkv.h). K, V: `layers` bf16
    pools, weights: `layers` float32 [pages][kv_heads][page_size]; cache_lens int32 [batch];
    kept int32 [layers][batch][kv_heads][budget]; new_lens: optional int32 [batch]."""
    dev = _device()
    i32, batch, layers = _Lazy.i32, cfg.batch, cfg.layers
    if len(K) != layers:
        raise ValueError(f"K: expected {layers} per-layer tensors, got {len(K)}")
    pages, shape = _check_pool(cfg, K[0], table, dev, "K[0]")
    kp, vp = _check_caches(K, "K", layers, shape + (cfg.d,), dev), _check_caches(V, "V", layers, shape + (cfg.d,), dev)
    wp = _check_caches(weights, "weights", layers, shape, dev, _Lazy.f32)
    _check(_lib.bkv_evict_weight(
        cfg, pages, kp, vp, wp, _check_on_device(cache_lens, "cache_lens", i32, (batch,), dev),
        _check_on_device(kept, "kept", i32, (layers, batch, cfg.kv_heads, cfg.budget), dev),
        None if new_lens is None else _check_on_device(new_lens, "new_lens", i32, (batch,), dev),
        None if status is None else _check_on_device(status, "status", i32, (1,), dev), _stream_ptr(stream)),
        "bkv_evict_weight")


def bkv_get_stats(h: Handle) -> BkvStats:
    s = BkvStats()
    _check(_lib.bkv_get_stats(_vp(h.ptr), ctypes.byref(s)), "bkv_get_stats")
    return s


def bkv_destroy(h: Handle) -> None:
    if h.ptr:
        _lib.bkv_destroy(_vp(h.ptr))
        h.ptr = 0


def raw_status(fn_name: str, *args) -> int:
    """Calls a C entry point and returns its status code (tests of the error paths)."""
    return getattr(_lib, fn_name)(*args)


def library_path() -> str:
    return _LIB_PATH
