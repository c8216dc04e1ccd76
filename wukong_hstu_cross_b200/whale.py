"""Thin ctypes binding of libwhale_fusion.so (include/whale_fusion.h), same names.

Argument marshalling only: every step of the forward runs in the library's CUDA kernels.
Tensors are torch tensors (device memory and streams come from PyTorch); a plain int is
taken as a raw pointer. Importing this module loads the library and raises ImportError
if it has not been built (python -m wukong_hstu_cross_b200.build) — there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
from ctypes import POINTER, c_double, c_float, c_int, c_longlong, c_size_t, c_uint, c_void_p

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libwhale_fusion.so")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "whale_fusion.h")

WHALE_FP32, WHALE_BF16 = 0, 1
WHALE_SHARED_KV, WHALE_TIED_GATE, WHALE_DEBUG, WHALE_PREPARED_WEIGHTS = 1, 2, 4, 8
WHALE_MATERIALIZED_KV = 16
WHALE_DEVERR_TIMEOUT, WHALE_DEVERR_OFFSETS, WHALE_DEVERR_PAGES = 1, 2, 4
WHALE_ROTATE_HALVES, WHALE_ROTATE_ADJACENT = 0, 1
WHALE_CACHE_BF16, WHALE_CACHE_E4M3 = 0, 1
WHALE_ATTEND_CAUSAL = 1
WHALE_NOALLOC_SCRATCH_BYTES = 32 << 20
STATUS = {0: "WHALE_OK", 1: "WHALE_ERR_INVALID_ARG", 2: "WHALE_ERR_UNSUPPORTED", 3: "WHALE_ERR_CUDA",
          4: "WHALE_ERR_WORKSPACE", 5: "WHALE_ERR_DEVICE_CHECK"}


class whale_config(ctypes.Structure):
    _fields_ = [("n_layers", c_int), ("d", c_int), ("n_heads", c_int), ("n_tokens", c_int),
                ("ffn_hidden", c_int), ("fusion_hidden", c_int), ("dtype", c_int), ("flags", c_uint),
                ("eps", c_float)]


_WNAMES = ("g_q", "g_kv", "w_q", "w_kv", "w_f1", "w_f2", "g_ffn", "w_upgate", "w_down", "w_kabs")


class whale_layer_weights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in _WNAMES]


_GNAMES = ("g_q", "g_kv", "w_q", "w_kv", "w_f1", "w_f2", "g_ffn", "w_upgate", "w_down")


class whale_layer_grads(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in _GNAMES]


class whale_shape_hint(ctypes.Structure):
    _fields_ = [("B", c_int), ("max_L", c_int), ("total_L", c_longlong)]


class whale_kernel_time(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("ms", c_float)]


class whale_rotary(ctypes.Structure):
    _fields_ = [("rotary_dim", c_int), ("layout", c_int), ("base", c_double)]


class whale_head_rows(ctypes.Structure):
    _device = None  # of the tensors, where the binding made it
    _fields_ = [("x", c_void_p), ("y", c_void_p), ("gain", c_void_p), ("positions", c_void_p), ("rows", c_longlong),
                ("ld_x", c_longlong), ("ld_y", c_longlong), ("n_heads", c_int)]


class whale_head_grads(ctypes.Structure):
    _device = None  # of the tensors, where the binding made it
    _fields_ = [("dy", c_void_p), ("dx", c_void_p), ("d_gain", c_void_p), ("ld_dy", c_longlong), ("ld_dx", c_longlong)]


class whale_cache(ctypes.Structure):
    _device = None  # of the tensors, where the binding made it
    _fields_ = [("pages", c_void_p), ("scales", c_void_p), ("n_pages", c_int), ("page_size", c_int),
                ("n_kv_heads", c_int), ("format", c_int)]


class whale_chunk(ctypes.Structure):
    _device = None  # of the tensors, where the binding made it
    _fields_ = [("offsets", c_void_p), ("lengths", c_void_p), ("page_table", c_void_p), ("table_stride", c_int),
                ("B", c_int), ("max_new", c_int), ("max_length", c_int), ("total_new", c_longlong)]


class WhaleError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m wukong_hstu_cross_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)

_P = c_void_p
_SIGS = {
    "whale_status_string": ([c_int], ctypes.c_char_p),
    "whale_profile_begin": ([c_int], c_int),
    "whale_profile_end": ([POINTER(whale_kernel_time), c_int, POINTER(c_int)], c_int),
    "whale_workspace_size": ([POINTER(whale_config), POINTER(whale_shape_hint)], c_size_t),
    "whale_host_workspace_size": ([POINTER(whale_config), POINTER(whale_shape_hint)], c_size_t),
    "whale_fusion_forward": ([POINTER(whale_config), _P, _P, _P, POINTER(whale_layer_weights), _P,
                              POINTER(whale_shape_hint), _P, c_size_t, _P], c_int),
    "whale_fusion_forward_host": ([POINTER(whale_config), _P, _P, _P, POINTER(whale_layer_weights), _P,
                                   POINTER(whale_shape_hint), _P, c_size_t, _P], c_int),
    "whale_fusion_layer_forward": ([POINTER(whale_config), _P, _P, _P, POINTER(whale_layer_weights), _P,
                                    POINTER(whale_shape_hint), _P, c_size_t, _P], c_int),
    "whale_project_queries": ([POINTER(whale_config), c_longlong, _P, _P, _P, _P, _P, c_size_t, _P], c_int),
    "whale_project_kv": ([POINTER(whale_config), c_longlong, _P, _P, _P, _P, _P, c_size_t, _P], c_int),
    "whale_cross_attention": ([POINTER(whale_config), _P, _P, _P, _P, POINTER(whale_shape_hint), _P, c_size_t,
                               _P], c_int),
    "whale_attend_states": ([POINTER(whale_config), _P, _P, _P, POINTER(whale_layer_weights), _P,
                             POINTER(whale_shape_hint), _P, c_size_t, _P], c_int),
    "whale_fusion_mlp": ([POINTER(whale_config), c_longlong, _P, _P, _P, _P, _P, _P, c_size_t, _P], c_int),
    "whale_swiglu_ffn": ([POINTER(whale_config), c_longlong, _P, _P, _P, _P, _P, _P, c_size_t, _P], c_int),
    "whale_get_device_error": ([_P, POINTER(c_int)], c_int),
    "whale_prepared_weights_size": ([POINTER(whale_config)], c_size_t),
    "whale_prepare_weights": ([POINTER(whale_config), POINTER(whale_layer_weights), _P, c_size_t,
                               POINTER(whale_layer_weights), _P], c_int),
    "whale_cross_attention_noalloc": ([POINTER(whale_config), _P, _P, _P, _P, POINTER(whale_shape_hint), _P], c_int),
    "whale_test_bounded_waits": ([ctypes.c_ulonglong, _P], c_int),
    "whale_backward_workspace_size": ([POINTER(whale_config), POINTER(whale_shape_hint)], c_size_t),
    "whale_fusion_layer_backward": ([POINTER(whale_config), _P, _P, _P, POINTER(whale_layer_weights), _P, _P, _P,
                                     POINTER(whale_layer_grads), POINTER(whale_shape_hint), _P, c_size_t, _P], c_int),
    "whale_fusion_backward": ([POINTER(whale_config), _P, _P, _P, POINTER(whale_layer_weights), _P, _P, _P,
                               POINTER(whale_layer_grads), POINTER(whale_shape_hint), _P, c_size_t, _P], c_int),
    "whale_norm_rotate": ([POINTER(whale_config), POINTER(whale_rotary), POINTER(whale_head_rows),
                           POINTER(whale_head_rows), _P], c_int),
    "whale_norm_rotate_workspace_size": ([POINTER(whale_config), POINTER(whale_head_rows), POINTER(whale_head_rows)],
                                         c_size_t),
    "whale_norm_rotate_backward": ([POINTER(whale_config), POINTER(whale_rotary), POINTER(whale_head_rows),
                                    POINTER(whale_head_rows), POINTER(whale_head_grads), POINTER(whale_head_grads),
                                    c_int, _P, c_size_t, _P], c_int),
    "whale_cache_pages_size": ([POINTER(whale_config), POINTER(whale_cache)], c_size_t),
    "whale_cache_scales_size": ([POINTER(whale_config), POINTER(whale_cache)], c_size_t),
    "whale_cache_append": ([POINTER(whale_config), POINTER(whale_cache), POINTER(whale_chunk), _P, c_longlong, _P],
                           c_int),
    "whale_cache_read": ([POINTER(whale_config), POINTER(whale_cache), POINTER(whale_chunk), _P, c_longlong, _P], c_int),
    "whale_cache_attention_workspace_size": ([POINTER(whale_config), POINTER(whale_cache), POINTER(whale_chunk)],
                                             c_size_t),
    "whale_cache_attention": ([POINTER(whale_config), POINTER(whale_cache), POINTER(whale_chunk), _P, c_longlong, _P,
                               c_longlong, c_uint, _P, c_size_t, _P], c_int),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes, _f.restype = _args, _res


def header_functions() -> list:
    """Names of the functions include/whale_fusion.h declares."""
    with open(HEADER) as fh:
        text = fh.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(whale_\w+)\s*\(", text, flags=re.M)))


# ------------------------------------------------------------------------------------------------
# marshalling helpers
# ------------------------------------------------------------------------------------------------
def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != 0:
        raise WhaleError(status, where)


def make_config(n_layers, d, n_heads, n_tokens, ffn_hidden, fusion_hidden, dtype, flags=0, eps=1e-6) -> whale_config:
    return whale_config(n_layers, d, n_heads, n_tokens, ffn_hidden, fusion_hidden, dtype, flags, eps)


def make_hint(B, max_L, total_L) -> whale_shape_hint:
    return whale_shape_hint(int(B), int(max_L), int(total_L))


def layer_weights(lw) -> whale_layer_weights:
    """A whale_layer_weights from a dict of tensors (None allowed for w_f1)."""
    if isinstance(lw, whale_layer_weights):
        return lw
    return whale_layer_weights(*[_ptr(lw.get(n)) for n in _WNAMES])


def weights_array(layers) -> ctypes.Array:
    arr = (whale_layer_weights * len(layers))()
    for i, lw in enumerate(layers):
        arr[i] = layer_weights(lw)
    return arr


# ------------------------------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ------------------------------------------------------------------------------------------------
def whale_status_string(status: int) -> str:
    return _lib.whale_status_string(status).decode()


def whale_workspace_size(cfg: whale_config, hint: whale_shape_hint) -> int:
    return int(_lib.whale_workspace_size(ctypes.byref(cfg), ctypes.byref(hint)))


def whale_host_workspace_size(cfg: whale_config, hint: whale_shape_hint) -> int:
    return int(_lib.whale_host_workspace_size(ctypes.byref(cfg), ctypes.byref(hint)))


def _ws_bytes(workspace, nbytes):
    if nbytes is not None:
        return int(nbytes)
    if workspace is None:
        return 0
    return workspace.numel() * workspace.element_size()


def whale_prepared_weights_size(cfg: whale_config) -> int:
    return int(_lib.whale_prepared_weights_size(ctypes.byref(cfg)))


def whale_prepare_weights(cfg, weights, prepared, prepared_bytes=None, stream=None, raw=False):
    """Fold gains / pack up|gate once; returns the ctypes array of prepared layer weights (use it
    with cfg.flags | WHALE_PREPARED_WEIGHTS). The array points into `prepared` and, for the matrices
    that are not re-packed (w_f1, w_f2, w_down, the gains), into the caller's original tensors: it
    keeps references to both, so neither is freed while the array is alive."""
    w = weights if isinstance(weights, ctypes.Array) else weights_array(weights)
    out = (whale_layer_weights * len(w))()
    st = _lib.whale_prepare_weights(ctypes.byref(cfg), w, _ptr(prepared), _ws_bytes(prepared, prepared_bytes), out,
                                    _stream(stream))
    if raw:
        return st
    _check(st, "whale_prepare_weights")
    out._keepalive = (weights, w, prepared)
    return out


def whale_fusion_forward(cfg, wukong_tokens, seq_states, seq_offsets, weights, out, hint, workspace,
                         workspace_bytes=None, stream=None, raw=False):
    w = weights if isinstance(weights, ctypes.Array) else weights_array(weights)
    st = _lib.whale_fusion_forward(ctypes.byref(cfg), _ptr(wukong_tokens), _ptr(seq_states), _ptr(seq_offsets), w,
                                   _ptr(out), ctypes.byref(hint), _ptr(workspace),
                                   _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_fusion_forward")


def whale_fusion_forward_host(cfg, host_tokens, host_seq_states, host_offsets, weights, host_out, hint, workspace,
                              workspace_bytes=None, stream=None, raw=False):
    w = weights if isinstance(weights, ctypes.Array) else weights_array(weights)
    st = _lib.whale_fusion_forward_host(ctypes.byref(cfg), _ptr(host_tokens), _ptr(host_seq_states),
                                        _ptr(host_offsets), w, _ptr(host_out), ctypes.byref(hint), _ptr(workspace),
                                        _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_fusion_forward_host")


def whale_fusion_layer_forward(cfg, tokens_in, layer_states, seq_offsets, layer_weights_, tokens_out, hint, workspace,
                               workspace_bytes=None, stream=None, raw=False):
    lw = layer_weights(layer_weights_)
    st = _lib.whale_fusion_layer_forward(ctypes.byref(cfg), _ptr(tokens_in), _ptr(layer_states), _ptr(seq_offsets),
                                         ctypes.byref(lw), _ptr(tokens_out), ctypes.byref(hint), _ptr(workspace),
                                         _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_fusion_layer_forward")


def whale_project_queries(cfg, rows, x, g_q, w_q, q, workspace, workspace_bytes=None, stream=None, raw=False):
    st = _lib.whale_project_queries(ctypes.byref(cfg), int(rows), _ptr(x), _ptr(g_q), _ptr(w_q), _ptr(q),
                                    _ptr(workspace), _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_project_queries")


def whale_project_kv(cfg, rows, s, g_kv, w_kv, kv, workspace, workspace_bytes=None, stream=None, raw=False):
    st = _lib.whale_project_kv(ctypes.byref(cfg), int(rows), _ptr(s), _ptr(g_kv), _ptr(w_kv), _ptr(kv),
                               _ptr(workspace), _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_project_kv")


def whale_cross_attention(cfg, q, kv, seq_offsets, a, hint, workspace, workspace_bytes=None, stream=None, raw=False):
    st = _lib.whale_cross_attention(ctypes.byref(cfg), _ptr(q), _ptr(kv), _ptr(seq_offsets), _ptr(a),
                                    ctypes.byref(hint), _ptr(workspace), _ws_bytes(workspace, workspace_bytes),
                                    _stream(stream))
    if raw:
        return st
    _check(st, "whale_cross_attention")


def whale_attend_states(cfg, q, layer_states, seq_offsets, weights, a, hint, workspace, workspace_bytes=None,
                        stream=None, raw=False):
    """S2 + S3 in absorbed form (no K|V tensor): `weights` is one layer's dict or whale_layer_weights."""
    lw = layer_weights(weights)
    st = _lib.whale_attend_states(ctypes.byref(cfg), _ptr(q), _ptr(layer_states), _ptr(seq_offsets),
                                  ctypes.byref(lw), _ptr(a), ctypes.byref(hint), _ptr(workspace),
                                  _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_attend_states")


def whale_cross_attention_noalloc(cfg, q, kv, seq_offsets, a, hint, stream=None, raw=False):
    """Eq. (4) without a workspace: the partials live in the library's fixed device array
    (WHALE_NOALLOC_SCRATCH_BYTES); see include/whale_fusion.h."""
    st = _lib.whale_cross_attention_noalloc(ctypes.byref(cfg), _ptr(q), _ptr(kv), _ptr(seq_offsets), _ptr(a),
                                            ctypes.byref(hint), _stream(stream))
    if raw:
        return st
    _check(st, "whale_cross_attention_noalloc")


def whale_fusion_mlp(cfg, rows, a, x, w_f1, w_f2, f, workspace, workspace_bytes=None, stream=None, raw=False):
    st = _lib.whale_fusion_mlp(ctypes.byref(cfg), int(rows), _ptr(a), _ptr(x), _ptr(w_f1), _ptr(w_f2), _ptr(f),
                               _ptr(workspace), _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_fusion_mlp")


def whale_swiglu_ffn(cfg, rows, f, g_ffn, w_upgate, w_down, y, workspace, workspace_bytes=None, stream=None,
                     raw=False):
    st = _lib.whale_swiglu_ffn(ctypes.byref(cfg), int(rows), _ptr(f), _ptr(g_ffn), _ptr(w_upgate), _ptr(w_down),
                               _ptr(y), _ptr(workspace), _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_swiglu_ffn")


def whale_profile_begin(max_kernels: int = 4096) -> None:
    _check(_lib.whale_profile_begin(max_kernels), "whale_profile_begin")


def whale_profile_end(capacity: int = 4096) -> list:
    """[(kernel name, ms), ...] in launch order (see include/whale_fusion.h)."""
    buf = (whale_kernel_time * capacity)()
    n = c_int(0)
    _check(_lib.whale_profile_end(buf, capacity, ctypes.byref(n)), "whale_profile_end")
    return [((buf[i].kernel or b"?").decode(), float(buf[i].ms)) for i in range(min(n.value, capacity))]


def whale_backward_workspace_size(cfg: whale_config, hint: whale_shape_hint) -> int:
    return int(_lib.whale_backward_workspace_size(ctypes.byref(cfg), ctypes.byref(hint)))


def layer_grads(g) -> whale_layer_grads:
    """A whale_layer_grads from a dict of fp32 tensors (w_f1 may be absent or None)."""
    if isinstance(g, whale_layer_grads):
        return g
    return whale_layer_grads(*[_ptr(g.get(n)) for n in _GNAMES])


def whale_fusion_layer_backward(cfg, tokens_in, layer_states, seq_offsets, layer_weights_, d_out, d_tokens, d_states,
                                grads, hint, workspace, workspace_bytes=None, stream=None, raw=False):
    """Gradients of one fusion layer (see include/whale_fusion.h); `grads` is a dict of fp32 tensors."""
    lw = layer_weights(layer_weights_)
    gr = layer_grads(grads)
    st = _lib.whale_fusion_layer_backward(ctypes.byref(cfg), _ptr(tokens_in), _ptr(layer_states), _ptr(seq_offsets),
                                          ctypes.byref(lw), _ptr(d_out), _ptr(d_tokens), _ptr(d_states),
                                          ctypes.byref(gr), ctypes.byref(hint), _ptr(workspace),
                                          _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_fusion_layer_backward")


def whale_fusion_backward(cfg, wukong_tokens, seq_states, seq_offsets, weights, d_out, d_tokens, d_states, grads,
                          hint, workspace, workspace_bytes=None, stream=None, raw=False):
    """Gradients of the whole stack (see include/whale_fusion.h): `weights` one dict per layer (raw),
    `grads` one dict of fp32 tensors per layer."""
    w = weights if isinstance(weights, ctypes.Array) else weights_array(weights)
    g = (whale_layer_grads * len(grads))(*[layer_grads(x) for x in grads])
    st = _lib.whale_fusion_backward(ctypes.byref(cfg), _ptr(wukong_tokens), _ptr(seq_states), _ptr(seq_offsets), w,
                                    _ptr(d_out), _ptr(d_tokens), _ptr(d_states), g, ctypes.byref(hint),
                                    _ptr(workspace), _ws_bytes(workspace, workspace_bytes), _stream(stream))
    if raw:
        return st
    _check(st, "whale_fusion_backward")


def whale_test_bounded_waits(limit_ns: int, stream=None, raw=False):
    """Enqueue the self-test of the bounded device waits (see include/whale_fusion.h)."""
    st = _lib.whale_test_bounded_waits(int(limit_ns), _stream(stream))
    if raw:
        return st
    _check(st, "whale_test_bounded_waits")


def whale_get_device_error(stream=None) -> int:
    code = c_int(0)
    st = _lib.whale_get_device_error(_stream(stream), ctypes.byref(code))
    if st not in (0, 5):
        _check(st, "whale_get_device_error")
    return code.value


# ------------------------------------------------------------------------------------------------
# norm and rotation, cached histories: descriptors (each keeps its tensors alive) and entry points
# ------------------------------------------------------------------------------------------------
def _rows_of(name, t, dtypes, ndim=2, device=None):
    """Checks a tensor that the library reads as rows: innermost stride 1, on the current device. Returns it."""
    if t.dtype not in dtypes or t.dim() != ndim:
        raise ValueError(f"{name}: {ndim} dimensions of {' or '.join(map(str, dtypes))} expected, got {t.dim()} of {t.dtype}")
    if t.numel() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if device is None:
        import torch
        device = torch.cuda.current_device()
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, not on the current CUDA device")
    return t


def _stream_on(stream):
    """(stream handle, device of the call; None: the current one, not looked up)."""
    if stream is None:
        import torch
        device = torch.cuda.current_device()  # given to current_stream, it halves the look-up (1.5 us for 3.2)
        return torch.cuda.current_stream(device).cuda_stream, device
    return _stream(stream), None


def _same_device(device, workspace, *parts):
    """Descriptors and workspace are on the device that the call runs on (None: the current one); when a descriptor was
    made another may have been current. Those that were filled in by hand are not looked at."""
    for p in parts:
        if p is not None and p._device != device and p._device is not None:
            device = _on(p._device, device)
    if workspace is not None and not isinstance(workspace, int) and workspace.get_device() != device:
        _on(workspace.get_device(), device)


def _on(made, device):
    if device is None:
        import torch
        device = torch.cuda.current_device()
    if made != device:
        raise ValueError(f"tensors on device {made}, a call on device {device}")
    return device


def _ld(t) -> int:
    return int(t.stride(0)) if t.shape[0] > 1 and t.shape[1] > 0 else int(t.shape[1])


def _ints(name, t, n=None):
    import torch
    _rows_of(name, t, (torch.int32,), 1)
    if n is not None and t.numel() != n:
        raise ValueError(f"{name}: {n} entries expected, got {t.numel()}")
    return t


def make_rotary(rotary_dim, base=10000.0, layout=WHALE_ROTATE_HALVES) -> whale_rotary:
    return whale_rotary(int(rotary_dim), int(layout), float(base))


def head_rows(x, gain, positions, y=None) -> whale_head_rows:
    """The queries (or keys) of one norm-and-rotation call: x and y [rows, n_heads * d_head] (any row
    stride), gain fp32 [d_head], positions int32 [rows]. y is the forward's output (x itself: in place)."""
    import torch
    _rows_of("x", x, (torch.bfloat16, torch.float32))
    _rows_of("gain", gain, (torch.float32,), 1)
    _ints("positions", positions, x.shape[0])
    if x.shape[1] < gain.numel() or gain.numel() == 0 or x.shape[1] % gain.numel():
        raise ValueError(f"x: {x.shape[1]} columns are no whole number of heads of {gain.numel()}")
    if y is not None:
        _rows_of("y", y, (x.dtype,))
        if y.shape != x.shape:
            raise ValueError(f"y: {tuple(y.shape)} for x {tuple(x.shape)}")
    r = whale_head_rows(_ptr(x), _ptr(y), _ptr(gain), _ptr(positions), x.shape[0], _ld(x), 0 if y is None else _ld(y),
                        x.shape[1] // gain.numel())
    r._keepalive, r._device = (x, gain, positions, y), x.get_device()
    return r


def head_grads(dy, dx, d_gain) -> whale_head_grads:
    """The gradients of one part: dy and dx [rows, n_heads * d_head] of the call's grad_dtype, d_gain fp32 [d_head]."""
    import torch
    _rows_of("dy", dy, (torch.bfloat16, torch.float32))
    _rows_of("dx", dx, (dy.dtype,))
    _rows_of("d_gain", d_gain, (torch.float32,), 1)
    if dx.shape != dy.shape:
        raise ValueError(f"dx: {tuple(dx.shape)} for dy {tuple(dy.shape)}")
    r = whale_head_grads(_ptr(dy), _ptr(dx), _ptr(d_gain), _ld(dy), _ld(dx))
    r._keepalive, r._device = (dy, dx, d_gain), dy.get_device()
    return r


def _types(cfg, rows, grads=None, grad_dtype=None):
    """Rows and gradients agree with the call's types and with each other (the C ABI cannot see a tensor's type)."""
    import torch
    for r, g in zip(rows, grads or (None,) * len(rows)):
        if r is None or not hasattr(r, "_keepalive"):
            continue
        x, gain = r._keepalive[:2]
        if x.dtype != (torch.bfloat16 if cfg.dtype == WHALE_BF16 else torch.float32):
            raise ValueError(f"rows of {x.dtype} for this configuration's type")
        if gain.numel() * cfg.n_heads != cfg.d:
            raise ValueError(f"gain: {gain.numel()} entries for d_head {cfg.d // max(cfg.n_heads, 1)}")
        if g is not None and hasattr(g, "_keepalive"):
            dy, _, dg = g._keepalive
            if dy.dtype != (torch.bfloat16 if grad_dtype == WHALE_BF16 else torch.float32) or dy.shape != x.shape \
                    or dg.numel() != gain.numel():
                raise ValueError(f"gradients {tuple(dy.shape)} of {dy.dtype} for rows {tuple(x.shape)}")


def _ref(s):
    return None if s is None else ctypes.byref(s)


def whale_norm_rotate(cfg, rotary, q, k, stream=None, raw=False):
    """Per-head RMS norm and rotation by position (see include/whale_fusion.h); q, k: head_rows or None."""
    handle, device = _stream_on(stream)
    _types(cfg, (q, k))
    _same_device(device, None, q, k)
    st = _lib.whale_norm_rotate(ctypes.byref(cfg), ctypes.byref(rotary), _ref(q), _ref(k), handle)
    if raw:
        return st
    _check(st, "whale_norm_rotate")


def whale_norm_rotate_workspace_size(cfg, q, k) -> int:
    return int(_lib.whale_norm_rotate_workspace_size(ctypes.byref(cfg), _ref(q), _ref(k)))


def whale_norm_rotate_backward(cfg, rotary, q, k, dq, dk, grad_dtype, workspace, workspace_bytes=None, stream=None,
                               raw=False):
    handle, device = _stream_on(stream)
    _types(cfg, (q, k), (dq, dk), grad_dtype)
    _same_device(device, workspace, q, k, dq, dk)
    st = _lib.whale_norm_rotate_backward(ctypes.byref(cfg), ctypes.byref(rotary), _ref(q), _ref(k), _ref(dq), _ref(dk),
                                         int(grad_dtype), _ptr(workspace), _ws_bytes(workspace, workspace_bytes), handle)
    if raw:
        return st
    _check(st, "whale_norm_rotate_backward")


def make_cache(pages, scales=None) -> whale_cache:
    """A cache over pages [n_pages, planes, n_kv_heads, page_size, d_head] (bf16, or e4m3 as uint8 or
    float8_e4m3fn with scales uint8 [n_pages, planes, n_kv_heads, page_size]); both contiguous."""
    import torch
    e4m3 = scales is not None
    _rows_of("pages", pages, (torch.uint8, torch.float8_e4m3fn) if e4m3 else (torch.bfloat16,), 5)
    if e4m3:
        _rows_of("scales", scales, (torch.uint8,), 4)
        if scales.shape != pages.shape[:4]:
            raise ValueError(f"scales: {tuple(scales.shape)} for pages {tuple(pages.shape)}")
    if not pages.is_contiguous() or (e4m3 and not scales.is_contiguous()):
        raise ValueError("pages and scales must be contiguous")
    k = whale_cache(_ptr(pages), _ptr(scales), pages.shape[0], pages.shape[3], pages.shape[2],
                    WHALE_CACHE_E4M3 if e4m3 else WHALE_CACHE_BF16)
    k._keepalive, k._device = (pages, scales), pages.get_device()
    return k


def make_chunk(offsets, lengths, page_table, max_new, max_length, total_new) -> whale_chunk:
    """A batch of sequences (see whale_chunk): offsets int32 [B+1], lengths int32 [B], page_table int32
    [B, table_stride], and the host's bounds of rows per sequence, of lengths, and of rows in all."""
    import torch
    _ints("lengths", lengths)
    _ints("offsets", offsets, lengths.numel() + 1)
    _rows_of("page_table", page_table, (torch.int32,))
    if page_table.shape[0] != lengths.numel():
        raise ValueError(f"page_table: {page_table.shape[0]} sequences, lengths has {lengths.numel()}")
    if not page_table.is_contiguous():
        raise ValueError("page_table must be contiguous")
    c = whale_chunk(_ptr(offsets), _ptr(lengths), _ptr(page_table), page_table.shape[1], lengths.numel(), int(max_new),
                    int(max_length), int(total_new))
    c._keepalive, c._device = (offsets, lengths, page_table), offsets.get_device()
    return c


def _packed(name, t, cfg, cache, chunk, width, device):
    """A packed [total_new, width] bf16 tensor's row stride, and the cache's planes and d_head, checked."""
    import torch
    if isinstance(t, int) or t is None:
        return width
    _rows_of(name, t, (torch.bfloat16,), 2, device)
    if t.shape[0] < chunk.total_new or t.shape[1] != width:
        raise ValueError(f"{name}: {tuple(t.shape)}, [{chunk.total_new}, {width}] expected")
    pages = getattr(cache, "_keepalive", (None,))[0]
    if pages is not None and (pages.shape[4] * cfg.n_heads != cfg.d
                              or pages.shape[1] != (1 if cfg.flags & WHALE_SHARED_KV else 2)):
        raise ValueError(f"pages {tuple(pages.shape)} do not fit the configuration")
    return _ld(t)


def _kv_width(cfg, cache):
    return (1 if cfg.flags & WHALE_SHARED_KV else 2) * cache.n_kv_heads * (cfg.d // max(cfg.n_heads, 1))


def whale_cache_pages_size(cfg, cache) -> int:
    return int(_lib.whale_cache_pages_size(ctypes.byref(cfg), ctypes.byref(cache)))


def whale_cache_scales_size(cfg, cache) -> int:
    return int(_lib.whale_cache_scales_size(ctypes.byref(cfg), ctypes.byref(cache)))


def whale_cache_append(cfg, cache, chunk, kv, stream=None, raw=False):
    """Write the chunk's K|V rows to the cache, in its format."""
    handle, device = _stream_on(stream)
    _same_device(device, None, cache, chunk)
    ld = _packed("kv", kv, cfg, cache, chunk, _kv_width(cfg, cache), device)
    st = _lib.whale_cache_append(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(chunk), _ptr(kv), ld, handle)
    if raw:
        return st
    _check(st, "whale_cache_append")


def whale_cache_read(cfg, cache, chunk, kv, stream=None, raw=False):
    """Read the chunk's K|V rows back from the cache, as bf16."""
    handle, device = _stream_on(stream)
    _same_device(device, None, cache, chunk)
    ld = _packed("kv", kv, cfg, cache, chunk, _kv_width(cfg, cache), device)
    st = _lib.whale_cache_read(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(chunk), _ptr(kv), ld, handle)
    if raw:
        return st
    _check(st, "whale_cache_read")


def whale_cache_attention_workspace_size(cfg, cache, chunk) -> int:
    return int(_lib.whale_cache_attention_workspace_size(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(chunk)))


def whale_cache_attention(cfg, cache, chunk, q, a, workspace, workspace_bytes=None, flags=0, stream=None, raw=False):
    """Attention of the chunk's rows q over the cached histories (flags: WHALE_ATTEND_CAUSAL) into a."""
    handle, device = _stream_on(stream)
    _same_device(device, workspace, cache, chunk)
    ldq, lda = _packed("q", q, cfg, cache, chunk, cfg.d, device), _packed("a", a, cfg, cache, chunk, cfg.d, device)
    st = _lib.whale_cache_attention(ctypes.byref(cfg), ctypes.byref(cache), ctypes.byref(chunk), _ptr(q), ldq, _ptr(a),
                                    lda, int(flags), _ptr(workspace), _ws_bytes(workspace, workspace_bytes), handle)
    if raw:
        return st
    _check(st, "whale_cache_attention")
