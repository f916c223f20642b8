"""ctypes binding of libfp8mlp.so (include/fp8mlp.h), same names as the C ABI.

Argument marshalling only: torch tensors are passed as their device pointers
(after a contiguity/device check), streams as their CUDA handles, and a
non-zero return code raises :class:`Fp8MlpError` with the library's detail
text.  Every step of the computation runs in the library's CUDA kernels;
there is no fallback: if the library cannot be loaded, importing this module
raises.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8mlp.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "fp8mlp.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m fp8_relu_mlp_b200.build`")
lib = ctypes.CDLL(LIB_PATH)

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED_SHAPE = 2
ERR_CUDA = 3
ERR_TIMEOUT = 4
ERR_NO_DEVICE = 5
STATUS_TIMEOUT = 1
STATUS_NONFINITE_AMAX = 2
STATUS_W2_DEGENERATE = 4
STATUS_STEP_SKIPPED = 8
STATE_KEPT_SCALE = 1
FWD_EVAL_BF16 = 1
FWD_CALIBRATE = 2
CE_SUM = 0
CE_MEAN = 1
LAUNCH_OVERLAP_PREVIOUS = 1
DEBUG_STALL_PRODUCER = 1
DEBUG_STALL_AUX = 2
E4M3_MAX = 448.0


class Fp8MlpError(RuntimeError):
    def __init__(self, code, fn):
        self.code = code
        detail = lib.fp8mlp_last_error_detail().decode()
        msg = lib.fp8mlp_error_string(code).decode()
        super().__init__(f"{fn}: {msg} ({code}){': ' + detail if detail else ''}")


_i, _u64, _f, _p, _sz = ctypes.c_int, ctypes.c_ulonglong, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_u32 = ctypes.c_uint32

_SIGS = {
    "fp8mlp_up_proj_fused": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _i, _p],
    "fp8mlp_down_proj_fp8": [_i, _i, _i, _p, _p, _p, _p, _p, _p],
    "fp8mlp_down_proj_bf16": [_i, _i, _i, _p, _p, _p, _p],
    "fp8mlp_mlp_fwd": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _p],
    "fp8mlp_partial_amax_shape": [_i, _i, _p, _p, _p, _p],
    "fp8mlp_partial_amax_count": [_i, _i],
    "fp8mlp_mlp_train_step": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_scale_state_init": [_p, _f, _f, _p],
    "fp8mlp_amax_reduce_update_scale": [_p, _i, _p, _p],
    "fp8mlp_w2_fp8_cache_refresh": [_i, _i, _p, _p, _p, _p, _p],
    "fp8mlp_w2_fp8_cache_refresh_noalloc": [_i, _i, _p, _p, _p, _p],
    "fp8mlp_bwd_dpre": [_i, _i, _i, _p, _p, _p, _p, _i, _p],
    "fp8mlp_quantize_x": [_i, _i, _p, _p, _p, _p, _p],
    "fp8mlp_x_partial_amax_count": [_i, _i],
    "fp8mlp_w1_fp8_cache_refresh": [_i, _i, _p, _p, _p, _p, _p],
    "fp8mlp_up_proj_fused_fp8": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i, _p],
    "fp8mlp_linear_fwd_fp8": [_i, _i, _i, _p, _p, _p, _p, _p, _p],
    "fp8mlp_weight_fp8_cache_refresh": [_i, _i, _p, _p, _p, _p, _p],
    "fp8mlp_linear_bwd": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _i, _p],
    "fp8mlp_ce_fwd": [_i, _i, _i, _i, _p, _p, _p, _p, _f, _p, _p, _p, _p, _p],
    "fp8mlp_ce_fwd_fp8": [_i, _i, _i, _i, _p, _p, _p, _p, _p, _p, _f, _p, _p, _p, _p, _p],
    "fp8mlp_ce_bwd_dlogits": [_i, _i, _i, _i, _p, _p, _p, _p, _f, _p, _p, _p, _i, _p, _p],
    "fp8mlp_ce_bwd_dlogits_fp8": [_i, _i, _i, _i, _p, _p, _p, _p, _p, _p, _f, _p, _p, _p, _i, _p, _p],
    "fp8mlp_bwd_dx": [_i, _i, _i, _p, _p, _p, _p],
    "fp8mlp_bwd_dw": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _i, _p],
    "fp8mlp_mlp_bwd": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_rmsnorm_fwd": [_i, _i, _p, _p, _p, _p],
    "fp8mlp_rmsnorm_fwd_quant": [_i, _i, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_rmsnorm_bwd": [_i, _i, _p, _p, _p, _p, _p, _p],
    "fp8mlp_residual_add": [_i, _i, _p, _p, _p, _p],
    "fp8mlp_quantize_block": [_i, _i, _p, _p, _p, _p],
    "fp8mlp_weight_block_cache_refresh": [_i, _i, _p, _p, _p, _p, _p, _p],
    "fp8mlp_linear_fwd_block": [_i, _i, _i, _p, _p, _p, _p, _p, _p],
    "fp8mlp_linear_block": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_up_proj_block": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_mlp_fwd_block": [_i, _i, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_norm_gate_fwd": [_i, _i, _p, _p, _p, _p, _i, _p, _p, _f, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_norm_gate_bwd": [_i, _i, _p, _p, _p, _p, _i, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p],
    "fp8mlp_adamw_state_init": [_p, _f, _u32, _i, _p],
    "fp8mlp_grad_norm": [_i, _p, _f, _p, _p, _p],
    "fp8mlp_adamw_check": [_i, _p, _p, _i, _p],
    "fp8mlp_adamw_step": [_i, _p, _p, _i, _f, _f, _f, _p, _p],
    "fp8mlp_get_device_status": [_p, _p],
    "fp8mlp_clear_device_status": [_p],
    "fp8mlp_set_wait_timeout_ns": [_u64],
    "fp8mlp_set_debug_flags": [_i],
    "fp8mlp_set_programmatic_launch": [_i],
}
for _n, _a in _SIGS.items():
    _fn = getattr(lib, _n)
    _fn.argtypes = _a
    _fn.restype = ctypes.c_int
lib.fp8mlp_workspace_size.argtypes = [_i, _i, _i]
lib.fp8mlp_workspace_size.restype = _sz
lib.fp8mlp_ce_workspace_size.argtypes = [_i, _i, _i]
lib.fp8mlp_ce_workspace_size.restype = _sz
lib.fp8mlp_linear_bwd_workspace_size.argtypes = [_i, _i, _i]
lib.fp8mlp_linear_bwd_workspace_size.restype = _sz
lib.fp8mlp_norm_gate_bwd_workspace_size.argtypes = [_i, _i, _i]
lib.fp8mlp_norm_gate_bwd_workspace_size.restype = _sz
lib.fp8mlp_grad_norm_workspace_size.argtypes = [_i, _p]
lib.fp8mlp_grad_norm_workspace_size.restype = _sz
lib.fp8mlp_kernel_launch_count.argtypes = []
lib.fp8mlp_kernel_launch_count.restype = ctypes.c_ulonglong
for _n in ("fp8mlp_error_string",):
    getattr(lib, _n).argtypes = [_i]
    getattr(lib, _n).restype = ctypes.c_char_p
for _n in ("fp8mlp_last_error_detail", "fp8mlp_version"):
    getattr(lib, _n).argtypes = []
    getattr(lib, _n).restype = ctypes.c_char_p


def header_symbols() -> list[str]:
    """Every function the public header declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"\b(fp8mlp_[a-z0-9_]+)\s*\(", text)))


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("tensor arguments must be contiguous")
        return t.data_ptr()
    raise TypeError(f"cannot pass {type(t)} as a pointer")


_current = None  # () -> (device index, raw stream of the current stream); set once a GPU has been seen


def _find_current():
    """Sets ``_current``.  torch's own accessors build a Stream object per call
    and ask again whether there is a GPU, several microseconds; the ones below
    them are taken where this torch has them."""
    global _current
    import torch
    if not torch.cuda.is_available():
        return False
    torch.cuda.current_stream()  # initialises the context
    get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def fast():
        d = get_device()
        return d, raw(d)

    def plain():
        return torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream

    _current = plain if raw is None else fast
    _find_marshal(torch)
    return True


_marshal = None  # the compiled marshalling of the per-layer calls; set with _current


def _find_marshal(torch):
    """Sets ``_marshal`` where the module is built, for this very torch."""
    global _marshal
    try:
        from . import _marshal as m
    except ImportError:
        return
    if m.TORCH_VERSION != torch.__version__.split("+")[0]:
        return
    for name in m.names():
        m.bind(name, ctypes.cast(getattr(lib, name), _p).value)
    _marshal = m


def _done(rc, name):
    if rc != OK:
        raise Fp8MlpError(rc, name)
    return rc


def _stream(s):
    if s is None:
        try:
            if _current is not None or _find_current():
                return _current()[1]
        except Exception:
            pass
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


_functions = {}


def _call(name, *args):
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(lib, name)
    rc = fn(*args)
    if rc != OK:
        raise Fp8MlpError(rc, name)
    return rc


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def fp8mlp_up_proj_fused(M, d, h, x, W1, st, post, post_fp8, partial_amax, pre_debug=None, flags=0, stream=None):
    return _call("fp8mlp_up_proj_fused", M, d, h, _ptr(x), _ptr(W1), _ptr(st), _ptr(post), _ptr(post_fp8),
                 _ptr(partial_amax), _ptr(pre_debug), flags, _stream(stream))


def fp8mlp_down_proj_fp8(M, d, h, post_fp8, W2q_t, w2_scale_inv, st, out, stream=None):
    return _call("fp8mlp_down_proj_fp8", M, d, h, _ptr(post_fp8), _ptr(W2q_t), _ptr(w2_scale_inv), _ptr(st),
                 _ptr(out), _stream(stream))


def fp8mlp_down_proj_bf16(M, d, h, post, W2, out, stream=None):
    return _call("fp8mlp_down_proj_bf16", M, d, h, _ptr(post), _ptr(W2), _ptr(out), _stream(stream))


def fp8mlp_mlp_fwd(M, d, h, x, W1, W2q_t, w2_scale_inv, W2, st, post, post_fp8, partial_amax, out,
                   pre_debug=None, flags=0, stream=None):
    return _call("fp8mlp_mlp_fwd", M, d, h, _ptr(x), _ptr(W1), _ptr(W2q_t), _ptr(w2_scale_inv), _ptr(W2),
                 _ptr(st), _ptr(post), _ptr(post_fp8), _ptr(partial_amax), _ptr(out), _ptr(pre_debug), flags,
                 _stream(stream))


def fp8mlp_partial_amax_shape(M, h):
    """-> (row_blocks, col_blocks, block_rows, block_cols)"""
    v = [ctypes.c_int() for _ in range(4)]
    _call("fp8mlp_partial_amax_shape", M, h, *[ctypes.addressof(x) for x in v])
    return tuple(x.value for x in v)


def fp8mlp_mlp_train_step(M, d, h, x, W1, W2, dOut, W2q_t, w2_scale_inv, st, post, post_fp8, partial_amax, out,
                          dPre, dX, dW1, dW2, workspace, stream=None):
    return _call("fp8mlp_mlp_train_step", M, d, h, _ptr(x), _ptr(W1), _ptr(W2), _ptr(dOut), _ptr(W2q_t),
                 _ptr(w2_scale_inv), _ptr(st), _ptr(post), _ptr(post_fp8), _ptr(partial_amax), _ptr(out), _ptr(dPre),
                 _ptr(dX), _ptr(dW1), _ptr(dW2), _ptr(workspace), _stream(stream))


def fp8mlp_partial_amax_count(M, h):
    return int(lib.fp8mlp_partial_amax_count(M, h))


def fp8mlp_scale_state_init(st, margin, initial_scale, stream=None):
    return _call("fp8mlp_scale_state_init", _ptr(st), margin, initial_scale, _stream(stream))


def fp8mlp_amax_reduce_update_scale(partial_amax, n, st, stream=None):
    return _call("fp8mlp_amax_reduce_update_scale", _ptr(partial_amax), n, _ptr(st), _stream(stream))


def fp8mlp_w2_fp8_cache_refresh(h, d, W2, W2q_t, w2_scale_inv, workspace, stream=None):
    return _call("fp8mlp_w2_fp8_cache_refresh", h, d, _ptr(W2), _ptr(W2q_t), _ptr(w2_scale_inv), _ptr(workspace),
                 _stream(stream))


def fp8mlp_w2_fp8_cache_refresh_noalloc(h, d, W2, W2q_t, w2_scale_inv, stream=None):
    """W2 cache refresh without a workspace: for callers that cannot hand the
    library device memory (see include/fp8mlp.h)."""
    return _call("fp8mlp_w2_fp8_cache_refresh_noalloc", h, d, _ptr(W2), _ptr(W2q_t), _ptr(w2_scale_inv),
                 _stream(stream))


def fp8mlp_workspace_size(M, d, h):
    return int(lib.fp8mlp_workspace_size(M, d, h))


def fp8mlp_quantize_x(M, d, x, st_x, x_fp8, partial_amax_x, stream=None):
    return _call("fp8mlp_quantize_x", M, d, _ptr(x), _ptr(st_x), _ptr(x_fp8), _ptr(partial_amax_x), _stream(stream))


def fp8mlp_x_partial_amax_count(M, d):
    return int(lib.fp8mlp_x_partial_amax_count(M, d))


def fp8mlp_w1_fp8_cache_refresh(h, d, W1, W1q, w1_scale_inv, workspace, stream=None):
    return _call("fp8mlp_w1_fp8_cache_refresh", h, d, _ptr(W1), _ptr(W1q), _ptr(w1_scale_inv), _ptr(workspace),
                 _stream(stream))


def fp8mlp_up_proj_fused_fp8(M, d, h, x_fp8, W1q, w1_scale_inv, st_x, st, post, post_fp8, partial_amax,
                             pre_debug=None, flags=0, stream=None):
    return _call("fp8mlp_up_proj_fused_fp8", M, d, h, _ptr(x_fp8), _ptr(W1q), _ptr(w1_scale_inv), _ptr(st_x),
                 _ptr(st), _ptr(post), _ptr(post_fp8), _ptr(partial_amax), _ptr(pre_debug), flags, _stream(stream))


def fp8mlp_linear_fwd_fp8(M, K, N, x_fp8, Wq, w_scale_inv, st_x, y, stream=None):
    return _call("fp8mlp_linear_fwd_fp8", M, K, N, _ptr(x_fp8), _ptr(Wq), _ptr(w_scale_inv), _ptr(st_x), _ptr(y),
                 _stream(stream))


def fp8mlp_weight_fp8_cache_refresh(N, K, W, Wq, w_scale_inv, workspace, stream=None):
    return _call("fp8mlp_weight_fp8_cache_refresh", N, K, _ptr(W), _ptr(Wq), _ptr(w_scale_inv), _ptr(workspace),
                 _stream(stream))


def fp8mlp_linear_bwd_workspace_size(M, K, N):
    return int(lib.fp8mlp_linear_bwd_workspace_size(M, K, N))


def fp8mlp_linear_bwd(M, K, N, x, W, dY, dX, dW, flags=0, stream=None, workspace=None):
    return _call("fp8mlp_linear_bwd", M, K, N, _ptr(x), _ptr(W), _ptr(dY), _ptr(dX), _ptr(dW), _ptr(workspace), flags,
                 _stream(stream))


def _host_floats(seq):
    """A host float array for a C `const float*` (None stays NULL); the
    returned object must stay alive for the call."""
    if seq is None:
        return None
    vals = [float(v) for v in seq]
    return (ctypes.c_float * len(vals))(*vals)


def fp8mlp_ce_workspace_size(M, V, T):
    return int(lib.fp8mlp_ce_workspace_size(M, V, T))


def fp8mlp_ce_fwd(M, d, V, T, x, W, targets, target_weights, softcap, lse, row_loss, loss, workspace, stream=None):
    w = _host_floats(target_weights)
    return _call("fp8mlp_ce_fwd", M, d, V, T, _ptr(x), _ptr(W), _ptr(targets), ctypes.cast(w, _p) if w else None,
                 softcap, _ptr(lse), _ptr(row_loss), _ptr(loss), _ptr(workspace), _stream(stream))


def fp8mlp_ce_fwd_fp8(M, d, V, T, x_fp8, st_x, Wq, w_scale_inv, targets, target_weights, softcap, lse, row_loss,
                      loss, workspace, stream=None):
    w = _host_floats(target_weights)
    return _call("fp8mlp_ce_fwd_fp8", M, d, V, T, _ptr(x_fp8), _ptr(st_x), _ptr(Wq), _ptr(w_scale_inv),
                 _ptr(targets), ctypes.cast(w, _p) if w else None, softcap, _ptr(lse), _ptr(row_loss), _ptr(loss),
                 _ptr(workspace), _stream(stream))


def fp8mlp_ce_bwd_dlogits(M, d, V, T, x, W, targets, target_weights, softcap, lse, loss, dloss, reduction, dlogits,
                          stream=None):
    w = _host_floats(target_weights)
    return _call("fp8mlp_ce_bwd_dlogits", M, d, V, T, _ptr(x), _ptr(W), _ptr(targets),
                 ctypes.cast(w, _p) if w else None, softcap, _ptr(lse), _ptr(loss), _ptr(dloss), reduction,
                 _ptr(dlogits), _stream(stream))


def fp8mlp_ce_bwd_dlogits_fp8(M, d, V, T, x_fp8, st_x, Wq, w_scale_inv, targets, target_weights, softcap, lse, loss,
                              dloss, reduction, dlogits, stream=None):
    w = _host_floats(target_weights)
    return _call("fp8mlp_ce_bwd_dlogits_fp8", M, d, V, T, _ptr(x_fp8), _ptr(st_x), _ptr(Wq), _ptr(w_scale_inv),
                 _ptr(targets), ctypes.cast(w, _p) if w else None, softcap, _ptr(lse), _ptr(loss), _ptr(dloss),
                 reduction, _ptr(dlogits), _stream(stream))


def fp8mlp_bwd_dpre(M, d, h, dOut, W2, post, dPre, flags=0, stream=None):
    return _call("fp8mlp_bwd_dpre", M, d, h, _ptr(dOut), _ptr(W2), _ptr(post), _ptr(dPre), flags, _stream(stream))


def fp8mlp_bwd_dx(M, d, h, dPre, W1, dX, stream=None):
    return _call("fp8mlp_bwd_dx", M, d, h, _ptr(dPre), _ptr(W1), _ptr(dX), _stream(stream))


def fp8mlp_bwd_dw(M, d, h, x, dPre, post, dOut, dW1, dW2, flags=0, stream=None):
    return _call("fp8mlp_bwd_dw", M, d, h, _ptr(x), _ptr(dPre), _ptr(post), _ptr(dOut), _ptr(dW1), _ptr(dW2),
                 flags, _stream(stream))


def fp8mlp_mlp_bwd(M, d, h, x, W1, W2, post, dOut, dPre, dX, dW1, dW2, stream=None):
    return _call("fp8mlp_mlp_bwd", M, d, h, _ptr(x), _ptr(W1), _ptr(W2), _ptr(post), _ptr(dOut), _ptr(dPre),
                 _ptr(dX), _ptr(dW1), _ptr(dW2), _stream(stream))


def fp8mlp_rmsnorm_fwd_quant(M, d, r, x, rstd, st_x, x_fp8, row_amax, stream=None):
    return _call("fp8mlp_rmsnorm_fwd_quant", M, d, _ptr(r), _ptr(x), _ptr(rstd), _ptr(st_x), _ptr(x_fp8),
                 _ptr(row_amax), _stream(stream))


def fp8mlp_rmsnorm_fwd(M, d, r, x, rstd, stream=None):
    return _call("fp8mlp_rmsnorm_fwd", M, d, _ptr(r), _ptr(x), _ptr(rstd), _stream(stream))


def fp8mlp_rmsnorm_bwd(M, d, r, rstd, dx, dr_in, dr_out, stream=None):
    return _call("fp8mlp_rmsnorm_bwd", M, d, _ptr(r), _ptr(rstd), _ptr(dx), _ptr(dr_in), _ptr(dr_out),
                 _stream(stream))


def fp8mlp_residual_add(M, d, r, out, r_next, stream=None):
    return _call("fp8mlp_residual_add", M, d, _ptr(r), _ptr(out), _ptr(r_next), _stream(stream))


# ---------------------------------------------------------------------------
# block-scaled FP8 products, gated norms, optimizer.  Tensors of these calls
# are also held to their sizes and to the current device: a kernel that is
# handed a short buffer, or one of another GPU, would write out of bounds.
# ---------------------------------------------------------------------------

def _here(stream):
    """Current device (None without a GPU) and the raw stream of a call."""
    dev, raw = (_current or _no_gpu)()
    if stream is None:
        return dev, raw
    return dev, _address(stream if stream.__class__ is int else stream.cuda_stream, "stream")


def _address(v, name):
    """An int that ctypes would cut to 64 bits is refused."""
    if v.__class__ is int and not -(1 << 63) <= v < 1 << 64:
        raise OverflowError(f"{name}: an address has 64 bits")
    return v


def _buf(t, need, name, dev):
    """Device address of ``t`` with at least ``need`` bytes on device ``dev``
    (None stays NULL; an int is an address the caller vouches for)."""
    if t is None or t.__class__ is int:
        return _address(t, name)
    try:
        ok = t.is_contiguous() and t.nbytes >= need and t.get_device() == dev
    except AttributeError:
        raise TypeError(f"{name}: cannot pass {type(t)} as a pointer") from None
    if not ok:
        _refuse(t, need, name, dev)
    return t.data_ptr()


def _no_gpu():
    """Stands in for ``_current`` until a GPU has been seen."""
    return _current() if _find_current() else (None, None)


def _refuse(t, need, name, dev):
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor arguments must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is needed")
    if t.nbytes < need:
        raise ValueError(f"{name}: {need} bytes are needed, the tensor has {t.nbytes}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the current device is {dev}")


def _kblocks(n):
    return -(-n // 128)


def fp8mlp_quantize_block(M, K, x, xq, xs, stream=None):
    if _marshal is not None:
        return _done(_marshal.quantize_block(M, K, x, xq, xs, stream), "fp8mlp_quantize_block")
    dev, raw = _here(stream)
    return _call("fp8mlp_quantize_block", M, K, _buf(x, 2 * M * K, "x", dev), _buf(xq, M * K, "xq", dev),
                 _buf(xs, 4 * M * _kblocks(K), "xs", dev), raw)


def fp8mlp_weight_block_cache_refresh(N, K, W, Wq, ws, Wq_t=None, ws_t=None, stream=None):
    if _marshal is not None:
        return _done(_marshal.weight_block_cache_refresh(N, K, W, Wq, ws, Wq_t, ws_t,
                                                         stream), "fp8mlp_weight_block_cache_refresh")
    dev, raw = _here(stream)
    sc = 4 * _kblocks(K) * _kblocks(N)
    return _call("fp8mlp_weight_block_cache_refresh", N, K, _buf(W, 2 * N * K, "W", dev), _buf(Wq, N * K, "Wq", dev),
                 _buf(ws, sc, "ws", dev), _buf(Wq_t, N * K, "Wq_t", dev), _buf(ws_t, sc, "ws_t", dev), raw)


def fp8mlp_linear_fwd_block(M, K, N, xq, xs, Wq, ws, y, stream=None):
    if _marshal is not None:
        return _done(_marshal.linear_fwd_block(M, K, N, xq, xs, Wq, ws, y, stream), "fp8mlp_linear_fwd_block")
    dev, raw = _here(stream)
    kb = _kblocks(K)
    return _call("fp8mlp_linear_fwd_block", M, K, N, _buf(xq, M * K, "xq", dev), _buf(xs, 4 * M * kb, "xs", dev),
                 _buf(Wq, N * K, "Wq", dev), _buf(ws, 4 * kb * _kblocks(N), "ws", dev), _buf(y, 2 * M * N, "y", dev),
                 raw)


def fp8mlp_linear_block(M, K, N, x, Wq, ws, xq, xs, y, stream=None):
    if _marshal is not None:
        return _done(_marshal.linear_block(M, K, N, x, Wq, ws, xq, xs, y, stream), "fp8mlp_linear_block")
    dev, raw = _here(stream)
    kb = _kblocks(K)
    return _call("fp8mlp_linear_block", M, K, N, _buf(x, 2 * M * K, "x", dev), _buf(Wq, N * K, "Wq", dev),
                 _buf(ws, 4 * kb * _kblocks(N), "ws", dev), _buf(xq, M * K, "xq", dev), _buf(xs, 4 * M * kb, "xs", dev),
                 _buf(y, 2 * M * N, "y", dev), raw)


def fp8mlp_up_proj_block(M, d, h, xq, xs, W1q, w1s, post, post_q, post_s, stream=None):
    if _marshal is not None:
        return _done(_marshal.up_proj_block(M, d, h, xq, xs, W1q, w1s, post, post_q, post_s,
                                            stream), "fp8mlp_up_proj_block")
    dev, raw = _here(stream)
    kd, kh = _kblocks(d), _kblocks(h)
    return _call("fp8mlp_up_proj_block", M, d, h, _buf(xq, M * d, "xq", dev), _buf(xs, 4 * M * kd, "xs", dev),
                 _buf(W1q, h * d, "W1q", dev), _buf(w1s, 4 * kd * kh, "w1s", dev), _buf(post, 2 * M * h, "post", dev),
                 _buf(post_q, M * h, "post_q", dev), _buf(post_s, 4 * M * kh, "post_s", dev), raw)


def fp8mlp_mlp_fwd_block(M, d, h, x, W1q, w1s, W2q_t, w2s_t, xq, xs, post, post_q, post_s, out, stream=None):
    if _marshal is not None:
        return _done(_marshal.mlp_fwd_block(M, d, h, x, W1q, w1s, W2q_t, w2s_t, xq, xs, post, post_q, post_s, out,
                                            stream), "fp8mlp_mlp_fwd_block")
    dev, raw = _here(stream)
    kd, kh = _kblocks(d), _kblocks(h)
    return _call("fp8mlp_mlp_fwd_block", M, d, h, _buf(x, 2 * M * d, "x", dev), _buf(W1q, h * d, "W1q", dev),
                 _buf(w1s, 4 * kd * kh, "w1s", dev), _buf(W2q_t, h * d, "W2q_t", dev), _buf(w2s_t, 4 * kd * kh, "w2s_t", dev),
                 _buf(xq, M * d, "xq", dev), _buf(xs, 4 * M * kd, "xs", dev), _buf(post, 2 * M * h, "post", dev),
                 _buf(post_q, M * h, "post_q", dev), _buf(post_s, 4 * M * kh, "post_s", dev), _buf(out, 2 * M * d, "out", dev),
                 raw)


def _gate_rows(M, rows_per_gate):
    return -(-M // rows_per_gate) if rows_per_gate > 0 else 0


def fp8mlp_norm_gate_fwd(M, d, r, y, w_post, gate, rows_per_gate, alpha, w_pre, eps, r_next, rstd_post, x, rstd_pre,
                         xq=None, xs=None, stream=None):
    if _marshal is not None:
        return _done(_marshal.norm_gate_fwd(M, d, r, y, w_post, gate, rows_per_gate, alpha, w_pre, eps, r_next,
                                            rstd_post, x, rstd_pre, xq, xs, stream), "fp8mlp_norm_gate_fwd")
    dev, raw = _here(stream)
    n = 2 * M * d
    return _call("fp8mlp_norm_gate_fwd", M, d, _buf(r, n, "r", dev), _buf(y, n, "y", dev), _buf(w_post, 2 * d, "w_post", dev),
                 _buf(gate, 2 * d * _gate_rows(M, rows_per_gate), "gate", dev), rows_per_gate, _buf(alpha, 4, "alpha", dev),
                 _buf(w_pre, 2 * d, "w_pre", dev), eps, _buf(r_next, n, "r_next", dev), _buf(rstd_post, 4 * M, "rstd_post", dev),
                 _buf(x, n, "x", dev), _buf(rstd_pre, 4 * M, "rstd_pre", dev), _buf(xq, M * d, "xq", dev),
                 _buf(xs, 4 * M * _kblocks(d), "xs", dev), raw)


def fp8mlp_norm_gate_bwd_workspace_size(M, d, rows_per_gate):
    return int(lib.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows_per_gate))


def fp8mlp_norm_gate_bwd(M, d, r, y, w_post, gate, rows_per_gate, alpha, rstd_post, r_next, w_pre, rstd_pre, dx,
                         dr_next, dr, dy, dw_post, dgate, dalpha, dw_pre, workspace, stream=None):
    if _marshal is not None:
        return _done(_marshal.norm_gate_bwd(M, d, r, y, w_post, gate, rows_per_gate, alpha, rstd_post, r_next, w_pre,
                                            rstd_pre, dx, dr_next, dr, dy, dw_post, dgate, dalpha, dw_pre, workspace,
                                            stream), "fp8mlp_norm_gate_bwd")
    dev, raw = _here(stream)
    n, g = 2 * M * d, _gate_rows(M, rows_per_gate)
    need = int(lib.fp8mlp_norm_gate_bwd_workspace_size(M, d, rows_per_gate))
    return _call("fp8mlp_norm_gate_bwd", M, d, _buf(r, n, "r", dev), _buf(y, n, "y", dev), _buf(w_post, 2 * d, "w_post", dev),
                 _buf(gate, 2 * d * g, "gate", dev), rows_per_gate, _buf(alpha, 4, "alpha", dev),
                 _buf(rstd_post, 4 * M, "rstd_post", dev), _buf(r_next, n, "r_next", dev), _buf(w_pre, 2 * d, "w_pre", dev),
                 _buf(rstd_pre, 4 * M, "rstd_pre", dev), _buf(dx, n, "dx", dev), _buf(dr_next, n, "dr_next", dev), _buf(dr, n, "dr", dev),
                 _buf(dy, n, "dy", dev), _buf(dw_post, 4 * d, "dw_post", dev), _buf(dgate, 4 * d * g, "dgate", dev),
                 _buf(dalpha, 4, "dalpha", dev), _buf(dw_pre, 4 * d, "dw_pre", dev), _buf(workspace, need, "workspace", dev),
                 raw)


class AdamwTensor(ctypes.Structure):
    """fp8mlp_adamw_tensor"""
    _fields_ = [("n", ctypes.c_int64), ("p", _p), ("p_bf16", _p), ("g", _p), ("m", _p), ("v", _p), ("m_scale", _p),
                ("v_scale", _p), ("lr_mult", _f), ("weight_decay", _f)]


def adamw_tensor(n, p, p_bf16, g, m, v, m_scale=None, v_scale=None, lr_mult=1.0, weight_decay=0.0, state_bits=32):
    """One descriptor for :func:`fp8mlp_adamw_step`, its tensors' sizes checked.
    It holds addresses: the tensors have to stay alive."""
    dev = (_current or _no_gpu)()[0]
    sb, nb = state_bits // 8, 4 * _kblocks(n)
    t = AdamwTensor(n, _buf(p, 4 * n, "p", dev), _buf(p_bf16, 2 * n, "p_bf16", dev), _buf(g, 4 * n, "g", dev),
                    _buf(m, sb * n, "m", dev), _buf(v, sb * n, "v", dev), _buf(m_scale, nb, "m_scale", dev),
                    _buf(v_scale, nb, "v_scale", dev), lr_mult, weight_decay)
    t.state_bits = state_bits
    return t


def adamw_tensors(descriptors):
    """The array the calls below take; build it once, use it every step."""
    arr = (AdamwTensor * len(descriptors))(*descriptors)
    arr.state_bits = {t.state_bits for t in descriptors if t.m and hasattr(t, "state_bits")}  # that their sizes were held to
    return arr


def _tensors(arr):
    if not isinstance(arr, ctypes.Array) or arr._type_ is not AdamwTensor:
        raise TypeError("tensors: an array from adamw_tensors() is needed")
    return len(arr), ctypes.addressof(arr)


def fp8mlp_adamw_state_init(st, lr, seed=0, step=0, stream=None):
    dev, raw = _here(stream)
    return _call("fp8mlp_adamw_state_init", _buf(st, 32, "st", dev), lr, seed, step, raw)


def fp8mlp_grad_norm_workspace_size(tensors):
    return int(lib.fp8mlp_grad_norm_workspace_size(*_tensors(tensors)))


def fp8mlp_grad_norm(tensors, max_norm, norm_coef, workspace, stream=None):
    if _marshal is not None:
        return _done(_marshal.grad_norm(*_tensors(tensors), max_norm, norm_coef, workspace, stream), "fp8mlp_grad_norm")
    dev, raw = _here(stream)
    need = int(lib.fp8mlp_grad_norm_workspace_size(*_tensors(tensors)))
    return _call("fp8mlp_grad_norm", *_tensors(tensors), max_norm, _buf(norm_coef, 8, "norm_coef", dev),
                 _buf(workspace, need, "workspace", dev), raw)


def fp8mlp_adamw_check(tensors, st, state_bits, grad_coef=None):
    """What :func:`fp8mlp_adamw_step` refuses about its arrays, without a GPU."""
    return _call("fp8mlp_adamw_check", *_tensors(tensors), _ptr(st), state_bits, _ptr(grad_coef))


def fp8mlp_adamw_step(tensors, st, state_bits, beta1, beta2, eps, grad_coef=None, stream=None):
    for bits in getattr(tensors, "state_bits", ()):
        if bits != state_bits:
            raise ValueError(f"the descriptors were made for {bits}-bit states, not {state_bits}")
    if _marshal is not None:
        return _done(_marshal.adamw_step(*_tensors(tensors), st, state_bits, beta1, beta2, eps, grad_coef, stream),
                     "fp8mlp_adamw_step")
    dev, raw = _here(stream)
    return _call("fp8mlp_adamw_step", *_tensors(tensors), _buf(st, 32, "st", dev), state_bits, beta1, beta2, eps,
                 _buf(grad_coef, 4, "grad_coef", dev), raw)


def fp8mlp_get_device_status(stream=None):
    v = ctypes.c_uint()
    _call("fp8mlp_get_device_status", ctypes.addressof(v), _stream(stream))
    return v.value


def fp8mlp_clear_device_status(stream=None):
    return _call("fp8mlp_clear_device_status", _stream(stream))


def fp8mlp_set_wait_timeout_ns(ns):
    return _call("fp8mlp_set_wait_timeout_ns", int(ns))


def fp8mlp_set_programmatic_launch(enable):
    return _call("fp8mlp_set_programmatic_launch", int(bool(enable)))


def fp8mlp_set_debug_flags(flags):
    return _call("fp8mlp_set_debug_flags", int(flags))


def fp8mlp_error_string(code):
    return lib.fp8mlp_error_string(code).decode()


def fp8mlp_last_error_detail():
    return lib.fp8mlp_last_error_detail().decode()


def fp8mlp_kernel_launch_count():
    return int(lib.fp8mlp_kernel_launch_count())


def fp8mlp_version():
    return lib.fp8mlp_version().decode()
