"""ctypes binding to the vidattn C ABI (``include/vidattn.h``).

Argument marshalling only: tensors become raw pointers, streams become
``cudaStream_t`` handles.  Every step of the attention runs in the library's
CUDA kernels.  There is no fallback: if the library is missing or the call
fails, these functions raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libvidattn.so"
_HEADER = os.path.join(os.path.dirname(_PKG), "include", "vidattn.h")

VIDATTN_OK = 0
_lib = None
# the device type the tensor helpers require (the library reads device memory)
_DEVICE_TYPE = "cuda"


def library_path() -> str:
    """The in-tree libvidattn.so, or the file named by VIDATTN_LIBRARY."""
    return os.environ.get("VIDATTN_LIBRARY") or os.path.join(_PKG, "csrc", _LIB_NAME)


def load_library():
    """Load libvidattn.so (built in-tree by ``build.py``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m video_diffusion_transformer_non_b200.build` "
            "(or __graft_entry__.build()); there is no fallback implementation")
    lib = ctypes.CDLL(path)
    p, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.vidattn_fwd.argtypes = [p, p, p, p, p, p, p, i32, i32, i32, i32, i32, f32, p]
    lib.vidattn_fwd.restype = i32
    lib.vidattn_fwd_ex.argtypes = [p, p, p, p, p, p, p, i32, i32, i32, i32, i32, f32, i32, p]
    lib.vidattn_fwd_ex.restype = i32
    lib.vidattn_fwd_noalloc.argtypes = [p, p, p, p, p, p, p, i32, i32, i32, i32, i32, f32, p]
    lib.vidattn_fwd_noalloc.restype = i32
    lib.vidattn_fwd_host.argtypes = [p, p, p, p, p, p, p,
                                     p, p, p, p, p, p, p,
                                     i32, i32, i32, i32, i32, f32, p]
    lib.vidattn_fwd_host.restype = i32
    lib.vidattn_status_string.argtypes = [i32]
    lib.vidattn_status_string.restype = ctypes.c_char_p
    lib.vidattn_release.argtypes = []
    lib.vidattn_release.restype = None
    lib.vidattn_device_status.argtypes = [p]
    lib.vidattn_device_status.restype = i32
    lib.vidattn_kernels_per_call.argtypes = [p, p, i32, i32, i32, i32, i32, i32]
    lib.vidattn_kernels_per_call.restype = i32
    lib.vidattn_split_count.argtypes = [p, i32, i32, i32, i32, i32]
    lib.vidattn_split_count.restype = i32
    ip = ctypes.POINTER(ctypes.c_int)
    lib.vidattn_launch_plan.argtypes = [p, i32, i32, i32, i32, i32, i32, ip, ip, ip]
    lib.vidattn_launch_plan.restype = i32
    lib.vidattn_selftest_timeout.argtypes = [i32, p]
    lib.vidattn_selftest_timeout.restype = i32
    lib.vidattn_fwd_window.argtypes = [p, p, p, p, p, p, p, i32, i32, i32, i32, i32, f32,
                                       i32, i32, i32, i32, i32, i32, i32, p]
    lib.vidattn_fwd_window.restype = i32
    i64, f64 = ctypes.c_longlong, ctypes.c_double
    lib.vidattn_rope3d.argtypes = [p, p, p, p, i32, i32, i32, i32, i64, i64, i64,
                                   i32, i32, i32, i32, i32, i32, i32, f64, i32, p]
    lib.vidattn_rope3d.restype = i32
    lib.vidattn_bwd.argtypes = [p] * 12 + [i32, i32, i32, i32, i32, f32, i32, p, i64, p]
    lib.vidattn_bwd.restype = i32
    lib.vidattn_bwd_workspace.argtypes = [i32] * 7
    lib.vidattn_bwd_workspace.restype = i64
    lib.vidattn_layernorm.argtypes = [p] * 6 + [i32] * 4 + [p, p, i32, i32, f64, p]
    lib.vidattn_layernorm.restype = i32
    lib.vidattn_layernorm_bwd.argtypes = [p] * 8 + [i32] * 4 + [p, p, p, i32, i32, p, i64, p]
    lib.vidattn_layernorm_bwd.restype = i32
    lib.vidattn_layernorm_bwd_workspace.argtypes = [i32] * 5
    lib.vidattn_layernorm_bwd_workspace.restype = i64
    lib.vidattn_rope3d_scaled.argtypes = [p, p, p, p, i32, i32, i32, i32, p, p, i32, i32, i32, i32,
                                          i32, i32, i32, p, p, f64, i32, p]
    lib.vidattn_rope3d_scaled.restype = i32
    lib.vidattn_version.argtypes = []
    lib.vidattn_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def exported_symbols() -> list[str]:
    """Names of the functions declared in include/vidattn.h."""
    with open(_HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"VIDATTN_API\s+[\w\s\*]+?\b(vidattn_\w+)\s*\(", text)))


def status_string(status: int) -> str:
    return load_library().vidattn_status_string(int(status)).decode()


def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        pass
    if hasattr(x, "ctypes"):          # numpy array (host buffer)
        return x.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(x)}")


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_tensors(named, dtype, ndim=None, contiguous=True):
    """Raise ValueError unless every tensor in ``named`` (name -> tensor or
    None) is a CUDA tensor of ``dtype`` on one device, ``ndim``-dimensional
    and (when asked) contiguous.  Runs before any pointer reaches the library,
    whose kernels read device memory in the documented layout only."""
    import torch
    device = None
    for name, t in named.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor, not {type(t).__name__}")
        here = t.device
        if here != device:
            if here.type != _DEVICE_TYPE:
                raise ValueError(f"{name} must be on a CUDA device (is on {here})")
            if device is not None:
                raise ValueError(f"{name} is on {here}, the other tensors on {device}")
            device = here
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype} (is {t.dtype})")
        if ndim is not None and t.dim() != ndim:
            raise ValueError(f"{name} must have {ndim} dims (has shape {tuple(t.shape)})")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _check_qkv(q, k, v):
    """q bf16 [B,H,S_q,D], k and v bf16 [B,H,S_kv,D], contiguous, on one GPU."""
    import torch
    _check_tensors(dict(q=q, k=k, v=v), torch.bfloat16, ndim=4)
    if k.shape != v.shape or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]:
        raise ValueError(f"shapes do not match: q {tuple(q.shape)}, k {tuple(k.shape)}, "
                         f"v {tuple(v.shape)}")


def _check_per_token(name_q, t_q, name_kv, t_kv, B, S_q, S_kv, device):
    """int32 [B,S_q] and [B,S_kv] per-token arrays (ids or coordinates), both
    or neither, contiguous, on the device of q."""
    import torch
    if (t_q is None) != (t_kv is None):
        raise ValueError(f"{name_q} and {name_kv} must both be given or both be None")
    if t_q is None:
        return
    _check_tensors({name_q: t_q, name_kv: t_kv}, torch.int32, ndim=2)
    if t_q.device != device:
        raise ValueError(f"{name_q} is on {t_q.device}, q on {device}")
    if tuple(t_q.shape) != (B, S_q) or tuple(t_kv.shape) != (B, S_kv):
        raise ValueError(f"{name_q} must be [B,S_q] = {(B, S_q)} and {name_kv} [B,S_kv] = "
                         f"{(B, S_kv)} (are {tuple(t_q.shape)}, {tuple(t_kv.shape)})")


def vidattn_fwd(q, k, v, seg_q, seg_kv, out, lse, B, H, S_q, S_kv, D, scale, stream=None) -> int:
    """Enqueue the forward on ``stream`` (device pointers).  Returns the status."""
    return load_library().vidattn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(seg_q), _ptr(seg_kv), _ptr(out), _ptr(lse),
        int(B), int(H), int(S_q), int(S_kv), int(D), float(scale), _stream(stream))


VIDATTN_CAUSAL = 1


def vidattn_fwd_ex(q, k, v, seg_q, seg_kv, out, lse, B, H, S_q, S_kv, D, scale, flags,
                   stream=None) -> int:
    """vidattn_fwd with flags (VIDATTN_CAUSAL).  Returns the status."""
    return load_library().vidattn_fwd_ex(
        _ptr(q), _ptr(k), _ptr(v), _ptr(seg_q), _ptr(seg_kv), _ptr(out), _ptr(lse),
        int(B), int(H), int(S_q), int(S_kv), int(D), float(scale), int(flags), _stream(stream))


def vidattn_fwd_noalloc(q, k, v, seg_q, seg_kv, out, lse, B, H, S_q, S_kv, D, scale,
                        stream=None) -> int:
    """vidattn_fwd without any device allocation (fixed library scratch, with a
    size limit); for callers that may not allocate.  Returns the status."""
    return load_library().vidattn_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(seg_q), _ptr(seg_kv), _ptr(out), _ptr(lse),
        int(B), int(H), int(S_q), int(S_kv), int(D), float(scale), _stream(stream))


def vidattn_fwd_host(h_q, h_k, h_v, h_seg_q, h_seg_kv, h_out, h_lse,
                     d_q, d_k, d_v, d_seg_q, d_seg_kv, d_out, d_lse,
                     B, H, S_q, S_kv, D, scale, stream=None) -> int:
    """Host buffers in and out, through caller-owned device staging buffers:
    copies in, forward, copies out, all enqueued on ``stream``."""
    return load_library().vidattn_fwd_host(
        _ptr(h_q), _ptr(h_k), _ptr(h_v), _ptr(h_seg_q), _ptr(h_seg_kv), _ptr(h_out), _ptr(h_lse),
        _ptr(d_q), _ptr(d_k), _ptr(d_v), _ptr(d_seg_q), _ptr(d_seg_kv), _ptr(d_out), _ptr(d_lse),
        int(B), int(H), int(S_q), int(S_kv), int(D), float(scale), _stream(stream))


def device_status(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the kernels' error word."""
    return load_library().vidattn_device_status(_stream(stream))


def selftest_timeout(timeout_us: int, stream=None) -> int:
    return load_library().vidattn_selftest_timeout(int(timeout_us), _stream(stream))


def kernels_per_call(seg_q, seg_kv, B, H, S_q, S_kv, D, flags=0) -> int:
    return load_library().vidattn_kernels_per_call(_ptr(seg_q), _ptr(seg_kv), int(B), int(H),
                                                   int(S_q), int(S_kv), int(D), int(flags))


def split_count(seg_q, B, H, S_q, S_kv, flags=0) -> int:
    """Key splits a vidattn_fwd_ex call with these arguments uses (the
    library's launch heuristic, or the VIDATTN_SPLIT_KV request in flags)."""
    return load_library().vidattn_split_count(_ptr(seg_q), int(B), int(H), int(S_q), int(S_kv),
                                              int(flags))


def launch_plan(seg_q, B, H, S_q, S_kv, D, flags=0) -> dict:
    """The launch a vidattn_fwd_ex call would make on the current device:
    dict(grid_ctas, key_splits, persistent).  Raises on an error status."""
    g, k, pe = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = load_library().vidattn_launch_plan(_ptr(seg_q), int(B), int(H), int(S_q), int(S_kv),
                                            int(D), int(flags), ctypes.byref(g), ctypes.byref(k),
                                            ctypes.byref(pe))
    if st != VIDATTN_OK:
        raise RuntimeError(f"vidattn_launch_plan: {status_string(st)}")
    return dict(grid_ctas=g.value, key_splits=k.value, persistent=bool(pe.value))


def VIDATTN_SPLIT_KV(n: int) -> int:
    """vidattn_fwd_ex flag: split every 256-row query block's keys into n ranges."""
    return (int(n) & 0xFF) << 8


def attention(q, k, v, seg_q=None, seg_kv=None, scale=None, stream=None, causal=False):
    """Allocate out/lse with torch and run ``vidattn_fwd``.
    q: bf16 [B,H,S_q,D]; k, v: bf16 [B,H,S_kv,D]; seg_*: int32 [B,S] or None.
    Returns (out bf16 [B,H,S_q,D], lse fp32 [B,H,S_q]); raises on error."""
    import torch
    _check_qkv(q, k, v)
    B, H, S_q, D = q.shape
    S_kv = k.shape[2]
    _check_per_token("seg_q", seg_q, "seg_kv", seg_kv, B, S_q, S_kv, q.device)
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q.device)
    st = vidattn_fwd_ex(q, k, v, seg_q, seg_kv, out, lse, B, H, S_q, S_kv, D, scale,
                        VIDATTN_CAUSAL if causal else 0, stream)
    if st != VIDATTN_OK:
        raise RuntimeError(f"vidattn_fwd failed: {status_string(st)} ({st})")
    return out, lse


def vidattn_bwd(q, k, v, out, dout, lse, dlse, seg_q, seg_kv, dq, dk, dv, B, H, S_q, S_kv, D,
                scale, flags, workspace, workspace_bytes, stream=None) -> int:
    """Enqueue the attention's backward pass on ``stream``.  Returns the status."""
    return load_library().vidattn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dlse), _ptr(seg_q),
        _ptr(seg_kv), _ptr(dq), _ptr(dk), _ptr(dv), int(B), int(H), int(S_q), int(S_kv), int(D),
        float(scale), int(flags), _ptr(workspace), int(workspace_bytes), _stream(stream))


def bwd_workspace(has_ids, B, H, S_q, S_kv, D, flags=0) -> int:
    """Bytes of workspace a vidattn_bwd call needs (-1: arguments it refuses)."""
    return load_library().vidattn_bwd_workspace(int(bool(has_ids)), int(B), int(H), int(S_q),
                                                int(S_kv), int(D), int(flags))


_HERE = contextlib.nullcontext()


def _place(tensor, stream):
    """Where a call on ``tensor`` runs: (the stream's handle, a context in which
    the tensor's device is current and allocations belong to that stream).
    The default is the current stream of the tensor's device."""
    import torch
    device = tensor.device
    if stream is None:
        here = torch.cuda.current_device() == device.index
        return (torch._C._cuda_getCurrentRawStream(device.index),
                _HERE if here else torch.cuda.device(device))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream \
            else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream, torch.cuda.stream(stream)   # makes its device current too


def attention_bwd(dout, q, k, v, out, lse, seg_q=None, seg_kv=None, scale=None, causal=False,
                  dlse=None, stream=None, n_split=0):
    """The gradients (dq, dk, dv) of ``attention``: dout is the gradient of its
    out, dlse (or None) that of its lse; out and lse are what it returned, the
    rest what it was given.  dout: bf16 [B,H,S_q,D] contiguous; dlse: fp32
    [B,H,S_q], not used where lse is -inf.  n_split (1 to 64) forces the split of units (0: the
    library's choice).  Returns bf16 tensors of the shapes of q, k, v; raises on error."""
    import torch
    _check_tensors(dict(q=q, k=k, v=v, dout=dout, out=out), torch.bfloat16, ndim=4)
    _check_tensors(dict(lse=lse, dlse=dlse), torch.float32, ndim=3)
    shape = q.shape
    B, H, S_q, D = shape
    S_kv = k.shape[2]
    for name, t, like in (("v", v, k.shape), ("k", k, (B, H, S_kv, D)), ("dout", dout, shape),
                          ("out", out, shape), ("lse", lse, (B, H, S_q)), ("dlse", dlse, (B, H, S_q))):
        if t is not None and t.shape != like:
            raise ValueError(f"{name} must be {tuple(like)} (is {tuple(t.shape)})")
    if lse.device != q.device:
        raise ValueError(f"lse is on {lse.device}, q on {q.device}")
    _check_per_token("seg_q", seg_q, "seg_kv", seg_kv, B, S_q, S_kv, q.device)
    if not 0 <= n_split <= 64:
        raise ValueError(f"n_split must be 0 to 64 (is {n_split})")
    if scale is None:
        scale = D ** -0.5
    flags = (VIDATTN_CAUSAL if causal else 0) | VIDATTN_SPLIT_KV(n_split)
    n = load_library().vidattn_bwd_workspace(seg_q is not None, B, H, S_q, S_kv, D, flags)
    handle, place = _place(q, stream)
    with place:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = q.new_empty(max(n, 0), dtype=torch.uint8)
        st = load_library().vidattn_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(),
            lse.data_ptr(), _ptr(dlse), _ptr(seg_q), _ptr(seg_kv), dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), B, H, S_q, S_kv, D, scale, flags, ws.data_ptr() if n > 0 else None, n,
            handle)
    if st != VIDATTN_OK:
        raise RuntimeError(f"vidattn_bwd failed: {status_string(st)} ({st})")
    return dq, dk, dv


VIDATTN_BF16, VIDATTN_F32 = 0, 1


_Strides = ctypes.c_int64 * 3


def _strides(values):
    return _Strides(*values)


def vidattn_layernorm(x, weight, bias, y, mean, rstd, B, H, S, N, x_strides, y_strides, x_type,
                      param_type, eps, stream=None) -> int:
    """Enqueue the layer norm on ``stream``.  Returns the status."""
    return load_library().vidattn_layernorm(
        _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), int(B), int(H), int(S),
        int(N), _strides(x_strides), _strides(y_strides), int(x_type), int(param_type), float(eps),
        _stream(stream))


def vidattn_layernorm_bwd(dy, x, mean, rstd, weight, dx, dweight, dbias, B, H, S, N, dy_strides,
                          x_strides, dx_strides, x_type, param_type, workspace, workspace_bytes,
                          stream=None) -> int:
    """Enqueue the layer norm's gradients on ``stream``.  Returns the status."""
    return load_library().vidattn_layernorm_bwd(
        _ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(dx), _ptr(dweight),
        _ptr(dbias), int(B), int(H), int(S), int(N), _strides(dy_strides), _strides(x_strides),
        _strides(dx_strides), int(x_type), int(param_type), _ptr(workspace), int(workspace_bytes),
        _stream(stream))


def layernorm_bwd_workspace(B, H, S, N, x_type) -> int:
    """Bytes of workspace a vidattn_layernorm_bwd call needs (-1: sizes it refuses)."""
    return load_library().vidattn_layernorm_bwd_workspace(int(B), int(H), int(S), int(N),
                                                          int(x_type))


def _type_code(t):
    import torch
    if t is torch.bfloat16:
        return VIDATTN_BF16
    if t is torch.float32:
        return VIDATTN_F32
    raise ValueError(f"dtype must be bfloat16 or float32 (is {t})")


def _rows(name, t, shape=None):
    """A tensor of 1 to 4 dims as rows of [B,H,S,N]: its last dim contiguous,
    any strides for the others.  Returns (B, H, S, N), (sb, sh, ss)."""
    mine, strides = t.shape, t.stride()
    if shape is not None and mine != shape:
        raise ValueError(f"{name} must be {tuple(shape)} (is {tuple(mine)})")
    dims = len(mine)
    if not 1 <= dims <= 4:
        raise ValueError(f"{name} must have 1 to 4 dims (has shape {tuple(mine)})")
    if strides[-1] != 1 and mine[-1] != 1:
        raise ValueError(f"the last dim of {name} must be contiguous")
    if dims < 4:
        mine, strides = (1,) * (4 - dims) + tuple(mine), (0,) * (4 - dims) + strides
    B, H, S, N = mine
    sb, sh, ss, _ = strides
    return (B, H, S, N), (sb if B > 1 else 0, sh if H > 1 else 0, ss if S > 1 else 0)


def _dense(B, H, S, N):
    """_rows' strides of a contiguous tensor."""
    return (H * S * N if B > 1 else 0, S * N if H > 1 else 0, N if S > 1 else 0)


def _like(t):
    """An uninitialised contiguous tensor of t's shape, type and device."""
    import torch
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _check_norm(x, named, weight, bias):
    """Common checks of layer_norm and layer_norm_bwd; returns the types."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"x must be a torch tensor, not {type(x).__name__}")
    x_type = _type_code(x.dtype)
    _check_tensors(dict(x=x, **named), x.dtype, contiguous=False)
    if weight is None and bias is None:
        return x_type, VIDATTN_F32
    p = weight if weight is not None else bias
    if not isinstance(p, torch.Tensor):
        raise ValueError(f"weight and bias must be torch tensors, not {type(p).__name__}")
    p_type = _type_code(p.dtype)
    _check_tensors(dict(weight=weight, bias=bias), p.dtype, ndim=1)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and (t.device != x.device or t.shape[0] != x.shape[-1]):
            raise ValueError(f"{name} must be [{x.shape[-1]}] on {x.device} (is "
                             f"{tuple(t.shape)} on {t.device})")
    return x_type, p_type


def layer_norm(x, weight=None, bias=None, eps=1e-6, out=None, stream=None):
    """Layer norm over the last dim.  x: bf16 or fp32 of 1 to 4 dims, the last
    contiguous, any other strides (the [B,S,H,D] projection's ``transpose(1, 2)``
    view works); weight, bias: [N], bf16 or fp32, or None.  ``out=x`` works in
    place.  Returns (y contiguous or out, mean, rstd), the statistics fp32 of
    x's shape without its last dim; raises on error."""
    import torch
    x_type, p_type = _check_norm(x, dict(out=out), weight, bias)
    (B, H, S, N), sx = _rows("x", x)
    handle, place = _place(x, stream)
    with place:
        if out is None:
            y, sy = _like(x), _dense(B, H, S, N)
        else:
            y, sy = out, _rows("out", out, x.shape)[1]
        mean, rstd = x.new_empty((2, *x.shape[:-1]), dtype=torch.float32).unbind(0)
        if N > 0 and B * H * S == 0:
            return y, mean, rstd
        st = load_library().vidattn_layernorm(
            x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            B, H, S, N, _Strides(*sx), _Strides(*sy), x_type, p_type, eps, handle)
    if st != VIDATTN_OK:
        raise RuntimeError(f"vidattn_layernorm failed: {status_string(st)} ({st})")
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, weight=None, out=None, stream=None, params=True):
    """The gradients of ``layer_norm``: (dx, dweight, dbias), the last two None
    without a weight or with ``params=False`` (then only dx is computed).  dy: as y, any
    strides; x, weight: as given to it; mean, rstd: as it returned them; dx is
    contiguous, or ``out`` (which may be dy or x); raises on error."""
    import torch
    x_type, p_type = _check_norm(x, dict(dy=dy, out=out), weight, None)
    (B, H, S, N), sx = _rows("x", x)
    _, sdy = _rows("dy", dy, x.shape)
    _check_tensors(dict(mean=mean, rstd=rstd), torch.float32)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.shape != x.shape[:-1] or t.device != x.device:
            raise ValueError(f"{name} must be {tuple(x.shape[:-1])} on {x.device} (is "
                             f"{tuple(t.shape)} on {t.device})")
    handle, place = _place(x, stream)
    with place:
        if out is None:
            dx, sdx = _like(x), _dense(B, H, S, N)
        else:
            dx, sdx = out, _rows("out", out, x.shape)[1]
        dw = db = ws = None
        n = 0
        if weight is not None and params:
            dw, db = torch.empty_like(weight), torch.empty_like(weight)
            if x.numel() == 0:
                return dx, dw.zero_(), db.zero_()
            n = layernorm_bwd_workspace(B, H, S, N, x_type)
            ws = x.new_empty(max(n, 0), dtype=torch.uint8)
        if N > 0 and B * H * S == 0:
            return dx, None, None
        st = load_library().vidattn_layernorm_bwd(
            dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(weight),
            dx.data_ptr(), _ptr(dw), _ptr(db), B, H, S, N, _Strides(*sdy), _Strides(*sx),
            _Strides(*sdx), x_type, p_type, _ptr(ws), n, handle)
    if st != VIDATTN_OK:
        raise RuntimeError(f"vidattn_layernorm_bwd failed: {status_string(st)} ({st})")
    return dx, dw, db


VIDATTN_ROPE_HALF_SPLIT = 1


def vidattn_rope3d(q_in, k_in, q_out, k_out, B, H, S, D, stride_b, stride_h, stride_s,
                   T, Hg, Wg, token_offset, d_t, d_h, d_w, theta, flags, stream=None) -> int:
    """Enqueue the 3D rotary embedding of q (and k) on ``stream``.  Returns the status."""
    return load_library().vidattn_rope3d(
        _ptr(q_in), _ptr(k_in), _ptr(q_out), _ptr(k_out), int(B), int(H), int(S), int(D),
        int(stride_b), int(stride_h), int(stride_s), int(T), int(Hg), int(Wg), int(token_offset),
        int(d_t), int(d_h), int(d_w), float(theta), int(flags), _stream(stream))


def rope3d(q, k=None, grid=None, bands=None, theta=10000.0, interleaved=True, token_offset=0,
           out_q=None, out_k=None, stream=None):
    """Rotate q (and k) by the 3D rotary embedding; returns (q_rot, k_rot or None),
    bf16 [B,H,S,D] contiguous.  q, k: bf16 [B,H,S,D] tensors whose last dim is
    contiguous, any other strides (a [B,S,H,D] tensor's ``transpose(1, 2)`` view
    works); grid = (T, Hg, Wg) of the video tokens; bands = (d_t, d_h, d_w).
    ``out_q=q`` (and ``out_k=k``) rotates a contiguous input in place."""
    import torch
    _check_tensors(dict(q=q, k=k, out_q=out_q, out_k=out_k), torch.bfloat16, ndim=4,
                   contiguous=False)
    if out_k is not None and k is None:
        raise ValueError("out_k without k")
    B, H, S, D = q.shape
    if k is not None and k.shape != q.shape:
        raise ValueError("q and k must have the same shape")
    if k is not None and k.stride() != q.stride():
        raise ValueError("q and k must have the same strides")
    if q.stride(3) != 1:
        raise ValueError("the feature dim must be contiguous")
    out_q = torch.empty((B, H, S, D), dtype=q.dtype, device=q.device) if out_q is None else out_q
    if k is not None and out_k is None:
        out_k = torch.empty((B, H, S, D), dtype=k.dtype, device=k.device)
    for o in (out_q, out_k):
        if o is not None and (tuple(o.shape) != (B, H, S, D) or not o.is_contiguous()):
            raise ValueError("outputs must be contiguous [B,H,S,D]")
    T, Hg, Wg = grid
    d_t, d_h, d_w = bands
    sb, sh, ss, _ = q.stride()
    st = vidattn_rope3d(q, k, out_q, out_k if k is not None else None, B, H, S, D, sb, sh, ss,
                        T, Hg, Wg, token_offset, d_t, d_h, d_w, theta,
                        0 if interleaved else VIDATTN_ROPE_HALF_SPLIT, stream)
    if st != VIDATTN_OK:
        raise RuntimeError(f"vidattn_rope3d failed: {status_string(st)} ({st})")
    return out_q, out_k


VIDATTN_ROPE_TRANSPOSE = 2


_doubles_types = {}   # length -> ctypes array type (making one costs as much as a launch)


def _doubles(values):
    n = max(len(values), 1)
    t = _doubles_types.get(n)
    if t is None:
        t = _doubles_types[n] = ctypes.c_double * n
    return t(*values)


def vidattn_rope3d_scaled(q_in, k_in, q_out, k_out, B, H, S, D, in_strides, out_strides, T, Hg, Wg,
                          token_offset, d_t, d_h, d_w, freqs, pos_scale, amplitude, flags,
                          stream=None) -> int:
    """Enqueue the scaled 3D rotary embedding of q (and k) on ``stream``.
    freqs, pos_scale: sequences of floats.  Returns the status."""
    return load_library().vidattn_rope3d_scaled(
        _ptr(q_in), _ptr(k_in), _ptr(q_out), _ptr(k_out), int(B), int(H), int(S), int(D),
        _strides(in_strides), _strides(out_strides), int(T), int(Hg), int(Wg), int(token_offset),
        int(d_t), int(d_h), int(d_w), _doubles(freqs), _doubles(pos_scale), float(amplitude),
        int(flags), _stream(stream))


def _rope_scaled(name, q, k, grid, bands, freqs, pos_scale, amplitude, interleaved, token_offset,
                 out_q, out_k, stream, transpose):
    import torch
    _check_tensors(dict(q=q, k=k, out_q=out_q, out_k=out_k), torch.bfloat16, ndim=4,
                   contiguous=False)
    if out_k is not None and k is None:
        raise ValueError("out_k without k")
    (B, H, S, D), s_in = _rows("q", q)
    if k is not None and _rows("k", k, q.shape)[1] != s_in:
        raise ValueError("q and k must have the same strides")
    if len(bands) != 3 or any(d < 0 or d % 2 for d in bands) or sum(bands) > D:
        raise ValueError(f"bands must be 3 even sizes of at most {D} together (are {bands})")
    if len(freqs) != sum(bands) // 2:
        raise ValueError(f"freqs must hold {sum(bands) // 2} values, one a pair (holds "
                         f"{len(freqs)})")
    if len(pos_scale) != 3:
        raise ValueError("pos_scale must hold 3 values")
    handle, place = _place(q, stream)
    with place:
        if out_q is None:
            out_q, s_out = _like(q), _dense(B, H, S, D)
        else:
            s_out = _rows("out_q", out_q, q.shape)[1]
        if k is not None:
            if out_k is None:
                out_k = torch.empty_like(out_q)   # of a dense out_q: the same strides
                if out_k.stride() != out_q.stride():
                    out_k = torch.empty_strided(out_q.shape, out_q.stride(), dtype=k.dtype,
                                                device=k.device)
            elif _rows("out_k", out_k, q.shape)[1] != s_out:
                raise ValueError("out_q and out_k must have the same strides")
        if q.numel() == 0 and D > 0:
            return out_q, out_k
        flags = (0 if interleaved else VIDATTN_ROPE_HALF_SPLIT) | \
            (VIDATTN_ROPE_TRANSPOSE if transpose else 0)
        T, Hg, Wg = grid
        d_t, d_h, d_w = bands
        st = load_library().vidattn_rope3d_scaled(
            q.data_ptr(), _ptr(k), out_q.data_ptr(), _ptr(out_k), B, H, S, D, _Strides(*s_in),
            _Strides(*s_out), T, Hg, Wg, token_offset, d_t, d_h, d_w, _doubles(freqs),
            _doubles(pos_scale), amplitude, flags, handle)
    if st != VIDATTN_OK:
        raise RuntimeError(f"{name} failed: {status_string(st)} ({st})")
    return out_q, out_k


def rope3d_scaled(q, k=None, grid=None, bands=None, freqs=None, pos_scale=(1.0, 1.0, 1.0),
                  amplitude=1.0, interleaved=True, token_offset=0, out_q=None, out_k=None,
                  stream=None):
    """Rotate q (and k) with the caller's frequencies: pair c of the bands turns
    by coord * pos_scale[axis] * freqs[c] and is scaled by amplitude; features
    behind the bands and tokens outside the video are copied.  q, k: bf16
    [B,H,S,D] of equal strides, the last dim contiguous; grid = (T, Hg, Wg);
    bands = (d_t, d_h, d_w), at most D together; freqs: one float a pair (see
    rope3d_frequencies).  Outputs are contiguous, or out_q and out_k of any
    equal strides (out_q=q, out_k=k: in place).  Returns (q_rot, k_rot or None)."""
    return _rope_scaled("vidattn_rope3d_scaled", q, k, grid, bands, freqs, pos_scale, amplitude,
                        interleaved, token_offset, out_q, out_k, stream, False)


def rope3d_scaled_bwd(dq, dk=None, grid=None, bands=None, freqs=None, pos_scale=(1.0, 1.0, 1.0),
                      amplitude=1.0, interleaved=True, token_offset=0, out_q=None, out_k=None,
                      stream=None):
    """The gradients of rope3d_scaled's inputs from those of its outputs: the
    transposed rotation, same arguments, same layouts."""
    return _rope_scaled("vidattn_rope3d_scaled", dq, dk, grid, bands, freqs, pos_scale, amplitude,
                        interleaved, token_offset, out_q, out_k, stream, True)


def rope3d_frequencies(bands, theta=10000.0, extent=None, factor=1.0, turns=(1.0, 8.0)):
    """Frequencies for rope3d_scaled: theta^(-2c/d) for pair c of a band of d
    features, as vidattn_rope3d's.  With ``extent`` = the trained volume
    (T, Hg, Wg), stretched by parts for one ``factor`` times as long on every
    axis: a pair that turns fewer than turns[0] times over the trained extent
    is interpolated (its frequency divided by factor), one that turns more than
    turns[1] times is kept, linear in between."""
    import math
    if len(bands) != 3 or any(d < 0 or d % 2 for d in bands):
        raise ValueError(f"bands must be 3 even sizes (are {bands})")
    if not (theta > 0 and factor > 0 and turns[1] > turns[0]):
        raise ValueError("theta and factor must be positive, turns ascending")
    out = []
    for a, d in enumerate(bands):
        for c in range(d // 2):
            w = theta ** (-2.0 * c / d)
            if extent is not None:
                n = extent[a] * w / (2 * math.pi)
                keep = min(1.0, max(0.0, (n - turns[0]) / (turns[1] - turns[0])))
                w = w * keep + w / factor * (1.0 - keep)
            out.append(w)
    return out


VIDATTN_WINDOW_CLAMPED = 1


def vidattn_fwd_window(q, k, v, coord_q, coord_kv, out, lse, B, H, S_q, S_kv, D, scale,
                       win_t, win_h, win_w, T, Hg, Wg, flags, stream=None) -> int:
    """Enqueue 3D neighbourhood attention on ``stream``.  Returns the status."""
    return load_library().vidattn_fwd_window(
        _ptr(q), _ptr(k), _ptr(v), _ptr(coord_q), _ptr(coord_kv), _ptr(out), _ptr(lse),
        int(B), int(H), int(S_q), int(S_kv), int(D), float(scale), int(win_t), int(win_h),
        int(win_w), int(T), int(Hg), int(Wg), int(flags), _stream(stream))


def attention_window(q, k, v, coord_q, coord_kv, size, extent, clamped=True, scale=None,
                     stream=None):
    """3D neighbourhood attention.  coord_*: int32 [B,S] packed t << 22 | h << 11 | w;
    size = (win_t, win_h, win_w), odd; extent = (T, Hg, Wg).  Returns (out, lse)."""
    import torch
    _check_qkv(q, k, v)
    B, H, S_q, D = q.shape
    S_kv = k.shape[2]
    if coord_q is None or coord_kv is None:
        raise ValueError("a window needs coord_q and coord_kv")
    _check_per_token("coord_q", coord_q, "coord_kv", coord_kv, B, S_q, S_kv, q.device)
    if scale is None:
        scale = D ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q.device)
    st = vidattn_fwd_window(q, k, v, coord_q, coord_kv, out, lse, B, H, S_q, S_kv, D, scale,
                            *size, *extent, VIDATTN_WINDOW_CLAMPED if clamped else 0, stream)
    if st != VIDATTN_OK:
        raise RuntimeError(f"vidattn_fwd_window failed: {status_string(st)} ({st})")
    return out, lse
