"""Python binding of libwqmm.so, the weight-resident quantized matmul for MI355X.

    y[s,o] = scale[o] * sum_i dequant(W[o,i]) * x[s,i]

(colibri "第 8 章 · 02 CUDA/Metal/Vulkan 三后端", section 四; colibri-analysis
"CUDA 后端", section 1.) Every function here has the name of the C entry point
it wraps (include/wqmm.h) and only marshals arguments: numpy arrays for host
buffers, torch tensors for device buffers and the current torch stream.
All computation happens in the HIP kernels of libwqmm.so; there is no CPU
fallback. A non-zero status becomes a WqError carrying the code.

The library is loaded after torch so that both use the same HIP runtime.
If libwqmm.so has not been built yet it is built once with hipcc; if that is
impossible the import fails loudly.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

try:  # torch first: its HIP runtime is the one the library must bind to
    import torch
except ImportError:  # pragma: no cover - host-only use (plan description, row bytes)
    torch = None

WQ_F32, WQ_I8, WQ_I4, WQ_I2 = 0, 1, 2, 3
WQ_OK = 0
WQ_E_INVAL = -1
WQ_E_NODEV = -2
WQ_E_NOTINIT = -3
WQ_E_OOM = -4
WQ_E_MISMATCH = -5
WQ_E_HIP = -6
WQ_E_FAULT = -7
WQ_E_UNSUPPORTED = -8
WQ_DT_F32, WQ_DT_BF16, WQ_DT_F16, WQ_DT_I8 = 0, 1, 2, 3
WQ_KV_F16, WQ_KV_I8, WQ_KV_I4 = 0, 1, 2
WQ_NORM_MAX_N = 32768
WQ_ROPE_MAX_ROT = 256
WQ_ROPE_MAX_AXES = 8
WQ_KV_MAX_HEADS = 1024
WQ_MAX_DEVICES = 16
WQ_GEMV_MAX_S = 8

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwqmm.so")

_c_int_p = ctypes.POINTER(ctypes.c_int)
_c_size_p = ctypes.POINTER(ctypes.c_size_t)


class _KvCacheC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("device", "kind", "pages", "heads", "page", "dim")] + [
        (n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [
        ("row_stride", ctypes.c_long * 3), ("scale_stride", ctypes.c_long * 3)]


class _KvBatchC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "width", "max_q", "max_kv")] + [
        ("table_stride", ctypes.c_long)] + [(n, ctypes.c_void_p) for n in ("q_start", "kv_len", "table")]


class WqError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (what, wq_strerror(code), code))


def _bind(lib):
    vp, ci, cl = ctypes.c_void_p, ctypes.c_int, ctypes.c_long
    cf, cachep, batchp = ctypes.c_float, ctypes.POINTER(_KvCacheC), ctypes.POINTER(_KvBatchC)
    sig = {
        "wq_init": (ci, [_c_int_p, ci]),
        "wq_mem_info": (ci, [ci, _c_size_p, _c_size_p]),
        "wq_row_bytes": (cl, [ci, cl]),
        "wq_tensor_upload": (ci, [ctypes.POINTER(vp), ci, ci, ci, ci, vp, vp]),
        "wq_tensor_upload_gs": (ci, [ctypes.POINTER(vp), ci, ci, ci, ci, ci, vp, vp]),
        "wq_matmul": (ci, [ctypes.POINTER(vp), ci, ci, ci, ci, vp, vp, vp, ci, vp]),
        "wq_matmul_t": (ci, [vp, vp, ci, vp]),
        "wq_matmul_dev": (ci, [vp, vp, ci, vp, vp]),
        "wq_grouped_create": (ci, [ctypes.POINTER(vp), ci, ctypes.POINTER(vp)]),
        "wq_grouped_matmul_dev": (ci, [vp, ctypes.POINTER(vp), _c_int_p, ctypes.POINTER(vp), vp]),
        "wq_grouped_free": (ci, [vp]),
        "wq_swiglu_create": (ci, [ctypes.POINTER(vp), ctypes.POINTER(vp), ci, ctypes.POINTER(vp)]),
        "wq_swiglu_matmul_dev": (ci, [vp, ctypes.POINTER(vp), _c_int_p, ctypes.POINTER(vp), vp]),
        "wq_swiglu_ffn_dev": (ci, [vp, vp, ctypes.POINTER(vp), _c_int_p, ctypes.POINTER(vp),
                                   ctypes.POINTER(vp), vp]),
        "wq_tensor_free": (ci, [vp]),
        "wq_strerror": (ctypes.c_char_p, [ci]),
        "wq_describe_plan": (ci, [ci, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t]),
        "wq_describe_plan_gs": (ci, [ci, ci, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t]),
        "wq_stream_read_dev": (ci, [vp, ctypes.c_size_t, ci, ci, vp, vp]),
        "wq_matmul_dev_noalloc": (ci, [vp, vp, ci, vp, vp]),
        "wq_noalloc_scratch_bytes": (ctypes.c_size_t, []),
        "wq_rmsnorm_dev": (ci, [ci, vp, ci, cl, vp, cl, vp, cf, ci, ci, vp, ci, cl, vp, vp, cl, vp]),
        "wq_rope_create": (ci, [ci, ci, ctypes.c_double, _c_int_p, ci, ctypes.POINTER(vp)]),
        "wq_rope_dev": (ci, [vp, ci, vp, ci, ci, ci, ci, cl, cl, vp, cl, vp, cl, cl, vp]),
        "wq_rope_free": (ci, [vp]),
        "wq_kv_append_dev": (ci, [cachep, batchp, vp, vp, ci, cl, cl, vp]),
        "wq_kv_read_dev": (ci, [cachep, batchp, vp, vp, ci, cl, cl, vp]),
        "wq_describe_attn": (ci, [cachep, batchp, ci, ci, ci, ci, ctypes.c_char_p, ctypes.c_size_t]),
        "wq_attn_paged_dev": (ci, [cachep, batchp, vp, ci, ci, cl, cl, cf, ci, ci, vp, cl, cl, vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


def _load():
    if not os.path.exists(LIB_PATH):
        from . import build as _build  # nothing built yet: build once, in-tree
        _build.build()
    return _bind(ctypes.CDLL(LIB_PATH))


lib = _load()


def _check(rc: int, what: str):
    if rc != WQ_OK:
        raise WqError(rc, what)


def _stream_handle(stream, device):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _host_f32(a, shape, what):
    a = np.ascontiguousarray(a, dtype=np.float32)
    if a.shape != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), a.shape))
    return a


def _dev_f32(t, shape, device, what):
    if torch is None or not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor on a GPU" % what)
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 GPU tensor" % what)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.device.index != device:
        raise ValueError("%s is on %s, tensor lives on cuda:%d" % (what, t.device, device))
    return ctypes.c_void_p(t.data_ptr())


class Tensor:
    """Handle of a resident weight tensor (the C wq_tensor*)."""

    def __init__(self, ptr: ctypes.c_void_p, device: int, fmt: int, O: int, I: int):
        self.ptr, self.device, self.fmt, self.O, self.I = ptr, device, fmt, O, I

    def __repr__(self):
        return "Tensor(device=%d, fmt=%d, O=%d, I=%d)" % (self.device, self.fmt, self.O, self.I)


class Group:
    """Handle of a tensor group (the C wq_group*); `ups` is set for a gated group."""

    def __init__(self, ptr: ctypes.c_void_p, tensors, ups=None):
        self.ptr, self.tensors = ptr, list(tensors)
        self.ups = None if ups is None else list(ups)


# ----------------------------------------------------------------------------
# C ABI wrappers


def wq_strerror(code: int) -> str:
    return lib.wq_strerror(int(code)).decode()


def wq_init(devices=None) -> None:
    if devices is None:
        _check(lib.wq_init(None, 0), "wq_init")
        return
    devs = list(devices)
    arr = (ctypes.c_int * max(1, len(devs)))(*devs)
    _check(lib.wq_init(arr, len(devs)), "wq_init")


def wq_mem_info(device: int = 0):
    f, t = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.wq_mem_info(int(device), ctypes.byref(f), ctypes.byref(t)), "wq_mem_info")
    return f.value, t.value


def wq_row_bytes(fmt: int, I: int) -> int:
    return int(lib.wq_row_bytes(int(fmt), int(I)))


def _weights(fmt, O, I, w, scales):
    rb = wq_row_bytes(fmt, I)
    if rb < 0:
        raise WqError(WQ_E_INVAL, "wq_row_bytes")
    w = np.ascontiguousarray(w, dtype=np.uint8)
    if w.size != O * rb:
        raise ValueError("w must hold O * row_bytes = %d bytes, got %d" % (O * rb, w.size))
    if scales is not None:
        scales = _host_f32(scales, (O,), "scales")
    return w, scales


def wq_tensor_upload(t, device: int, fmt: int, O: int, I: int, w, scales) -> Tensor:
    """Upload (t is None) or validate (t given) a resident tensor; returns the handle."""
    h = ctypes.c_void_p(t.ptr.value if t is not None else None)
    if t is None:
        w, scales = _weights(fmt, O, I, w, scales)
        wp, sp = w.ctypes.data, (scales.ctypes.data if scales is not None else None)
    else:
        wp, sp = None, None
    _check(lib.wq_tensor_upload(ctypes.byref(h), int(device), int(fmt), int(O), int(I), wp, sp),
           "wq_tensor_upload")
    return t if t is not None else Tensor(h, int(device), int(fmt), int(O), int(I))


def wq_tensor_upload_gs(t, device: int, fmt: int, O: int, I: int, gs: int, w, scales) -> Tensor:
    """Upload with group-wise scales (scales float32 [O, ceil(I/gs)]) or validate; returns the handle."""
    h = ctypes.c_void_p(t.ptr.value if t is not None else None)
    if t is None:
        w, _ = _weights(fmt, O, I, w, None)
        ng = (int(I) + int(gs) - 1) // int(gs) if int(gs) > 0 else 1
        scales = _host_f32(scales, (O, ng), "scales")
        wp, sp = w.ctypes.data, scales.ctypes.data
    else:
        wp, sp = None, None
    _check(lib.wq_tensor_upload_gs(ctypes.byref(h), int(device), int(fmt), int(O), int(I), int(gs), wp, sp),
           "wq_tensor_upload_gs")
    return t if t is not None else Tensor(h, int(device), int(fmt), int(O), int(I))


def wq_matmul(t, device: int, fmt: int, O: int, I: int, w, scales, x):
    """Lazy upload + synchronous host matmul; returns (handle, y [S, O])."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    if x.ndim != 2 or x.shape[1] != I:
        raise ValueError("x must be [S, I]")
    S = x.shape[0]
    y = np.empty((S, O), dtype=np.float32)
    h = ctypes.c_void_p(t.ptr.value if t is not None else None)
    if t is None:
        w, scales = _weights(fmt, O, I, w, scales)
        wp, sp = w.ctypes.data, (scales.ctypes.data if scales is not None else None)
    else:
        wp, sp = None, None
    _check(lib.wq_matmul(ctypes.byref(h), int(device), int(fmt), int(O), int(I), wp, sp,
                         x.ctypes.data, S, y.ctypes.data), "wq_matmul")
    return (t if t is not None else Tensor(h, int(device), int(fmt), int(O), int(I))), y


def wq_matmul_t(t: Tensor, x) -> np.ndarray:
    x = np.ascontiguousarray(x, dtype=np.float32)
    if x.ndim != 2 or x.shape[1] != t.I:
        raise ValueError("x must be [S, I]")
    y = np.empty((x.shape[0], t.O), dtype=np.float32)
    _check(lib.wq_matmul_t(t.ptr, x.ctypes.data, x.shape[0], y.ctypes.data), "wq_matmul_t")
    return y


def wq_matmul_dev(t: Tensor, x_dev, y_dev, stream=None) -> None:
    """y_dev[S, O] = matmul(t, x_dev[S, I]) as one launch on `stream` (default: current)."""
    S = x_dev.shape[0] if x_dev.dim() == 2 else -1
    xp = _dev_f32(x_dev, (S, t.I), t.device, "x_dev")
    yp = _dev_f32(y_dev, (S, t.O), t.device, "y_dev")
    _check(lib.wq_matmul_dev(t.ptr, xp, int(S), yp, _stream_handle(stream, t.device)), "wq_matmul_dev")


def wq_matmul_dev_noalloc(t: Tensor, x_dev, y_dev, stream=None) -> None:
    """As wq_matmul_dev, allocating nothing (the tiled workspace is the library's fixed
    per-device array of wq_noalloc_scratch_bytes() bytes)."""
    S = x_dev.shape[0] if x_dev.dim() == 2 else -1
    xp = _dev_f32(x_dev, (S, t.I), t.device, "x_dev")
    yp = _dev_f32(y_dev, (S, t.O), t.device, "y_dev")
    _check(lib.wq_matmul_dev_noalloc(t.ptr, xp, int(S), yp, _stream_handle(stream, t.device)),
           "wq_matmul_dev_noalloc")


def wq_noalloc_scratch_bytes() -> int:
    return int(lib.wq_noalloc_scratch_bytes())


def wq_grouped_create(tensors) -> Group:
    ts = list(tensors)
    arr = (ctypes.c_void_p * len(ts))(*[t.ptr.value for t in ts])
    h = ctypes.c_void_p(None)
    _check(lib.wq_grouped_create(arr, len(ts), ctypes.byref(h)), "wq_grouped_create")
    return Group(h, ts)


def wq_grouped_matmul_dev(g: Group, xs, ys, stream=None) -> None:
    """For each g: ys[g][S_g, O_g] = matmul(tensor g, xs[g][S_g, I_g]); xs[g] None means S_g = 0."""
    G = len(g.tensors)
    if len(xs) != G or len(ys) != G:
        raise ValueError("need one x and one y per tensor")
    xp = (ctypes.c_void_p * G)()
    yp = (ctypes.c_void_p * G)()
    Ss = (ctypes.c_int * G)()
    for i, (t, x, y) in enumerate(zip(g.tensors, xs, ys)):
        if x is None:
            Ss[i] = 0
            continue
        S = x.shape[0]
        xp[i] = _dev_f32(x, (S, t.I), t.device, "xs[%d]" % i).value
        yp[i] = _dev_f32(y, (S, t.O), t.device, "ys[%d]" % i).value
        Ss[i] = S
    dev = g.tensors[0].device
    _check(lib.wq_grouped_matmul_dev(g.ptr, xp, Ss, yp, _stream_handle(stream, dev)), "wq_grouped_matmul_dev")


def _per_problem(tensors, xs, outs, out_cols, what):
    G = len(tensors)
    if len(xs) != G or len(outs) != G:
        raise ValueError("need one x and one %s per problem" % what)
    xp = (ctypes.c_void_p * G)()
    op = (ctypes.c_void_p * G)()
    Ss = (ctypes.c_int * G)()
    for i, (t, x, o) in enumerate(zip(tensors, xs, outs)):
        if x is None:
            Ss[i] = 0
            continue
        S = x.shape[0]
        xp[i] = _dev_f32(x, (S, t.I), t.device, "xs[%d]" % i).value
        op[i] = _dev_f32(o, (S, out_cols[i]), t.device, "%s[%d]" % (what, i)).value
        Ss[i] = S
    return xp, Ss, op


def wq_swiglu_create(gates, ups) -> Group:
    """Gated group: expert e pairs gates[e] with ups[e] (same shape)."""
    gs, us = list(gates), list(ups)
    if len(gs) != len(us):
        raise ValueError("need one up tensor per gate tensor")
    ga = (ctypes.c_void_p * len(gs))(*[t.ptr.value for t in gs])
    ua = (ctypes.c_void_p * len(us))(*[t.ptr.value for t in us])
    h = ctypes.c_void_p(None)
    _check(lib.wq_swiglu_create(ga, ua, len(gs), ctypes.byref(h)), "wq_swiglu_create")
    return Group(h, gs, us)


def wq_swiglu_matmul_dev(g: Group, xs, hs, stream=None) -> None:
    """hs[e][S_e, O_e] = silu(gate_e . xs[e]) * (up_e . xs[e]); xs[e] None skips expert e."""
    xp, Ss, hp = _per_problem(g.tensors, xs, hs, [t.O for t in g.tensors], "hs")
    dev = g.tensors[0].device
    _check(lib.wq_swiglu_matmul_dev(g.ptr, xp, Ss, hp, _stream_handle(stream, dev)), "wq_swiglu_matmul_dev")


def wq_swiglu_ffn_dev(g: Group, down: Group, xs, hs, ys, stream=None) -> None:
    """Both halves of the gated feed-forward: hs as wq_swiglu_matmul_dev, then ys[e] = down_e . hs[e]."""
    xp, Ss, hp = _per_problem(g.tensors, xs, hs, [t.O for t in g.tensors], "hs")
    if len(ys) != len(down.tensors):
        raise ValueError("need one y per expert")
    E = len(g.tensors)
    yp = (ctypes.c_void_p * E)()
    for i in range(E):
        if Ss[i] > 0:
            t = down.tensors[i]
            yp[i] = _dev_f32(ys[i], (Ss[i], t.O), t.device, "ys[%d]" % i).value
    dev = g.tensors[0].device
    _check(lib.wq_swiglu_ffn_dev(g.ptr, down.ptr, xp, Ss, hp, yp, _stream_handle(stream, dev)),
           "wq_swiglu_ffn_dev")


def wq_grouped_free(g: Group) -> None:
    _check(lib.wq_grouped_free(g.ptr), "wq_grouped_free")
    g.ptr = ctypes.c_void_p(None)


def wq_tensor_free(t: Tensor) -> None:
    if t is None:
        return
    _check(lib.wq_tensor_free(t.ptr), "wq_tensor_free")
    t.ptr = ctypes.c_void_p(None)


def wq_describe_plan(fmt: int, O: int, I: int, S: int) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib.wq_describe_plan(int(fmt), int(O), int(I), int(S), buf, 256), "wq_describe_plan")
    return buf.value.decode()


def wq_describe_plan_gs(fmt: int, O: int, I: int, S: int, gs: int) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib.wq_describe_plan_gs(int(fmt), int(O), int(I), int(S), int(gs), buf, 256), "wq_describe_plan_gs")
    return buf.value.decode()


def wq_stream_read_dev(buf_dev, waves: int, loads_in_flight: int, out_dev, stream=None) -> None:
    """Read every byte of the device tensor buf_dev once (HBM read ceiling);
    out_dev: int32 device tensor of >= 64 * waves elements."""
    nbytes = buf_dev.numel() * buf_dev.element_size()
    if not buf_dev.is_cuda or not buf_dev.is_contiguous() or not out_dev.is_cuda:
        raise ValueError("device tensors expected")
    if out_dev.numel() * out_dev.element_size() < 4 * 64 * int(waves):
        raise ValueError("out_dev too small")
    _check(lib.wq_stream_read_dev(ctypes.c_void_p(buf_dev.data_ptr()), nbytes, int(waves), int(loads_in_flight),
                                  ctypes.c_void_p(out_dev.data_ptr()), _stream_handle(stream, buf_dev.device)),
           "wq_stream_read_dev")


# ----------------------------------------------------------------------------
# between a decoder layer's products: norm, rotary positions, cache, attention

_FLOATS = {} if torch is None else {torch.float32: WQ_DT_F32, torch.bfloat16: WQ_DT_BF16, torch.float16: WQ_DT_F16}
_OUTS = {} if torch is None else {torch.int8: WQ_DT_I8, **_FLOATS}

# The calls of one token's step are shorter than their checks if those are not kept lean: a tensor is checked once,
# in one condition, and the message is made only when it fails.


_INT_MAX = 0x7FFFFFFF


def _int(v):
    """v for a C int, which ctypes would take modulo 2^32: larger numbers become the largest one, smaller ones -1."""
    v = int(v)
    return v if -1 <= v <= _INT_MAX else _INT_MAX if v > 0 else -1


def _raw_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _first(t, dims, types, what):
    """(shape, type code, device, strides) of a GPU tensor with `dims` dimensions, the last one contiguous."""
    if torch is None or not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor on a GPU" % what)
    dt = types.get(t.dtype, -1)
    shape, st, dev = t.shape, t.stride(), t.get_device()
    if dt < 0 or dev < 0 or len(shape) != dims or (st[-1] != 1 and shape[-1] > 1) or max(shape) > _INT_MAX:
        raise ValueError("%s: a %s tensor of shape %s and strides %s on %s is not taken" % (what, t.dtype, tuple(shape), st, t.device))
    return shape, dt, dev, st


def _more(t, shape, dtype, dev, what):
    """The strides of a further tensor, with the shape, type and device asked for and its last dimension contiguous."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
        st = t.stride()
        if st[-1] == 1 or shape[-1] <= 1:
            return st
    raise ValueError("%s must be %s of shape %s on GPU %d, its last dimension contiguous; got %s, %s, %s" % (
        what, dtype, tuple(shape), dev, t.dtype, tuple(t.shape), t.device))


def wq_rmsnorm_dev(x, w, eps: float, y, residual=None, sum_out=None, y_scale=None, stream=None) -> None:
    """y[rows, n] = norm of x (+ residual) times w; sum_out receives x + residual in x's type.

    y float32, bfloat16, float16, or int8 codes with y_scale [rows] (y ~ code * y_scale)."""
    shape, dt, dev, xs = _first(x, 2, _FLOATS, "x")
    rows, n = shape
    ydt = _OUTS.get(y.dtype, -1)
    ys = _more(y, shape, y.dtype, dev, "y")
    _more(w, shape[1:], torch.float32, dev, "w")
    rp = rs = sp = ss = yp = None
    if residual is not None:
        rs = _more(residual, shape, x.dtype, dev, "residual")[0]
        rp = residual.data_ptr()
    if sum_out is not None:
        ss = _more(sum_out, shape, x.dtype, dev, "sum_out")[0]
        sp = sum_out.data_ptr()
    if (ydt == WQ_DT_I8) != (y_scale is not None):
        raise ValueError("y_scale goes with an int8 y")
    if y_scale is not None:
        _more(y_scale, shape[:1], torch.float32, dev, "y_scale")
        yp = y_scale.data_ptr()
    rc = lib.wq_rmsnorm_dev(dev, x.data_ptr(), dt, xs[0], rp, rs or 0, w.data_ptr(), eps, rows, n, y.data_ptr(), ydt,
                            ys[0], yp, sp, ss or 0, _raw_stream(stream, dev))
    if rc:
        _check(rc, "wq_rmsnorm_dev")


class Rope:
    """Plan of rotary positions (the C wq_rope*; host memory, released with the object or wq_rope_free)."""

    def __init__(self, ptr: ctypes.c_void_p, rot: int, axes: int):
        self.ptr, self.rot, self.axes = ptr, rot, axes

    def __del__(self):
        if self.ptr and lib is not None:
            lib.wq_rope_free(self.ptr)
            self.ptr = None


def wq_rope_create(rot: int, pairing: int, theta: float, sections) -> Rope:
    """Plan for heads whose first `rot` elements turn; sections[a] pairs follow axis a.

    pairing 0 pairs element i with i + rot/2, pairing 1 element 2i with 2i + 1."""
    sec = list(sections)
    arr = (ctypes.c_int * max(1, len(sec)))(*map(_int, sec))
    h = ctypes.c_void_p(None)
    _check(lib.wq_rope_create(_int(rot), _int(pairing), float(theta), arr, len(sec), ctypes.byref(h)), "wq_rope_create")
    return Rope(h, int(rot), len(sec))


def wq_rope_dev(rope: Rope, x, pos, y, stream=None) -> None:
    """y[T, H, D] = x turned by the positions pos [axes, T] (int32); y may be x."""
    shape, dt, dev, xs = _first(x, 3, _FLOATS, "x")
    ys = _more(y, shape, x.dtype, dev, "y")
    T, H, D = shape
    ps = _more(pos, (rope.axes, T), torch.int32, dev, "pos")
    rc = lib.wq_rope_dev(rope.ptr, dev, x.data_ptr(), dt, T, H, D, xs[0], xs[1], pos.data_ptr(), ps[0], y.data_ptr(),
                         ys[0], ys[1], _raw_stream(stream, dev))
    if rc:
        _check(rc, "wq_rope_dev")


def wq_rope_free(rope: Rope) -> None:
    if rope is None:
        return
    _check(lib.wq_rope_free(rope.ptr), "wq_rope_free")
    rope.ptr = None


class KvCache:
    """A paged, quantised key/value cache over the caller's pools.

    k, v: uint8 [pages, heads, page, row bytes] with the same strides, rows contiguous; a row holds D float16 codes
    (2 D bytes, WQ_KV_F16), D int8 codes (WQ_KV_I8) or two 4-bit codes a byte (D / 2 bytes, WQ_KV_I4).
    k_scale, v_scale: float32 [pages, heads, page] with the same strides."""

    def __init__(self, kind: int, k, v, k_scale, v_scale):
        if kind not in (WQ_KV_F16, WQ_KV_I8, WQ_KV_I4):
            raise ValueError("kind must be WQ_KV_F16, WQ_KV_I8 or WQ_KV_I4")
        for t, what, dt, dims in ((k, "k", torch.uint8, 4), (v, "v", torch.uint8, 4),
                                  (k_scale, "k_scale", torch.float32, 3), (v_scale, "v_scale", torch.float32, 3)):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch tensor on a GPU" % what)
            if t.dtype != dt or not t.is_cuda or t.dim() != dims or t.device != k.device:
                raise ValueError("%s must be a %s tensor with %d dimensions, on k's GPU" % (what, dt, dims))
        if k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same shape and strides, rows contiguous")
        if k_scale.shape != k.shape[:3] or v_scale.shape != k.shape[:3] or k_scale.stride() != v_scale.stride():
            raise ValueError("k_scale and v_scale must have the shape of k without its rows, and the same strides")
        pages, heads, page, rb = k.shape
        self.kind, self.dim, self.heads, self.page = kind, (rb // 2, rb, rb * 2)[kind], heads, page
        self.tensors = (k, v, k_scale, v_scale)
        self.device, self.dev = k.device, k.get_device()
        self.c = _KvCacheC(k.device.index, kind, pages, heads, page, self.dim, k.data_ptr(), v.data_ptr(),
                           k_scale.data_ptr(), v_scale.data_ptr(), (ctypes.c_long * 3)(*k.stride()[:3]),
                           (ctypes.c_long * 3)(*k_scale.stride()))
        self.ref = ctypes.byref(self.c)


class KvBatch:
    """The new tokens of B sequences: q_start int32 [B+1], kv_len int32 [B] (new tokens among them), table int32
    [B, width] of pages, all on the GPU; T = q_start[B] tokens. max_q, max_kv: the longest lengths, if known."""

    def __init__(self, q_start, kv_len, table, T: int, max_q: int = 0, max_kv: int = 0):
        for t, what, dims in ((q_start, "q_start", 1), (kv_len, "kv_len", 1), (table, "table", 2)):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch tensor on a GPU" % what)
            if t.dtype != torch.int32 or not t.is_cuda or t.dim() != dims or t.device != q_start.device:
                raise ValueError("%s must be an int32 GPU tensor with %d dimensions" % (what, dims))
            if t.stride(-1) != 1 and t.shape[-1] > 1:
                raise ValueError("%s must be contiguous" % what)
        B, width = table.shape
        if q_start.shape[0] != B + 1 or kv_len.shape[0] != B:
            raise ValueError("q_start, kv_len and table must hold B + 1, B and B rows")
        if max(B, width, int(T)) > _INT_MAX:
            raise ValueError("a batch of %d sequences, %d pages each and %d tokens is not taken" % (B, width, int(T)))
        self.B, self.T, self.device, self.dev = B, _int(T), q_start.device, q_start.get_device()
        self.tensors = (q_start, kv_len, table)
        self.c = _KvBatchC(B, self.T, width, _int(max_q), _int(max_kv), table.stride(0), q_start.data_ptr(),
                           kv_len.data_ptr(), table.data_ptr())
        self.ref = ctypes.byref(self.c)


def _tokens(cache, batch, a, b, what):
    """(type code, strides) of the tokens' keys and values a, b [T, heads, D]."""
    shape, dt, dev, st = _first(a, 3, _FLOATS, what)
    if shape != (batch.T, cache.heads, cache.dim) or dev != cache.dev or dev != batch.dev:
        raise ValueError("%s must have shape %s, on the GPU of the cache and the batch" % (what, (batch.T, cache.heads, cache.dim)))
    if _more(b, shape, a.dtype, dev, what) != st:
        raise ValueError("%s must have the same strides" % what)
    return dt, st


def wq_kv_append_dev(cache: KvCache, batch: KvBatch, k_new, v_new, stream=None) -> None:
    """Quantise the batch's keys and values [T, heads, D] into their slots of the cache."""
    dt, st = _tokens(cache, batch, k_new, v_new, "k_new and v_new")
    rc = lib.wq_kv_append_dev(cache.ref, batch.ref, k_new.data_ptr(), v_new.data_ptr(), dt, st[0], st[1],
                              _raw_stream(stream, cache.dev))
    if rc:
        _check(rc, "wq_kv_append_dev")


def wq_kv_read_dev(cache: KvCache, batch: KvBatch, k_out, v_out, stream=None) -> None:
    """The values of the batch's tokens in the cache, into k_out, v_out [T, heads, D]."""
    dt, st = _tokens(cache, batch, k_out, v_out, "k_out and v_out")
    rc = lib.wq_kv_read_dev(cache.ref, batch.ref, k_out.data_ptr(), v_out.data_ptr(), dt, st[0], st[1],
                            _raw_stream(stream, cache.dev))
    if rc:
        _check(rc, "wq_kv_read_dev")


def wq_attn_paged_dev(cache: KvCache, batch: KvBatch, q, o, scale: float, causal: bool = True, window: int = 0,
                      lse=None, stream=None) -> None:
    """o[T, H, D] = attention of the batch's tokens q [T, H, D] over the cache; lse float32 [T, H] if given."""
    shape, dt, dev, qs = _first(q, 3, _FLOATS, "q")
    os_ = _more(o, shape, q.dtype, dev, "o")
    T, H, D = shape
    if T != batch.T or D != cache.dim or dev != cache.dev or dev != batch.dev:
        raise ValueError("q must have shape [%d, H, %d] on %s" % (batch.T, cache.dim, cache.device))
    lp = None
    if lse is not None:
        if _more(lse, shape[:2], torch.float32, dev, "lse")[0] != H and T > 1:
            raise ValueError("lse must be contiguous")
        lp = lse.data_ptr()
    rc = lib.wq_attn_paged_dev(cache.ref, batch.ref, q.data_ptr(), dt, H, qs[0], qs[1], scale, 1 if causal else 0, _int(window),
                               o.data_ptr(), os_[0], os_[1], lp, _raw_stream(stream, dev))
    if rc:
        _check(rc, "wq_attn_paged_dev")


def wq_describe_attn(cache, batch, dtype: int, H: int, causal: bool = True, window: int = 0) -> str:
    """The plan of wq_attn_paged_dev for queries of H heads and type code dtype (WQ_DT_F32, ...)."""
    buf = ctypes.create_string_buffer(256)
    _check(lib.wq_describe_attn(cache.ref, batch.ref, dtype, H, 1 if causal else 0, _int(window), buf, len(buf)), "wq_describe_attn")
    return buf.value.decode()
